"""ds4g_paged_attention_status: a time-out is reported once, however many calls on the workspace
follow it, and nothing else is taken for one.  (No wait runs out here: the status word that a
CTA writes when one does is planted from the host.)"""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged_ref import fill_slots, paged_inputs, randn

pytestmark = pytest.mark.gpu

OK, ETIMEOUT = 0, pdl.ds4g.ETIMEOUT
TIMED_OUT = 0x54494d45   # the status word


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cta", [0, 5, 151, 319])
def test_a_time_out_stays_until_it_is_read(dtype, cta):
    p = paged_inputs([3000, 40], [1, 1], 1, 64, 16, dtype, seed=1)
    fill_slots(p, 2)
    q = randn((2, 4, 64), dtype, 3)
    kv, batch = pdl.PagedKV(p["k"], p["v"]), pdl.PagedBatch(p["table"], p["length"])
    ws = torch.full((pdl.paged_attention_workspace_bytes(kv, batch, 4),), 255, dtype=torch.uint8, device="cuda")
    want, out = torch.empty_like(q), torch.empty_like(q)
    pdl.paged_attention(kv, batch, q, want, ws)
    assert pdl.paged_attention_status(ws) == OK
    ws.view(torch.int32)[cta] = TIMED_OUT
    for _ in range(3):   # the next layers' calls
        pdl.paged_attention(kv, batch, q, out, ws)
    assert pdl.paged_attention_status(ws) == ETIMEOUT
    assert pdl.paged_attention_status(ws) == OK
    pdl.paged_attention(kv, batch, q, out, ws)
    assert pdl.paged_attention_status(ws) == OK and torch.equal(out, want)


@pytest.mark.parametrize("byte", [0, 1, 255])
def test_a_workspace_without_a_call_or_tokens_has_no_time_out(byte):
    p = paged_inputs([300], [1], 1, 64, 16, torch.bfloat16, seed=4)
    kv = pdl.PagedKV(p["k"], p["v"])
    none = pdl.PagedBatch(p["table"][:0], p["length"][:0])
    some = pdl.PagedBatch(p["table"], p["length"], torch.zeros(2, dtype=torch.int32, device="cuda"))
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((pdl.paged_attention_workspace_bytes(kv, some, 4),), byte, dtype=torch.uint8, device="cuda")
    assert pdl.paged_attention_status(ws) == OK
    for batch in (none, some):
        pdl.paged_attention(kv, batch, q, torch.empty_like(q), ws)
        assert pdl.paged_attention_status(ws) == OK
    stream = torch.cuda.Stream()
    assert pdl.paged_attention_status(ws, stream=stream) == OK


def test_what_is_no_workspace_is_refused():
    big = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    for ws in (big[:16], big[::2], big[:1].expand(1 << 16), big[128:], big.cpu()):
        try:
            rc = pdl.paged_attention_status(ws)
        except pdl.Ds4gError:
            continue
        assert rc == pdl.ds4g.EINVAL
