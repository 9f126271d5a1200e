"""An append to the 8-bit cache whose tokens and heads make more blocks of work than 32 bits count: the last
token's row is stored, and nothing else is touched."""
import ctypes as C

import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged8_ref import E4M3
from prefill_decode_layer_gb300 import ds4g

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [131073, 262145])
def test_more_work_than_32_bits_count(n):
    heads, dim = 65536, 16
    row = heads * dim
    codes = [torch.zeros(1, 1, heads, dim, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    kv = pdl.PagedKV8(*codes, *(torch.ones(1, 1, heads, device="cuda") for _ in range(2)))
    # the first sequence's tokens lie past its table and are not read; the second has one token and the page
    start = torch.tensor([0, n - 1, n], dtype=torch.int32, device="cuda")
    length = torch.tensor([n + 5, 1], dtype=torch.int32, device="cuda")
    table = torch.tensor([[-1], [0]], dtype=torch.int32, device="cuda")
    batch = pdl.PagedBatch(table, length, start, max_new=n)
    batch.struct.n_tokens = n
    x = torch.randn(2, heads, dim, device="cuda").to(torch.bfloat16)
    first = [(x[i].data_ptr() - (n - 1) * row * 2) % 2 ** 64 for i in range(2)]   # of rows that only the last one is there of
    rc = pdl.lib().ds4g_paged_append8(C.byref(kv.struct), C.byref(batch.struct), C.c_void_p(first[0]), row, C.c_void_p(first[1]), row,
                                      None, None, 0, None, 0, 0, ds4g.BF16, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    for c, s, y in zip((kv.k, kv.v), (kv.k_scale, kv.v_scale), x.float()):
        top = y.abs().amax(-1)
        m, e = torch.frexp(top)
        want = torch.exp2((e - 9 + (m > 0.875)).clamp(-64, 64).float())
        assert torch.equal(s[0, 0], want)
        assert torch.equal(c[0, 0].float(), (y / want[:, None]).to(E4M3).float())
