"""Rows of an 8-bit block that are taken back, as after rejected drafts: the scale that they asked for stays until
the block is begun again, and the rows beside them lose no more than that scale's rounding."""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged8_ref import E4M3, ask, f32
from paged_ref import randn

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PAGE = BLOCK = 16


class Cache:
    def __init__(self, heads, dim):
        codes = [torch.zeros(2, PAGE, heads, dim, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        self.kv = pdl.PagedKV8(*codes, *(torch.ones(2, 1, heads, device="cuda") for _ in range(2)))
        self.table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")

    def append(self, length, k, v):
        n = k.shape[0]
        batch = pdl.PagedBatch(self.table, torch.tensor([length], dtype=torch.int32, device="cuda"),
                               torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_new=n)
        pdl.paged_append(self.kv, batch, k, v)

    def rows(self, page, n):
        return [(f32(c[page, :n]) * s[page, 0][:, None]).double() for c, s in ((self.kv.k, self.kv.k_scale), (self.kv.v, self.kv.v_scale))]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("large", [2.0, 64.0, 2.0 ** 12, 2.0 ** 40])
def test_rejected_drafts_leave_their_scale(dtype, large):
    heads, dim = 2, 64
    rows = [randn((n, heads, dim), dtype, 10 + n) for n in (9, 2, 1, 16)]
    with_drafts, without = Cache(heads, dim), Cache(heads, dim)
    for c in (with_drafts, without):
        c.append(9, rows[0], -rows[0])
    with_drafts.append(11, large * rows[1], large * -rows[1])   # two drafts, not kept
    before = [x.clone() for x in with_drafts.rows(1, 9)]
    for c in (with_drafts, without):
        c.append(10, rows[2], -rows[2])                         # the token after them in the first one's slot
    x = torch.cat([rows[0], rows[2]]).double()
    for got, scale, sign in zip(with_drafts.rows(1, 10), (with_drafts.kv.k_scale, with_drafts.kv.v_scale), (1, -1)):
        for h in range(heads):
            asked = max(ask(float(rows[0][:, h].abs().max())), ask(float(large * rows[1][:, h].abs().max())))
            asked = max(asked, ask(float(rows[2][:, h].abs().max())))
            assert float(scale[1, 0, h]) == asked
            # each row's own rounding (2^-4 of it, or half a step of 2^-9 of its first scale, not above the last) and the last scale's
            off = (got[:, h] - sign * x[:, h]).abs()
            assert (off <= 2.0 ** -4 * x[:, h].abs() + 2 * 2.0 ** -10 * asked).all()
    assert all(torch.equal(a, b[:9]) for a, b in zip(before, with_drafts.rows(1, 10)))   # the token after them changes nothing more
    # blocks begun by a call do not know of them, and the same block begun again forgets
    for c in (with_drafts, without):
        c.append(16, rows[3], rows[3])
    for name in ("k", "v"):
        a, b = (getattr(c.kv, name)[1].view(torch.uint8) for c in (with_drafts, without))
        assert torch.equal(a, b)
        assert torch.equal(getattr(with_drafts.kv, name + "_scale")[1], getattr(without.kv, name + "_scale")[1])
