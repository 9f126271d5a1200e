"""Attention over the cache in 8 bits of items that are cut between CTAs: NaN codes of keys that only
some of a call's tokens see, on both sides of a cut, at the edges of windows and of shares without a
page; and the status of a call."""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged8_ref import NAN_CODE, inputs8, values
from paged_ref import randn, ref_attention
from test_gpu_paged8 import attend, bound_of, cache, close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

# (128 keys of the tensor-core form, 64 of the FP32 form: cuts at multiples of 128 are cuts of both)
LAYOUTS = [(1, 2, 64, 16, 16), (2, 16, 128, 64, 64), (1, 64, 128, 64, 32), (1, 8, 64, 48, 8), (2, 4, 128, 16, 16)]


def nan_at(p, b, j, dims, name="v8"):
    page = p["page"]
    p[name].view(torch.uint8)[int(p["table"][b, j // page]), j % page, :, dims] = NAN_CODE


def check(p, q, window=0, clean=None):
    """NaN exactly where the 64-bit form has one, everything else within the finite keys' bounds."""
    got = attend(p, q, window)
    ref, _, _ = ref_attention(values(p), q, window)
    fine = dict(p, k8=p["k8"].clone(), v8=p["v8"].clone())
    for name in ("k8", "v8"):
        codes = fine[name].view(torch.uint8)
        codes[(codes & 0x7f) == NAN_CODE] = 0
    some, err, mass = ref_attention(values(fine), q, window)
    assert torch.equal(got.isnan(), ref.isnan())
    bound = bound_of(fine, q, some, err, mass)
    bad = ~ref.isnan() & ~((got.double() - some).abs() <= bound)
    assert not bad.any(), float(((got.double() - some).abs() / bound)[bad].max())
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page,block", LAYOUTS)
def test_newest_keys_around_a_cut(dtype, kv_heads, heads, dim, page, block):
    """Tokens 5117 .. 5122, the cut at 5120; and all of them before or behind the last cut."""
    p = inputs8([5123, 2688, 4998], [6, 6, 5], kv_heads, dim, page, block, seed=dim + page)
    q = randn((17, heads, dim), dtype, 4)
    clean = check(p, q)
    for b, keys in ((0, (5118, 5121)), (1, (2684, 2687)), (2, (4995,))):
        for i, j in enumerate(keys):
            nan_at(p, b, j, [5 + i, 40])
    got = check(p, q)
    for t0, n, seen in ((0, 6, 1), (6, 6, 2), (12, 5, 2)):
        assert torch.equal(got[t0:t0 + seen], clean[t0:t0 + seen]) and got[t0 + seen:t0 + n, :, 40].isnan().all()
    nan_at(p, 0, 5119, [1], "k8")      # a score: nothing of the tokens that see it is left
    got = check(p, q)
    assert got[2:6].isnan().all() and torch.equal(got[:1], clean[:1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page,block", LAYOUTS)
def test_window_edges_around_a_cut(dtype, kv_heads, heads, dim, page, block):
    window = 1500
    p = inputs8([2046 + window + 3, 9000, 1400], [4, 3, 4], kv_heads, dim, page, block, seed=dim + page + 1)
    q = randn((11, heads, dim), dtype, 6)
    clean = check(p, q, window)
    a, c = 2046, 8997 - window + 1     # the first tokens' oldest keys
    for b, j, d in ((0, a + 1, 7), (0, a + 2, 8), (1, c, 7), (1, c + 1, 8)):
        nan_at(p, b, j, [d])
    nan_at(p, 0, a - 1, list(range(dim)))     # no token sees it
    nan_at(p, 0, a - 1, [0], "k8")
    got = check(p, q, window)
    sees = {(0, 7): [0, 1], (0, 8): [0, 1, 2], (1, 7): [4], (1, 8): [4, 5]}
    for t in range(11):
        b = 0 if t < 4 else 1 if t < 7 else 2
        for d in (7, 8):
            if t in sees.get((b, d), []):
                assert got[t, :, d].isnan().all()
            else:
                assert torch.equal(got[t, :, d], clean[t, :, d])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page,block", LAYOUTS)
def test_missing_pages_of_whole_shares(dtype, kv_heads, heads, dim, page, block):
    lengths, new = [6000, 4100, 3000, 2496], [3, 1, 4, 2]
    p = inputs8(lengths, new, kv_heads, dim, page, block, seed=dim + page + 2)
    table = p["table"]
    table[0, 640 // page:1920 // page] = -1                      # ten units and more
    table[0, (6000 - 1) // page] = p["k8"].shape[0]              # the newest keys' own page
    table[1, 1:] = -1                                            # all but the first page
    table[2, :] = -7                                             # nothing at all
    table[3, :2304 // page] = 2 ** 31 - 1                        # the newest ones alone
    q = randn((10, heads, dim), dtype, 8)
    got = check(p, q)
    assert (got[4:8] == 0).all()
    check(p, q, window=1300)   # sequence 1's window holds no key that is there
    p["length"][3] = table.shape[1] * page + 1                   # past the table's end
    check(p, q)


@pytest.mark.parametrize("kv_heads,heads,dim,page,block", LAYOUTS)
def test_a_share_whose_scores_are_all_nan(kv_heads, heads, dim, page, block):
    """Keys of one CTA's share with NaN codes alone: it has no maximum, and the row no value."""
    p = inputs8([9000, 500], [1, 1], kv_heads, dim, page, block, seed=dim + page + 3)
    q = randn((2, heads, dim), BF16, 9)
    clean = check(p, q)
    for i in range(3200 // page + 1, 6000 // page):
        p["k8"].view(torch.uint8)[int(p["table"][0, i])] = NAN_CODE
    got = check(p, q)
    assert got[0].isnan().all() and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cta", [0, 5, 151, 319])
def test_a_time_out_stays_until_it_is_read(dtype, cta):
    """The status word that a CTA writes when a wait runs out is planted from the host."""
    p = inputs8([3000, 40], [1, 1], 1, 64, 16, 16, seed=1)
    q = randn((2, 4, 64), dtype, 3)
    kv, batch = cache(p), pdl.PagedBatch(p["table"], p["length"])
    ws = torch.full((pdl.paged_attention_workspace_bytes(kv, batch, 4),), 255, dtype=torch.uint8, device="cuda")
    want, out = torch.empty_like(q), torch.empty_like(q)
    pdl.paged_attention(kv, batch, q, want, ws)
    assert pdl.paged_attention_status(ws) == 0
    ws.view(torch.int32)[cta] = 0x54494d45
    for _ in range(3):
        pdl.paged_attention(kv, batch, q, out, ws)
    assert pdl.paged_attention_status(ws) == pdl.ds4g.ETIMEOUT
    assert pdl.paged_attention_status(ws) == 0
    pdl.paged_attention(kv, batch, q, out, ws)
    assert pdl.paged_attention_status(ws) == 0 and torch.equal(out, want)


def test_one_workspace_for_both_caches():
    """A workspace as large as either cache asks for serves calls on both in turn."""
    p = inputs8([20000, 3000, 50], [1, 1, 1], 1, 128, 64, 64, seed=5)
    kv8, batch, q = cache(p), pdl.PagedBatch(p["table"], p["length"]), randn((3, 64, 128), BF16, 6)
    kv = pdl.PagedKV(*(values(p)[x].to(BF16) for x in "kv"))
    ws = torch.empty(max(pdl.paged_attention_workspace_bytes(c, batch, 64) for c in (kv, kv8)), dtype=torch.uint8, device="cuda")
    want = []
    for c in (kv, kv8):
        want.append(torch.empty_like(q))
        pdl.paged_attention(c, batch, q, want[-1], ws)
    for _ in range(3):
        for c, w in zip((kv, kv8), want):
            out = torch.empty_like(q)
            pdl.paged_attention(c, batch, q, out, ws)
            assert torch.equal(out, w)
    assert pdl.paged_attention_status(ws) == 0
