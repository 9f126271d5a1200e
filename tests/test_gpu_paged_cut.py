"""Paged attention of items that are cut between CTAs (tables of many units): keys that only
some of a call's tokens see with values that are not finite, on both sides of a cut, missing
pages that leave a whole share without a key, and infinities whose weight is far below the
sequence's largest."""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged_ref import HALF, fill_slots, paged_inputs, randn, ref_attention

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def attend(p, q, window=0):
    kv = pdl.PagedKV(p["k"], p["v"])
    batch = pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=int((p["start"][1:] - p["start"][:-1]).max()))
    ws = torch.full((pdl.paged_attention_workspace_bytes(kv, batch, q.shape[1]),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    pdl.paged_attention(kv, batch, q, out, ws, window=window)
    assert pdl.paged_attention_status(ws) == 0
    return out


def slot(p, b, j):
    return int(p["table"][b, j // p["page"]]), j % p["page"]


def check(p, q, window=0, kinds=True):
    """Against the 64-bit form, element by element: infinite and NaN where it is (kinds False: not
    finite where it is not), and otherwise within the bounds of the finite keys' sums."""
    got = attend(p, q, window).double()
    ref, _, _ = ref_attention(p, q, window)
    finite = dict(p, k=p["k"].nan_to_num(0.0, 0.0, 0.0), v=p["v"].nan_to_num(0.0, 0.0, 0.0))
    _, err, mass = ref_attention(finite, q, window)
    before = err + (HALF[BF16] if q.dtype == BF16 and p["k"].dtype == BF16 else 0.0) * mass
    some = ref.isfinite()
    assert torch.equal(got.isfinite(), some)
    if kinds:
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(torch.where(got.isinf(), got, 0.0), torch.where(ref.isinf(), ref, 0.0))
    bad = some & ~((got - ref).abs() <= before + HALF[q.dtype] * (ref.abs() + before))
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()))
    assert (got[mass.sum(-1) == 0] == 0).all()
    return got


# (128 keys of the tensor-core form, 64 of the FP32 form: cuts at multiples of 128 are cuts of both)
LAYOUTS = [(1, 4, 64, 16), (2, 16, 128, 64), (1, 64, 128, 64), (1, 40, 64, 48)]


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("kv_heads,heads,dim,page", LAYOUTS)
def test_newest_keys_around_a_cut(dtype, cache, kv_heads, heads, dim, page):
    """Tokens 5117 .. 5122, the cut at 5120; and all of them before or behind the last cut."""
    p = paged_inputs([5123, 2688, 4998], [6, 6, 5], kv_heads, dim, page, cache, seed=dim + page)
    fill_slots(p, 3)
    q = randn((17, heads, dim), dtype, 4)
    clean = check(p, q)
    for b, keys in ((0, (5118, 5121)), (1, (2684, 2687)), (2, (4995,))):
        for i, j in enumerate(keys):
            v = p["v"][slot(p, b, j)]
            v[:, 5 + i], v[:, 9 + i], v[:, 20] = float("nan"), float("inf"), float("-inf") if i else float("inf")
    got = check(p, q)
    for b, t0, first in ((0, 0, 5117), (1, 6, 2682), (2, 12, 4993)):
        bad = {0: 5118, 1: 2684, 2: 4995}[b]
        n = (6, 6, 5)[b]
        for i in range(n):   # tokens before the first bad key keep their values
            if first + i < bad:
                assert torch.equal(got[t0 + i], clean[t0 + i])
            else:
                assert got[t0 + i, :, 5].isnan().all() and (got[t0 + i, :, 9] == float("inf")).all()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("kv_heads,heads,dim,page", LAYOUTS)
def test_window_edges_around_a_cut(dtype, cache, kv_heads, heads, dim, page):
    """Windows of many units, the oldest keys of the tokens 2046 .. 2049 and 0 ..: not finite."""
    window = 1500
    p = paged_inputs([2046 + window + 3, 9000, 1400], [4, 3, 4], kv_heads, dim, page, cache, seed=dim + page + 1)
    fill_slots(p, 5)
    q = randn((11, heads, dim), dtype, 6)
    clean = check(p, q, window)
    a, c = 2046, 8997 - window + 1     # the first tokens' oldest keys
    for b, j, d in ((0, a + 1, 7), (0, a + 2, 8), (1, c, 7), (1, c + 1, 8)):
        p["v"][slot(p, b, j)][:, d] = float("nan") if d == 7 else float("inf")
    p["v"][slot(p, 0, a - 1)][:] = float("nan")     # no token sees it
    p["k"][slot(p, 0, a - 1)][:] = float("inf")
    got = check(p, q, window)
    sees = {(0, 7): [0, 1], (0, 8): [0, 1, 2], (1, 7): [4], (1, 8): [4, 5]}
    for t in range(11):
        b = 0 if t < 4 else 1 if t < 7 else 2
        for d in (7, 8):
            if t in sees.get((b, d), []):
                assert not got[t, :, d].isfinite().any()
            else:
                assert torch.equal(got[t, :, d], clean[t, :, d])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page", LAYOUTS)
def test_missing_pages_of_whole_shares(dtype, kv_heads, heads, dim, page):
    lengths, new = [6000, 4100, 3000, 2496], [3, 1, 4, 2]
    p = paged_inputs(lengths, new, kv_heads, dim, page, dtype, seed=dim + page + 2)
    fill_slots(p, 7)
    table = p["table"]
    table[0, 640 // page:1920 // page] = -1                      # ten units and more
    table[0, (6000 - 1) // page] = p["k"].shape[0]               # the newest keys' own page
    table[1, 1:] = -1                                            # all but the first page
    table[2, :] = -7                                             # nothing at all
    table[3, :2304 // page] = 2 ** 31 - 1                        # the newest ones alone
    q = randn((10, heads, dim), dtype, 8)
    check(p, q)
    check(p, q, window=1300)   # sequence 1's window holds no key that is there
    p["length"][3] = table.shape[1] * page + 1                   # past the table's end
    check(p, q)


def peaked(dtype, cache, lengths, new, peaks, kv_heads, heads, dim, page, seed):
    """Sequences in which one key has a score 400 above the others', whose weights (e^-400) are 0
    in 32 bits and not in 64."""
    p = paged_inputs(lengths, new, kv_heads, dim, page, cache, seed=seed)
    fill_slots(p, seed)
    q = randn((sum(new), heads, dim), dtype, seed + 1)
    q[..., 0] = 16.0
    p["k"][..., 0] = torch.where(p["k"][..., 0].isnan(), float("nan"), 0.0)
    for b, j in peaks:
        p["k"][slot(p, b, j)][:, 0] = 25.0 * dim ** 0.5
    return p, q


@pytest.mark.parametrize("kv_heads,heads,dim,page", LAYOUTS)
def test_infinities_of_partly_seen_keys_survive_the_join(kv_heads, heads, dim, page):
    """An infinity counts however far its key's weight lies below the largest, as it does where
    the item is whole."""
    window = 1500
    p, q = peaked(BF16, BF16, [2046 + window + 3, 5123], [4, 6], [(0, 3000), (1, 4700)], kv_heads, heads, dim, page, 9)
    p["v"][slot(p, 0, 2047)][:, 8] = float("inf")      # the oldest key of token 1
    p["v"][slot(p, 0, 3546)][:, 9] = float("-inf")     # the newest key of token 1
    p["v"][slot(p, 1, 5121)][:, 9] = float("inf")      # of token 4 of six
    got = check(p, q, window)
    assert (got[:2, :, 8] == float("inf")).all() and (got[1:4, :, 9] == float("-inf")).all()
    assert (got[8:, :, 9] == float("inf")).all() and got[4:8].isfinite().all()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("kv_heads,heads,dim,page", LAYOUTS + [(1, 3, 32, 16), (1, 2, 256, 16)])
def test_a_seen_key_counts_however_small_its_weight(dtype, cache, kv_heads, heads, dim, page):
    """What is not finite in the V row of a key that a token sees leaves nothing finite there, in
    whole and in cut items, beside the key with the large score and far from it."""
    p, q = peaked(dtype, cache, [100, 3549, 3000], [1, 1, 2], [(0, 4), (1, 2000), (2, 2999)], kv_heads, heads, dim, page, 11)
    for b, j, d in ((0, 6, 3), (0, 70, 4), (1, 2002, 3), (1, 2064, 4), (1, 3000, 5), (2, 2997, 6), (2, 0, 7)):
        p["v"][slot(p, b, j)][:, d] = float("inf") if d % 2 else float("nan")
    got = check(p, q, kinds=False)
    for t, dims in ((0, (3, 4)), (1, (3, 4, 5)), (2, (6, 7)), (3, (6, 7))):
        assert torch.equal(got[t].isfinite().all(0).cpu(), torch.tensor([d not in dims for d in range(dim)]))
