"""Paged attention at the ends of its ranges: up to 128 new tokens of a sequence, windows shorter
than a call's tokens, groups of more than 128 query heads, tables without pages; and rows of
probabilities that outnumber the clusters."""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged_ref import fill_slots, paged_inputs, randn
from test_gpu_paged_cut import attend, check, slot

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page", [(2, 2, 64, 16), (1, 4, 128, 64), (1, 64, 128, 64), (1, 40, 64, 48)])
@pytest.mark.parametrize("window", [0, 17, 300])
def test_128_new_tokens(dtype, kv_heads, heads, dim, page, window):
    p = paged_inputs([128, 131, 900, 60, 1280], [128, 128, 100, 60, 1], kv_heads, dim, page, dtype, seed=dim + window)
    fill_slots(p, 1)
    q = randn((417, heads, dim), dtype, 2)
    clean = check(p, q, window)
    # keys that some of a call's tokens see and others do not: the newest one, one that has left
    # the window of some and is not there yet for others, and one at a tile's end
    for b, j, d in ((0, 127, 3), (0, 40, 4), (1, 64, 5), (2, 895, 6), (2, 850, 7), (3, 59, 8)):
        p["v"][slot(p, b, j)][:, d] = float("nan") if d % 2 else float("inf")
    got = check(p, q, window)
    for t, pos, b in ((0, 0, 0), (39, 39, 0), (128, 3, 1), (188, 63, 1), (256, 800, 2), (416, 1279, 4)):
        assert torch.equal(got[t], clean[t])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page", [(1, 129, 64, 16), (2, 512, 128, 32)])
def test_groups_of_more_than_128_heads(dtype, kv_heads, heads, dim, page):
    p = paged_inputs([700, 3, 1600], [2, 3, 1], kv_heads, dim, page, dtype, seed=heads)
    fill_slots(p, 3)
    check(p, randn((6, heads, dim), dtype, 4))
    check(p, randn((6, heads, dim), dtype, 5), window=100)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tables_without_pages(dtype):
    p = paged_inputs([5, 0, 2000], [1, 1, 3], 1, 64, 16, dtype, seed=6)
    fill_slots(p, 7)
    p["table"] = p["table"][:, :0]
    assert (attend(p, randn((5, 4, 64), dtype, 8)) == 0).all()


# rows and sizes of every kind of cluster, more rows than fit at once
@pytest.mark.parametrize("rows,n", [(4000, 2700), (1000, 5000), (700, 16384), (300, 40000), (130, 100000), (60, 262144),
                                    (2100, 4096)])
@pytest.mark.parametrize("t", [0.7, 0.0])
def test_more_rows_than_clusters(rows, n, t):
    z = randn((rows, n + 4), F32, rows + n, 3.0)[:, :n]
    z[1, 3], z[2, :], z[rows - 1, n - 1] = float("nan"), float("-inf"), float("inf")
    z[rows // 2, 5:] = z[rows // 2, 4]
    out = torch.full_like(z, float("nan"))
    pdl.probs(z, t, out)
    for r0 in range(0, rows, 256):
        x = z[r0:r0 + 256].double().nan_to_num(nan=float("-inf"), posinf=float("inf"), neginf=float("-inf"))
        top = x.amax(-1, keepdim=True)
        if t <= 0:
            want = torch.zeros_like(x)
            some = top[:, 0] > float("-inf")
            want[some, (x == top).int().argmax(-1)[some]] = 1.0
        else:
            e = torch.where(top == float("inf"), (x == top).double(), torch.exp((x - top) / t)).nan_to_num(0.0)
            want = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
        got = out[r0:r0 + 256].double()
        # the bound of a single row: at most 120 half steps, and values below the smallest normal number
        assert ((got - want).abs() <= 120 * 2.0 ** -24 * want + 2.0 ** -126).all()
    pdl.probs(z, t, z)
    assert torch.equal(z, out)
