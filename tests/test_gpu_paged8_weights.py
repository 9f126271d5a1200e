"""How many bits the attention over the cache in 8 bits keeps of its weights, by the rows of a tile: 2^-9 of each
(pairs of E4M3 values) up to 32 rows, 2^-11 (FP16) above, where values that cancel leave nothing else in the
output."""
import pytest
import torch

from paged8_ref import E4M3, inputs8, nearest8, values
from paged_ref import HALF, ref_attention
from test_gpu_paged8 import attend, close

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
SEQS = 150


def tile_rows(group, max_new):
    """Rows of a K/V head in a tile: as few tiles of up to 64 as hold them, of equal size."""
    rows = group * max_new
    return -(-rows // -(-rows // 64))


def cancelling(kv_heads, heads, dim):
    """Three keys a sequence: one of score 0 and V 0, the largest weight; two a little apart at about half of its weight,
    of V v and -v."""
    p = inputs8([3] * SEQS, [1] * SEQS, kv_heads, dim, 8, 8, seed=heads)
    for x in ("k8", "v8"):
        p[x].view(torch.uint8)[:] = 0
    p["ks"][:], p["vs"][:] = 1.0, 2.0 ** -3
    pg = p["table"][:, 0].long()
    p["k8"][pg, 1, :, :2] = torch.tensor([-1.0, 1.0], device="cuda").to(E4M3)
    p["k8"][pg, 2, :, :2] = torch.tensor([-1.0, 1.125], device="cuda").to(E4M3)
    p["v8"][pg, 1], p["v8"][pg, 2] = (torch.full((dim,), s * 448.0, device="cuda").to(E4M3) for s in (1, -1))
    g = torch.Generator(device="cuda").manual_seed(heads)
    q = torch.zeros(SEQS, heads, dim, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    q[..., 1] = (0.25 * torch.rand(SEQS, heads, generator=g, device="cuda")).to(BF16)
    return p, q


def bound(weight, ref, err, mass):
    """`weight` of each weight; 2^-16 of their arguments (2^-22 of the query's largest times three keys' codes, the scales'
    logarithms); the output's rounding."""
    before = err + mass * (weight + 2.0 ** -16)
    return before + HALF[BF16] * (ref.abs() + before)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_heads,heads", [(1, 8), (2, 16), (1, 16), (1, 32), (1, 33), (1, 48), (1, 64), (1, 100), (2, 80)])
def test_bits_of_the_weights(kv_heads, heads, dim):
    p, q = cancelling(kv_heads, heads, dim)
    ref, err, mass = ref_attention(values(p), q, 0, 0.6)
    weight = 2.0 ** -9 if tile_rows(heads // kv_heads, 1) <= 32 else 2.0 ** -11
    close(attend(p, q, scale=0.6), ref, bound(weight, ref, err, mass))


def test_the_inputs_tell_the_two_apart():
    """With weights as pairs of E4M3 values the outputs are outside the bound of FP16's."""
    p, q = cancelling(1, 64, 64)
    ref, err, mass = ref_attention(values(p), q, 0, 0.6)
    x = q[..., :2].double()
    score = torch.stack([torch.zeros_like(x[..., 0]), x[..., 1] - x[..., 0], 1.125 * x[..., 1] - x[..., 0]], -1) * 0.6
    w = 32.0 * torch.exp(score - score.amax(-1, keepdim=True))
    hi = nearest8(w)
    pair = hi + nearest8(16 * (w - hi)) / 16
    assert float(((pair - w).abs() / w).max()) <= 2.0 ** -9
    out = (pair[..., 1] - pair[..., 2]) * 448.0 / 8 / w.sum(-1)
    assert torch.allclose((w[..., 1] - w[..., 2]) * 448.0 / 8 / w.sum(-1), ref[..., 0], rtol=1e-9, atol=1e-9)
    out = out.to(BF16).double()
    assert ((out - ref[..., 0]).abs() > bound(2.0 ** -11, ref, err, mass)[..., 0]).any()
    assert ((out - ref[..., 0]).abs() <= bound(2.0 ** -9, ref, err, mass)[..., 0]).all()
