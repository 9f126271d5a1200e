"""Attention over the cache in 8 bits where one V block's scale is 2^64 and the others' are 2^-64 (blocks of
zeros): their keys add nothing to the sum of V, but count in the sum of the weights, whichever comes first and
however the item is cut."""
import math

import pytest
import torch

from paged8_ref import E4M3, inputs8, values
from paged_ref import randn, ref_attention
from test_gpu_paged8 import attend, bound_of, close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("length,at", [(100, 99), (700, 0), (700, 380), (700, 699), (20000, 3), (20000, 12345), (20000, 19999)])
@pytest.mark.parametrize("kv_heads,heads,dim,score", [(1, 4, 128, 0.0), (1, 64, 128, 0.0), (2, 16, 64, -9.0), (1, 20, 64, 4.0)])
def test_zeros_beside_a_large_value(dtype, length, at, kv_heads, heads, dim, score):
    """One key of V 2^64 and a score of its own, all others zeros of score 0: out = 2^64 w / (w + length - 1)."""
    p = inputs8([length], [1], kv_heads, dim, 16, 16, seed=length + at)
    for x in ("k8", "v8"):
        p[x].view(torch.uint8)[:] = 0
    p["ks"][:], p["vs"][:] = 1.0, 2.0 ** -64
    pg = int(p["table"][0, at // 16])
    p["vs"][pg] = 2.0 ** 64
    p["v8"][pg, at % 16] = torch.ones(kv_heads, dim, device="cuda").to(E4M3)
    p["k8"][pg, at % 16, :, 0] = torch.full((kv_heads,), score, device="cuda").to(E4M3)
    q = torch.zeros(1, heads, dim, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    got = attend(p, q, scale=1.0)
    w = math.exp(score)
    # the score and its weight in FP32 (2^-16 with the logarithms of the scales, up to 64 in FP32), 2^-8 of the
    # weight, the output's rounding
    want = 2.0 ** 64 * w / (w + length - 1)
    assert float((got.double() / want - 1).abs().max()) <= 2.0 ** -16 + 2.0 ** -8 + 2.0 ** -8


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,block", [(1, 64, 128, 16), (4, 16, 128, 4), (1, 24, 64, 16)])
def test_scales_over_the_whole_range(dtype, kv_heads, heads, dim, block):
    """V scales from 2^-64 to 2^64, in rising, falling and random order along the sequences."""
    lengths = [900, 900, 6000, 40]
    p = inputs8(lengths, [1, 2, 1, 1], kv_heads, dim, 16, block, seed=7)
    for b, n in enumerate(lengths):
        pages = p["table"][b, :-(-n // 16)].long()
        steps = torch.linspace(-64, 64, len(pages) * (16 // block), device="cuda").round()
        steps = [steps, steps.flip(0), steps[torch.randperm(len(steps), generator=torch.Generator().manual_seed(3)).cuda()], steps][b]
        p["vs"][pages] = torch.exp2(steps).view(len(pages), 16 // block, 1).expand(-1, -1, kv_heads).contiguous()
    q = randn((5, heads, dim), dtype, 8)
    ref, err, mass = ref_attention(values(p), q)
    close(attend(p, q), ref, bound_of(p, q, ref, err, mass))
