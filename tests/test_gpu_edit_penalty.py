"""The repetition penalty of ds4g_edit_logits alone: z / r for z > 0, z r otherwise, each rounded once."""
import numpy as np
import pytest
import torch

import prefill_decode_layer_gb300 as pdl

pytestmark = pytest.mark.gpu

FLT_MAX = 3.4028234663852886e38


def penalised(z, r):
    rows, vocab = z.shape
    ids = torch.arange(vocab, dtype=torch.int32).repeat(rows, 1).cuda()
    out = torch.empty(rows, vocab, device="cuda")
    pdl.edit_logits(z.cuda(), out, pdl.LogitEdits(history=ids, n_prompt=torch.full((rows,), vocab, dtype=torch.int32).cuda(),
                                                  repetition=r.cuda()))
    return out.double().cpu().numpy()


@pytest.mark.parametrize("vocab", [1500, 40000])
def test_each_logit_is_rounded_once(vocab):
    """Off by half a step (2^-24 of the value, 2^-150 below the normal ones), and 2^-20 of that more for quotients between
    two steps."""
    g = torch.Generator().manual_seed(vocab)
    z = 3 * torch.randn(60, vocab, generator=g)
    r = 1.0 + 0.3 * torch.rand(60, generator=g)
    r[40:] = torch.exp(torch.empty(20).uniform_(-8, 8, generator=g))
    got = penalised(z, r)
    z, r = z.double().numpy(), r.double().numpy()[:, None]
    ref = np.where(z > 0, z / r, z * r)
    off = np.abs(got - ref) / (2.0 ** (np.floor(np.log2(np.abs(ref))) - 24))   # in half steps
    assert off.max() <= 1 + 2.0 ** -20, off.max()


TINY, SMALL = 2.0 ** -149, 2.0 ** -126
ENDS = [0.0, -0.0, TINY, 5 * TINY, -7 * TINY, SMALL, 1.5 * SMALL, -SMALL, 1e-30, -1e-30, 1e-10, 0.9, 1.0, -1.0, 123.456, 1e30, -1e30,
        FLT_MAX, -FLT_MAX, float("inf"), float("-inf"), float("nan")]


@pytest.mark.parametrize("r", [2.0 ** -60, 1e-10, 0.3, 1.0, 1.7, 3.0, 1e10, 2.0 ** 60])
def test_logits_at_the_ends(r):
    """As a division or product in FP32, to infinities too; quotients below 2^-100 a unit off at most (2^-149 where
    they are subnormal)."""
    z, r = torch.tensor([ENDS * 20]), torch.tensor([r])
    got = penalised(z, r)[0]
    z, r = z.numpy()[0], r.numpy()[0]
    with np.errstate(all="ignore"):
        ref = np.where(z > 0, z / r, z * r)                                          # in FP32
        near = np.where(z > 0, z.astype(np.float64) / r, z.astype(np.float64) * r)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    got, near, above = got[fine], near[fine], z[fine] > 0
    unit = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(near), 1e-300))) - 23), TINY)
    most = np.where(above & (near <= 2.0 ** -100), unit, unit / 2 * (1 + 2.0 ** -20))
    assert (np.abs(got - near) <= most).all()
    assert np.array_equal(got[near == 0], near[near == 0])


@pytest.mark.parametrize("r", [TINY, 1e-39, 2.0 ** -127, SMALL, 1e-30, 2.0 ** -61, 2.0 ** 61, 1e30, 2.0 ** 126, 3e38, FLT_MAX])
def test_penalties_at_the_ends(r):
    """Products with the rounded reciprocal."""
    z, r = torch.tensor([ENDS]), torch.tensor([r])
    got = penalised(z, r)[0].astype(np.float32)
    z, r = z.numpy()[0], r.numpy()[0]
    with np.errstate(all="ignore"):
        ref = np.where(z > 0, z * (np.float32(1) / r), z * r)
    assert np.array_equal(got, ref, equal_nan=True)
