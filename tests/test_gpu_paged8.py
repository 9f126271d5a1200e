"""The paged K/V cache in 8 bits (ds4g_paged_append8, ds4g_paged_attention8) against 64-bit forms:
head layouts, page and block sizes, strides, ragged and empty sequences, windows, missing pages, NaN
codes and scales in every place that is masked, scales far apart, captured graphs, and the append
and the attention as they are used together."""
import math

import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged8_ref import E4M3, NAN_CODE, check_append8, f32, inputs8, values
from paged_ref import HALF, randn, ref_attention

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def close(got, ref, bound):
    """Every element within `bound` of ref, NaN exactly where ref has one."""
    got = got.double()
    assert torch.equal(got.isnan(), ref.isnan())
    bad = ~((got - ref).abs() <= bound) & ~ref.isnan()
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()), float(((got - ref).abs() / bound)[bad].max()))


def cache(p):
    return pdl.PagedKV8(p["k8"], p["v8"], p["ks"], p["vs"])


def attend(p, q, window=0, scale=0.0, max_new=None, out=None, ws=None, start=True):
    kv = cache(p)
    new = int((p["start"][1:] - p["start"][:-1]).max())
    batch = pdl.PagedBatch(p["table"], p["length"], p["start"] if start else None, max_new=max_new or max(1, new))
    out = torch.full_like(q, float("nan")) if out is None else out
    if ws is None:
        ws = torch.full((pdl.paged_attention_workspace_bytes(kv, batch, q.shape[1]),), 255, dtype=torch.uint8,
                        device="cuda")
    pdl.paged_attention(kv, batch, q, out, ws, scale=scale, window=window)
    assert pdl.paged_attention_status(ws) == 0
    return out


def bound_of(p, q, ref, err, mass, scale=None):
    """What the outputs may be off by: `err` of the FP32 form; in the tensor-core form also the
    queries' second halves (2^-22 of a row's largest for each dim, once more for the weights'
    maximum), the scales' logarithms (up to 64 in FP32: 2^-18) and the weights: 2^-8 of each (E4M3 pairs; 2^-11 as
    FP16), or 2^-32 of the largest times the largest V that its scales allow."""
    dim = q.shape[2]
    before = err
    if q.dtype == BF16 and dim in (64, 128) and p["page"] % 8 == 0:
        scale = 1.0 / math.sqrt(dim) if scale is None else scale
        fine = values(p)["k"].nan_to_num(0.0)
        k_sum = float(fine.abs().sum(-1).max())
        ds = 2.0 ** -22 * q.double().abs().amax(-1, keepdim=True) * k_sum * scale
        tiny = 2.0 ** -32 * float(p["length"].max()) * 448.0 * float(p["vs"].nan_to_num(0.0).max())
        before = err + mass * (4 * ds + 2.0 ** -17 + 2.0 ** -8) + (mass > 0) * tiny
    return before + HALF[q.dtype] * (ref.abs() + before)


def check_attention(p, heads, dtype, window=0, scale=None, seed=1, q_scale=1.0):
    q = randn((p["tokens"], heads, p["k8"].shape[3]), dtype, seed, q_scale)
    ref, err, mass = ref_attention(values(p), q, window, scale)
    got = attend(p, q, window, scale or 0.0)
    n = int(p["start"][-1])
    assert got[n:].isnan().all()          # rows behind the last sequence
    close(got[:n], ref[:n], bound_of(p, q, ref, err, mass, scale)[:n])
    assert (got[:n][mass[:n].sum(-1) == 0] == 0).all()
    return got


LENGTHS = [1, 127, 128, 129, 5, 640, 0, 64, 255, 1000]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page,block", [
    (1, 64, 128, 64, 64), (8, 32, 128, 16, 16), (2, 8, 64, 48, 8), (4, 4, 64, 8, 1), (1, 128, 128, 128, 32), (3, 15, 128, 24, 3),
    (1, 8, 32, 16, 16), (2, 6, 48, 7, 7), (1, 3, 256, 1, 1), (2, 10, 96, 32, 4), (2, 16, 128, 256, 64), (2, 64, 64, 192, 96),
    (1, 200, 64, 16, 16), (2, 34, 128, 40, 20)])
def test_attention_one_token(dtype, kv_heads, heads, dim, page, block):
    p = inputs8(LENGTHS, [1] * len(LENGTHS), kv_heads, dim, page, block, seed=dim + heads)
    check_attention(p, heads, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,page,block,window", [
    (1, 64, 128, 64, 64, 0), (1, 64, 128, 64, 16, 100), (8, 32, 128, 16, 16, 0), (2, 14, 64, 40, 8, 33),
    (1, 100, 128, 16, 8, 129), (1, 8, 32, 16, 16, 16), (2, 6, 64, 16, 16, 1)])
def test_attention_several_tokens_and_windows(dtype, kv_heads, heads, dim, page, block, window):
    new = [1, 5, 3, 8, 5, 2, 0, 7, 1, 4]
    p = inputs8(LENGTHS, new, kv_heads, dim, page, block, seed=dim + window, pad_rows=3)
    check_attention(p, heads, dtype, window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [5, 8, 9, 16, 17, 32, 33, 48, 64, 65])
def test_attention_of_any_number_of_rows(heads, dim):
    p = inputs8([700, 200, 2], [1, 1, 1], 1, dim, 16, 16, seed=heads)
    p["v8"].copy_((f32(p["v8"]) * 2.0 ** -14).to(E4M3))   # codes of 2^-9 .. 2^-6: subnormal
    check_attention(p, heads, BF16)


@pytest.mark.parametrize("window", [1, 2, 128, 1000000])
def test_attention_window_of_one_token(window):
    p = inputs8([4097, 130, 1, 128], [1] * 4, 1, 128, 64, 16, seed=window)
    check_attention(p, 64, BF16, window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [3, 2 ** 31 - 1])
def test_attention_window_with_tokens_before_position_0(dtype, window):
    p = inputs8([3, 150, 0], [7, 4, 2], 2, 64, 16, 8, seed=22)   # positions -4 .. 2; 146 ..; -2, -1
    check_attention(p, 8, dtype, window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_missing_pages_and_empty_rows(dtype):
    lengths = [200, 64, 300, 90, 0, 33]
    p = inputs8(lengths, [2, 1, 3, 1, 2, 1], 2, 64, 16, 16, seed=8)
    p["table"][0, 3] = -1
    p["table"][0, 7] = p["k8"].shape[0]
    p["table"][1, :] = -1                    # nothing is there
    p["table"][2, 0] = -2 ** 31
    p["length"][3] = 16 * p["table"].shape[1] + 40   # past the table's end: as long as the table
    p["length"][4] = -5
    check_attention(p, 8, dtype)
    check_attention(p, 8, dtype, window=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["head", "both"])
def test_attention_strides(dtype, layout):
    p = inputs8([700, 33, 257], [1, 4, 2], 2, 64, 16, 8, seed=3, layout=layout)
    q = randn((7, 3, 8, 64), dtype, 9)
    got = attend(p, q[:, 1], out=torch.full_like(q, float("nan"))[:, 2])
    assert torch.equal(got, attend(p, q[:, 1].contiguous()))
    check_attention(p, 8, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_nan_codes(dtype, window):
    """NaN codes in V of keys that some tokens see and others do not, and in K of such a key."""
    p = inputs8([70, 300], [6, 6], 1, 128, 16, 16, seed=12)
    q = randn((12, 16, 128), dtype, 13)
    clean = attend(p, q, window)
    ats = [(0, 67), (1, 297)] + ([(1, 294 - 40 + 3)] if window else [])
    sees = torch.zeros(12, dtype=torch.bool, device="cuda")
    for b, at in ats:
        p["v8"].view(torch.uint8)[int(p["table"][b, at // 16]), at % 16, 0, 7] = NAN_CODE | 0x80
        for i in range(6):
            pos = (64 if b == 0 else 294) + i
            sees[6 * b + i] |= at <= pos and (not window or at > pos - window)
    got = attend(p, q, window)
    assert torch.equal(got[~sees], clean[~sees]) and got[sees][..., 7].isnan().all()
    keep = [d for d in range(128) if d != 7]
    assert torch.equal(got[..., keep], clean[..., keep])
    for b, at in ats:
        p["k8"].view(torch.uint8)[int(p["table"][b, at // 16]), at % 16, 0, 3] = NAN_CODE
    got = attend(p, q, window)
    assert torch.equal(got[~sees], clean[~sees]) and got[sees].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_nan_in_v_of_a_key_without_weight(dtype):
    p = inputs8([9000], [1], 1, 64, 16, 16, seed=19)
    q = randn((1, 4, 64), dtype, 20)
    at = 4321
    pg = int(p["table"][0, at // 16])
    p["ks"][pg] = 2.0 ** 20               # a score of about -1e8 or 1e8
    s = torch.einsum("hd,d->h", q[0].float(), f32(p["k8"][pg, at % 16, 0]))
    p["k8"].view(torch.uint8)[pg, :] = 0
    p["k8"][pg, at % 16, 0] = (-200.0 * q[0, 0].float().sign()).to(E4M3)
    p["v8"].view(torch.uint8)[pg, at % 16, 0, 5] = NAN_CODE
    got = attend(p, q)
    assert float(s.abs().max()) < math.inf and got[0, 0, 5].isnan() and got[0, 0, 6].isfinite()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_queries_that_are_not_finite(dtype):
    p = inputs8([300, 300], [1, 1], 2, 64, 16, 16, seed=25)
    q = randn((2, 8, 64), dtype, 26)
    clean = attend(p, q)
    q[0, 1, 5], q[1, 6, 9] = float("nan"), float("inf")
    got = attend(p, q)
    assert got[0, 1].isnan().all() and got[1, 6].isnan().all()
    same = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    same[0, 1] = same[1, 6] = False
    assert torch.equal(got[same], clean[same])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_large_scores(dtype):
    """Scores of hundreds, growing along the sequence, so that the running maximum moves."""
    p = inputs8([1500, 700], [1, 2], 2, 64, 32, 32, seed=16)
    blocks = torch.arange(47, device="cuda")
    p["ks"][p["table"][0].long()[blocks]] *= torch.exp2(blocks // 8.0)[:, None, None]
    check_attention(p, 8, dtype, q_scale=4.0)
    check_attention(p, 8, dtype, scale=0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_much_that_is_small(dtype, dim):
    """One key with half of the weight, and 40,000 that share the other half (2^-16 of it each)."""
    n = 40000
    p = inputs8([n], [1], 1, dim, 16, 16, seed=33)
    p["k8"].view(torch.uint8)[:] = 0
    pg, slot = int(p["table"][0, 1000 // 16]), 1000 % 16
    p["k8"][pg, slot, 0, :] = torch.ones(dim, device="cuda").to(E4M3)
    p["ks"][:] = math.log(n) / math.sqrt(dim)
    p["v8"].copy_((f32(p["v8"]).nan_to_num(0.0) + 100.0).clamp(-448, 448).to(E4M3))
    q = torch.ones(1, 4, dim, dtype=dtype, device="cuda")
    ref, err, mass = ref_attention(values(p), q)
    close(attend(p, q), ref, bound_of(p, q, ref, err, mass))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_scales_far_apart(dtype):
    """V scales of 2^-60 to 2^60 and K scales of zero (2^-64): the sum is the large ones' but where only small ones
    are in a window."""
    p = inputs8([600, 64], [1, 1], 2, 64, 16, 8, seed=34)
    p["vs"][:] = torch.exp2(torch.randint(-60, 61, p["vs"].shape, generator=torch.Generator().manual_seed(1)).float()).cuda()
    p["ks"][::3] = 2.0 ** -64
    check_attention(p, 8, dtype)
    p["vs"][:] = 2.0 ** -64
    check_attention(p, 8, dtype, window=17)


@pytest.mark.parametrize("dtype,kv_heads,heads,dim", [(BF16, 1, 64, 128), (BF16, 8, 32, 128), (BF16, 2, 64, 64), (F32, 2, 8, 64)])
def test_attention_long_and_ragged(dtype, kv_heads, heads, dim):
    """Items split over many CTAs beside short ones."""
    lengths = [30001, 3, 700, 9000, 128, 12345, 1]
    p = inputs8(lengths, [2, 1, 3, 1, 1, 2, 1], kv_heads, dim, 16, 16, seed=31)
    got = check_attention(p, heads, dtype, seed=32)
    again = attend(p, randn((p["tokens"], heads, dim), dtype, 32))
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_many_sequences(dtype):
    lengths = [(i * 37) % 90 for i in range(700)]
    new = [min(n, 1 + i % 2) for i, n in enumerate(lengths)]
    p = inputs8(lengths, new, 1, 64, 8, 8, seed=41)
    check_attention(p, 4, dtype, seed=42)


def test_attention_of_a_full_prompt_chunk():
    """128 new tokens of a sequence, 64 heads: 128 row tiles."""
    p = inputs8([128, 300, 5], [128, 100, 5], 1, 128, 64, 64, seed=43, pad_rows=2)
    check_attention(p, 64, BF16)
    check_attention(p, 64, BF16, window=50)


def test_attention_offsets_past_32_bits():
    n_pages, page = 33600, 1024
    k = torch.zeros(n_pages, page, 1, 128, dtype=torch.uint8, device="cuda")
    v, ks = torch.zeros_like(k), torch.ones(n_pages, page // 64, 1, device="cuda")
    vs = ks.clone()
    for pg, s in ((33599, 1), (33598, 2), (5, 3)):
        for x, o in ((k, 0), (v, 10)):
            x[pg] = (100 * randn((page, 1, 128), F32, s + o)).clamp(-448, 448).to(E4M3).view(torch.uint8)
    ks[:], vs[:] = 0.01, 0.5
    p = dict(k8=k.view(E4M3), v8=v.view(E4M3), ks=ks, vs=vs, page=page, block=64, tokens=1,
             table=torch.tensor([[33599, 5, 33598]], dtype=torch.int32).cuda(),
             length=torch.tensor([2500], dtype=torch.int32).cuda(), start=torch.tensor([0, 1], dtype=torch.int32).cuda())
    few = dict(p, k8=k[[5, 33598, 33599]].view(E4M3), v8=v[[5, 33598, 33599]].view(E4M3), ks=ks[:3], vs=vs[:3],
               table=torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda())
    for dtype in (BF16, F32):
        q = randn((1, 8, 128), dtype, 7)
        ref, err, mass = ref_attention(values(few), q)
        close(attend(p, q), ref, bound_of(few, q, ref, err, mass))
    x, y = randn((1, 1, 128), BF16, 50), randn((1, 1, 128), BF16, 51)
    p["length"][0] = 2049   # the first slot of a block
    pdl.paged_append(cache(p), pdl.PagedBatch(p["table"], p["length"]), x, y)
    for c, s, z in ((k, ks, x), (v, vs, y)):
        got = f32(c[33598, 0].view(E4M3)) * s[33598, 0][:, None]
        assert float((got - z[0].float()).abs().max()) <= 2.0 ** -4 * float(z.float().abs().max())


# ------------------------------------------------------------------ append

def append8(p, heads, dim, rot, dtype, seed=5, n_pos=None, fused=False, scale=1.0):
    n, kvh = p["tokens"], p["k8"].shape[2]
    if fused:
        buf = randn((n, (heads + 2 * kvh) * dim + 16), dtype, seed)
        q = buf[:, :heads * dim].unflatten(1, (heads, dim))
        k = buf[:, heads * dim:(heads + kvh) * dim].unflatten(1, (kvh, dim))
        v = buf[:, (heads + kvh) * dim:(heads + 2 * kvh) * dim].unflatten(1, (kvh, dim))
    else:
        q = randn((n, heads, dim), dtype, seed) if heads else None
        k, v = randn((n, kvh, dim), dtype, seed + 1, scale), randn((n, kvh, dim), dtype, seed + 2, scale)
    rope = pdl.Rope.fill(n_pos or max(1, int(p["length"].max())), rot) if rot else None
    before = {x: p[x].clone() for x in ("k8", "v8", "ks", "vs")}
    batch = pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=10 ** 6)
    out = torch.full((n, heads, dim), float("nan"), dtype=dtype, device="cuda") if heads else None
    pdl.paged_append(cache(p), batch, k, v, rope, q=q, q_out=out)
    torch.cuda.synchronize()
    check_append8(p, before, k, v, rope.cs if rope else None, rot)
    if heads:   # as the append into a cache without scales turns them
        plain = torch.zeros(p["k8"].shape, dtype=dtype, device="cuda")
        other = torch.full_like(out, float("nan"))
        pdl.paged_append(pdl.PagedKV(plain, plain.clone()), batch, k, v, rope, q=q, q_out=other)
        assert torch.equal(out.nan_to_num(7.0), other.nan_to_num(7.0))
    return k, v


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv_heads,heads,dim,rot,page,block", [
    (1, 64, 128, 128, 64, 64), (8, 32, 128, 64, 16, 16), (2, 8, 64, 64, 48, 24), (3, 0, 48, 24, 7, 7), (1, 5, 256, 30, 1, 1),
    (4, 4, 16, 0, 5, 5), (2, 2, 128, 128, 256, 256), (5, 3, 64, 32, 32, 2)])
def test_append(dtype, kv_heads, heads, dim, rot, page, block):
    p = inputs8([1, 130, 17, 64, 0, 300], [1, 7, 17, 0, 0, 33], kv_heads, dim, page, block, seed=dim + page)
    append8(p, heads, dim, rot, dtype)


@pytest.mark.parametrize("scale", [1e-3, 30.0, 1e-30, 1e30])
def test_append_rounds_the_block_again(scale):
    """Scales that grow, and ones that stay, over four appends to the same blocks."""
    lengths = [5, 20, 33]
    p = inputs8(lengths, [5, 5, 5], 2, 64, 16, 16, seed=71, width_extra=2)
    for b in range(3):
        p["table"][b] = torch.arange(b * p["table"].shape[1], (b + 1) * p["table"].shape[1])
    n = 3 * p["table"].shape[1]
    for x in ("k8", "v8"):
        p[x] = torch.zeros(n, 16, 2, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    for x in ("ks", "vs"):
        p[x] = torch.full((n, 1, 2), 2.0 ** -64, device="cuda")
    for step in range(4):
        append8(p, 0, 64, 64, BF16, seed=80 + step, scale=scale ** (step / 2))
        p["length"] += 5


@pytest.mark.parametrize("layout", ["head", "both"])
def test_append_strides(layout):
    p = inputs8([100, 33, 257], [3, 33, 1], 2, 64, 16, 8, seed=3, layout=layout)
    append8(p, 6, 64, 64, BF16, fused=True)


def test_append_leaves_out_missing_pages_positions_and_rows():
    p = inputs8([40, 20, 9, 3, 50], [40, 8, 2, 5, 20], 1, 64, 8, 4, seed=9, pad_rows=6)
    p["table"][0, 1] = -1
    p["table"][0, 3] = p["k8"].shape[0]
    p["table"][1, 2] = 2 ** 31 - 1
    p["length"][3] = 3                      # five new tokens at positions -2 .. 2
    p["length"][4] = 8 * p["table"].shape[1] + 11   # past the table's end
    append8(p, 3, 64, 64, BF16, n_pos=35)   # and positions without an angle


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_values_that_are_not_finite(dtype):
    """They count for no scale; zeros have the least one."""
    p = inputs8([20, 16], [20, 16], 2, 64, 16, 16, seed=15)
    k, v = randn((36, 2, 64), dtype, 1), randn((36, 2, 64), dtype, 2)
    k[3, 0, 5], k[4, 1, 6], v[30, 1, 7] = float("nan"), float("inf"), float("-inf")
    v[20:, 0] = 0.0
    k[0, 0, 0] = 3e38
    before = {x: p[x].clone() for x in ("k8", "v8", "ks", "vs")}
    pdl.paged_append(cache(p), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=20), k, v)
    check_append8(p, before, k, v, None, 0)
    assert float(p["vs"][int(p["table"][1, 0]), 0, 0]) == 2.0 ** -64


@pytest.mark.parametrize("page,block", [(64, 64), (16, 16)])
def test_append_many_tokens(page, block):
    lengths = [1500 + 611 * i for i in range(6)]
    p = inputs8(lengths, [n - 7 * i for i, n in enumerate(lengths)], 1, 16, page, block, seed=21)
    append8(p, 1, 16, 16, F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_keeps_a_callers_scale(dtype):
    """A scale that is no power of two stays while it is large enough, and codes are rounded from x / s."""
    p = inputs8([30], [1], 1, 64, 32, 32, seed=16)
    pg = int(p["table"][0, 0])
    p["ks"][pg], p["vs"][pg] = 0.3, 0.7
    k, v = randn((1, 1, 64), dtype, 1), randn((1, 1, 64), dtype, 2)
    before = {x: p[x].clone() for x in ("k8", "v8")}
    pdl.paged_append(cache(p), pdl.PagedBatch(p["table"], p["length"]), k, v)
    for c, s, x, was in (("k8", 0.3, k, before["k8"]), ("v8", 0.7, v, before["v8"])):
        want = (x[0, 0].float() / torch.tensor(s, device="cuda")).to(E4M3)
        assert torch.equal(f32(p[c][pg, 29, 0]), want.float())
        assert torch.equal(p[c].view(torch.uint8)[pg, :29], was.view(torch.uint8)[pg, :29])


# ------------------------------------------------------------------ as they are used

@pytest.mark.parametrize("heads,kv_heads,dim", [(64, 1, 128), (8, 2, 64)])
def test_append_and_attention_in_a_graph(heads, kv_heads, dim):
    p = inputs8([900, 40, 333], [1, 2, 1], kv_heads, dim, 16, 16, seed=51, width_extra=4)
    q, k, v = randn((4, heads, dim), BF16, 52), randn((4, kv_heads, dim), BF16, 53), randn((4, kv_heads, dim), BF16, 54)
    kv, batch = cache(p), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=2)
    rope = pdl.Rope.fill(2000, dim)
    ws = torch.empty(pdl.paged_attention_workspace_bytes(kv, batch, heads), dtype=torch.uint8, device="cuda")
    out, turned = torch.empty_like(q), torch.empty_like(q)

    def step():
        pdl.paged_append(kv, batch, k, v, rope, q, turned)
        pdl.paged_attention(kv, batch, turned, out, ws)
    names = ("k8", "v8", "ks", "vs")
    saved = {x: p[x].clone() for x in names}

    def restore():
        for x in names:
            p[x].view(torch.uint8).copy_(saved[x].view(torch.uint8))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for shorter in (0, 35, 5):
        restore()
        p["length"].copy_(torch.tensor([900 - shorter, 40, 333 - 2 * shorter], dtype=torch.int32))
        q.copy_(randn((4, heads, dim), BF16, 60 + shorter))
        g.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        restore()
        step()
        assert torch.equal(replayed, out)
        check_append8(p, saved, k, v, rope.cs, dim)
        ref, err, mass = ref_attention(values(p), turned)
        close(replayed, ref, bound_of(p, turned, ref, err, mass))


def test_attention_on_two_streams_with_their_own_workspaces():
    ps = [inputs8([20000, 3000, 50], [1, 1, 1], 1, 128, 64, 64, seed=61 + i) for i in range(2)]
    qs = [randn((3, 64, 128), BF16, 63 + i) for i in range(2)]
    want = [attend(p, q) for p, q in zip(ps, qs)]
    kvs, bs = [cache(p) for p in ps], [pdl.PagedBatch(p["table"], p["length"]) for p in ps]
    wss = [torch.empty(pdl.paged_attention_workspace_bytes(kv, b, 64), dtype=torch.uint8, device="cuda")
           for kv, b in zip(kvs, bs)]
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            pdl.paged_attention(kvs[i], bs[i], qs[i], outs[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("seqs", ["few", "many"])
def test_append_finds_every_token_among_empty_sequences(seqs):
    """Long runs of sequences without a new token beside short and long ones: as a call for each sequence."""
    new = {"few": [0] * 9 + [900, 0, 1, 1, 0, 33, 5] + [0] * 11 + [2500, 2],
           "many": [0] * 60 + [900] + [0] * 45 + [1] * 100 + [7] * 33 + [0, 1] * 40 + [0] * 70 + [3000, 0, 2] + [0] * 35}[seqs]
    p = inputs8([n + 5 * i % 90 for i, n in enumerate(new)], new, 32, 16, 32, 32, seed=91)
    k, v = randn((p["tokens"], 32, 16), BF16, 92), randn((p["tokens"], 32, 16), BF16, 93)
    rope = pdl.Rope.fill(4000, 16)
    names = ("k8", "v8", "ks", "vs")
    one = {x: p[x].clone() for x in names}
    pdl.paged_append(cache(p), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=4000), k, v, rope)
    at, kv = 0, pdl.PagedKV8(*(one[x] for x in names))
    for b, n in enumerate(new):
        if n:
            start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            pdl.paged_append(kv, pdl.PagedBatch(p["table"][b:b + 1], p["length"][b:b + 1], start, max_new=4000),
                             k[at:at + n], v[at:at + n], rope)
        at += n
    for x in names:
        bits = [t.view(torch.uint8) if x in ("k8", "v8") else t.view(torch.int32) for t in (p[x], one[x])]
        assert torch.equal(*bits), x


def test_operators_on_two_streams_at_once():
    """Appends, page tables and edits have no memory in common."""
    ps = [inputs8([300, 64, 1000, 17], [4, 64, 1, 17], 2, 64, 16, 16, seed=95 + i, width_extra=2) for i in range(2)]
    ks, vs = [randn((86, 2, 64), BF16, 97 + i) for i in range(2)], [randn((86, 2, 64), BF16, 99 + i) for i in range(2)]
    zs = [randn((40, 30000), F32, 101 + i) for i in range(2)]
    edits = [pdl.LogitEdits(history=torch.randint(0, 30000, (40, 3000), generator=torch.Generator().manual_seed(i)).int().cuda(),
                            frequency=torch.full((40,), 0.5, device="cuda")) for i in range(2)]
    names, n_pages = ("k8", "v8", "ks", "vs"), 64
    want_len = torch.tensor([400, 7, 0, 33], dtype=torch.int32, device="cuda")

    def state():
        return [dict({x: p[x].clone() for x in names}, out=torch.zeros_like(z), slots=torch.zeros(600, dtype=torch.int64, device="cuda"),
                     pool=pdl.PagePool(torch.arange(n_pages, dtype=torch.int32, device="cuda"), torch.full((1,), n_pages, dtype=torch.int32, device="cuda"), 16),
                     batch=pdl.PagedBatch(torch.full((4, 30), -1, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"),
                                          torch.zeros(5, dtype=torch.int32, device="cuda"))) for p, z in zip(ps, zs)]

    def work(i, s, stream=None):
        for _ in range(5):
            pdl.paged_append(pdl.PagedKV8(*(s[x] for x in names)), pdl.PagedBatch(ps[i]["table"], ps[i]["length"], ps[i]["start"], max_new=64),
                             ks[i], vs[i], stream=stream)
            pdl.edit_logits(zs[i], s["out"], edits[i], stream=stream)
            pdl.paged_resize(s["pool"], s["batch"], want_len, s["slots"], stream=stream)
    alone = state()
    for i in range(2):
        work(i, alone[i])
        torch.cuda.synchronize()
    both, streams = state(), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        work(i, both[i], streams[i])
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for x in names:
            assert torch.equal(a[x].contiguous().view(torch.uint8), b[x].contiguous().view(torch.uint8))
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["slots"], b["slots"])
        assert torch.equal(a["batch"].table, b["batch"].table) and torch.equal(a["pool"].free, b["pool"].free)
