"""Paged K/V cache operators (ds4g_paged_append, ds4g_paged_attention) against their 64-bit
forms: types, head layouts, page sizes, strides, ragged and empty sequences, windows,
missing pages, NaN in every place that is masked, captured graphs, and a session's own
cache read as pages."""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
import synth
from helpers import gpu_model
from paged_ref import HALF, fill_slots, paged_inputs, randn, ref_append, ref_attention

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def close(got, ref, bound):
    """Every element within `bound` of ref, NaN exactly where ref has one."""
    got = got.double()
    assert torch.equal(got.isnan(), ref.isnan())
    bad = ~((got - ref).abs() <= bound) & ~ref.isnan()
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()))


# ------------------------------------------------------------------ append

def check_append(p, kv_heads, heads, dim, rot, dtype, n_pos=None, seed=5, pad=0, fused=False, inplace=False):
    n, cache = p["tokens"], p["k"].dtype
    per = (heads + 2 * kv_heads) * dim
    if fused:   # rows of one projection: queries, keys, values
        buf = randn((n, per + 16), dtype, seed)
        q = buf[:, :heads * dim].unflatten(1, (heads, dim))
        k = buf[:, heads * dim:(heads + kv_heads) * dim].unflatten(1, (kv_heads, dim))
        v = buf[:, (heads + kv_heads) * dim:per].unflatten(1, (kv_heads, dim))
    else:
        q = randn((n, heads, dim), dtype, seed) if heads else None
        k, v = randn((n, kv_heads, dim), dtype, seed + 1), randn((n, kv_heads, dim), dtype, seed + 2)
    longest = int(p["length"].max())
    rope = pdl.Rope.fill(n_pos or max(1, longest), rot) if rot else None
    kc, vc, qo, mag_k, mag_q = ref_append(p, k, v, q if heads else None, rope.cs if rope else None, rot)
    out = (q if inplace else torch.full((n, heads, dim), float("nan"), dtype=dtype, device="cuda")) if heads else None
    if inplace:
        qo = torch.where(qo.isnan(), q.double(), qo)
    pdl.paged_append(pdl.PagedKV(p["k"], p["v"]), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=10 ** 6),
                     k, v, rope, q=q if heads else None, q_out=out)
    torch.cuda.synchronize()
    # two products and a sum in FP32 (three roundings at most of the magnitudes), then one
    # rounding to the stored type
    close(p["k"], kc, 3 * 2.0 ** -24 * mag_k + HALF[cache] * (kc.abs() + 3 * 2.0 ** -24 * mag_k))
    close(p["v"], vc, HALF[cache] * vc.abs() if cache != dtype else 0 * vc)
    if heads:
        close(out, qo, 3 * 2.0 ** -24 * mag_q + HALF[dtype] * (qo.abs() + 3 * 2.0 ** -24 * mag_q))


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("kv_heads,heads,dim,rot,page", [(1, 64, 128, 128, 64), (8, 32, 128, 64, 16), (2, 8, 64, 64, 48),
                                                         (3, 0, 40, 24, 7), (1, 5, 256, 30, 1), (4, 4, 8, 0, 5)])
def test_append(dtype, cache, kv_heads, heads, dim, rot, page):
    lengths, new = [1, 130, 17, 64, 0, 300], [1, 7, 17, 0, 0, 33]
    p = paged_inputs(lengths, new, kv_heads, dim, page, cache, seed=dim + page)
    check_append(p, kv_heads, heads, dim, rot, dtype)


@pytest.mark.parametrize("layout", ["head", "both"])
def test_append_strides_and_in_place_queries(layout):
    p = paged_inputs([100, 33, 257], [3, 33, 1], 2, 64, 16, BF16, seed=3, layout=layout)
    check_append(p, 2, 6, 64, 64, BF16, fused=True)
    p = paged_inputs([100, 33, 257], [3, 33, 1], 2, 64, 16, BF16, seed=4, layout=layout)
    check_append(p, 2, 6, 64, 32, BF16, fused=True, inplace=True)


def test_append_leaves_out_missing_pages_positions_and_rows():
    p = paged_inputs([40, 20, 9, 3, 50], [40, 8, 2, 5, 20], 1, 64, 8, BF16, seed=9, pad_rows=6)
    p["table"][0, 1] = -1
    p["table"][0, 3] = p["k"].shape[0]      # one past the last page
    p["table"][1, 2] = 2 ** 31 - 1
    p["length"][3] = 3                      # five new tokens at positions -2 .. 2
    p["length"][4] = 8 * p["table"].shape[1] + 11   # past the table's end
    check_append(p, 1, 3, 64, 64, BF16, n_pos=35)   # and positions without an angle


def test_append_one_token_each_without_starts():
    p = paged_inputs([5, 1, 128, 64], [1] * 4, 2, 128, 32, BF16, seed=11)
    k, v, q = (randn((4, h, 128), BF16, s) for h, s in ((2, 1), (2, 2), (4, 3)))
    rope = pdl.Rope.fill(128, 128)
    a, out_a, out_b = {x: p[x].clone() for x in "kv"}, torch.empty_like(q), torch.empty_like(q)
    pdl.paged_append(pdl.PagedKV(p["k"], p["v"]), pdl.PagedBatch(p["table"], p["length"]), k, v, rope, q, out_a)
    pdl.paged_append(pdl.PagedKV(a["k"], a["v"]), pdl.PagedBatch(p["table"], p["length"], p["start"]), k, v, rope, q,
                     out_b)
    assert torch.equal(out_a, out_b)
    for x in "kv":
        assert torch.equal(p[x].nan_to_num(9.0), a[x].nan_to_num(9.0))


def test_append_many_tokens():
    """Enough tokens for several of them per CTA."""
    lengths = [1500 + 611 * i for i in range(12)]
    new = [n - 7 * i for i, n in enumerate(lengths)]
    p = paged_inputs(lengths, new, 1, 16, 64, BF16, seed=21)
    n = p["tokens"]
    k, v = randn((n, 1, 16), F32, 1), randn((n, 1, 16), F32, 2)
    pdl.paged_append(pdl.PagedKV(p["k"], p["v"]), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=n), k, v)
    start, table = p["start"].tolist(), p["table"].long()
    for b, (length, m) in enumerate(zip(lengths, new)):
        pos = torch.arange(length - m, length, device="cuda")
        for cache, x in ((p["k"], k), (p["v"], v)):
            assert torch.equal(cache[table[b][pos // 64], pos % 64], x[start[b]:start[b + 1]].bfloat16())


@pytest.mark.parametrize("seqs", [256, 257, 700, 9000])
def test_append_finds_the_sequence_among_many(seqs):
    new = [(i * 7919) % 5 for i in range(seqs)]   # 0 .. 4 tokens; some sequences have none
    new[0], new[-1] = 0, 0
    lengths = [n + i % 3 for i, n in enumerate(new)]
    p = paged_inputs(lengths, new, 1, 8, 8, F32, seed=13, pad_rows=3)
    n, owner = p["tokens"] - 3, torch.repeat_interleave(torch.arange(seqs), torch.tensor(new))
    first = torch.tensor([0] + new[:-1]).cumsum(0)
    at = torch.tensor(lengths)[owner] - torch.tensor(new)[owner] + torch.arange(n) - first[owner]
    k = torch.arange(n + 3, dtype=F32, device="cuda")[:, None, None].expand(-1, 1, 8).contiguous()
    want = p["k"].clone()
    want[p["table"].cpu()[owner, 0].long(), at] = k[:n]
    pdl.paged_append(pdl.PagedKV(p["k"], p["v"]), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=4), k, k)
    assert torch.equal(p["k"].nan_to_num(-1.0), want.nan_to_num(-1.0))
    assert torch.equal(p["v"].nan_to_num(-1.0), want.nan_to_num(-1.0))


def test_rope_table_matches_the_formula():
    t = pdl.Rope.fill(70000, 64, base=10000.0)
    pos = torch.arange(70000, dtype=torch.float64, device="cuda")[:, None]
    ang = pos * 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64, device="cuda") / 64)
    # FP64 angles (one rounding of up to 7e4, 2^-53 of it, and pow's) stored as FP32
    for i, f in ((0, torch.cos), (1, torch.sin)):
        assert float((t.cs[:, :, i].double() - f(ang)).abs().max()) <= 2.0 ** -24 + 7e4 * 2.0 ** -50


# ------------------------------------------------------------------ attention

def attend(p, q, window=0, scale=0.0, start=True, max_new=None, out=None, ws=None):
    kv = pdl.PagedKV(p["k"], p["v"])
    new = (p["start"][1:] - p["start"][:-1]).max()
    batch = pdl.PagedBatch(p["table"], p["length"], p["start"] if start else None, max_new=max_new or max(1, int(new)))
    out = torch.full_like(q, float("nan")) if out is None else out
    if ws is None:
        ws = torch.full((pdl.paged_attention_workspace_bytes(kv, batch, q.shape[1]),), 255, dtype=torch.uint8,
                        device="cuda")
    pdl.paged_attention(kv, batch, q, out, ws, scale=scale, window=window)
    assert pdl.paged_attention_status(ws) == 0
    return out


def check_attention(p, heads, dtype, window=0, scale=None, seed=1, q_scale=1.0):
    q = randn((p["tokens"], heads, p["k"].shape[3]), dtype, seed, q_scale)
    ref, err, mass = ref_attention(p, q, window, scale)
    got = attend(p, q, window, scale or 0.0)
    n = int(p["start"][-1])
    assert got[n:].isnan().all()          # rows behind the last sequence
    got, ref, err, mass = got[:n], ref[:n], err[:n], mass[:n]
    # BF16 throughout: the weights are rounded to BF16 as well
    p_round = HALF[BF16] if dtype == BF16 and p["k"].dtype == BF16 else 0.0
    before = err + p_round * mass
    close(got, ref, before + HALF[dtype] * (ref.abs() + before))
    empty = mass.sum(-1) == 0
    assert (got[empty] == 0).all()
    return got


LENGTHS = [1, 127, 128, 129, 5, 640, 0, 64, 255, 1000]


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("kv_heads,heads,dim,page", [(1, 64, 128, 64), (8, 32, 128, 16), (2, 8, 64, 48), (4, 4, 64, 8),
                                                     (1, 128, 128, 128), (3, 15, 128, 24), (1, 8, 32, 16),
                                                     (2, 6, 40, 7), (1, 3, 256, 1), (2, 10, 96, 32), (2, 16, 128, 256),
                                                     (2, 8, 64, 192)])
def test_attention_one_token(dtype, cache, kv_heads, heads, dim, page):
    p = paged_inputs(LENGTHS, [1] * len(LENGTHS), kv_heads, dim, page, cache, seed=dim + heads)
    fill_slots(p, seed=2)
    check_attention(p, heads, dtype)


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("kv_heads,heads,dim,page,window", [(1, 64, 128, 64, 0), (1, 64, 128, 64, 100), (8, 32, 128, 16, 0),
                                                            (2, 14, 64, 40, 33), (1, 100, 128, 16, 129), (1, 8, 32, 16, 16)])
def test_attention_several_tokens_and_windows(dtype, cache, kv_heads, heads, dim, page, window):
    new = [1, 5, 3, 8, 5, 2, 0, 7, 1, 4]
    p = paged_inputs(LENGTHS, new, kv_heads, dim, page, cache, seed=dim + window, pad_rows=3)
    fill_slots(p, seed=3)
    check_attention(p, heads, dtype, window)


@pytest.mark.parametrize("window", [1, 2, 128, 1000000])
def test_attention_window_of_one_token(window):
    p = paged_inputs([4097, 130, 1, 128], [1] * 4, 1, 128, 64, BF16, seed=window)
    fill_slots(p, seed=5)
    check_attention(p, 64, BF16, window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [3, 2 ** 31 - 1])
def test_attention_window_with_tokens_before_position_0(dtype, window):
    p = paged_inputs([3, 150, 0], [7, 4, 2], 2, 64, 16, dtype, seed=22)   # positions -4 .. 2; 146 ..; -2, -1
    fill_slots(p, 23)
    check_attention(p, 8, dtype, window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_missing_pages_and_empty_rows(dtype):
    lengths = [200, 64, 300, 90, 0, 33]
    p = paged_inputs(lengths, [2, 1, 3, 1, 2, 1], 2, 64, 16, dtype, seed=8)
    fill_slots(p, seed=6)
    p["table"][0, 3] = -1
    p["table"][0, 7] = p["k"].shape[0]
    p["table"][1, :] = -1                    # nothing is there
    p["table"][2, 0] = -2 ** 31
    p["length"][3] = 16 * p["table"].shape[1] + 40   # past the table's end: as long as the table
    p["length"][4] = -5
    check_attention(p, 8, dtype)
    check_attention(p, 8, dtype, window=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["head", "both"])
def test_attention_strides(dtype, layout):
    p = paged_inputs([700, 33, 257], [1, 4, 2], 2, 64, 16, dtype, seed=3, layout=layout)
    fill_slots(p, seed=4)
    q = randn((7, 3, 8, 64), dtype, 9)
    got = attend(p, q[:, 1], out=torch.full_like(q, float("nan"))[:, 2])
    assert torch.equal(got, attend(p, q[:, 1].contiguous()))
    check_attention(p, 8, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_nan_and_inf_in_keys_only_later_tokens_see(dtype):
    """A key that is masked for some of the call's tokens and not for others, with K and V
    that are not finite: the tokens before it keep their values."""
    p = paged_inputs([70, 200], [6, 6], 1, 64, 16, dtype, seed=12)
    fill_slots(p, seed=12)
    q = randn((12, 4, 64), dtype, 13)
    clean = attend(p, q)
    for b, at in ((0, 67), (1, 197)):
        page, slot = int(p["table"][b, at // 16]), at % 16
        p["k"][page, slot, 0, 3] = float("inf")
        p["v"][page, slot, 0, 5] = float("nan")
        p["v"][page, slot, 0, 9] = float("inf")
    got = attend(p, q)
    rows = torch.tensor([0, 1, 2, 6, 7, 8], device="cuda")
    assert torch.equal(got[rows], clean[rows])
    assert not got[3:6].isfinite().all() and not got[9:].isfinite().all()
    # V alone: weights stay finite, so the places of the row say what was there
    for b, at in ((0, 67), (1, 197)):
        p["k"][int(p["table"][b, at // 16]), at % 16, 0, 3] = 0.5
    got = attend(p, q)
    seen = torch.tensor([3, 4, 5, 9, 10, 11], device="cuda")
    assert torch.equal(got[rows], clean[rows])
    assert got[seen][..., 5].isnan().all() and (got[seen][..., 9] == float("inf")).all()
    keep = [d for d in range(64) if d not in (5, 9)]
    assert got[seen][..., keep].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_window_edge_holds_nan(dtype):
    """Keys that left the window of the later tokens only."""
    p = paged_inputs([300], [4], 1, 128, 16, dtype, seed=14)
    fill_slots(p, seed=14)
    q = randn((4, 16, 128), dtype, 15)
    clean = attend(p, q, window=40)
    at = 296 - 40 + 1 + 1          # seen by tokens 0 and 1 (positions 296, 297), not by 2 and 3
    p["v"][int(p["table"][0, at // 16]), at % 16, 0, 7] = float("nan")
    got = attend(p, q, window=40)
    assert got[:2, :, 7].isnan().all() and torch.equal(got[2:], clean[2:])
    keep = [d for d in range(128) if d != 7]
    assert torch.equal(got[:2][..., keep], clean[:2][..., keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_large_scores(dtype):
    """Scores of hundreds, growing along the sequence, so that the running maximum moves."""
    p = paged_inputs([1500, 700], [1, 2], 2, 64, 32, dtype, seed=16)
    fill_slots(p, seed=16)
    pos = torch.arange(1500, device="cuda")
    pages = p["table"][0].long()[pos // 32]
    p["k"][pages, pos % 32] = (p["k"][pages, pos % 32].float() * (0.2 + pos / 100.0)[:, None, None]).to(dtype)
    check_attention(p, 8, dtype, q_scale=4.0)
    check_attention(p, 8, dtype, scale=0.5)


@pytest.mark.parametrize("dtype,kv_heads,heads,dim", [(BF16, 1, 64, 128), (BF16, 8, 32, 128), (F32, 2, 8, 64)])
def test_attention_long_and_ragged(dtype, kv_heads, heads, dim):
    """Items split over many CTAs beside short ones."""
    lengths = [30001, 3, 700, 9000, 128, 12345, 1]
    p = paged_inputs(lengths, [2, 1, 3, 1, 1, 2, 1], kv_heads, dim, 16, dtype, seed=31)
    fill_slots(p, seed=31)
    got = check_attention(p, heads, dtype, seed=32)
    again = attend(p, randn((p["tokens"], heads, dim), dtype, 32))
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_many_sequences(dtype):
    """More sequences than threads of a CTA, most of them short."""
    lengths = [(i * 37) % 90 for i in range(700)]
    new = [min(n, 1 + i % 2) for i, n in enumerate(lengths)]
    p = paged_inputs(lengths, new, 1, 64, 8, dtype, seed=41)
    fill_slots(p, seed=41)
    check_attention(p, 4, dtype, seed=42)


def test_attention_offsets_past_32_bits():
    """A cache whose last pages start beyond 2^32 elements."""
    n_pages, page = 33000, 1024
    k = torch.zeros(n_pages, page, 1, 128, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    for pg, s in ((32999, 1), (32998, 2), (5, 3)):
        k[pg], v[pg] = randn((page, 1, 128), BF16, s), randn((page, 1, 128), BF16, s + 10)
    p = dict(k=k, v=v, table=torch.tensor([[32999, 5, 32998]], dtype=torch.int32).cuda(), page=page, tokens=1,
             length=torch.tensor([2500], dtype=torch.int32).cuda(), start=torch.tensor([0, 1], dtype=torch.int32).cuda())
    check_attention(p, 8, BF16)
    new_k, new_v = randn((1, 1, 128), BF16, 50), randn((1, 1, 128), BF16, 51)
    pdl.paged_append(pdl.PagedKV(k, v), pdl.PagedBatch(p["table"], p["length"]), new_k, new_v)
    assert torch.equal(k[32998, 2499 % page], new_k[0]) and torch.equal(v[32998, 2499 % page], new_v[0])
    check_attention(p, 8, F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_in_a_graph_follows_lengths_and_pages(dtype):
    p = paged_inputs([900, 40, 333], [1, 2, 1], 2, 64, 16, dtype, seed=51, width_extra=4)
    fill_slots(p, seed=51)
    q = randn((4, 8, 64), dtype, 52)
    kv, batch = pdl.PagedKV(p["k"], p["v"]), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=2)
    rope = pdl.Rope.fill(2000, 64)
    k, v = randn((4, 2, 64), dtype, 53), randn((4, 2, 64), dtype, 54)
    ws = torch.empty(pdl.paged_attention_workspace_bytes(kv, batch, 8), dtype=torch.uint8, device="cuda")
    out, turned = torch.empty_like(q), torch.empty_like(q)

    def step():
        pdl.paged_append(kv, batch, k, v, rope, q, turned)
        pdl.paged_attention(kv, batch, turned, out, ws)
    saved = p["k"].clone(), p["v"].clone()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for shorter in (0, 35, 5):
        p["k"].copy_(saved[0])
        p["v"].copy_(saved[1])
        p["length"].copy_(torch.tensor([900 - shorter, 40, 333 - 2 * shorter], dtype=torch.int32))
        q.copy_(randn((4, 8, 64), dtype, 60 + shorter))
        g.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        p["k"].copy_(saved[0])
        p["v"].copy_(saved[1])
        step()
        assert torch.equal(replayed, out)
        ref, err, mass = ref_attention(p, turned)
        before = err + (HALF[BF16] if dtype == BF16 else 0.0) * mass
        close(replayed, ref, before + HALF[dtype] * (ref.abs() + before))


def test_attention_on_two_streams_with_their_own_workspaces():
    ps = [paged_inputs([20000, 3000, 50], [1, 1, 1], 1, 128, 64, BF16, seed=61 + i) for i in range(2)]
    qs = [randn((3, 64, 128), BF16, 63 + i) for i in range(2)]
    for i, p in enumerate(ps):
        fill_slots(p, seed=65 + i)
    want = [attend(p, q) for p, q in zip(ps, qs)]
    torch.cuda.synchronize()
    kvs = [pdl.PagedKV(p["k"], p["v"]) for p in ps]
    bs = [pdl.PagedBatch(p["table"], p["length"]) for p in ps]
    wss = [torch.empty(pdl.paged_attention_workspace_bytes(kv, b, 64), dtype=torch.uint8, device="cuda")
           for kv, b in zip(kvs, bs)]
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            pdl.paged_attention(kvs[i], bs[i], qs[i], outs[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_sessions_cache_read_as_pages():
    """The session's own attention of its last decoded token, from its K/V rows as pages
    of 16 that follow one another."""
    shape = synth.LAYER.with_(name="paged_session", n_layers=1, hidden=512, n_heads=8, head_dim=128, q_rank=256,
                              kv_rank=128, window=100, n_experts=128, top_k=4, expert_inter=128, vocab=1000)
    sess = pdl.Session(gpu_model(shape), 256)
    assert sess.prefill(synth.host_tokens(180, shape.vocab, stream=91)) == 0
    assert sess.decode_layers(int(synth.host_tokens(1, shape.vocab, stream=92)[0])) == 0
    k, v = sess.kv(0)
    q, attn = (sess.debug(n, 1024).view(1, 8, 128) for n in ("q", "attn"))
    kv = pdl.PagedKV(k.view(16, 16, 1, 128), v.view(16, 16, 1, 128))
    batch = pdl.PagedBatch(torch.arange(16, dtype=torch.int32, device="cuda")[None],
                           torch.tensor([sess.len], dtype=torch.int32, device="cuda"))
    ws = torch.empty(pdl.paged_attention_workspace_bytes(kv, batch, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty(1, 8, 128, device="cuda")
    pdl.paged_attention(kv, batch, q.clone(), out, ws, window=100)
    # both in FP32 from the same BF16 rows: sums of 128 products, then of 100 keys
    scale = float(attn.abs().max())
    assert float((out - attn).abs().max()) <= 1e-5 * scale
