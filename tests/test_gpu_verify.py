"""Rows of probabilities (ds4g_probs) and draft verification (ds4g_verify_draft) against their
64-bit and integer forms, and the run in which they meet the paged cache: drafts appended,
attended, scored and verified."""
import numpy as np
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged_ref import paged_inputs, randn, ref_attention, ref_probs, ref_verify

pytestmark = pytest.mark.gpu

VOCABS = [1, 3, 100, 1000, 4095, 4097, 8193, 50257, 129280, 131073, 262141, 262145]


# ------------------------------------------------------------------ probabilities

def check_probs(z, t, out=None):
    want = ref_probs(z, t)
    out = torch.full_like(z, float("nan")) if out is None else out
    pdl.probs(z, t, out)
    got = out.double().cpu().numpy()
    # exp2f within 2 ulp, six roundings around it, a sum of at most 100 in a row, and the
    # quotient: 120 half steps; values below the smallest normal number are absolute
    assert np.all(np.abs(got - want) <= 120 * 2.0 ** -24 * want + 2.0 ** -126), np.max(np.abs(got - want))
    return out


@pytest.mark.parametrize("n", VOCABS)
@pytest.mark.parametrize("t", [0.0, -1.0, 0.3, 1.0, 5.0])
def test_probs(n, t):
    check_probs(randn((3, n), torch.float32, n, 3.0), t)


def test_probs_extremes():
    z = randn((9, 5000), torch.float32, 5, 2.0)
    z[0, 100:4900] = float("-inf")
    z[1] = float("-inf")
    z[2, 17] = float("inf")
    z[3, 17] = z[3, 4000] = float("inf")
    z[4, ::2] = float("nan")
    z[5] = float("nan")
    z[6] = 3e38
    z[6, ::3] = -3e38
    z[7] = 0.0
    z[7, 1::2] = -0.0
    z[8, :] = torch.finfo(torch.float32).min
    for t in (0.0, 1.0, 1e-6, 1e-38, 1e30):
        check_probs(z, t)


def test_probs_strides_and_in_place():
    buf = randn((5, 40003), torch.float32, 6, 2.0)
    check_probs(buf[:, 1:30000], 0.8)           # rows and results at different places of a 16-byte line
    check_probs(buf[:, 1:30000].contiguous(), 0.8)
    for at in (1, 2, 3):                        # at the same one
        check_probs(buf[:, at:at + 30000], 0.8, out=torch.full_like(buf, float("nan"))[:, at:at + 30000])
        check_probs(buf[:, at:at + 30000], 0.0, out=torch.full_like(buf, float("nan"))[:, at:at + 30000])
    wide = torch.full((5, 40003), 7.0, device="cuda")
    check_probs(buf[:, 5:20006], 0.8, out=wide[:, 9:20010])
    assert (wide[:, :9] == 7).all() and (wide[:, 20010:] == 7).all()   # nothing beside the rows
    for n in (40000, 29999):
        z = buf[:, :n].contiguous()
        want = torch.empty_like(z)
        pdl.probs(z, 0.8, want)
        check_probs(z.clone(), 0.8)
        pdl.probs(z, 0.8, z)
        assert torch.equal(z, want)
    big = randn((2, 300001), torch.float32, 7, 2.0)   # more than a cluster keeps in registers
    want = check_probs(big, 1.0)
    pdl.probs(big, 1.0, big)
    assert torch.equal(big, want)


def test_probs_ties_take_the_lowest_id():
    z = torch.zeros(3, 20000, device="cuda")
    z[0, [19999, 777, 12000]] = 2.0
    z[1, 5:] = -0.0
    out = check_probs(z, 0.0)
    assert out.argmax(-1).tolist() == [777, 0, 0]


# ------------------------------------------------------------------ verification

def draft_inputs(b, d, n, given, seed, near=0.5):
    z = randn((b, d + 1, n), torch.float32, seed, 2.0)
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :d] + near * randn((b, d, n), torch.float32, seed + 1), -1) if given else None
    g = torch.Generator().manual_seed(seed)
    like = (q if given else p[:, :d]).flatten(0, 1)
    drafts = torch.multinomial(like.cpu() + 1e-9, 1, generator=g).view(b, d).to(torch.int32).cuda() if d else \
        torch.zeros(b, 0, dtype=torch.int32, device="cuda")
    u = torch.randint(0, 1 << 24, (b, d + 1), generator=g).to(torch.int32).cuda()
    n_drafts = torch.randint(0, d + 1, (b,), generator=g).to(torch.int32).cuda()
    return p, q, drafts, u, n_drafts


def check_verify(p, q, drafts, u, n_drafts=None):
    b, d1 = u.shape
    acc = torch.full((b,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((b, d1), -7, dtype=torch.int32, device="cuda")
    pdl.verify_draft(p, q, drafts, u, acc, tok, n_drafts=n_drafts)
    want_acc, want_tok = ref_verify(p, q, drafts, None if n_drafts is None else n_drafts.tolist(), u)
    assert acc.tolist() == want_acc
    assert np.array_equal(tok.cpu().numpy(), want_tok)
    return acc, tok


@pytest.mark.parametrize("n", VOCABS)
@pytest.mark.parametrize("given", [True, False])
def test_verify(n, given):
    check_verify(*draft_inputs(7, 4, n, given, seed=n))


@pytest.mark.parametrize("b,d", [(1, 0), (1, 1), (3, 64), (200, 2)])
@pytest.mark.parametrize("given", [True, False])
def test_verify_sizes(b, d, given):
    p, q, drafts, u, n_drafts = draft_inputs(b, d, 500, given and d > 0, seed=b + d, near=0.02)
    check_verify(p, q, drafts, u)
    check_verify(p, q, drafts, u, n_drafts)


def test_verify_every_boundary_uniform():
    """u at both ends and at the steps of a small distribution."""
    n, us = 6, [0, 1, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 2 ** 23 - 1, 2 ** 23, 2 ** 23 + 1, 2 ** 24 - 1]
    row = torch.tensor([0.25, 0.0, 0.25, 0.125, 0.375, 0.0])
    other = torch.tensor([0.5, 0.25, 0.0, 0.125, 0.125, 0.0])
    rows = [(a, c, t) for a in us for c in us for t in range(n)]
    b = len(rows)
    p = row.expand(b, 2, n).contiguous().cuda()
    q = other.expand(b, 1, n).contiguous().cuda()
    u = torch.tensor([[a, c] for a, c, _ in rows], dtype=torch.int32, device="cuda")
    drafts = torch.tensor([[t] for _, _, t in rows], dtype=torch.int32, device="cuda")
    check_verify(p, q, drafts, u)
    check_verify(p, None, drafts, u)


def test_verify_odd_values():
    """Ids outside the vocabulary, counts outside [0, max_drafts], values that are no
    probabilities, rows without any weight, equal rows, u with high bits set."""
    p, q, drafts, u, n_drafts = draft_inputs(8, 3, 9000, True, seed=77)
    drafts[0, 0], drafts[1, 1], drafts[2, 0] = -1, 9000, 2 ** 31 - 1
    n_drafts[:] = torch.tensor([3, 3, 9, -4, 3, 3, 3, 2])
    p[3], q[4] = 0.0, float("nan")
    p[5, :, ::2] = -1.0
    p[5, :, 1] = float("inf")
    p[6, :3] = q[6]                       # every draft is accepted
    q[7] = 1.0                            # nothing is left of the target
    u[7] = 2 ** 24 - 1
    u[4] |= -2 ** 31
    check_verify(p, q, drafts, u, n_drafts)
    check_verify(p, None, drafts, u, n_drafts)


@pytest.mark.parametrize("n", [1001, 70000])
def test_verify_strides(n):
    p, q, drafts, u, n_drafts = draft_inputs(5, 3, n, True, seed=n)
    wide_p, wide_q = (torch.full((5, 6, n + 3), float("nan"), device="cuda") for _ in range(2))
    wide_p[:, 1:5, 2:n + 2], wide_q[:, 2:5, 1:n + 1] = p, q
    a = check_verify(p, q, drafts, u, n_drafts)
    b = check_verify(wide_p[:, 1:5, 2:n + 2], wide_q[:, 2:5, 1:n + 1], drafts, u, n_drafts)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_verified_tokens_follow_the_targets_distribution():
    """The first token of a verified draft is distributed as the target's own draw."""
    n, b = 8, 200000
    target = torch.tensor([0.3, 0.05, 0.2, 0.0, 0.15, 0.1, 0.15, 0.05])
    draft = torch.tensor([0.1, 0.2, 0.2, 0.1, 0.05, 0.15, 0.1, 0.1])
    g = torch.Generator().manual_seed(3)
    p, q = target.expand(b, 2, n).contiguous().cuda(), draft.expand(b, 1, n).contiguous().cuda()
    drafts = torch.multinomial(draft, b, replacement=True, generator=g).view(b, 1).to(torch.int32).cuda()
    u = torch.randint(0, 1 << 24, (b, 2), generator=g).to(torch.int32).cuda()
    acc, tok = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, 2, dtype=torch.int32, device="cuda")
    pdl.verify_draft(p, q, drafts, u, acc, tok)
    count = torch.bincount(tok[:, 0].cpu(), minlength=n).double()
    for i in range(n):   # six standard deviations of a binomial count
        mean = b * float(target[i])
        assert abs(float(count[i]) - mean) <= 6 * (mean * (1 - float(target[i]))) ** 0.5 + 1


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_drafts_through_the_paged_cache(dtype):
    """Steps of a server with drafted tokens: the last drawn token and its drafts are
    appended and attended together, their logits become probabilities, the drafts are
    verified, and the next step begins behind the accepted ones, over the rows that rejected
    drafts left."""
    heads, kv_heads, dim, page, n_vocab, d = 8, 2, 64, 16, 3000, 3
    lengths = [40, 7, 130, 1]
    b = len(lengths)
    p = paged_inputs([n + 40 for n in lengths], [d + 1] * b, kv_heads, dim, page, dtype, seed=71)
    embed, head = randn((n_vocab, heads + 2 * kv_heads, dim), dtype, 72), randn((n_vocab, heads * dim), dtype, 73, 0.2)
    rope, kv = pdl.Rope.fill(300, dim), pdl.PagedKV(p["k"], p["v"])
    history = [torch.randint(0, n_vocab, (n,), generator=torch.Generator().manual_seed(74 + i)).tolist()
               for i, n in enumerate(lengths)]
    # the prompts, all but their last tokens
    tokens = torch.tensor(sum((h[:-1] for h in history), []), device="cuda")
    start = torch.tensor([0] + [len(h) - 1 for h in history]).cumsum(0).to(torch.int32).cuda()
    x = embed[tokens]
    pdl.paged_append(kv, pdl.PagedBatch(p["table"], torch.tensor([len(h) - 1 for h in history], dtype=torch.int32).cuda(),
                                        start, max_new=200),
                     x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], rope)
    length = torch.tensor([len(h) + d for h in history], dtype=torch.int32, device="cuda")
    p["length"], p["tokens"] = length, b * (d + 1)
    batch = pdl.PagedBatch(p["table"], length, p["start"], max_new=d + 1)
    ws = torch.empty(pdl.paged_attention_workspace_bytes(kv, batch, heads), dtype=torch.uint8, device="cuda")
    q, out = (torch.empty(b * (d + 1), heads, dim, dtype=dtype, device="cuda") for _ in range(2))
    probs = torch.empty(b * (d + 1), n_vocab, device="cuda")
    accepted = torch.empty(b, dtype=torch.int32, device="cuda")
    got = torch.empty(b, d + 1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(79)
    taken = 0
    for step in range(6):
        drafts = torch.randint(0, n_vocab, (b, d), generator=g).to(torch.int32).cuda()
        last = torch.tensor([[h[-1]] for h in history], dtype=torch.int32, device="cuda")
        if step:   # some drafts that the target likes: what it liked best at these places before
            drafts[::2] = probs.view(b, d + 1, n_vocab)[::2, :d].argmax(-1).to(torch.int32)
        for again in range(2):   # the second time with the first pass's likeliest tokens as drafts
            x = embed[torch.cat([last, drafts], 1).flatten().long()]
            pdl.paged_append(kv, batch, x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], rope, x[:, :heads], q)
            pdl.paged_attention(kv, batch, q, out, ws)
            logits = (out.flatten(1).float() @ head.float().T).contiguous()
            pdl.probs(logits, 0.7, probs)
            if not again:
                drafts[1::2] = probs.view(b, d + 1, n_vocab)[1::2, :d].argmax(-1).to(torch.int32)
        u = torch.randint(0, 1 << 24, (b, d + 1), generator=g).to(torch.int32).cuda()
        pdl.verify_draft(probs.view(b, d + 1, n_vocab), None, drafts, u, accepted, got)
        # every stage against its own form on what it was given
        ref, err, mass = ref_attention(p, q)
        half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
        before = err + (half if dtype == torch.bfloat16 else 0.0) * mass
        assert ((out.double() - ref).abs() <= before + half * (ref.abs() + before)).all()
        want = ref_probs(logits, 0.7)
        assert np.all(np.abs(probs.double().cpu().numpy() - want) <= 120 * 2.0 ** -24 * want + 2.0 ** -126)
        want_acc, want_tok = ref_verify(probs.view(b, d + 1, n_vocab), None, drafts, None, u)
        assert accepted.tolist() == want_acc and np.array_equal(got.cpu().numpy(), want_tok)
        for i, k in enumerate(want_acc):
            history[i] += got[i, :k + 1].tolist()
            taken += k
        length += accepted + 1
    assert taken > 0
    # the cache holds the accepted tokens' rows, whatever was rejected on the way
    fresh = paged_inputs([len(h) - 1 for h in history], [len(h) - 1 for h in history], kv_heads, dim, page, dtype, seed=80)
    x = embed[torch.tensor(sum((h[:-1] for h in history), []), device="cuda")]
    pdl.paged_append(pdl.PagedKV(fresh["k"], fresh["v"]),
                     pdl.PagedBatch(fresh["table"], fresh["length"], fresh["start"], max_new=1000),
                     x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], rope)
    for i, h in enumerate(history):
        pos = torch.arange(len(h) - 1, device="cuda")
        for name in "kv":
            a = p[name][p["table"][i].long()[pos // page], pos % page]
            c = fresh[name][fresh["table"][i].long()[pos // page], pos % page]
            assert torch.equal(a, c)
