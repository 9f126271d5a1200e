"""Cases of the operators that serve several sequences from a paged K/V cache:

  append   K/V rows of new tokens into the pages of their sequences, with the
           position rotation of the keys and queries on the way;
  attend   attention of each sequence's newest tokens over its pages;
  probs    probabilities of a row of logits at a temperature;
  verify   drafted tokens against the target's probabilities, from given random
           numbers.

``run`` computes a case with plain torch operations, or, where ``own`` is true, with
the calls of the package."""
import math

import torch

own = False

DEV = "cuda"
ROPE_BASE = 10000.0


def listed():
    return [
        # one sequence of the layer's own shape (64 heads, one K/V head, window 128): a
        # single user's decode step, where latency counts
        dict(name="attend-one-window", op="attend", seqs=1, heads=64, kv_heads=1, dim=128, page=64, length=4097,
             drafts=1, window=128, dtype="bf16", cache="bf16"),
        # a server's decode step: many users at lengths of their own, grouped heads
        dict(name="attend-batch", op="attend", seqs=64, heads=32, kv_heads=8, dim=128, page=16, length=8191,
             drafts=1, window=0, dtype="bf16", cache="bf16"),
        # few users with long documents: the cache is much larger than L2
        dict(name="attend-long", op="attend", seqs=4, heads=64, kv_heads=8, dim=128, page=64, length=131072,
             drafts=1, window=0, dtype="bf16", cache="bf16"),
        # drafted tokens scored together: 1 to 5 new tokens a sequence, all 64 heads on one
        # K/V head, lengths up to the resync workload's
        dict(name="attend-drafts", op="attend", seqs=32, heads=64, kv_heads=1, dim=128, page=64, length=16994,
             drafts=5, window=0, dtype="bf16", cache="bf16"),
        # a small model kept in FP32 throughout
        dict(name="attend-f32", op="attend", seqs=16, heads=8, kv_heads=2, dim=64, page=16, length=2000,
             drafts=1, window=0, dtype="f32", cache="f32"),
        # one new token of each of 64 sequences
        dict(name="append-step", op="append", seqs=64, tokens=1, heads=64, kv_heads=1, dim=128, rot=128, page=64,
             length=4097, dtype="bf16", cache="bf16"),
        # a prefill chunk: a few prompts of thousands of tokens
        dict(name="append-prompt", op="append", seqs=4, tokens=4096, heads=64, kv_heads=1, dim=128, rot=128, page=64,
             length=16994, dtype="bf16", cache="bf16"),
        # FP32 projections rounded into a BF16 cache, half of each head rotated, grouped heads
        dict(name="append-f32-rows", op="append", seqs=33, tokens=37, heads=32, kv_heads=8, dim=128, rot=64, page=16,
             length=3001, dtype="f32", cache="bf16"),
        # logits of one sampled token of the layer's vocabulary
        dict(name="probs-one", op="probs", rows=1, vocab=129280, temperature=0.7),
        # logits of a batch of drafted positions
        dict(name="probs-batch", op="probs", rows=320, vocab=129280, temperature=1.0),
        # one user with a draft model's probabilities
        dict(name="verify-one", op="verify", seqs=1, drafts=4, vocab=129280, given=True),
        # a batch of users
        dict(name="verify-batch", op="verify", seqs=64, drafts=8, vocab=129280, given=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "probs", "verify"])
    if op == "probs":
        vocab = _log(rng, 1000, 262144)
        return dict(op=op, rows=_log(rng, 1, max(1, 320 * 129280 // vocab)), vocab=vocab,
                    temperature=rng.choice([0.0, 0.5, 0.7, 1.0, 1.3]))
    if op == "verify":
        vocab, drafts = _log(rng, 1000, 262144), rng.randint(1, 8)
        most = max(1, 64 * 8 * 129280 // (vocab * drafts))
        return dict(op=op, seqs=_log(rng, 1, min(most, 512)), drafts=drafts, vocab=vocab, given=rng.random() < 0.7)
    heads, kv = rng.choice([(64, 1), (32, 8), (64, 8), (16, 2), (8, 8), (28, 4), (8, 1), (40, 8)])
    dim, page = rng.choice([64, 128]), rng.choice([16, 16, 32, 48, 64, 128])
    f32 = rng.random() < 0.25
    if op == "append":
        seqs = _log(rng, 1, 256)
        tokens = rng.choice([1, _log(rng, 1, 4096)])
        tokens = max(1, min(tokens, (4 << 23) // (seqs * (heads + 2 * kv) * dim * (2 if f32 else 1))))
        most = max(1, (1 << 28) // (seqs * kv * dim))
        return dict(op=op, seqs=seqs, tokens=tokens, heads=rng.choice([0, heads, heads, heads]), kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 0]), page=page, length=tokens + _log(rng, 1, min(8192, most)),
                    dtype="f32" if f32 else "bf16", cache=rng.choice(["f32", "bf16"]) if f32 else "bf16")
    drafts = rng.choice([1, 1, rng.randint(2, 8)])
    seqs = _log(rng, 1, 16 if f32 else 256)
    most = (16 * 2000 * 2 * 64 if f32 else 4 * 131072 * 8 * 128) // (seqs * kv * dim)
    if not f32:   # the scores of the plain form fit as well
        most = min(most, (1 << 28) // (seqs * heads * drafts), (1 << 33) // (seqs * heads * dim * drafts))
    length = _log(rng, 1, max(drafts, min(most, 131072)))
    return dict(op=op, seqs=seqs, heads=heads, kv_heads=kv, dim=dim, page=page, length=max(length, drafts),
                drafts=drafts, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
                dtype="f32" if f32 else "bf16", cache="f32" if f32 else "bf16")


# ------------------------------------------------------------------ sizes of a case

def _spread(b):
    """A share in [0.25, 1] for sequence b: the first has all of it, the rest are spread evenly."""
    return 1.0 if b == 0 else 0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0)


def _counts(case):
    """(new tokens, length) of every sequence, before they are put in the seed's order."""
    out = []
    for b in range(case["seqs"]):
        if case["op"] == "attend":
            n = case["drafts"] - b % case["drafts"]
        else:
            n = max(1, int(case["tokens"] * _spread(b)))
        out.append((n, max(n, int(case["length"] * _spread(b)))))
    return out


_BYTES = {"bf16": 2, "f32": 4}
_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def work(case):
    op = case["op"]
    if op == "probs":
        n = case["rows"] * case["vocab"]
        return {"bytes": 8.0 * n, "flops": 4.0 * n}
    if op == "verify":
        # the rows of a draw: the target's and, where a draft was rejected, the draft's
        # (0 to `drafts` of them, each accepted about four times in five)
        most = case["drafts"]
        all_taken = sum(0.8 ** n for n in range(most + 1)) / (most + 1)
        rows = case["seqs"] * (2.0 - all_taken if case["given"] else 1.0)
        return {"bytes": rows * case["vocab"] * 4.0 + case["seqs"] * case["drafts"] * 16.0,
                "flops": 2.0 * rows * case["vocab"]}
    es, cs = _BYTES[case["dtype"]], _BYTES[case["cache"]]
    kvd, hd = case["kv_heads"] * case["dim"], case["heads"] * case["dim"]
    if op == "append":
        n = sum(c for c, _ in _counts(case))
        return {"bytes": float(n * (2 * kvd * (es + cs) + 2 * hd * es + case["rot"] * 4)),
                "flops": 3.0 * n * (case["heads"] + case["kv_heads"]) * case["rot"]}
    w, data, flops = case["window"], 0, 0
    for n, length in _counts(case):
        data += (min(length, w + n - 1) if w else length) * 2 * kvd * cs + 2 * n * hd * es
        for i in range(n):
            seen = length - n + i + 1
            flops += 4 * hd * (min(seen, w) if w else seen)
    return {"bytes": float(data), "flops": float(flops)}


# ------------------------------------------------------------------ inputs

def _paged(case, g, cpu):
    """Cache, page table, lengths and token starts of a case's sequences, in the seed's order."""
    counts = _counts(case)
    order = torch.randperm(len(counts), generator=cpu).tolist()
    counts = [counts[i] for i in order]
    page = case["page"]
    need = [-(-length // page) for _, length in counts]
    n_pages, width = sum(need) + 3, max(need)
    ids = torch.randperm(n_pages, generator=cpu)
    table = torch.full((len(counts), width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k].to(torch.int32)
        at += k
    starts = torch.zeros(len(counts) + 1, dtype=torch.int32)
    starts[1:] = torch.tensor([n for n, _ in counts]).cumsum(0)
    shape = (n_pages, page, case["kv_heads"], case["dim"])
    ct = _TYPE[case["cache"]]
    return dict(k_cache=torch.randn(shape, generator=g, device=DEV, dtype=ct),
                v_cache=torch.randn(shape, generator=g, device=DEV, dtype=ct), table=table.to(DEV),
                lengths=torch.tensor([n for _, n in counts], dtype=torch.int32, device=DEV),
                starts=starts.to(DEV), tokens=int(starts[-1]), most_new=max(n for n, _ in counts),
                most_length=max(n for _, n in counts))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op == "probs":
        s["logits"] = 2.5 * torch.randn(case["rows"], case["vocab"], generator=g, device=DEV)
        s["out"] = torch.empty_like(s["logits"])
        return s
    if op == "verify":
        b, d, v = case["seqs"], case["drafts"], case["vocab"]
        target = 2.5 * torch.randn(b, d + 1, v, generator=g, device=DEV)
        s["p"] = torch.softmax(target, -1)
        if case["given"]:   # a draft model near the target, and tokens drawn from it
            target[:, :d] += 0.5 * torch.randn(b, d, v, generator=g, device=DEV)
            s["q"] = torch.softmax(target[:, :d], -1)
        else:               # a draft without probabilities: tokens the target likes
            s["q"] = None
        like = s["q"] if case["given"] else s["p"][:, :d].sqrt().sqrt()
        noise = torch.empty(b, d, v, device=DEV).exponential_(generator=g)
        s["drafts"] = (like / noise).argmax(-1).to(torch.int32)
        if not case["given"]:   # every other sequence's drafts are the target's first choice
            s["drafts"][::2] = s["p"][::2, :d].argmax(-1).to(torch.int32)
        del target, noise, like
        s["n_drafts"] = torch.randint(0, d + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        s["n_drafts"][0] = d
        s["u24"] = torch.randint(0, 1 << 24, (b, d + 1), generator=g, device=DEV, dtype=torch.int32)
        s["accepted"] = torch.empty(b, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(b, d + 1, dtype=torch.int32, device=DEV)
        return s
    s.update(_paged(case, g, cpu))
    dt, n, hd = _TYPE[case["dtype"]], s["tokens"], case["dim"]
    if case["heads"]:
        s["q"] = torch.randn(n, case["heads"], hd, generator=g, device=DEV, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
    if op == "append":
        s["k"] = torch.randn(n, case["kv_heads"], hd, generator=g, device=DEV, dtype=dt)
        s["v"] = torch.randn(n, case["kv_heads"], hd, generator=g, device=DEV, dtype=dt)
        half = case["rot"] // 2
        s["rope"] = None
        if half:
            theta = ROPE_BASE ** (-2.0 * torch.arange(half, dtype=torch.float64, device=DEV) / case["rot"])
            angle = torch.arange(s["most_length"], dtype=torch.float64, device=DEV)[:, None] * theta
            s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    if own:
        import prefill_decode_layer_gb300 as pdl
        one = s["most_new"] == 1
        s["kv"] = pdl.PagedKV(s["k_cache"], s["v_cache"])
        s["batch"] = pdl.PagedBatch(s["table"], s["lengths"], None if one else s["starts"], max_new=s["most_new"])
        if op == "append":
            s["turn"] = pdl.Rope(s["rope"]) if s["rope"] is not None else None
        else:
            s["ws"] = torch.empty(pdl.paged_attention_workspace_bytes(s["kv"], s["batch"], case["heads"]),
                                  dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    return {"attend": _attend, "append": _append, "probs": _probs, "verify": _verify}[op](s)


def _places(s):
    """Sequence and position of every token."""
    t = torch.arange(s["tokens"], device=DEV)
    starts = s["starts"].long()
    seq = torch.searchsorted(starts, t, right=True) - 1
    pos = s["lengths"].long()[seq] - starts[seq + 1] + t
    return seq, pos


def _attend(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.paged_attention(s["kv"], s["batch"], s["q"], s["out"], s["ws"], window=c["window"])
        return s["out"]
    b, n, kv, group, hd = c["seqs"], s["most_new"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    at = torch.arange(s["most_length"], device=DEV)
    page = s["table"][:, at // c["page"]].long()
    there = (page >= 0) & (at < s["lengths"][:, None])                       # [b][L]
    keys = s["k_cache"][page.clamp(min=0), at % c["page"]].float()           # [b][L][kv][hd]
    values = s["v_cache"][page.clamp(min=0), at % c["page"]].float()
    values = torch.where(there[:, :, None, None], values, 0.0)
    starts = s["starts"].long()
    token = (starts[:-1, None] + torch.arange(n, device=DEV)).clamp(max=s["tokens"] - 1)   # [b][n]
    pos = s["lengths"].long()[:, None] - (starts[1:] - starts[:-1])[:, None] + torch.arange(n, device=DEV)
    seen = there[:, None] & (at <= pos[:, :, None])                          # [b][n][L]
    if c["window"]:
        seen &= at > pos[:, :, None] - c["window"]
    q = s["q"][token].float().view(b, n, kv, group, hd).permute(0, 2, 1, 3, 4).reshape(b, kv, n * group, hd)
    score = (q @ keys.permute(0, 2, 3, 1)).view(b, kv, n, group, -1) * (1.0 / math.sqrt(hd))
    score = torch.where(seen[:, None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = weight.view(b, kv, n * group, -1) @ values.permute(0, 2, 1, 3)
    out = out.view(b, kv, n, group, hd) / torch.where(total == 0, 1.0, total)
    seq, tpos = _places(s)
    i = tpos - (s["lengths"].long()[seq] - (starts[seq + 1] - starts[seq]))
    return out.permute(0, 2, 1, 3, 4).reshape(b, n, c["heads"], hd)[seq, i].to(s["q"].dtype)


def _turned(x, cs):
    """Pairs (2i, 2i+1) of the leading part of x [n][heads][hd] turned by cs [n][rot/2][2], in 32 bits."""
    x = x.float()
    if cs is None:
        return x
    rot = 2 * cs.shape[1]
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.paged_append(s["kv"], s["batch"], s["k"], s["v"], s["turn"], q=s.get("q"), q_out=s.get("out"))
        return {"k": s["k_cache"], "v": s["v_cache"], "q": s["out"] if c["heads"] else None}
    seq, pos = _places(s)
    page = s["table"][seq, pos // c["page"]].long()
    slot = pos % c["page"]
    cs = s["rope"][pos] if s["rope"] is not None else None
    s["k_cache"][page, slot] = _turned(s["k"], cs).to(s["k_cache"].dtype)
    s["v_cache"][page, slot] = s["v"].to(s["v_cache"].dtype)
    return {"k": s["k_cache"], "v": s["v_cache"],
            "q": _turned(s["q"], cs).to(s["q"].dtype) if c["heads"] else None}


def _probs(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.probs(s["logits"], c["temperature"], s["out"])
        return s["out"]
    z = s["logits"]
    if c["temperature"] <= 0:
        # first index of the largest logit
        top = (z == z.amax(-1, keepdim=True))
        first = (top.cumsum(-1, dtype=torch.int32) == 1) & top
        return first.float()
    e = torch.exp((z - z.amax(-1, keepdim=True)) / c["temperature"])
    return e / e.sum(-1, keepdim=True)


def _verify(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.verify_draft(s["p"], s["q"], s["drafts"], s["u24"], s["accepted"], s["tokens"], n_drafts=s["n_drafts"])
        return {"accepted": s["accepted"], "tokens": s["tokens"]}
    b, d, v = c["seqs"], c["drafts"], c["vocab"]
    p, q, draft, n = s["p"], s["q"], s["drafts"].long(), s["n_drafts"].long()
    rows = torch.arange(b, device=DEV)
    step = torch.arange(d, device=DEV)
    u = s["u24"].double() * 2.0 ** -24
    pd = p[:, :d].gather(2, draft[:, :, None])[:, :, 0].double()
    qd = q.gather(2, draft[:, :, None])[:, :, 0].double() if q is not None else 1.0
    ok = (u[:, :d] * qd < pd) & (step < n[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    rejected = accepted < n
    row = p[rows, accepted].clone()
    at = accepted.clamp(max=d - 1)
    if q is not None:
        rest = (row - q[rows, at]).clamp(min=0)
    else:
        rest = row.scatter(1, draft[rows, at][:, None], 0.0)
    weight = torch.where(rejected[:, None], rest, row)
    fixed = (weight * 2.0 ** 40).round().long()
    total = fixed.sum(1)
    alone = (row * 2.0 ** 40).round().long()   # nothing left of the target: its own probabilities
    fixed = torch.where(total[:, None] > 0, fixed, alone)
    run_sum = fixed.cumsum(1)
    total = run_sum[:, -1]
    u24 = s["u24"].long()[:, d]   # the draw's own number: those before it decided on the drafts
    goal = (u24 * (total >> 24) + ((u24 * (total & 0xffffff) + 0xffffff) >> 24)).clamp(min=1)
    token = torch.where(total > 0, torch.searchsorted(run_sum, goal[:, None])[:, 0], -1)
    step1 = torch.arange(d + 1, device=DEV)
    padded = torch.cat([draft, draft[:, :1]], 1)
    tokens = torch.where(step1 < accepted[:, None], padded,
                         torch.where(step1 == accepted[:, None], token[:, None], -1))
    return {"accepted": accepted.to(torch.int32), "tokens": tokens.to(torch.int32)}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "probs":
        z, t = s["logits"].double(), case["temperature"]
        if t <= 0:
            out = torch.zeros_like(z)
            for r in range(z.shape[0]):
                out[r, int(torch.nonzero(z[r] == z[r].max())[0])] = 1.0
            return out
        return torch.softmax(z / t, -1)
    if op == "verify":
        return _exact_verify(case, s)
    lengths, starts = s["lengths"].tolist(), s["starts"].tolist()
    page, table, hd = case["page"], s["table"].tolist(), case["dim"]
    if op == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        q = s["q"].double() if case["heads"] else None
        rot, half = case["rot"], case["rot"] // 2
        theta = ROPE_BASE ** (-2.0 * torch.arange(half, dtype=torch.float64, device=DEV) / max(rot, 1))
        for b, length in enumerate(lengths):
            n = starts[b + 1] - starts[b]
            pos = torch.arange(length - n, length, device=DEV)
            turn = torch.polar(torch.ones(n, half, dtype=torch.float64, device=DEV), pos[:, None].double() * theta)
            rows = slice(starts[b], starts[b + 1])

            def turned(x):
                y = x.clone()
                if half:
                    z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], half, 2).contiguous())
                    y[..., :rot] = torch.view_as_real(z * turn[:, None]).flatten(-2)
                return y
            where = torch.tensor(table[b], device=DEV)[pos // page] * page + pos % page
            kc.view(-1, *kc.shape[2:])[where] = turned(s["k"][rows].double())
            vc.view(-1, *vc.shape[2:])[where] = s["v"][rows].double()
            if q is not None:
                q[rows] = turned(s["q"][rows].double())
        return {"k": kc, "v": vc, "q": q}
    kv, group, w = case["kv_heads"], case["heads"] // case["kv_heads"], case["window"]
    if work(case)["flops"] > 4e11:   # too long in 64 bits
        return None
    out = torch.zeros(s["tokens"], case["heads"], hd, dtype=torch.float64, device=DEV)
    for b, length in enumerate(lengths):
        ids = torch.tensor(table[b], device=DEV)
        at = torch.arange(length, device=DEV)
        where = ids[at // page] * page + at % page
        keys = s["k_cache"].view(-1, kv, hd)[where].double()
        values = s["v_cache"].view(-1, kv, hd)[where].double()
        n = starts[b + 1] - starts[b]
        for i in range(n):
            pos = length - n + i
            lo = max(0, pos - w + 1) if w else 0
            t = starts[b] + i
            for h in range(kv):
                heads = slice(h * group, (h + 1) * group)
                p = torch.softmax(s["q"][t, heads].double() @ keys[lo:pos + 1, h].T / math.sqrt(hd), -1)
                out[t, heads] = p @ values[lo:pos + 1, h]
    return out


def _exact_verify(case, s):
    accepted, tokens = [], []
    drafts, n_drafts, u24 = s["drafts"].tolist(), s["n_drafts"].tolist(), s["u24"].tolist()
    for b in range(case["seqs"]):
        k = 0
        while k < n_drafts[b]:
            d = drafts[b][k]
            q = float(s["q"][b, k, d]) if s["q"] is not None else 1.0
            if not u24[b][k] / 2.0 ** 24 * q < float(s["p"][b, k, d]):
                break
            k += 1
        row = s["p"][b, k]
        left = row.clone()
        if k < n_drafts[b]:
            if s["q"] is not None:
                left = torch.clamp(row - s["q"][b, k], min=0.0)
            else:
                left[drafts[b][k]] = 0.0
        fixed = torch.round(left.double() * 2.0 ** 40).cpu().numpy().astype("int64")
        if not fixed.any():
            fixed = torch.round(row.double() * 2.0 ** 40).cpu().numpy().astype("int64")
        sums = fixed.cumsum()
        total = int(sums[-1])
        goal = max(1, -(-u24[b][case["drafts"]] * total // (1 << 24)))
        token = int(sums.searchsorted(goal)) if total else -1
        accepted.append(k)
        tokens.append(drafts[b][:k] + [token] + [-1] * (case["drafts"] - k))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device=DEV),
            "tokens": torch.tensor(tokens, dtype=torch.int32, device=DEV)}
