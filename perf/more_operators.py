"""Cases of the operators that serve many sequences from a K/V cache in 8 bits:

  attend8  attention of each sequence's newest tokens over pages of E4M3 codes with a
           scale for each block of slots and head;
  append8  K/V rows of new tokens rounded into such pages, with the position rotation
           of the keys and queries on the way;
  resize   the sequences' page tables, lengths, starts and slots from the lengths they
           are to have, pages taken from and given back to a pool;
  edit     penalties for repeated tokens, biases and a grammar's mask on rows of logits.

``run`` computes a case with plain torch operations, or, where ``own`` is true, with
the calls of the package."""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
ROPE_BASE = 10000.0
LEAST = 2.0 ** -64   # a block's scale at least; at most 2^64


def listed():
    return [
        # one user's decode step of the layer's own shape (64 heads, one K/V head, window 128)
        dict(name="attend8-one-window", op="attend8", seqs=1, heads=64, kv_heads=1, dim=128, page=64, block=64,
             length=4097, drafts=1, window=128, dtype="bf16"),
        # a server's decode step: many users at lengths of their own, grouped heads
        dict(name="attend8-batch", op="attend8", seqs=64, heads=32, kv_heads=8, dim=128, page=16, block=16, length=8191,
             drafts=1, window=0, dtype="bf16"),
        # few users with long documents: the cache is much larger than L2
        dict(name="attend8-long", op="attend8", seqs=4, heads=64, kv_heads=8, dim=128, page=64, block=32, length=131072,
             drafts=1, window=0, dtype="bf16"),
        # drafted tokens scored together: 1 to 5 new tokens a sequence, all 64 heads on one
        # K/V head, lengths up to the resync workload's
        dict(name="attend8-drafts", op="attend8", seqs=32, heads=64, kv_heads=1, dim=128, page=64, block=64,
             length=16994, drafts=5, window=0, dtype="bf16"),
        # a small model whose activations stay in FP32
        dict(name="attend8-f32", op="attend8", seqs=16, heads=8, kv_heads=2, dim=64, page=16, block=16, length=2000,
             drafts=1, window=0, dtype="f32"),
        # one new token of each of 64 sequences, into blocks that are partly full
        dict(name="append8-step", op="append8", seqs=64, tokens=1, heads=64, kv_heads=1, dim=128, rot=128, page=64,
             block=64, length=4097, dtype="bf16"),
        # a prefill chunk: a few prompts of thousands of tokens
        dict(name="append8-prompt", op="append8", seqs=4, tokens=4096, heads=64, kv_heads=8, dim=128, rot=128, page=64,
             block=16, length=16994, dtype="bf16"),
        # FP32 projections, half of each head rotated, without queries
        dict(name="append8-f32-rows", op="append8", seqs=33, tokens=37, heads=0, kv_heads=8, dim=64, rot=32, page=16,
             block=16, length=3001, dtype="f32"),
        # a decode step with four drafted tokens a user: pages for them, and back what was not kept
        dict(name="resize-drafts", op="resize", seqs=64, most_new=5, page=16, length=8191, prompts=0),
        # thousands of requests, some of them new: prompts come in as others grow or end
        dict(name="resize-many", op="resize", seqs=4096, most_new=8, page=16, length=2000, prompts=256),
        # one user's next token: a history of 2000, no grammar
        dict(name="edit-one", op="edit", rows=1, vocab=129280, history=2000, biases=0, grammar=False),
        # a batch with long histories, biases and a grammar each
        dict(name="edit-batch", op="edit", rows=256, vocab=129280, history=8192, biases=100, grammar=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend8", "attend8", "attend8", "append8", "append8", "resize", "edit"])
    if op == "edit":
        vocab = _log(rng, 1000, 262144)
        return dict(op=op, rows=_log(rng, 1, max(1, min(1024, 256 * 129280 // vocab))), vocab=vocab,
                    history=rng.choice([0, _log(rng, 1, 8192), _log(rng, 1, 8192)]), biases=rng.choice([0, _log(rng, 1, 300)]),
                    grammar=rng.random() < 0.5)
    if op == "resize":
        seqs = _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, most_new=rng.choice([1, rng.randint(2, 8), _log(rng, 8, 256)]),
                    page=rng.choice([1, 7, 16, 16, 32, 64, 128]), length=_log(rng, 16, max(64, min(131072, 8192000 // seqs))),
                    prompts=rng.choice([0, _log(rng, 1, max(1, seqs // 16))]))
    heads, kv = rng.choice([(64, 1), (32, 8), (64, 8), (16, 2), (8, 8), (28, 4), (8, 1), (40, 8)])
    dim, page = rng.choice([64, 128]), rng.choice([16, 16, 32, 48, 64, 128])
    block = rng.choice([page, 16, 8])
    f32 = rng.random() < 0.25
    if op == "append8":
        seqs = _log(rng, 1, 256)
        tokens = rng.choice([1, _log(rng, 1, 4096)])
        tokens = max(1, min(tokens, (4 << 23) // (seqs * (heads + 2 * kv) * dim * (2 if f32 else 1))))
        most = max(1, (1 << 28) // (seqs * kv * dim))
        return dict(op=op, seqs=seqs, tokens=tokens, heads=rng.choice([0, heads, heads, heads]), kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 0]), page=page, block=block,
                    length=tokens + _log(rng, 1, min(8192, most)), dtype="f32" if f32 else "bf16")
    drafts = rng.choice([1, 1, rng.randint(2, 8)])
    seqs = _log(rng, 1, 16 if f32 else 256)
    most = (16 * 2000 * 2 * 64 if f32 else 4 * 131072 * 8 * 128) // (seqs * kv * dim)
    if not f32:   # the scores of the plain form fit as well
        most = min(most, (1 << 28) // (seqs * heads * drafts), (1 << 33) // (seqs * heads * dim * drafts))
    length = _log(rng, 1, max(drafts, min(most, 131072)))
    return dict(op=op, seqs=seqs, heads=heads, kv_heads=kv, dim=dim, page=page, block=block, length=max(length, drafts),
                drafts=drafts, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), dtype="f32" if f32 else "bf16")


# ------------------------------------------------------------------ sizes of a case

def _spread(b):
    """A share in [0.25, 1] for sequence b: the first has all of it, the rest are spread evenly."""
    return 1.0 if b == 0 else 0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0)


def _counts(case):
    """(new tokens, length) of every sequence, before they are put in the seed's order."""
    out = []
    for b in range(case["seqs"]):
        if case["op"] == "attend8":
            n = case["drafts"] - b % case["drafts"]
        else:
            n = max(1, int(case["tokens"] * _spread(b)))
        out.append((n, max(n, int(case["length"] * _spread(b)))))
    return out


def _sizes(case):
    """Of a resize: (length now, length wanted, length kept after it) of every sequence.  The last
    `prompts` sequences come in with nothing; every 16th of the others ends."""
    out = []
    for b in range(case["seqs"]):
        n, new = max(1, int(case["length"] * _spread(b))), 1 + b % case["most_new"]
        if b >= case["seqs"] - case["prompts"]:
            out.append((0, n, max(1, n - b % 3)))
        elif b % 16 == 15:
            out.append((n, 0, 0))
        else:
            out.append((n, n + new, n + (b * 7 % (new + 1))))
    return out


_BYTES = {"bf16": 2, "f32": 4}
_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def work(case):
    op = case["op"]
    if op == "edit":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (8.0 + (0.125 if case["grammar"] else 0.0)) +
                case["rows"] * (4.0 * case["history"] + 8.0 * case["biases"]), "flops": 4.0 * n}
    if op == "resize":
        page, total = case["page"], 0.0
        for n, want, kept in _sizes(case):
            pages = [-(-x // page) for x in (n, want, kept)]
            moved = abs(pages[1] - pages[0]) + abs(pages[2] - pages[1])
            # a page: its table entry and its place in the pool; a new token: its slot
            total += 8.0 * moved + 8.0 * (max(0, want - n) + max(0, kept - want)) + 2 * 16.0
        return {"bytes": total, "flops": 0.0}
    es = _BYTES[case["dtype"]]
    kvd, hd, kv = case["kv_heads"] * case["dim"], case["heads"] * case["dim"], case["kv_heads"]
    if op == "append8":
        n = sum(c for c, _ in _counts(case))
        return {"bytes": float(n * (2 * kvd * (es + 1) + 2 * hd * es + case["rot"] * 4 + 8.0 * kv / case["block"])),
                "flops": 3.0 * n * (case["heads"] + kv) * case["rot"] + 4.0 * n * kvd}
    w, data, flops = case["window"], 0, 0
    for n, length in _counts(case):
        keys = min(length, w + n - 1) if w else length
        data += keys * 2 * (kvd + 4.0 * kv / case["block"]) + 2 * n * hd * es
        for i in range(n):
            seen = length - n + i + 1
            flops += 4 * hd * (min(seen, w) if w else seen)
    return {"bytes": float(data), "flops": float(flops)}


# ------------------------------------------------------------------ inputs

def _scale_for(top):
    """The least power of two s with top <= 448 s (within the scales' bounds), for FP32 top >= 0."""
    mant, expo = torch.frexp(top)          # top = mant 2^expo, mant in [0.5, 1); 448 = 0.875 2^9
    expo = expo - 9 + (mant > 0.875)
    s = torch.ldexp(torch.ones_like(top), expo.clamp(-64, 64))
    return torch.where(top > 0, s, LEAST)


def _full_cache(case, n_pages, g):
    """Codes and scales of random rows whose sizes differ by head and block."""
    kv, hd, page, block = case["kv_heads"], case["dim"], case["page"], case["block"]
    codes = torch.empty(n_pages, page, kv, hd, dtype=E4M3, device=DEV)
    scale = torch.empty(n_pages, page // block, kv, device=DEV)
    per = max(1, (1 << 25) // (page * kv * hd))
    head = torch.exp(0.3 * torch.randn(kv, generator=g, device=DEV))
    for a in range(0, n_pages, per):
        m = min(per, n_pages - a)
        x = torch.randn(m, page // block, block, kv, hd, generator=g, device=DEV)
        x *= (head * torch.exp(0.3 * torch.randn(m, page // block, kv, generator=g, device=DEV)))[:, :, None, :, None]
        s = _scale_for(x.abs().amax((2, 4)))
        scale[a:a + m] = s
        codes[a:a + m] = (x / s[:, :, None, :, None]).to(E4M3).view(m, page, kv, hd)
    return codes, scale


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
    k, ks = _full_cache(case, n_pages, g)
    v, vs = _full_cache(case, n_pages, g)
    return dict(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, table=table.to(DEV),
                lengths=torch.tensor([n for _, n in counts], dtype=torch.int32, device=DEV),
                starts=starts.to(DEV), tokens=int(starts[-1]), most_new=max(n for n, _ in counts),
                most_length=max(n for _, n in counts))


def _prepare_resize(case, cpu):
    sizes = _sizes(case)
    order = torch.randperm(len(sizes), generator=cpu).tolist()
    now, want, kept = (torch.tensor([sizes[i][j] for i in order], dtype=torch.int64) for j in range(3))
    page = case["page"]
    held = (now + page - 1) // page
    most = int(((torch.maximum(torch.maximum(now, want), kept) + page - 1) // page).max())
    grow = ((torch.maximum(want, now) + page - 1) // page - held).sum()
    n_pages = int(held.sum() + grow) + 5
    ids = torch.randperm(n_pages, generator=cpu).to(torch.int32)
    table = torch.full((len(sizes), most), -1, dtype=torch.int32)
    seq = torch.repeat_interleave(torch.arange(len(sizes)), held)
    index = torch.arange(int(held.sum())) - (held.cumsum(0) - held)[seq]
    table[seq, index] = ids[:len(seq)]
    free = torch.full((n_pages,), -1, dtype=torch.int32)
    free[:n_pages - len(seq)] = ids[len(seq):]
    tokens = int((want - now).clamp(min=0).sum() + (kept - want).clamp(min=0).sum())
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(table=table.to(DEV), lengths=now.to(**i32), wanted=want.to(**i32), kept=kept.to(**i32),
                free=free.to(DEV), n_free=torch.tensor([n_pages - len(seq)], **i32), tokens=max(1, tokens),
                starts=torch.zeros(len(sizes) + 1, **i32), n_pages=n_pages)


def _prepare_edit(case, g, cpu):
    rows, v, most = case["rows"], case["vocab"], case["history"]
    s = dict(logits=2.5 * torch.randn(rows, v, generator=g, device=DEV), out=torch.empty(rows, v, device=DEV))
    i32 = dict(dtype=torch.int32, device=DEV)
    if most:
        # few tokens make up most of a text: ids fall off as a power of their rank
        u = torch.rand(rows, most, generator=g, device=DEV)
        rank = (v ** u.double()).long().clamp(1, v) - 1
        s["history"] = (rank * 7919 % v).to(torch.int32)
        length = (most * (0.25 + 0.75 * torch.rand(rows, generator=g, device=DEV))).int()
        length[0] = most
        s["n_history"] = length
        s["n_prompt"] = (length * torch.rand(rows, generator=g, device=DEV)).int()
        s["repetition"] = 1.0 + 0.3 * torch.rand(rows, generator=g, device=DEV)
        s["frequency"] = 0.5 * torch.rand(rows, generator=g, device=DEV)
        s["presence"] = 0.5 * torch.rand(rows, generator=g, device=DEV)
    if case["biases"]:
        n = case["biases"]
        s["bias_ids"] = torch.randint(0, v, (rows, n), generator=g, **i32)
        s["bias"] = 4.0 * torch.randn(rows, n, generator=g, device=DEV)
        s["n_bias"] = torch.randint(0, n + 1, (rows,), generator=g, **i32)
    if case["grammar"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (rows, (v + 31) // 32), generator=g, device=DEV)
        more = torch.randint(-2 ** 31, 2 ** 31, (rows, (v + 31) // 32), generator=g, device=DEV)
        s["allowed"] = (words & more).to(torch.int32)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op == "edit":
        s.update(_prepare_edit(case, g, cpu))
        if own:
            import prefill_decode_layer_gb300 as pdl
            keys = ("history", "n_history", "n_prompt", "repetition", "frequency", "presence", "bias_ids", "bias",
                    "n_bias", "allowed")
            s["edits"] = pdl.LogitEdits(**{k: s[k] for k in keys if k in s})
        return s
    if op == "resize":
        s.update(_prepare_resize(case, cpu))
        s["slots"] = [torch.full((s["tokens"],), -1, dtype=torch.int64, device=DEV) for _ in range(2)]
        if own:
            import prefill_decode_layer_gb300 as pdl
            s["pool"] = pdl.PagePool(s["free"], s["n_free"], case["page"])
            s["batch"] = pdl.PagedBatch(s["table"], s["lengths"], s["starts"], max_new=s["tokens"])
        return s
    s.update(_paged(case, g, cpu))
    dt, n, hd = _TYPE[case["dtype"]], s["tokens"], case["dim"]
    if case["heads"]:
        s["q"] = torch.randn(n, case["heads"], hd, generator=g, device=DEV, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
    if op == "append8":
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
        s["kv"] = pdl.PagedKV8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["batch"] = pdl.PagedBatch(s["table"], s["lengths"], None if one else s["starts"], max_new=s["most_new"])
        if op == "append8":
            s["turn"] = pdl.Rope(s["rope"]) if s["rope"] is not None else None
        else:
            s["ws"] = torch.empty(pdl.paged_attention_workspace_bytes(s["kv"], s["batch"], case["heads"]),
                                  dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    return {"attend8": _attend8, "append8": _append8, "resize": _resize, "edit": _edit}[op](s)


def _places(s):
    """Sequence and position of every token."""
    t = torch.arange(s["tokens"], device=DEV)
    starts = s["starts"].long()
    seq = torch.searchsorted(starts, t, right=True) - 1
    pos = s["lengths"].long()[seq] - starts[seq + 1] + t
    return seq, pos


def _rows8(codes, scale, page, slot, block):
    """The rows that codes and scales stand for, in 32 bits."""
    rows = codes.view(torch.uint8)[page, slot].view(E4M3).float()
    return rows * scale[page, slot // block][..., None]


def _attend8(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.paged_attention(s["kv"], s["batch"], s["q"], s["out"], s["ws"], window=c["window"])
        return s["out"]
    b, n, kv, group, hd = c["seqs"], s["most_new"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    at = torch.arange(s["most_length"], device=DEV)
    page = s["table"][:, at // c["page"]].long()
    there = (page >= 0) & (at < s["lengths"][:, None])                       # [b][L]
    page, slot = page.clamp(min=0), (at % c["page"]).expand_as(page)
    keys = _rows8(s["k_cache"], s["k_scale"], page, slot, c["block"])        # [b][L][kv][hd]
    values = _rows8(s["v_cache"], s["v_scale"], page, slot, c["block"])
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


def _store8(codes, scale, x, page, slot, block, pos, first):
    """Rows x [n][kv][hd] into (page, slot).  A block that the call begins (its first slot is among
    the new tokens) gets the scale its rows ask for; another one keeps its scale unless they
    ask for a larger one, and then the rows it holds already are rounded again."""
    n_pages, blocks, kv = scale.shape
    place = page * blocks + slot // block                                    # [n]: block of each token
    top = torch.zeros(n_pages * blocks, kv, device=DEV).scatter_reduce_(
        0, place[:, None].expand(-1, kv), x.abs().amax(-1), "amax")
    old = scale.view(-1, kv)
    begun = pos - slot % block >= first                                      # the block's first slot is new
    fresh = torch.zeros(n_pages * blocks, dtype=torch.bool, device=DEV)
    fresh[place[begun]] = True
    touched = torch.zeros_like(fresh)
    touched[place] = True
    ask = _scale_for(top)
    new = torch.where(fresh[:, None], ask, torch.maximum(old, ask))
    new = torch.where(touched[:, None], new, old)
    # the rows before them in the blocks that new tokens go on with
    go_on = ~begun & (pos == first)
    before = torch.arange(block, device=DEV) < (slot % block)[go_on][:, None]
    go_on = place[go_on]
    held = codes.view(torch.uint8).view(n_pages * blocks, block, kv, -1)
    bits = held[go_on]
    rows = (bits.view(E4M3).float() * (old[go_on] / new[go_on])[:, None, :, None]).to(E4M3)
    held[go_on] = torch.where(before[:, :, None, None], rows.view(torch.uint8), bits)
    old.copy_(new)
    x = (x / new[place][..., None]).to(E4M3)
    codes.view(torch.uint8)[page, slot] = x.view(torch.uint8)


def _append8(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.paged_append(s["kv"], s["batch"], s["k"], s["v"], s["turn"], q=s.get("q"), q_out=s.get("out"))
        return {"k": s["k_cache"], "v": s["v_cache"], "ks": s["k_scale"], "vs": s["v_scale"],
                "q": s["out"] if c["heads"] else None}
    seq, pos = _places(s)
    starts = s["starts"].long()
    first = (s["lengths"].long() - starts[1:] + starts[:-1])[seq]            # of the sequence's new tokens
    page = s["table"][seq, pos // c["page"]].long()
    slot = pos % c["page"]
    cs = s["rope"][pos] if s["rope"] is not None else None
    _store8(s["k_cache"], s["k_scale"], _turned(s["k"], cs), page, slot, c["block"], pos, first)
    _store8(s["v_cache"], s["v_scale"], s["v"].float(), page, slot, c["block"], pos, first)
    return {"k": s["k_cache"], "v": s["v_cache"], "ks": s["k_scale"], "vs": s["v_scale"],
            "q": _turned(s["q"], cs).to(s["q"].dtype) if c["heads"] else None}


def _resize_once(s, want, slots):
    """Lengths to `want`: pages above the shorter ones go back to the pool (the first one given back
    on top), and the longer ones take from its top, sequence by sequence."""
    page, table, lengths, free, n_free = s["case"]["page"], s["table"], s["lengths"], s["free"], s["n_free"]
    width = table.shape[1]
    now, want = lengths.long(), want.long().clamp(min=0)
    want = torch.where(want > width * page, now, want)
    held, need = (now + page - 1) // page, (want + page - 1) // page
    index = torch.arange(width, device=DEV)
    back = (index >= need[:, None]) & (index < held[:, None])
    n_back = back.sum()
    order = back.view(-1).cumsum(0).view_as(back) - 1
    top = n_free.long() + n_back
    place = torch.where(back, top - 1 - order, free.numel())                 # the last place is a spare
    pool = torch.cat([free, free[:1]]).scatter_(0, place.view(-1), table.view(-1))[:-1]
    table.masked_fill_(back, -1)
    more, grown = (need - held).clamp(min=0), (want - now).clamp(min=0)
    fits = ((more == 0) | (more.cumsum(0) <= top)) & ((grown == 0) | (grown.cumsum(0) <= slots.numel()))
    more, grown = torch.where(fits, more, 0), torch.where(fits, grown, 0)
    taken = (index >= held[:, None]) & (index < (held + more)[:, None])
    order = taken.view(-1).cumsum(0).view_as(taken) - 1
    table.copy_(torch.where(taken, pool[(top - 1 - order).clamp(min=0)], table))
    free.copy_(pool)
    n_free.copy_(top - more.sum())
    lengths.copy_(torch.where(want < now, want, now + grown))
    starts = s["starts"]
    starts[1:] = grown.cumsum(0)
    t = torch.arange(slots.numel(), device=DEV)
    ends = starts.long()
    seq = (torch.searchsorted(ends, t, right=True) - 1).clamp(max=len(now) - 1)
    pos = (lengths.long()[seq] - ends[seq + 1] + t).clamp(min=0, max=width * page - 1)
    slots.copy_(torch.where(t < ends[-1], table[seq, pos // page].long() * page + pos % page, slots))


def _resize(s):
    starts = []
    for want, slots in zip((s["wanted"], s["kept"]), s["slots"]):
        if own:
            import prefill_decode_layer_gb300 as pdl
            pdl.paged_resize(s["pool"], s["batch"], want, slots)
        else:
            _resize_once(s, want, slots)
        starts.append(s["starts"].clone())
    return {"table": s["table"], "lengths": s["lengths"], "free": s["free"], "n_free": s["n_free"], "starts": starts,
            "slots": s["slots"]}


def _edit(s):
    c = s["case"]
    if own:
        import prefill_decode_layer_gb300 as pdl
        pdl.edit_logits(s["logits"], s["out"], s["edits"])
        return s["out"]
    z, (rows, v) = s["logits"], s["logits"].shape
    if c["history"]:
        at = torch.arange(s["history"].shape[1], device=DEV)
        inside = at < s["n_history"][:, None]
        made = inside & (at >= s["n_prompt"][:, None])
        ids = s["history"].long()
        seen = torch.zeros(rows, v, dtype=torch.int32, device=DEV).scatter_add_(1, ids, inside.int()) > 0
        count = torch.zeros(rows, v, dtype=torch.int32, device=DEV).scatter_add_(1, ids, made.int())
        r = s["repetition"][:, None]
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - (s["frequency"][:, None] * count + torch.where(count > 0, s["presence"][:, None], 0.0))
    if c["biases"]:
        n = torch.arange(s["bias"].shape[1], device=DEV) < s["n_bias"][:, None]
        add = torch.zeros(rows, v, dtype=torch.float64, device=DEV).scatter_add_(
            1, s["bias_ids"].long(), torch.where(n, s["bias"], 0.0).double())
        z = z + add.float()
    if c["grammar"]:
        bit = torch.arange(v, device=DEV)
        allowed = (s["allowed"][:, bit // 32] >> (bit % 32)) & 1
        z = torch.where(allowed != 0, z, -math.inf)
    return z if z is not s["logits"] else z.clone()


# ------------------------------------------------------------------ from the definition, in 64 bits

def _nearest8(x):
    """x, in 64 bits, to the nearest of 3 bits behind the first, in steps of 2^-9 at least, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "resize":
        return None   # whole numbers throughout
    if op == "edit":
        return _exact_edit(case, s)
    lengths, starts = s["lengths"].tolist(), s["starts"].tolist()
    page, table, hd, block = case["page"], s["table"].tolist(), case["dim"], case["block"]
    if op == "append8":
        out = {"k": s["k_cache"].double(), "v": s["v_cache"].double(), "ks": s["k_scale"].double(),
               "vs": s["v_scale"].double(), "q": s["q"].double() if case["heads"] else None}
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
            if out["q"] is not None:
                out["q"][rows] = turned(s["q"][rows].double())
            # whole blocks side by side: the rows before the new ones, and none behind them
            a0, per = (length - n) // block * block, -(-length // block) - (length - n) // block
            ids = torch.tensor(table[b], device=DEV)
            at = torch.arange(a0, a0 + per * block, device=DEV).clamp(max=length - 1)
            where = ids[at // page] * page + at % page
            blk = ids[at[::block] // page] * (page // block) + at[::block] % page // block
            held = (torch.arange(a0, a0 + per * block, device=DEV) < length - n).view(per, block)
            live = (torch.arange(a0, a0 + per * block, device=DEV) < length).view(per, block)
            for name, x in (("k", turned(s["k"][rows].double())), ("v", s["v"][rows].double())):
                codes, scale = out[name].view(-1, case["kv_heads"], hd), out[name + "s"].view(-1, case["kv_heads"])
                old = scale[blk]                                             # [per][kv]
                full = torch.zeros(per * block, case["kv_heads"], hd, dtype=torch.float64, device=DEV)
                full[length - n - a0:length - a0] = x
                full = full.view(per, block, case["kv_heads"], hd)
                ask = torch.exp2(torch.ceil(torch.log2(full.abs().amax((1, 3)).clamp(min=2.0 ** -300) / 448.0))
                                 .clamp(-64, 64))
                new = torch.where(held.any(1)[:, None], torch.maximum(old, ask), ask)
                before = codes[where].view(per, block, case["kv_heads"], hd) * old[:, None, :, None]
                rounded = _nearest8(torch.where(held[:, :, None, None], before, full) / new[:, None, :, None])
                keep = live.view(-1)
                codes[where[keep]] = rounded.view(per * block, case["kv_heads"], hd)[keep]
                scale[blk] = new
        return out
    kv, group, w = case["kv_heads"], case["heads"] // case["kv_heads"], case["window"]
    if work(case)["flops"] > 4e11:   # too long in 64 bits
        return None
    out = torch.zeros(s["tokens"], case["heads"], hd, dtype=torch.float64, device=DEV)
    for b, length in enumerate(lengths):
        n = starts[b + 1] - starts[b]
        first = max(0, length - n - w + 1) if w else 0
        ids = torch.tensor(table[b], device=DEV)
        at = torch.arange(first, length, device=DEV)
        where, blk = ids[at // page] * page + at % page, ids[at // page] * (page // block) + at % page // block
        keys, values = ((x.view(torch.uint8).view(-1, kv, hd)[where].view(E4M3).double() *
                         f.view(-1, kv)[blk].double()[..., None]) for x, f in
                        ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        for i in range(n):
            pos = length - n + i
            lo = max(0, pos - w + 1) if w else 0
            for h in range(kv):
                heads = slice(h * group, (h + 1) * group)
                p = torch.softmax(s["q"][starts[b] + i, heads].double() @ keys[lo - first:pos + 1 - first, h].T /
                                  math.sqrt(hd), -1)
                out[starts[b] + i, heads] = p @ values[lo - first:pos + 1 - first, h]
    return out


def _exact_edit(case, s):
    out = s["logits"].double()
    for r in range(case["rows"]):
        z = out[r]
        if case["history"]:
            n, m = int(s["n_history"][r]), int(s["n_prompt"][r])
            ids = s["history"][r, :n].long()
            rep, freq, pres = (float(s[k][r]) for k in ("repetition", "frequency", "presence"))
            seen = torch.unique(ids)
            z[seen] = torch.where(z[seen] > 0, z[seen] / rep, z[seen] * rep)
            made, count = torch.unique(ids[m:], return_counts=True)
            z[made] -= freq * count.double() + pres
        if case["biases"]:
            n = int(s["n_bias"][r])
            z.index_add_(0, s["bias_ids"][r, :n].long(), s["bias"][r, :n].double())
        if case["grammar"]:
            words = s["allowed"][r].long() & 0xffffffff
            bits = (words[:, None] >> torch.arange(32, device=DEV)) & 1
            z[bits.view(-1)[:case["vocab"]] == 0] = -math.inf
    return out
