"""Random paged inputs of a cache in 8 bits and the plain 64-bit forms of its append and of the
page tables' bookkeeping, for the tests.  No code is shared with the library."""
from __future__ import annotations

import math

import torch

from paged_ref import paged_inputs

E4M3 = torch.float8_e4m3fn
NAN_CODE = 0x7f


def f32(codes: torch.Tensor) -> torch.Tensor:
    return codes.view(torch.uint8).view(E4M3).float()


def inputs8(lengths, new, kv_heads, dim, page, block, seed, layout="slot", pad_rows=0, width_extra=0, spare=3, spread=2):
    """A cache whose codes are all NaN and whose scales are NaN, with a shuffled page table, lengths and
    starts; then random codes, and scales that differ by up to 2^spread, in the slots the sequences use."""
    p = paged_inputs(lengths, new, 1, 1, page, torch.float32, seed, spare=spare, pad_rows=pad_rows,
                     width_extra=width_extra)
    n_pages = p["k"].shape[0]
    shape = (n_pages, page, kv_heads, dim)
    if layout == "both":     # K and V of a page next to one another, scales alike
        buf = torch.full((n_pages, 2, page, kv_heads, dim), NAN_CODE, dtype=torch.uint8, device="cuda")
        sc = torch.full((n_pages, 2, page // block, kv_heads), float("nan"), device="cuda")
        k, v, ks, vs = buf[:, 0], buf[:, 1], sc[:, 0], sc[:, 1]
    else:
        k, v = (torch.full(shape, NAN_CODE, dtype=torch.uint8, device="cuda") for _ in range(2))
        if layout == "head":
            k, v = (x.view(n_pages, kv_heads, page, dim).transpose(1, 2) for x in (k, v))
        ks, vs = (torch.full((n_pages, page // block, kv_heads), float("nan"), device="cuda") for _ in range(2))
    p.update(k8=k.view(E4M3) if layout == "slot" else k.view(E4M3), v8=v.view(E4M3), ks=ks, vs=vs, block=block)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    table = p["table"].tolist()
    for b, n in enumerate(lengths):
        for i in range(-(-max(n, 0) // page)):
            pg, m = table[b][i], min(page, n - i * page)
            if not 0 <= pg < n_pages:
                continue
            for c, s in ((k, ks), (v, vs)):
                x = 130.0 * torch.randn(m, kv_heads, dim, generator=g, device="cuda")
                c[pg, :m] = x.clamp(-448, 448).to(E4M3).view(torch.uint8)
                used = -(-m // block)
                s[pg, :used] = torch.exp2(torch.randint(-7 - spread, -6, (used, kv_heads), generator=g, device="cuda").float())
    return p


def values(p):
    """The cache as ref_attention takes it: the values of its codes in FP32 (exact)."""
    out = dict(p)
    for name in "kv":
        s = p[name + "s"].repeat_interleave(p["block"], 1)
        out[name] = f32(p[name + "8"]) * s[..., None]
    return out


def nearest8(x):
    """x in 64 bits to the nearest E4M3 value of its range, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def half_step(x):
    """Half the distance of the E4M3 values around x."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 4)


def ask(top: float) -> float:
    if top <= 0:
        return 2.0 ** -64
    m, e = math.frexp(top)
    return 2.0 ** max(-64, min(64, e - 9 + (m > 0.875)))


def check_append8(p, before, k, v, cs, rot):
    """Compare the cache that an append left with the cache `before` it, row by row."""
    lengths, start, table, page, block = (p["length"].tolist(), p["start"].tolist(), p["table"].tolist(), p["page"],
                                          p["block"])
    n_pages, kvh = p["k8"].shape[0], p["k8"].shape[2]
    want = {n: before[n].clone() for n in ("k8", "v8", "ks", "vs")}   # what no token touches
    for b, n in enumerate(lengths):
        new = start[b + 1] - start[b]
        first = n - new
        end = min(n, len(table[b]) * page)
        if cs is not None:
            end = min(end, cs.shape[0])
        pos = max(first, 0)
        while pos < end:
            stop = min(end, (pos // block + 1) * block)
            pg, slot = table[b][pos // page], pos % page
            if 0 <= pg < n_pages:
                t0, m, blk, skip = start[b] + pos - first, stop - pos, slot // block, slot % block
                for name, src in (("k", k), ("v", v)):
                    x = src[t0:t0 + m].double()
                    mag = x.abs()
                    if name == "k" and cs is not None:
                        c, s = cs[pos:stop, None, :, 0].double(), cs[pos:stop, None, :, 1].double()
                        a, d = x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()
                        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - d * s, a * s + d * c
                        mag[..., 0:rot:2] = mag[..., 1:rot:2] = a.abs() + d.abs()
                    # two products and a sum in FP32: three roundings at most of the magnitudes
                    off = 3 * 2.0 ** -24 * mag if name == "k" and cs is not None else torch.zeros_like(mag)
                    codes, scale = p[name + "8"], p[name + "s"]
                    got = f32(codes[pg, slot:slot + m]).double()
                    fine = x.isfinite()
                    assert torch.equal(got.isnan(), ~fine)
                    for h in range(kvh):
                        xh = torch.where(fine[:, h], x[:, h].abs(), 0.0)
                        tops = [float(xh.max()), float((xh + torch.where(fine[:, h], off[:, h], 0.0)).max()),
                                float((xh - torch.where(fine[:, h], off[:, h], 0.0)).max())]
                        s = float(scale[pg, blk, h])
                        old = float(before[name + "s"][pg, blk, h])
                        asked = [ask(t) for t in tops]
                        begun = pos - skip >= first
                        assert s in (asked if begun else [max(old, t) for t in asked]), (b, pos, h, s, asked, old)
                        y, d = x[:, h] / s, off[:, h] / s
                        bad = ~((got[:, h] - y.clamp(-448, 448)).abs() <= half_step(y.abs() + d) + d) & fine[:, h]
                        assert not bad.any(), (b, pos, h, name)
                        want[name + "s"][pg, blk, h] = s
                        want[name + "8"].view(torch.uint8)[pg, slot:slot + m, h] = codes.view(torch.uint8)[pg, slot:slot + m, h]
                        if not begun and s > old and skip:   # rows that the block held
                            held = f32(before[name + "8"][pg, slot - skip:slot, h]).double()
                            r = nearest8(held * old / s).float().to(E4M3)
                            want[name + "8"].view(torch.uint8)[pg, slot - skip:slot, h] = torch.where(
                                held.isnan(), before[name + "8"].view(torch.uint8)[pg, slot - skip:slot, h], r.view(torch.uint8))
            pos = stop
    for name in ("k8", "v8"):
        assert torch.equal(f32(p[name]).nan_to_num(1e9), f32(want[name]).nan_to_num(1e9)), name
    for name in ("ks", "vs"):
        assert torch.equal(p[name].nan_to_num(-1.0), want[name].nan_to_num(-1.0)), name


def resize(table, length, want, free, page, max_tokens):
    """The bookkeeping of a resize with lists: (table, length, free, start, slots)."""
    width, n = len(table[0]) if table else 0, len(length)
    table, free = [list(r) for r in table], list(free)
    want = [max(w, 0) for w in want]
    want = [now if w > width * page else w for w, now in zip(want, length)]

    def pages(x):
        return min(-(-x // page), width)
    back = [(b, i) for b in range(n) for i in range(pages(want[b]), pages(length[b]))]
    for b, i in reversed(back):
        free.append(table[b][i])
    for b, i in back:
        table[b][i] = -1
    asked_pages = asked_tokens = 0
    had = len(free)
    out, start, slots = list(length), [0], []
    for b in range(n):
        more, grown = max(0, pages(want[b]) - pages(length[b])), max(0, want[b] - length[b])
        asked_pages, asked_tokens = asked_pages + more, asked_tokens + grown
        fits = (more == 0 or asked_pages <= had) and (grown == 0 or asked_tokens <= max_tokens)
        if want[b] < length[b] or fits:
            out[b] = want[b]
        new = grown if fits else 0
        if fits:
            for i in range(pages(length[b]), pages(length[b]) + more):
                table[b][i] = free.pop()
        start.append(start[-1] + new)
        slots += [table[b][p // page] * page + p % page for p in range(out[b] - new, out[b])]
    return table, out, free, start, slots
