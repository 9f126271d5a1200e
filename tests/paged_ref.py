"""Plain 64-bit forms of the paged-cache operators, probabilities and draft verification,
with random paged inputs, for the tests.  One loop per formula; no code is shared with the
library."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # largest relative rounding error


def paged_inputs(lengths, new, kv_heads, dim, page, dtype, seed, spare=3, layout="slot", fill=float("nan"),
                 pad_rows=0, width_extra=0):
    """Caches whose every slot holds `fill`, a shuffled page table, lengths and starts.
    layout: "slot" [page][slot][head][dim], "head" [page][head][slot][dim] in memory, or
    "both": K and V of a page next to one another."""
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-n // page)) for n in lengths]
    n_pages, width = sum(need) + spare, max(need + [1]) + width_extra
    ids = torch.randperm(n_pages, generator=g)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k].to(torch.int32)
        at += k
    if layout == "both":
        buf = torch.full((n_pages, 2, page, kv_heads, dim), fill, dtype=dtype, device="cuda")
        k, v = buf[:, 0], buf[:, 1]
    elif layout == "head":
        k, v = (torch.full((n_pages, kv_heads, page, dim), fill, dtype=dtype, device="cuda").transpose(1, 2)
                for _ in range(2))
    else:
        k, v = (torch.full((n_pages, page, kv_heads, dim), fill, dtype=dtype, device="cuda") for _ in range(2))
    start = torch.zeros(len(new) + 1, dtype=torch.int32)
    start[1:] = torch.tensor(new).cumsum(0)
    return dict(k=k, v=v, table=table.cuda(), length=torch.tensor(lengths, dtype=torch.int32).cuda(),
                start=start.cuda(), tokens=int(start[-1]) + pad_rows, page=page)


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def fill_slots(p, seed):
    """Random K and V in the slots the sequences use; the rest stays as it was."""
    lengths, table, page = p["length"].tolist(), p["table"].tolist(), p["page"]
    n_pages = p["k"].shape[0]
    for b, n in enumerate(lengths):
        for i in range(-(-n // page)):
            if i >= len(table[b]) or not 0 <= table[b][i] < n_pages:
                continue
            m = min(page, n - i * page)
            for x, s in ((p["k"], 0), (p["v"], 1)):
                x[table[b][i], :m] = randn((m,) + x.shape[2:], x.dtype, seed + 7919 * (2 * (b * 131 + i) + s))


def ref_append(p, k, v, q, cs, rot):
    """(K cache, V cache, q rows, bound on |error| before the rounding) in 64 bits."""
    kc, vc = p["k"].double().clone(), p["v"].double().clone()
    qo = None if q is None else torch.full_like(q, float("nan")).double()
    mag_k, mag_q = torch.zeros_like(kc), None if q is None else torch.zeros_like(qo)
    lengths, start, table = p["length"].tolist(), p["start"].tolist(), p["table"].tolist()
    for b, n in enumerate(lengths):
        new = start[b + 1] - start[b]
        for i in range(new):
            pos, t = n - new + i, start[b] + i
            if pos < 0 or (cs is not None and pos >= cs.shape[0]):
                continue

            def turn(x):
                y, mag = x.double().clone(), x.double().abs()
                if cs is not None:
                    c, s = cs[pos, :, 0].double(), cs[pos, :, 1].double()
                    a, d = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
                    y[..., 0:rot:2], y[..., 1:rot:2] = a * c - d * s, a * s + d * c
                    m = a.abs() + d.abs()
                    mag[..., 0:rot:2], mag[..., 1:rot:2] = m, m
                return y, mag
            if q is not None:
                qo[t], mag_q[t] = turn(q[t])
            j = pos // p["page"]
            if j < len(table[b]) and 0 <= table[b][j] < kc.shape[0]:
                g, s = table[b][j], pos % p["page"]
                kc[g, s], mag_k[g, s] = turn(k[t])
                vc[g, s] = v[t].double()
    return kc, vc, qo, mag_k, mag_q


def ref_attention(p, q, window=0, scale=None):
    """(out, E): out in 64 bits and a bound of the FP32 form's error per element, from
    the sizes of the sums: a score of D products is off by at most (D + 4) 2^-24 of the sum of
    their magnitudes, which moves a weight by twice that (the maximum moves too), and sums
    over n keys by (n + 64) 2^-24 of the sum of their terms (streams, parts and rescales
    included).  Third: sum of p |v|, what a relative error of the weights acts on."""
    n_tok, heads, dim = q.shape
    kv = p["k"].shape[2]
    group, page = heads // kv, p["page"]
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    out = torch.zeros(n_tok, heads, dim, dtype=torch.float64, device="cuda")
    err, mass = torch.zeros_like(out), torch.zeros_like(out)
    lengths, start, table = p["length"].tolist(), p["start"].tolist(), p["table"].tolist()
    n_pages = p["k"].shape[0]
    for b, n in enumerate(lengths):
        new = start[b + 1] - start[b]
        for i in range(new):
            pos = n - new + i
            keys = [j for j in range(max(0, pos - window + 1) if window > 0 else 0, pos + 1)
                    if j // page < len(table[b]) and 0 <= table[b][j // page] < n_pages]
            if not keys:
                continue
            j = torch.tensor(keys, device="cuda")
            pg = p["table"][b].long()[j // page]
            k, v = p["k"][pg, j % page].double(), p["v"][pg, j % page].double()
            k = k.repeat_interleave(group, 1)     # [n][heads][dim]
            v = v.repeat_interleave(group, 1)
            x = q[start[b] + i].double()
            s = torch.einsum("hd,nhd->hn", x, k) * scale
            ds = (dim + 4) * 2.0 ** -24 * torch.einsum("hd,nhd->hn", x.abs(), k.abs()).amax(-1) * abs(scale)
            w = torch.softmax(s, -1)
            out[start[b] + i] = torch.einsum("hn,nhd->hd", w, v)
            m = torch.einsum("hn,nhd->hd", w, v.abs())
            err[start[b] + i] = m * (4 * ds + (len(keys) + 64) * 2.0 ** -23)[:, None]
            mass[start[b] + i] = m
    return out, err, mass


def ref_probs(z, t):
    z = z.double().cpu().numpy().copy()
    z[np.isnan(z)] = -np.inf
    out = np.zeros_like(z)
    for r in range(z.shape[0]):
        m = z[r].max()
        if m == -np.inf:
            continue
        if t <= 0:
            out[r, int(np.argmax(z[r]))] = 1.0
        elif m == np.inf:
            out[r] = (z[r] == np.inf) / np.sum(z[r] == np.inf)
        else:
            e = np.exp((z[r] - m) / t)
            out[r] = e / e.sum()
    return out


def _unit(x):
    x = np.where(np.isnan(x), np.float32(0), x)
    return np.clip(x, np.float32(0), np.float32(1)).astype(np.float32)


def ref_verify(p, q, drafts, n_drafts, u24):
    """Accepted counts and tokens with integers of Python's own size."""
    p, drafts, u24 = p.cpu().numpy(), drafts.cpu().numpy(), u24.cpu().numpy()
    q = None if q is None else q.cpu().numpy()
    b, d1, v = p.shape
    acc, tok = [], np.full((b, d1), -1, dtype=np.int64)
    for s in range(b):
        n = d1 - 1 if n_drafts is None else min(max(int(n_drafts[s]), 0), d1 - 1)
        k = 0
        while k < n:
            d = int(drafts[s, k])
            if not 0 <= d < v:
                break
            qd = 1.0 if q is None else float(_unit(q[s, k, d]))
            if not (int(u24[s, k]) & 0xffffff) * qd < float(_unit(p[s, k, d])) * 2.0 ** 24:
                break
            k += 1
        row = _unit(p[s, k])
        w = row.copy()
        if k < n:
            if q is not None:
                w = np.maximum(row - _unit(q[s, k]), np.float32(0))
            elif 0 <= drafts[s, k] < v:
                w[drafts[s, k]] = 0

        def fixed(x):
            return np.rint(x.astype(np.float64) * 2.0 ** 40).astype(np.int64)
        f = fixed(w)
        if not f.any() and k < n:
            f = fixed(row)
        acc.append(k)
        tok[s, :k] = drafts[s, :k]
        total = sum(int(x) for x in f[f > 0])
        if total:
            goal = max(1, -(-(int(u24[s, d1 - 1]) & 0xffffff) * total // (1 << 24)))
            tok[s, k] = int(np.searchsorted(np.cumsum(f), goal))
    return acc, tok
