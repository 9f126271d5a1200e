"""Steps of a server over the paged cache in 8 bits, every operator's result checked on what it was given:
the lengths of a step are taken, pages with them; the last drawn token and its drafts are
appended and attended; their logits are edited and become probabilities; the drafts are verified; and
the rejected ones' slots are given back.  Sequences come, wait for pages, and end."""
import numpy as np
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged8_ref import E4M3, NAN_CODE, check_append8, resize, values
from paged_ref import randn, ref_attention, ref_probs, ref_verify
from test_gpu_edit import compare, reference
from test_gpu_paged8 import bound_of, close

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
NAMES = ("k8", "v8", "ks", "vs")


@pytest.mark.parametrize("heads,kv_heads,dim,page,block", [(8, 2, 64, 16, 16), (16, 1, 128, 8, 4), (6, 2, 96, 5, 5)])
def test_steps_of_a_server(heads, kv_heads, dim, page, block):
    vocab, d, width, temperature = 1500, 3, 160 // page, 0.7
    prompts, joins, ends = [40, 7, 100, 1, 30], [0, 0, 0, 2, 1], [9, 9, 3, 9, 9]   # steps
    b, most, n_pages = len(prompts), 256, 184 // page
    g = torch.Generator().manual_seed(74)
    history = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in prompts]
    pages = torch.randperm(n_pages, generator=g).to(I32)
    pool = pdl.PagePool(pages.clone().cuda(), torch.tensor([n_pages], dtype=I32).cuda(), page)
    model = [[-1] * width for _ in range(b)], [0] * b, pages.tolist()
    p = {"k8": torch.full((n_pages, page, kv_heads, dim), NAN_CODE, dtype=torch.uint8, device="cuda").view(E4M3),
         "ks": torch.full((n_pages, page // block, kv_heads), float("nan"), device="cuda"), "page": page, "block": block,
         "table": torch.full((b, width), -1, dtype=I32, device="cuda"), "length": torch.zeros(b, dtype=I32, device="cuda"),
         "start": torch.zeros(b + 1, dtype=I32, device="cuda")}
    p["v8"], p["vs"] = p["k8"].clone(), p["ks"].clone()
    kv, batch = pdl.PagedKV8(*(p[x] for x in NAMES)), pdl.PagedBatch(p["table"], p["length"], p["start"], max_new=128)
    embed, head = randn((vocab, heads + 2 * kv_heads, dim), BF16, 72), randn((vocab, heads * dim), BF16, 73)
    rope = pdl.Rope.fill(200, dim)
    slots = torch.full((most,), -1, dtype=torch.int64, device="cuda")
    rows = b * (d + 1)
    ws = torch.empty(pdl.paged_attention_workspace_bytes(kv, batch, heads), dtype=torch.uint8, device="cuda")
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, (vocab + 31) // 32), generator=g).to(I32)
    mask |= torch.randint(-2 ** 31, 2 ** 31 - 1, mask.shape, generator=g).to(I32)

    def take(want):
        nonlocal model
        before = slots.tolist()
        pdl.paged_resize(pool, batch, torch.tensor(want, dtype=I32, device="cuda"), slots)
        table, length, free, start, places = resize(*model[:2], want, model[2], page, most)
        assert p["table"].tolist() == table and p["length"].tolist() == length and p["start"].tolist() == start
        assert int(pool.n_free[0]) == len(free) and pool.free.tolist()[:len(free)] == free
        assert slots.tolist() == places + before[len(places):]
        model = table, length, free
        return start

    def append(x, q_out):
        before = {name: p[name].clone() for name in NAMES}
        k, v = x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
        pdl.paged_append(kv, batch, k, v, rope, x[:, :heads] if q_out is not None else None, q_out)
        check_append8(p, before, k, v, rope.cs, dim)

    taken, waited = 0, 0
    holds = [0] * b      # tokens of a sequence that the cache has
    for step in range(5):
        # prompts, all but their last tokens
        want = [(len(h) - 1 if joins[i] <= step < ends[i] else 0) for i, h in enumerate(history)]
        start = take(want)
        fed = torch.tensor(sum((history[i][holds[i]:model[1][i]] for i in range(b)), []), dtype=torch.long, device="cuda")
        assert len(fed) == start[-1]
        append(embed[fed], None)
        holds = list(model[1])
        runs = [joins[i] <= step < ends[i] and holds[i] == len(h) - 1 for i, h in enumerate(history)]
        # the last token and its drafts
        start = take([len(history[i]) + d if runs[i] else holds[i] for i in range(b)])
        runs = [start[i + 1] - start[i] == d + 1 for i in range(b)]
        waited += sum(joins[i] <= step < ends[i] and not runs[i] for i in range(b))
        n, ran = start[-1], [i for i in range(b) if runs[i]]
        drafts = torch.randint(0, vocab, (b, d), generator=g).to(I32).cuda()
        p["tokens"] = rows
        for _ in range(2):   # the second time with the first pass's likeliest tokens as drafts
            ids = torch.zeros(rows, dtype=torch.long, device="cuda")
            for i in ran:
                ids[start[i]:start[i + 1]] = torch.tensor([history[i][-1]] + drafts[i].tolist(), device="cuda")
            x, q = embed[ids], torch.full((rows, heads, dim), 3.0, dtype=BF16, device="cuda")
            out = torch.full_like(q, 7.0)
            append(x, q)
            pdl.paged_attention(kv, batch, q, out, ws)
            ref, err, mass = ref_attention(values(p), q)
            close(out[:n], ref[:n], bound_of(p, q, ref, err, mass)[:n])
            assert (out[n:] == 7).all() and (q[n:] == 3).all()
            at = torch.tensor([start[i] + j for i in ran for j in range(d + 1)], device="cuda")
            logits = (out[at].flatten(1).float() @ head.float().T).contiguous()
            # a row's history: the sequence's tokens up to the row's own
            hist = [history[i] + drafts[i].tolist()[:j] for i in ran for j in range(d + 1)]
            e = {"history": torch.tensor([h + [-1] * (200 - len(h)) for h in hist], dtype=I32),
                 "n_history": torch.tensor([len(h) for h in hist], dtype=I32),
                 "n_prompt": torch.tensor([prompts[i] for i in ran for _ in range(d + 1)], dtype=I32),
                 "repetition": torch.full((len(hist),), 1.1), "frequency": torch.full((len(hist),), 0.2),
                 "presence": torch.full((len(hist),), 0.3), "allowed": mask,
                 "bias_ids": torch.randint(0, vocab, (len(hist), 5), generator=g, dtype=I32), "bias": torch.randn(len(hist), 5, generator=g)}
            before = logits.cpu()
            pdl.edit_logits(logits, logits, pdl.LogitEdits(**{k: t.cuda() for k, t in e.items()}))
            compare(logits, *reference(before, e))
            probs = torch.empty_like(logits)
            pdl.probs(logits, temperature, probs)
            want_p = ref_probs(logits, temperature)
            assert np.all(np.abs(probs.double().cpu().numpy() - want_p) <= 120 * 2.0 ** -24 * want_p + 2.0 ** -126)
            likely = drafts.clone()
            likely[ran] = probs.view(len(ran), d + 1, vocab)[:, :d].argmax(-1).to(I32)
            used, drafts = drafts, likely
        drafts = used[ran].contiguous()
        u = torch.randint(0, 1 << 24, (len(ran), d + 1), generator=g).to(I32).cuda()
        accepted, got = torch.empty(len(ran), dtype=I32, device="cuda"), torch.empty(len(ran), d + 1, dtype=I32, device="cuda")
        pdl.verify_draft(probs.view(len(ran), d + 1, vocab), None, drafts, u, accepted, got)
        want_acc, want_tok = ref_verify(probs.view(len(ran), d + 1, vocab), None, drafts, None, u)
        assert accepted.tolist() == want_acc and np.array_equal(got.cpu().numpy(), want_tok)
        for i, a, row in zip(ran, want_acc, got.tolist()):
            history[i] += row[:a + 1]
            taken += a
            holds[i] += a + 1
        start = take(holds)      # the rejected ones' slots
        assert start[-1] == 0
    assert taken > 0 and waited > 0 and pdl.paged_attention_status(ws) == 0
    # the accepted tokens' rows are there, as they were rounded under the scales of their blocks: half a step
    # of each value, and half of the smallest step of each scale that the block had, which double
    table = p["table"].long()
    stored = values(p)
    for i, h in enumerate(history):
        pos = torch.arange(holds[i], device="cuda")
        if not holds[i]:
            continue
        x = embed[torch.tensor(h[:holds[i]], device="cuda")]
        k, v = x[:, heads:heads + kv_heads].double(), x[:, heads + kv_heads:].double()
        c, s = rope.cs[pos, None, :, 0].double(), rope.cs[pos, None, :, 1].double()
        k = torch.stack([k[..., 0::2] * c - k[..., 1::2] * s, k[..., 0::2] * s + k[..., 1::2] * c], -1).flatten(2)
        for name, y in (("k", k), ("v", v)):
            pg = table[i][pos // page]
            scale = p[name + "s"][pg, pos % page // block].double()[..., None]
            off = 2.0 ** -4 * y.abs() * (1 + 2.0 ** -20) + 2.0 ** -9 * scale + 2.0 ** -20
            assert ((stored[name][pg, pos % page].double() - y).abs() <= off).all()
