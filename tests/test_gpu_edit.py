"""ds4g_edit_logits against the definition in 64 bits: repetitions, counts, biases of the same id,
masks, logits that are not finite, strides, rows in place and ids outside the vocabulary."""
import numpy as np
import pytest
import torch

import prefill_decode_layer_gb300 as pdl

pytestmark = pytest.mark.gpu


def inputs(rows, vocab, history, biases, grammar, seed, prompt=True, penalties=True):
    g = torch.Generator().manual_seed(seed)
    e = {}
    if history:
        e["history"] = (torch.rand(rows, history, generator=g) ** 3 * (vocab + 2)).int() - 1   # some ids outside
        e["n_history"] = torch.randint(0, history + 1, (rows,), generator=g, dtype=torch.int32)
        e["n_history"][0] = history
        if prompt:
            e["n_prompt"] = (torch.rand(rows, generator=g) * e["n_history"]).int()
        if penalties:
            e["repetition"] = 0.7 + torch.rand(rows, generator=g)
            e["frequency"] = torch.randn(rows, generator=g)
            e["presence"] = torch.randn(rows, generator=g)
    if biases:
        e["bias_ids"] = torch.randint(-1, vocab + 1, (rows, biases), generator=g, dtype=torch.int32)
        e["bias_ids"][:, biases // 2] = e["bias_ids"][:, 0]     # the same id twice
        e["bias"] = 5 * torch.randn(rows, biases, generator=g)
        e["n_bias"] = torch.randint(0, biases + 1, (rows,), generator=g, dtype=torch.int32)
        e["n_bias"][-1] = biases
    if grammar:
        e["allowed"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, (vocab + 31) // 32), generator=g).to(torch.int32)
    z = 3 * torch.randn(rows, vocab, generator=g)
    return z, e


def reference(z, e):
    """(the result in 64 bits, a bound of the FP32 form's error)."""
    z = z.double().numpy().copy()
    size = np.abs(z)
    rows, vocab = z.shape
    for r in range(rows):
        if "history" in e:
            n = int(e["n_history"][r]) if "n_history" in e else e["history"].shape[1]
            m = min(max(int(e["n_prompt"][r]), 0), n) if "n_prompt" in e else 0
            ids = e["history"][r, :max(n, 0)].numpy()
            rep, freq, pres = (float(e[k][r]) if k in e else d for k, d in (("repetition", 1), ("frequency", 0), ("presence", 0)))
            count, seen = {}, set()
            for i, t in enumerate(ids):
                if 0 <= t < vocab:
                    seen.add(t)
                    if i >= m:
                        count[t] = count.get(t, 0) + 1
            for t in seen:
                z[r, t] = z[r, t] / rep if z[r, t] > 0 else z[r, t] * rep
            size[r] = np.maximum(size[r], np.abs(z[r]))
            for t, c in count.items():
                size[r, t] += abs(freq) * c + abs(pres)
                z[r, t] -= freq * c + pres
        if "bias" in e:
            n = int(e["n_bias"][r]) if "n_bias" in e else e["bias"].shape[1]
            for t, b in zip(e["bias_ids"][r, :n].tolist(), e["bias"][r, :n].tolist()):
                if 0 <= t < vocab:
                    z[r, t] += b
                    size[r, t] += abs(b)
        if "allowed" in e:
            words = e["allowed"][r if e["allowed"].shape[0] > 1 else 0].numpy().view(np.uint32)
            bits = (words[:, None] >> np.arange(32, dtype=np.uint32)) & 1
            z[r, bits.reshape(-1)[:vocab] == 0] = -np.inf
    # reciprocal, its product, product, sum, difference, the bias' rounding and its sum: seven roundings of sizes up to `size`
    return z, 7 * 2.0 ** -24 * size


def compare(got, ref, bound):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = ~np.isfinite(ref)
    assert np.array_equal(got[inf & ~np.isnan(ref)], ref[inf & ~np.isnan(ref)])
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - ref)[~inf] <= bound[~inf]).all(), float(np.max((np.abs(got - ref) / bound)[~inf]))


def edit(z, e, out=None):
    z = z if z.is_cuda else z.cuda()
    out = torch.full_like(z, float("nan")) if out is None else out
    pdl.edit_logits(z, out, pdl.LogitEdits(**{k: v.cuda() for k, v in e.items()}))
    return out


@pytest.mark.parametrize("rows,vocab,history,biases,grammar", [
    (1, 129280, 2000, 0, False), (3, 129280, 300, 40, True), (5, 1000, 0, 0, True), (4, 33, 100, 5, True), (7, 1, 3, 1, False),
    (2, 16385, 5000, 300, False), (300, 517, 50, 1, True), (2, 262144, 1, 1024, True), (3, 4099, 0, 2, False), (2, 1 << 20, 70, 0, True)])
def test_edits(rows, vocab, history, biases, grammar):
    z, e = inputs(rows, vocab, history, biases, grammar, seed=rows + vocab)
    ref, bound = reference(z, e)
    compare(edit(z, e), ref, bound)
    dev = z.cuda()
    compare(edit(dev, e, out=dev), ref, bound)   # in place


@pytest.mark.parametrize("rows,vocab,history,biases,grammar", [
    (64, 40000, 3000, 20, True), (400, 9000, 2500, 0, False), (40, 129280, 8192, 100, True), (130, 20001, 2049, 7, True)])
def test_long_histories(rows, vocab, history, biases, grammar):
    """Histories that several CTAs share."""
    z, e = inputs(rows, vocab, history, biases, grammar, seed=rows)
    e["n_history"][1], e["n_history"][2], e["n_prompt"][3] = 0, 1, 0
    ref, bound = reference(z, e)
    compare(edit(z, e), ref, bound)


@pytest.mark.parametrize("left_out", ["n_history", "n_prompt", "repetition", "frequency", "presence", "n_bias"])
def test_parts_that_are_not_there(left_out):
    z, e = inputs(3, 2000, 80, 7, True, seed=4)
    del e[left_out]
    ref, bound = reference(z, e)
    compare(edit(z, e), ref, bound)


def test_nothing_to_edit_and_one_mask_for_all_rows():
    z, _ = inputs(3, 5000, 0, 0, False, seed=5)
    assert torch.equal(edit(z, {}).cpu(), z)
    empty = {"history": torch.empty(3, 0, dtype=torch.int32), "n_history": torch.zeros(3, dtype=torch.int32),
             "bias_ids": torch.empty(3, 0, dtype=torch.int32), "bias": torch.empty(3, 0)}
    assert torch.equal(edit(z, empty).cpu(), z)
    one = {"allowed": torch.randint(-2 ** 31, 2 ** 31 - 1, (1, 200)).to(torch.int32)}
    ref, bound = reference(z, one)
    compare(edit(z, one), ref, bound)
    assert (edit(z, {"allowed": torch.zeros(3, 157, dtype=torch.int32)}) == float("-inf")).all()


def test_counts_out_of_range_are_clamped():
    z, e = inputs(4, 700, 20, 6, False, seed=6)
    e["n_history"] = torch.tensor([-3, 2 ** 31 - 1, 20, 0], dtype=torch.int32)
    e["n_prompt"] = torch.tensor([5, -1, 2 ** 31 - 1, 7], dtype=torch.int32)
    e["n_bias"] = torch.tensor([-1, 2 ** 31 - 1, 0, 6], dtype=torch.int32)
    got = edit(z, e)
    e["n_history"], e["n_prompt"], e["n_bias"] = (torch.tensor(x, dtype=torch.int32) for x in ([0, 20, 20, 0], [0, 0, 20, 0], [0, 6, 0, 6]))
    ref, bound = reference(z, e)
    compare(got, ref, bound)


def test_logits_that_are_not_finite():
    z, e = inputs(3, 900, 60, 10, True, seed=7)
    z[0, ::3], z[1, ::4], z[2, ::5] = float("-inf"), float("nan"), float("inf")
    z[0, 7] = -torch.finfo(torch.float32).max
    e["allowed"][0, 0] = -1
    ref, bound = reference(z, e)
    masked = ref == -np.inf
    bound[~np.isfinite(bound)] = 0
    got = edit(z, e)
    compare(got, ref, np.where(masked, 0, bound))


def test_strides_and_odd_alignment():
    z, e = inputs(5, 1001, 33, 9, True, seed=8)
    ref, bound = reference(z, e)
    store = torch.full((5, 1010), 5.0, device="cuda")
    store[:, 3:1004] = z.cuda()
    out = torch.full((5, 1007), 6.0, device="cuda")
    wide = {k: v.cuda() for k, v in e.items()}
    wide["history"] = torch.cat([wide["history"], wide["history"] + 1], 1)[:, :33]
    wide["allowed"] = torch.cat([wide["allowed"], ~wide["allowed"]], 1)[:, :32]
    wide["bias"], wide["bias_ids"] = (torch.cat([wide[k], wide[k]], 1)[:, :9] for k in ("bias", "bias_ids"))
    pdl.edit_logits(store[:, 3:1004], out[:, 1:1002], pdl.LogitEdits(**wide))
    compare(out[:, 1:1002], ref, bound)
    assert (out[:, 0] == 6).all() and (out[:, 1002:] == 6).all()


def test_rows_of_a_history_that_is_one_token():
    """65,000 times the same token: every thread counts in one place."""
    z = torch.zeros(2, 5000)
    e = {"history": torch.full((2, 65000), 4321, dtype=torch.int32), "frequency": torch.tensor([0.5, 0.25]),
         "n_prompt": torch.tensor([0, 65000], dtype=torch.int32)}
    ref, bound = reference(z, e)
    got = edit(z, e)
    compare(got, ref, bound)
    assert float(got[0, 4321]) == -32500.0 and float(got[1, 4321]) == 0.0


def test_in_a_graph():
    z, e = inputs(4, 3000, 100, 10, True, seed=9)
    dev, edits = z.cuda(), {k: v.cuda() for k, v in e.items()}
    out, le = torch.empty_like(dev), pdl.LogitEdits(**edits)
    pdl.edit_logits(dev, out, le)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pdl.edit_logits(dev, out, le)
    for s in (10, 11):
        z, e = inputs(4, 3000, 100, 10, True, seed=s)
        dev.copy_(z)
        for k, v in e.items():
            edits[k].copy_(v)
        g.replay()
        ref, bound = reference(z, e)
        compare(out, ref, bound)
