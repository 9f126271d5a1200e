"""Biases of ds4g_edit_logits whose ids lie near each other or repeat: results, and the time of a call, which
follows the number of biases and not where they lie."""
import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from test_gpu_edit import compare, edit, inputs, reference

pytestmark = pytest.mark.gpu

KINDS = ["one", "pairs", "neighbours", "twice", "reversed", "two ends"]


def ids_of(kind, rows, n, vocab, g):
    if kind == "one":                # all of one token
        return torch.full((rows, n), vocab // 2, dtype=torch.int32)
    if kind == "pairs":              # every id twice, the second time far behind the first
        half = torch.arange((n + 1) // 2).repeat(2)[:n]
        return (vocab - 1 - half).clamp(min=0).int().repeat(rows, 1)
    if kind == "twice":              # half of the ids often, in any order
        return torch.randint(0, max(1, min(vocab, n // 2)), (rows, n), generator=g, dtype=torch.int32)
    if kind == "two ends":
        return torch.where(torch.arange(n) % 2 == 0, torch.arange(n) // 2, vocab - 1 - torch.arange(n) // 2).clamp(0, vocab - 1).int().repeat(rows, 1)
    near = torch.arange(n) if kind == "neighbours" else torch.arange(n).flip(0)
    return ((vocab * 2 // 3 + near) % vocab).int().repeat(rows, 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,vocab,history,biases,grammar", [
    (1, 129280, 2000, 1024, False), (5, 129280, 5000, 300, True), (3, 700, 90, 1024, False), (40, 20001, 0, 1023, True), (300, 9000, 33, 64, False)])
def test_ids_that_lie_near_each_other(kind, rows, vocab, history, biases, grammar):
    z, e = inputs(rows, vocab, history, biases, grammar, seed=rows + vocab)
    e["bias_ids"] = ids_of(kind, rows, biases, vocab, torch.Generator().manual_seed(3))
    if history:                      # biased tokens that were seen, and generated
        e["history"][:, ::2] = e["bias_ids"][:, torch.arange((history + 1) // 2) % biases]
    ref, bound = reference(z, e)
    got = edit(z, e)
    compare(got, ref, bound)
    assert torch.equal(got, edit(z, e))


def device_us(z, e):
    z, out = z.cuda(), torch.empty(z.shape, device="cuda")
    edits = pdl.LogitEdits(**{k: v.cuda() for k, v in e.items()})
    pdl.edit_logits(z, out, edits)
    torch.cuda.synchronize()
    g, best = torch.cuda.CUDAGraph(), 1e9
    with torch.cuda.graph(g):
        for _ in range(10):
            pdl.edit_logits(z, out, edits)
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


@pytest.mark.parametrize("rows,kind", [(1, "neighbours"), (64, "neighbours"), (1, "pairs")])
def test_the_time_does_not_follow_where_they_lie(rows, kind):
    """1024 ids side by side against the same number all over the vocabulary (a search for each biased token took 12
    times as long, and 240 us for one row's pairs)."""
    z, e = inputs(rows, 129280, 0, 1024, False, seed=1)
    e["n_bias"][:] = 1024
    spread = device_us(z, e)
    e["bias_ids"] = ids_of(kind, rows, 1024, 129280, None)
    near = device_us(z, e)
    print("%d rows: %.1f us all over, %.1f us %s" % (rows, spread, near, kind))
    assert near <= 8 * spread + 10
