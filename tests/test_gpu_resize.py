"""ds4g_paged_resize against the same bookkeeping with lists: lengths that go up and down, pools and token
rows that run out, pools without room, strides, large prompts and page numbers, captured graphs."""
import random

import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from paged8_ref import resize

pytestmark = pytest.mark.gpu


def pool_of(pages, page, capacity=None):
    free = torch.full((capacity or max(1, len(pages)),), -7, dtype=torch.int32)
    free[:len(pages)] = torch.tensor(pages, dtype=torch.int32)
    return pdl.PagePool(free.cuda(), torch.tensor([len(pages)], dtype=torch.int32).cuda(), page)


def run(page, width, seqs, steps, n_pages, max_tokens, rng, slots=True, stride=None):
    pages = list(range(n_pages))
    rng.shuffle(pages)
    pool = pool_of(pages, page, n_pages)
    store = torch.full((seqs, stride or width), -1, dtype=torch.int32, device="cuda")
    table = store[:, :width]
    batch = pdl.PagedBatch(table, torch.zeros(seqs, dtype=torch.int32, device="cuda"),
                           torch.full((seqs + 1,), 99, dtype=torch.int32, device="cuda"), max_new=10 ** 6)
    out = torch.full((max_tokens,), -5, dtype=torch.int64, device="cuda") if slots else None
    model = [[-1] * width for _ in range(seqs)], [0] * seqs, pages
    for want in steps(rng):
        was = out.clone() if slots else None
        pdl.paged_resize(pool, batch, torch.tensor(want, dtype=torch.int32, device="cuda"), out,
                         max_tokens=None if slots else max_tokens)
        t, length, free, start, places = resize(*model[:2], want, model[2], page, max_tokens)
        assert batch.length.tolist() == length
        assert batch.start.tolist() == start
        assert table.tolist() == t
        assert int(pool.n_free[0]) == len(free) and pool.free.tolist()[:len(free)] == free
        if slots:
            assert out.tolist() == places + was.tolist()[len(places):]
        if stride:
            assert (store[:, width:] == -1).all()
        model = t, length, free
        held = [x for row in t for x in row if x >= 0] + free
        assert sorted(held) == sorted(pages)   # every page has one owner


@pytest.mark.parametrize("page", [1, 16, 7, 128])
@pytest.mark.parametrize("seqs", [1, 3, 64, 512, 513, 1500])
def test_lengths_that_go_up_and_down(page, seqs):
    width = 9

    def steps(rng):
        now = [0] * seqs
        for _ in range(6):
            now = [max(0, min(width * page, n + rng.randint(-2 * page, 3 * page))) if rng.random() < 0.8 else n for n in now]
            yield now
        yield [0] * seqs
    run(page, width, seqs, steps, seqs * width, seqs * 3 * page + 1, random.Random(page + seqs))


@pytest.mark.parametrize("seqs", [5, 700])
@pytest.mark.parametrize("slots", [True, False])
def test_pools_and_rows_that_run_out(seqs, slots):
    width, page = 6, 8

    def steps(rng):
        for _ in range(8):
            yield [rng.randint(-3, (width + 1) * page) for _ in range(seqs)]   # (some above the table)
    run(page, width, seqs, steps, seqs * 2, seqs * 10, random.Random(seqs), slots, stride=8)


def test_taking_and_giving_back_restores_the_pool():
    pages = list(range(100))
    pool = pool_of(pages, 16, 100)
    batch = pdl.PagedBatch(torch.full((4, 20), -1, dtype=torch.int32, device="cuda"),
                           torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"))
    for want in ([100, 3, 0, 17], [100, 20, 33, 17], [100, 3, 0, 17], [0, 0, 0, 0]):
        pdl.paged_resize(pool, batch, torch.tensor(want, dtype=torch.int32, device="cuda"))
        if want == [100, 3, 0, 17]:
            after = pool.free.clone(), pool.n_free.clone(), batch.table.clone()
            if pool.n_free.item() != 100 - 10:
                raise AssertionError
    assert pool.free.tolist() == pages and (batch.table == -1).all()
    assert after[0].tolist()[:90] == pages[:90]


def test_no_sequences_no_room_and_long_prompts():
    none = pdl.PagedBatch(torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                          torch.full((1,), 9, dtype=torch.int32, device="cuda"))
    pool = pool_of([], 16)
    pdl.paged_resize(pool, none, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert none.start.tolist() == [0] and int(pool.n_free[0]) == 0
    # a pool without room loses what is given back, and hands out no page that it has not
    table = torch.tensor([[4, 5, 6]], dtype=torch.int32, device="cuda")
    batch = pdl.PagedBatch(table, torch.tensor([48], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
    pool = pool_of([1], 16, capacity=2)
    pdl.paged_resize(pool, batch, torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert table.tolist() == [[4, -1, -1]] and int(pool.n_free[0]) == 2 and pool.free.tolist() == [1, 6]
    # one prompt of a million tokens beside an empty sequence
    n = 1 << 20
    pool = pool_of(list(range(n // 16)), 16)
    batch = pdl.PagedBatch(torch.full((2, n // 16), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, dtype=torch.int32, device="cuda"))
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    pdl.paged_resize(pool, batch, torch.tensor([0, n], dtype=torch.int32, device="cuda"), slots)
    pages = torch.arange(n // 16 - 1, -1, -1, device="cuda")
    assert torch.equal(slots, (pages[:, None] * 16 + torch.arange(16, device="cuda")).view(-1))
    assert batch.start.tolist() == [0, 0, n] and int(pool.n_free[0]) == 0


def test_pages_past_32_bits_of_slots():
    pool = pool_of([2 ** 31 - 1, 2 ** 30], 128)
    batch = pdl.PagedBatch(torch.full((1, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                           torch.zeros(2, dtype=torch.int32, device="cuda"))
    slots = torch.zeros(130, dtype=torch.int64, device="cuda")
    pdl.paged_resize(pool, batch, torch.tensor([130], dtype=torch.int32, device="cuda"), slots)
    assert slots[:2].tolist() == [2 ** 37, 2 ** 37 + 1] and slots[128].item() == (2 ** 31 - 1) * 128


def test_in_a_graph_with_another_stream():
    pool = pool_of(list(range(200)), 16, 200)
    batch = pdl.PagedBatch(torch.full((10, 20), -1, dtype=torch.int32, device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda"),
                           torch.zeros(11, dtype=torch.int32, device="cuda"))
    want, slots = torch.zeros(10, dtype=torch.int32, device="cuda"), torch.zeros(400, dtype=torch.int64, device="cuda")
    pdl.paged_resize(pool, batch, want, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pdl.paged_resize(pool, batch, want, slots)
    model = [[-1] * 20 for _ in range(10)], [0] * 10, list(range(200))
    rng = random.Random(5)
    for _ in range(5):
        w = [rng.randint(0, 300) for _ in range(10)]
        want.copy_(torch.tensor(w, dtype=torch.int32))
        g.replay()
        t, length, free, start, _ = resize(*model[:2], w, model[2], 16, 400)
        assert batch.table.tolist() == t and batch.length.tolist() == length and batch.start.tolist() == start
        model = t, length, free


@pytest.mark.parametrize("seqs", [2, 600])
def test_pages_that_the_pool_lost_are_not_taken(seqs):
    """Three pages given back to a pool with room for one: another sequence finds one."""
    table = torch.full((seqs, 4), -1, dtype=torch.int32)
    table[0] = torch.tensor([10, 11, 12, 13])
    length = torch.zeros(seqs, dtype=torch.int32)
    length[0] = 32
    for more, takes in ((9, False), (8, True)):
        pool = pool_of([], 8, capacity=1)
        batch = pdl.PagedBatch(table.cuda(), length.cuda(), torch.zeros(seqs + 1, dtype=torch.int32, device="cuda"))
        want = torch.zeros(seqs, dtype=torch.int32)
        want[0], want[-1] = 8, more
        pdl.paged_resize(pool, batch, want.cuda())
        assert batch.table[0].tolist() == [10, -1, -1, -1] and batch.length.tolist()[:-1] == want.tolist()[:-1]
        assert batch.table[-1].tolist() == [13 if takes else -1, -1, -1, -1]
        assert int(batch.length[-1]) == (8 if takes else 0) and int(pool.n_free[0]) == (0 if takes else 1)
