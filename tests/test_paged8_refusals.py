"""What the 8-bit cache's operators, ds4g_paged_resize and ds4g_edit_logits refuse, before any device
work (no GPU needed: pointers are host addresses that are never read), and what the binding passes on."""
import ctypes as C

import pytest
import torch

EINVAL, ESIZE, OK = -1, -6, 0
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from prefill_decode_layer_gb300 import build
    build.build()
    import prefill_decode_layer_gb300 as pdl
    return pdl.lib()


def structs(**kw):
    from prefill_decode_layer_gb300 import ds4g
    kv = dict(k=4096, v=8192, k_scale=4, v_scale=8, page_stride=16 * 2 * 64, slot_stride=128, head_stride=64,
              scale_stride=8, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, block=4)
    b = dict(table=4096, length=4096, start=4096, n_seqs=3, n_tokens=7, max_new=4, width=5, table_stride=5)
    kv.update({k: v for k, v in kw.items() if k in kv})
    b.update({k: v for k, v in kw.items() if k in b})
    return ds4g.PagedKV8Struct(**kv), ds4g.PagedBatchStruct(**b)


BAD = [dict(k=None), dict(v=4104), dict(k_scale=None), dict(v_scale=None), dict(k_scale=6), dict(v_scale=9),
       dict(page_stride=16), dict(page_stride=2040), dict(slot_stride=136), dict(head_stride=0), dict(head_stride=48),
       dict(scale_stride=7), dict(n_pages=0), dict(page_size=0), dict(n_kv_heads=0), dict(n_kv_heads=65537), dict(head_dim=0),
       dict(head_dim=12), dict(head_dim=264), dict(block=0), dict(block=-4), dict(block=3), dict(block=32), dict(table=None),
       dict(length=None), dict(start=None), dict(n_seqs=-1), dict(n_tokens=-1), dict(max_new=0), dict(width=-1), dict(table_stride=4),
       dict(width=2 ** 28, table_stride=2 ** 28)]


def append(lib, kv, b, k=4096, ks=128, v=8192, vs=128, rope=None, q=16384, qs=512, qo=32768, qos=512, heads=8, dtype=1):
    return lib.ds4g_paged_append8(C.byref(kv) if kv else None, C.byref(b) if b else None, k, ks, v, vs,
                                  C.byref(rope) if rope else None, q, qs, qo, qos, heads, dtype, None)


def attention(lib, kv, b, q=4096, qs=512, out=8192, os=512, heads=8, dtype=1, scale=0.0, window=0, ws=4096, n=1 << 40):
    return lib.ds4g_paged_attention8(C.byref(kv) if kv else None, C.byref(b) if b else None, q, qs, out, os, heads,
                                     dtype, scale, window, ws, n, None)


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_caches_and_batches(lib, bad):
    kv, b = structs(**bad)
    assert append(lib, kv, b) == EINVAL
    assert attention(lib, kv, b) == EINVAL
    assert lib.ds4g_paged_attention8_workspace_bytes(C.byref(kv), C.byref(b), 8) == 0


def test_append_and_attention_refuse(lib):
    from prefill_decode_layer_gb300 import ds4g
    kv, b = structs()
    assert append(lib, None, b) == EINVAL and append(lib, kv, None) == EINVAL
    for bad in (dict(k=None), dict(k=4104), dict(v=None), dict(ks=127), dict(ks=132), dict(vs=64), dict(dtype=2), dict(dtype=3),
                dict(qo=None), dict(q=None), dict(q=8), dict(qs=256), dict(qos=513), dict(heads=0), dict(heads=70000),
                dict(qo=16384, qos=520)):
        assert append(lib, kv, b, **bad) == EINVAL, bad
    for cs, n_pos, rot in ((None, 5, 64), (4100, 5, 64), (4096, 0, 64), (4096, 5, 63), (4096, 5, 66)):
        assert append(lib, kv, b, rope=ds4g.RopeStruct(cs, n_pos, rot)) == EINVAL
    assert append(lib, *structs(n_tokens=0), k=None, v=None) == OK
    need = lib.ds4g_paged_attention8_workspace_bytes(C.byref(kv), C.byref(b), 8)
    assert need > 0
    for bad in (dict(q=None), dict(q=8), dict(out=None), dict(out=4100), dict(qs=511), dict(os=64), dict(heads=0), dict(heads=7),
                dict(dtype=2), dict(scale=float("nan")), dict(scale=3e38), dict(scale=-1.0), dict(ws=None), dict(ws=4096 + 128), dict(out=4096)):
        assert attention(lib, kv, b, **bad) == EINVAL, bad
    assert attention(lib, kv, b, n=need - 1) == ESIZE
    assert attention(lib, kv, structs(max_new=129)[1]) == EINVAL
    assert attention(lib, kv, structs(n_seqs=0, n_tokens=0)[1]) == OK


def resize(lib, pool=True, free=4096, n_free=4096, capacity=10, page=16, table=4096, width=5, stride=5, length=4096, want=8192, n=3,
           start=4096, slots=4096, tokens=100):
    from prefill_decode_layer_gb300 import ds4g
    p = ds4g.PagePoolStruct(free, n_free, capacity, page)
    return lib.ds4g_paged_resize(C.byref(p) if pool else None, table, width, stride, length, want, n, start, slots, tokens, None)


def test_resize_refuses(lib):
    for bad in (dict(pool=False), dict(free=None), dict(n_free=None), dict(capacity=-1), dict(page=0), dict(table=None), dict(width=-1),
                dict(stride=4), dict(length=None), dict(want=None), dict(n=-1), dict(start=None), dict(slots=4100), dict(tokens=-1),
                dict(width=2 ** 28, stride=2 ** 28), dict(width=2 ** 24, stride=2 ** 24, page=1, n=200)):
        assert resize(lib, **bad) == EINVAL, bad
    assert resize(lib, n=65537) == ESIZE


def edit(lib, z=4096, zs=100, rows=2, n=100, out=8192, os=100, edits=True, **kw):
    from prefill_decode_layer_gb300 import ds4g
    e = dict(history=4096, n_history=4096, n_prompt=None, history_stride=10, repetition=4096, frequency=None, presence=None,
             bias_ids=4096, n_bias=None, bias=4096, bias_stride=5, allowed=4096, allowed_stride=4, max_history=10, max_bias=5)
    e.update(kw)
    return lib.ds4g_edit_logits(z, zs, rows, n, C.byref(ds4g.LogitEditsStruct(**e)) if edits else None, out, os, None)


def test_edit_refuses(lib):
    for bad in (dict(z=None), dict(out=None), dict(zs=99), dict(os=99), dict(rows=-1), dict(n=0), dict(edits=False), dict(out=4096, os=104),
                dict(rows=(1 << 24) + 1), dict(history=None), dict(max_history=-1), dict(max_history=11), dict(bias=None), dict(bias_ids=None),
                dict(max_bias=-1), dict(max_bias=6), dict(allowed_stride=3)):
        assert edit(lib, **bad) == EINVAL, bad
    assert edit(lib, n=(1 << 20) + 1, zs=1 << 21, os=1 << 21) == ESIZE
    assert edit(lib, max_bias=1025, bias_stride=1025) == ESIZE
    assert edit(lib, max_history=1 << 30, history_stride=1 << 30) == ESIZE
    assert edit(lib, rows=0, z=None) == OK


def test_the_binding_refuses_tensors_that_do_not_fit():
    import prefill_decode_layer_gb300 as pdl
    E = pdl.Ds4gError
    k, s = torch.zeros(4, 8, 2, 64, dtype=torch.uint8).view(E4M3), torch.ones(4, 2, 2)
    good = pdl.PagedKV8(k, k.clone(), s, s.clone())
    assert (good.block, good.struct.block, good.struct.scale_stride) == (4, 4, 4)
    for args in ((k.view(torch.uint8), k.view(torch.uint8), s, s), (k, k[:3], s, s), (k, k, s, s[:3]), (k, k, s[:3], s[:3]), (k, k, s.half(), s.half()),
                 (k, k, torch.ones(4, 3, 2), torch.ones(4, 3, 2)), (k, k, torch.ones(4, 2, 1), torch.ones(4, 2, 1)),
                 (k, k, torch.ones(4, 2, 4)[..., ::2], torch.ones(4, 2, 4)[..., ::2]), (k, k, torch.ones(4, 4, 2)[:, ::2], torch.ones(4, 4, 2)[:, ::2]),
                 (k, k, torch.ones(4, 0, 2), torch.ones(4, 0, 2)), (k.transpose(2, 3), k.transpose(2, 3), s, s)):
        with pytest.raises(E):
            pdl.PagedKV8(*args)
    # K's and V's scales of a page side by side
    both = torch.ones(4, 2, 2, 2)
    assert pdl.PagedKV8(k, k.clone(), both[:, 0], both[:, 1]).struct.scale_stride == 8
    table, length = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    start, want = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    free, n_free = torch.zeros(9, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for args in ((free.long(), n_free, 16), (free, n_free.long(), 16), (free, torch.zeros(2, dtype=torch.int32), 16), (free, n_free, 0),
                 (free, n_free, 2 ** 31), (free[::2], n_free, 16), (free[None], n_free, 16)):
        with pytest.raises(E):
            pdl.PagePool(*args)
    pool, batch = pdl.PagePool(free, n_free, 16), pdl.PagedBatch(table, length, start)
    for args in ((pdl.PagedBatch(table, length), want), (batch, want.long()), (batch, want[:2]), (batch, length),
                 (batch, torch.zeros(6, dtype=torch.int32)[::2]), (batch, want, torch.zeros(5)), (batch, want, torch.zeros(5, dtype=torch.int64)[::2]),
                 (batch, want, torch.zeros(5, dtype=torch.int64), 6)):
        with pytest.raises(E):
            pdl.paged_resize(pool, *args)
    z = torch.zeros(2, 50)
    ids, two = torch.zeros(2, 7, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(n_history=two), dict(repetition=torch.ones(2)), dict(history=ids.long()), dict(history=ids[0]), dict(history=ids, n_history=two.long()),
               dict(history=ids, n_history=torch.zeros(3, dtype=torch.int32)), dict(history=ids, repetition=torch.ones(2).double()),
               dict(history=ids.t()), dict(history=ids, frequency=torch.ones(4)[::2]), dict(bias_ids=ids), dict(bias=torch.zeros(2, 7)),
               dict(bias_ids=ids, bias=torch.zeros(2, 6)), dict(bias_ids=ids, bias=torch.zeros(2, 8)[:, :7]), dict(bias_ids=ids, bias=torch.zeros(3, 7)),
               dict(n_bias=two), dict(allowed=torch.zeros(2, 2)), dict(history=ids, allowed=torch.zeros(3, 2, dtype=torch.int32)),
               dict(history=ids[:1].expand(2, 7))):
        with pytest.raises(E):
            pdl.LogitEdits(**kw)
    edits = pdl.LogitEdits(history=ids)
    for args in ((z, z.double()), (z[0], z[0]), (z, torch.zeros(50, 2).t()), (torch.zeros(3, 50), torch.zeros(3, 50)), (z, z.clone())):
        with pytest.raises(E):
            pdl.edit_logits(*args, edits)
    with pytest.raises(E):   # a mask of one word for 50 tokens
        pdl.edit_logits(z, z.clone(), pdl.LogitEdits(allowed=torch.zeros(2, 1, dtype=torch.int32)))


@pytest.mark.parametrize("given,slots,passed", [(None, None, 2 ** 31 - 1), (None, 7, 7), (5, 7, 5), (2 ** 32 + 3, None, 2 ** 31 - 1), (-1, None, 0)])
def test_tokens_of_a_resize(monkeypatch, given, slots, passed):
    import prefill_decode_layer_gb300 as pdl
    from prefill_decode_layer_gb300 import ds4g
    args = []
    monkeypatch.setattr(ds4g, "_call", lambda name, index, stream, *a: args.extend(a))
    pool = pdl.PagePool(torch.zeros(9, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 16)
    batch = pdl.PagedBatch(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    out = torch.zeros(slots, dtype=torch.int64) if slots else None
    pdl.paged_resize(pool, batch, torch.zeros(3, dtype=torch.int32), out, max_tokens=given)
    assert args[-1] == passed and args[-2] == (out.data_ptr() if slots else None)


def test_either_cache_by_the_same_calls(monkeypatch):
    import prefill_decode_layer_gb300 as pdl
    from prefill_decode_layer_gb300 import ds4g
    names = []
    monkeypatch.setattr(ds4g, "_call", lambda name, index, stream, *a: names.append(name))
    batch = pdl.PagedBatch(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    k = torch.zeros(4, 8, 2, 64)
    k8, s = k.to(E4M3), torch.ones(4, 1, 2)
    x, q = torch.zeros(3, 2, 64), torch.zeros(3, 4, 64)
    for kv in (pdl.PagedKV(k, k.clone()), pdl.PagedKV8(k8, k8.clone(), s, s.clone())):
        pdl.paged_append(kv, batch, x, x)
        pdl.paged_append(kv, batch, x, x, None, q, q)
        pdl.paged_attention(kv, batch, q, q.clone(), torch.zeros(16, dtype=torch.uint8))
    assert names == ["ds4g_paged_append"] * 2 + ["ds4g_paged_attention"] + ["ds4g_paged_append8"] * 2 + ["ds4g_paged_attention8"]
