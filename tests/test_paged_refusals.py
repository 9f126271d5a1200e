"""What the paged-cache operators, ds4g_probs and ds4g_verify_draft refuse, before any device
work (no GPU needed: pointers are host addresses that are never read)."""
import ctypes as C

import pytest
import torch

EINVAL, ESIZE, OK = -1, -6, 0


@pytest.fixture(scope="module")
def lib():
    from prefill_decode_layer_gb300 import build
    build.build()
    import prefill_decode_layer_gb300 as pdl
    return pdl.lib()


def structs(**kw):
    from prefill_decode_layer_gb300 import ds4g
    kv = dict(k=4096, v=8192, page_stride=16 * 2 * 64, slot_stride=128, head_stride=64, n_pages=10, page_size=16,
              n_kv_heads=2, head_dim=64, dtype=1)
    b = dict(table=4096, length=4096, start=4096, n_seqs=3, n_tokens=7, max_new=4, width=5, table_stride=5)
    kv.update({k: v for k, v in kw.items() if k in kv})
    b.update({k: v for k, v in kw.items() if k in b})
    return ds4g.PagedKVStruct(**kv), ds4g.PagedBatchStruct(**b)


BAD = [dict(k=None), dict(v=4104), dict(page_stride=4), dict(slot_stride=129), dict(head_stride=0), dict(n_pages=0),
       dict(page_size=0), dict(n_kv_heads=0), dict(n_kv_heads=65537), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264), dict(dtype=2),
       dict(table=None), dict(length=None), dict(start=None), dict(n_seqs=-1), dict(n_tokens=-1), dict(max_new=0),
       dict(width=-1), dict(table_stride=4), dict(width=2 ** 28, table_stride=2 ** 28)]


def append(lib, kv, b, k=4096, ks=128, v=8192, vs=128, rope=None, q=16384, qs=512, qo=32768, qos=512, heads=8, dtype=1):
    return lib.ds4g_paged_append(C.byref(kv) if kv else None, C.byref(b) if b else None, k, ks, v, vs,
                                 C.byref(rope) if rope else None, q, qs, qo, qos, heads, dtype, None)


def attention(lib, kv, b, q=4096, qs=512, out=8192, os=512, heads=8, dtype=1, scale=0.0, window=0, ws=4096, n=1 << 40):
    return lib.ds4g_paged_attention(C.byref(kv) if kv else None, C.byref(b) if b else None, q, qs, out, os, heads,
                                    dtype, scale, window, ws, n, None)


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_caches_and_batches(lib, bad):
    kv, b = structs(**bad)
    assert append(lib, kv, b) == EINVAL
    assert attention(lib, kv, b) == EINVAL
    assert lib.ds4g_paged_attention_workspace_bytes(C.byref(kv), C.byref(b), 8) == 0


def test_append_refuses(lib):
    from prefill_decode_layer_gb300 import ds4g
    kv, b = structs()
    assert append(lib, None, b) == EINVAL and append(lib, kv, None) == EINVAL
    for bad in (dict(k=None), dict(k=4104), dict(v=None), dict(ks=127), dict(ks=132), dict(vs=64), dict(dtype=3),
                dict(qo=None), dict(q=None), dict(q=8), dict(qs=256), dict(qos=513), dict(heads=0), dict(heads=70000),
                dict(qo=16384, qos=520)):
        assert append(lib, kv, b, **bad) == EINVAL, bad
    for cs, n_pos, rot in ((None, 5, 64), (4100, 5, 64), (4096, 0, 64), (4096, 5, 0), (4096, 5, 63), (4096, 5, 66)):
        assert append(lib, kv, b, rope=ds4g.RopeStruct(cs, n_pos, rot)) == EINVAL
    assert lib.ds4g_rope_fill(None, 4, 4, 10.0, None) == EINVAL
    assert lib.ds4g_rope_fill(4096, 0, 4, 10.0, None) == EINVAL
    assert lib.ds4g_rope_fill(4096, 4, 3, 10.0, None) == EINVAL
    assert lib.ds4g_rope_fill(4096, 4, 4, 0.0, None) == EINVAL
    kv, b = structs(n_tokens=0)
    assert append(lib, kv, b, k=None, v=None) == OK        # nothing to do


def test_attention_refuses(lib):
    kv, b = structs()
    need = lib.ds4g_paged_attention_workspace_bytes(C.byref(kv), C.byref(b), 8)
    assert need > 0
    assert attention(lib, None, b) == EINVAL and attention(lib, kv, None) == EINVAL
    for bad in (dict(q=None), dict(q=8), dict(out=None), dict(out=4100), dict(qs=511), dict(os=64), dict(heads=0),
                dict(heads=7), dict(dtype=9), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(scale=-1.0), dict(ws=None),
                dict(ws=4096 + 128), dict(out=4096)):
        assert attention(lib, kv, b, **bad) == EINVAL, bad
    assert attention(lib, kv, b, n=need - 1) == ESIZE
    assert lib.ds4g_paged_attention_status(None, None) == EINVAL
    assert attention(lib, kv, structs(max_new=129)[1]) == EINVAL
    assert lib.ds4g_paged_attention_workspace_bytes(C.byref(kv), C.byref(b), 7) == 0
    assert attention(lib, kv, structs(n_seqs=0, n_tokens=0)[1]) == OK
    assert attention(lib, kv, structs(start=None, n_tokens=3, max_new=2)[1]) == EINVAL
    assert attention(lib, kv, structs(start=None, n_tokens=2, max_new=1)[1]) == EINVAL


def test_probs_refuses(lib):
    f = lib.ds4g_probs
    assert f(None, 10, 1, 10, 1.0, 4096, 10, None) == EINVAL
    assert f(4096, 10, 1, 10, 1.0, None, 10, None) == EINVAL
    assert f(4096, 9, 1, 10, 1.0, 8192, 10, None) == EINVAL
    assert f(4096, 10, 1, 10, 1.0, 8192, 9, None) == EINVAL
    assert f(4096, 10, -1, 10, 1.0, 8192, 10, None) == EINVAL
    assert f(4096, 10, 1, 0, 1.0, 8192, 10, None) == EINVAL
    assert f(4096, 10, 1, 10, float("nan"), 8192, 10, None) == EINVAL
    assert f(4096, 10, 2, 10, 1.0, 4096, 12, None) == EINVAL
    assert f(4096, 1 << 21, 1, (1 << 20) + 1, 1.0, 8192, 1 << 21, None) == ESIZE
    assert f(None, 10, 0, 10, 1.0, None, 10, None) == OK


def test_verify_refuses(lib):
    def call(p=4096, ps=300, pp=100, q=4096, qs=200, qp=100, d=4096, nd=None, u=4096, b=2, D=2, n=100, a=4096, t=4096):
        return lib.ds4g_verify_draft(p, ps, pp, q, qs, qp, d, nd, u, b, D, n, a, t, None)
    for bad in (dict(p=None), dict(pp=99), dict(ps=99), dict(qp=99), dict(qs=10), dict(d=None), dict(u=None), dict(b=-1),
                dict(D=-1), dict(D=65), dict(n=0), dict(a=None), dict(t=None)):
        assert call(**bad) == EINVAL, bad
    assert call(n=(1 << 20) + 1) == ESIZE
    assert call(b=0, p=None) == OK


def test_the_binding_refuses_tensors_that_do_not_fit():
    import prefill_decode_layer_gb300 as pdl
    k = torch.zeros(4, 8, 2, 64)
    table, length = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    E = pdl.Ds4gError
    for a, b in ((k, k[:3]), (k, k.double()), (k.double(), k.double()), (k[0], k[0]), (k, k.transpose(0, 1).contiguous()),
                 (k.transpose(2, 3), k.transpose(2, 3))):
        with pytest.raises(E):
            pdl.PagedKV(a, b)
    for args in ((table.long(), length), (table, length.long()), (table[:2], length), (table, length, length),
                 (table.t().contiguous().t(), length), (table[:1].expand(3, 2), length), (table, torch.zeros(6, dtype=torch.int32)[::2])):
        with pytest.raises(E):
            pdl.PagedBatch(*args)
    with pytest.raises(E):
        pdl.Rope(torch.zeros(4, 3))
    kv, batch = pdl.PagedKV(k, k.clone()), pdl.PagedBatch(table, length)
    x, q = torch.zeros(3, 2, 64), torch.zeros(3, 4, 64)
    ws = torch.zeros(16, dtype=torch.uint8)
    for args in ((x[:2], x), (x, x.bfloat16()), (x, torch.zeros(3, 2, 32)), (x.double(), x.double()),
                 (x, x, None, q), (x, x, None, q, q[:, :2]), (x, x, None, q.bfloat16(), q.bfloat16())):
        with pytest.raises(E):
            pdl.paged_append(kv, batch, *args)
    for args in ((q, q[:2]), (q, q.bfloat16()), (q.double(), q.double()), (q[..., :32], q[..., :32])):
        with pytest.raises(E):
            pdl.paged_attention(kv, batch, *args, ws)
    with pytest.raises(E):
        pdl.paged_attention(kv, batch, q, q.clone(), ws[:1].expand(1 << 30))
    z = torch.zeros(2, 10)
    for args in ((z, z.double()), (z[0], z[0]), (z, torch.zeros(10, 2).t())):
        with pytest.raises(E):
            pdl.probs(args[0], 1.0, args[1])
    p, d, u = torch.zeros(2, 3, 10), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    a = torch.zeros(2, dtype=torch.int32)
    for args in ((p, p, d, u, a, u), (p, None, d.long(), u, a, u), (p, None, d, d, a, u), (p.double(), None, d, u, a, u),
                 (p, None, d, u, u, u), (p[0], None, d, u, a, u)):
        with pytest.raises(E):
            pdl.verify_draft(*args)
