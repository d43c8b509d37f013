"""Plain paged cache without a GPU: layouts, and what the C ABI and the binding
refuse before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from decode_attention_strided_b200 import build as dkv_build
from decode_attention_strided_b200 import deltakv as dkv
from kv_util import KvCase, attend64, evict64, few_bounds, few_queries, unit_rows

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    dkv_build.build()
    return dkv.load_library()


def _plan(**kw):
    base = dict(batch=2, kv_heads=2, q_heads=8, d_h=128, max_T=1000, stride_s=16, k=4, d_c=32, hidden=256)
    base.update(kw)
    return dkv.plan(dkv.Config(**base))


def test_layout(lib):
    p = _plan()
    lay = dkv.kv_pool_layout(p, 10, 64, 1000)
    assert lay["k_offset"] == 0 and lay["v_offset"] == 10 * 64 * 128 * 2 and lay["pool_bytes"] == 2 * lay["v_offset"]
    assert lay["weights_workspace_bytes"] >= 4 * 1000 * 4 * 4  # a logit per pair, row and head
    assert lay["workspace_bytes"] >= 2 * 4 * 500 * 4           # both lists of moves
    assert dkv.kv_pool_layout(_plan(dtype=dkv.F32), 10, 64, 1)["v_offset"] == 10 * 64 * 128 * 4
    # no part of the workspace depends on the pool, all of it on max_len
    assert dkv.kv_pool_layout(p, 99999, 16, 1000)["workspace_bytes"] == lay["workspace_bytes"]
    assert dkv.kv_pool_layout(p, 10, 64, 10)["weights_workspace_bytes"] < lay["weights_workspace_bytes"]


@pytest.mark.parametrize("args,code", [
    ((0, 64, 10), INVALID), ((-3, 64, 10), INVALID), ((4, 64, 0), INVALID), ((4, 64, 1001), INVALID),
    ((4, 8, 10), UNSUPPORTED), ((4, 48, 10), UNSUPPORTED), ((4, 512, 10), UNSUPPORTED), ((4, 0, 10), UNSUPPORTED),
    ((4, -16, 10), UNSUPPORTED), ((2**31 - 1, 16, 10), UNSUPPORTED), ((2**27, 16, 10), UNSUPPORTED),
])
def test_layout_refuses(lib, args, code):
    with pytest.raises(dkv.DeltaKVError) as e:
        dkv.kv_pool_layout(_plan(), *args)
    assert e.value.code == code
    assert lib.deltakv_kv_pool_layout(None, 4, 64, 10, ctypes.byref(dkv._KvLayout())) == INVALID
    p = _plan()
    assert lib.deltakv_kv_pool_layout(p.handle, 4, 64, 10, None) == INVALID


FAKE = 1 << 20  # never dereferenced: validation fails first


def _view(**kw):
    v = dict(pool=FAKE, n_pages=64, tokens_per_page=64, page_table=FAKE, max_pages=16, lens=FAKE, max_len=1000)
    v.update(kw)
    return dkv._KvCache(*v.values())


VIEWS = [
    (dict(pool=None), INVALID), (dict(page_table=None), INVALID), (dict(lens=None), INVALID),
    (dict(n_pages=0), INVALID), (dict(max_len=0), INVALID), (dict(max_len=1001), INVALID),
    (dict(max_pages=15), INVALID), (dict(tokens_per_page=24), UNSUPPORTED), (dict(n_pages=2**25), UNSUPPORTED),
    (dict(pool=FAKE + 8), ALIGNMENT), (dict(page_table=FAKE + 2), ALIGNMENT), (dict(lens=FAKE + 1), ALIGNMENT),
]


def _calls(lib, p, view, ws=FAKE, nbytes=1 << 40):
    s3, s2 = (ctypes.c_int64 * 3)(4096, 2048, 128), (ctypes.c_int64 * 2)(1024, 128)
    v = None if view is None else ctypes.byref(view)
    return [
        lib.deltakv_kv_append(p, v, 3, FAKE, FAKE, s3, None, None, None, None, 0, None, ws, nbytes, None),
        lib.deltakv_kv_decode_attention(p, v, FAKE, s2, FAKE, s2, None, None, 0, 1.0, ws, nbytes, None),
        lib.deltakv_kv_evict(p, v, FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, 1000, FAKE, ws, nbytes, None),
    ]


@pytest.mark.parametrize("change,code", VIEWS)
def test_calls_refuse_a_bad_cache(lib, change, code):
    p = _plan()
    assert _calls(lib, p.handle, _view(**change)) == [code] * 3


def test_calls_refuse_missing_plan_cache_and_workspace(lib):
    p = _plan()
    assert _calls(lib, None, _view()) == [INVALID] * 3
    assert _calls(lib, p.handle, None) == [INVALID] * 3
    assert _calls(lib, p.handle, _view(), ws=None) == [INVALID] * 3
    assert _calls(lib, p.handle, _view(), ws=FAKE + 4) == [ALIGNMENT] * 3
    assert _calls(lib, p.handle, _view(), nbytes=255) == [WORKSPACE] * 3
    lay = dkv.kv_pool_layout(p, 64, 64, 1000)
    s2 = (ctypes.c_int64 * 2)(1024, 128)
    v = ctypes.byref(_view())
    assert lib.deltakv_kv_decode_attention(p.handle, v, FAKE, s2, FAKE, s2, None, FAKE, 1000, 1.0, FAKE,
                                           lay["weights_workspace_bytes"] - 256, None) == WORKSPACE


def test_append_refuses(lib):
    plan, v = _plan(), ctypes.byref(_view())
    p = plan.handle

    def call(n_new=3, K=FAKE, V=FAKE, st=(4096, 2048, 128), nt=None, fp=None, w=None, pos=None, cap=1000, tw=None):
        return lib.deltakv_kv_append(p, v, n_new, K, V, (ctypes.c_int64 * 3)(*st), nt, fp, w, pos, cap, tw, FAKE,
                                     1 << 40, None)

    assert call(n_new=-1) == INVALID
    assert lib.deltakv_kv_append(p, None, 0, None, None, None, None, None, None, None, 0, None, None, 0, None) == OK
    assert call(K=None) == INVALID and call(V=None) == INVALID
    assert call(pos=FAKE) == INVALID                                  # positions without first_pos
    assert call(w=FAKE, cap=999) == INVALID and call(pos=FAKE, fp=FAKE, cap=999) == INVALID
    assert call(st=(4096, 2048, 64)) == INVALID                       # token stride below d_h
    assert call(st=(4096, 2048, 129)) == ALIGNMENT and call(st=(-4096, 2048, 128)) == ALIGNMENT
    assert call(K=FAKE + 8) == ALIGNMENT and call(w=FAKE + 4) == ALIGNMENT
    assert call(nt=FAKE + 2) == ALIGNMENT and call(fp=FAKE + 1) == ALIGNMENT and call(tw=FAKE + 2) == ALIGNMENT


def test_decode_refuses(lib):
    plan, v = _plan(), ctypes.byref(_view())
    p = plan.handle

    def call(q=FAKE, qs=(1024, 128), out=FAKE, os_=(1024, 128), lse=None, w=None, cap=1000, decay=1.0):
        return lib.deltakv_kv_decode_attention(p, v, q, (ctypes.c_int64 * 2)(*qs), out, (ctypes.c_int64 * 2)(*os_),
                                               lse, w, cap, decay, FAKE, 1 << 40, None)

    assert call(q=None) == INVALID and call(out=None) == INVALID
    assert call(qs=(-1024, 128)) == INVALID and call(os_=(1024, -128)) == INVALID
    assert call(qs=(1024, 124)) == ALIGNMENT and call(os_=(1024, 130)) == ALIGNMENT
    assert call(q=FAKE + 2) == ALIGNMENT and call(out=FAKE + 4) == ALIGNMENT and call(lse=FAKE + 2) == ALIGNMENT
    assert call(w=FAKE, cap=999) == INVALID and call(w=FAKE + 4) == ALIGNMENT
    for bad in (-0.5, math.nan, math.inf):
        assert call(w=FAKE, decay=bad) == INVALID


def test_evict_refuses(lib):
    plan, v = _plan(), ctypes.byref(_view())
    p = plan.handle

    def call(budget=FAKE, first=0, recent=0, ptrs=(FAKE,) * 4, cap=1000, lo=FAKE):
        return lib.deltakv_kv_evict(p, v, budget, first, recent, *ptrs, cap, lo, FAKE, 1 << 40, None)

    assert call(budget=None) == INVALID and call(lo=None) == INVALID
    for i in range(4):
        assert call(ptrs=tuple(None if j == i else FAKE for j in range(4))) == INVALID
        assert call(ptrs=tuple(FAKE + 4 if j == i else FAKE for j in range(4))) == ALIGNMENT
    assert call(first=-1) == INVALID and call(recent=-1) == INVALID and call(first=500, recent=501) == INVALID
    assert call(first=2**31 - 1, recent=2**31 - 1) == INVALID
    assert call(cap=999) == INVALID
    assert call(budget=FAKE + 2) == ALIGNMENT and call(lo=FAKE + 2) == ALIGNMENT


def _cpu_cache(p, page=64, dtype=torch.bfloat16, B=2, H=2, per=16):
    return (torch.zeros(2, 64, page, 128, dtype=dtype), torch.zeros(B, H, per, dtype=torch.int32),
            torch.zeros(B, H, dtype=torch.int32))


def test_binding_refuses_a_cache_of_other_shapes(lib):
    p = _plan()
    pool, table, lens = _cpu_cache(p)
    dkv.KVCache(p, pool, table, lens)
    for bad in ((pool.float(), table, lens), (pool[0], table, lens), (pool.transpose(0, 1), table, lens),
                (pool, table.long(), lens), (pool, table[0], lens), (pool, table, lens[0]),
                (pool, table, lens.float()), (pool, table[:, :, ::2], lens), (pool[..., :64], table, lens)):
        with pytest.raises(ValueError):
            dkv.KVCache(p, *bad)
    with pytest.raises(dkv.DeltaKVError):
        dkv.KVCache(p, torch.zeros(2, 4, 24, 128, dtype=torch.bfloat16), table, lens)


def test_binding_refuses_what_the_kernels_would_misread(lib):
    """Types, shapes and layouts first; a cache that is not on the current
    CUDA device last, so none of these calls reaches the library."""
    p = _plan()
    cache = dkv.KVCache(p, *_cpu_cache(p))
    ws = torch.zeros(16, dtype=torch.uint8)
    q, out = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 128)
    w, pos = torch.zeros(2, 2, 1000), torch.zeros(2, 2, 1000, dtype=torch.int32)
    bud = torch.zeros(2, 2, dtype=torch.int32)
    K = torch.zeros(2, 2, 5, 128, dtype=torch.bfloat16)
    for kw in (dict(), dict(q=q.float()), dict(q=q[:, :4]), dict(out=out.bfloat16()), dict(w=w[..., 0]),
               dict(w=w.double()), dict(lse=torch.zeros(2, 4)), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            dkv.kv_decode_attention(p, cache, 10, kw.get("q", q), kw.get("out", out), ws, weights=kw.get("w"),
                                    lse=kw.get("lse"))
    for kw in (dict(), dict(K=K.float()), dict(K=K[..., :64]), dict(K=K[:1]), dict(V=K[:, :, :4]),
               dict(nt=torch.zeros(3, dtype=torch.int32)), dict(nt=torch.zeros(2)), dict(fp=torch.zeros(2)),
               dict(tw=torch.zeros(2, 2, 4)), dict(w=w, pos=pos[..., :999].contiguous(), fp=bud[0]),
               dict(V=K.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            dkv.kv_append(p, cache, 10, kw.get("K", K), kw.get("V", K), ws, n_tokens=kw.get("nt"),
                          first_pos=kw.get("fp"), weights=kw.get("w"), pos=kw.get("pos"), token_weights=kw.get("tw"))
    for kw in (dict(), dict(bud=bud.long()), dict(bud=bud[0]), dict(w=w.double()), dict(pos=pos.long()),
               dict(wo=w[..., :999]), dict(po=pos.float()), dict(lo=bud[0])):
        with pytest.raises(ValueError):
            dkv.kv_evict(p, cache, 10, kw.get("bud", bud), kw.get("w", w), kw.get("pos", pos), ws,
                         weights_out=kw.get("wo"), pos_out=kw.get("po"), lens_out=kw.get("lo"))
    # what does not fit 32 bits is refused, not wrapped round
    for kw in (dict(max_len=2**32 + 10), dict(max_len=0), dict(n_first=2**32), dict(n_recent=-1)):
        with pytest.raises((ValueError, dkv.DeltaKVError)) as e:
            dkv.kv_evict(p, cache, kw.pop("max_len", 10), bud, w, pos, ws, **kw)
        assert e.type is dkv.DeltaKVError and e.value.code == INVALID
    other = _plan(q_heads=4)
    with pytest.raises(ValueError):
        dkv.kv_evict(other, cache, 10, bud, w, pos, ws)


def test_the_plain_implementations():
    """The tests' own 64-bit forms on examples small enough to check by hand."""
    out, lse, p = attend64(np.zeros((1, 4)), np.ones((2, 4)), np.array([[1.0, 0, 0, 0], [3.0, 0, 0, 0]]))
    assert out[0, 0] == 2.0 and abs(lse[0] - math.log(2)) < 1e-15 and (p == 0.5).all()
    # rows 1 and 4 are guarded (position 0, and the last one); of the others 3 is the heaviest, and 0 wins its
    # tie with 2: kept 0, 1, 3, 4 and so rows 3, 4 fill row 2 and stay
    m, src = evict64(5, 4, 1, 1, np.array([0.5, 0, 0.5, 0.9, 0], np.float32), np.array([3, 0, 4, 6, 8]))
    assert m == 4 and src.tolist() == [0, 1, 4, 3]
    m, src = evict64(3, 9, 0, 0, np.zeros(3, np.float32), np.arange(3))
    assert m == 3 and src.tolist() == [0, 1, 2]
    m, src = evict64(4, 2, 0, 0, np.array([np.nan, -np.inf, np.nan, 1], np.float32), np.arange(4))
    assert m == 2 and src.tolist() == [3, 1]


def _pointers(view):
    return view.pool, view.n_pages, view.tokens_per_page, view.page_table, view.max_pages, view.lens, view.max_len


def _of(pool, table, lens, max_len):
    return (pool.data_ptr(), pool.shape[1], pool.shape[2], table.data_ptr(), table.shape[2], lens.data_ptr(), max_len)


def test_a_cache_passes_the_tensors_it_shows(lib):
    """Assigning pool, page_table or lens takes effect, as does replacing the
    storage of one; what the constructor refuses is refused, with the cache
    left as it was."""
    p = _plan()
    pool, table, lens = _cpu_cache(p)
    cache = dkv.KVCache(p, pool, table, lens)
    assert _pointers(cache._view(10)) == _of(pool, table, lens, 10)
    held = cache._view(10)
    cache.lens = more = lens + 1
    assert cache.lens is more and _pointers(cache._view(10)) == _of(pool, table, more, 10)
    assert _pointers(held) == _of(pool, table, lens, 10)  # a view in another thread's hands stays what it was
    cache.page_table = wide = torch.zeros(2, 2, 20, dtype=torch.int32)
    cache.pool = small = torch.zeros(2, 9, 128, 128, dtype=torch.bfloat16)
    for max_len in (1000, 10, 10):
        assert _pointers(cache._view(max_len)) == _of(small, wide, more, max_len)
    for name, bad in (("pool", small.float()), ("pool", small[0]), ("pool", None), ("page_table", wide.long()),
                      ("page_table", wide[..., ::2]), ("page_table", 3), ("lens", lens[0]), ("lens", lens.float()),
                      ("lens", "lens")):
        with pytest.raises((ValueError, TypeError)):
            setattr(cache, name, bad)
        assert _pointers(cache._view(10)) == _of(small, wide, more, 10)
        assert cache.pool is small and cache.page_table is wide and cache.lens is more
    moved = torch.ones(2, 2, dtype=torch.int32)
    more.set_(moved)
    assert _pointers(cache._view(10)) == _of(small, wide, moved, 10)
    bigger = torch.zeros(2, 30, 128, 128, dtype=torch.bfloat16)
    small.data = bigger
    assert _pointers(cache._view(10)) == _of(bigger, wide, moved, 10)
    more.set_(torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        cache._view(10)


@pytest.mark.parametrize("batch,max_len", [(2**27 - 1, 256), (2**27 - 64, 256), (2**21 - 1, 2**14)])
def test_calls_refuse_more_rows_than_their_unit_counts_hold(lib, batch, max_len):
    """A little below 2^31 units of 16 rows the look ahead past the last unit
    would wrap round: refused before any launch."""
    p = _plan(batch=batch, kv_heads=1, q_heads=1, max_T=max_len, dtype=dkv.F32)
    view = _view(max_len=max_len, max_pages=max_len // 64)
    got = _calls(lib, p.handle, view)[:2]
    got.append(lib.deltakv_kv_evict(p.handle, ctypes.byref(view), FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, max_len, FAKE,
                                    FAKE, 1 << 40, None))
    assert got == [UNSUPPORTED] * 3


@pytest.mark.parametrize("B,Hq,strides,code", [
    (2, 8, (0, 128), INVALID), (2, 8, (1024, 0), INVALID), (2, 8, (0, 0), INVALID), (2, 8, (128, 128), INVALID),
    (2, 8, (1020, 128), INVALID), (2, 8, (1024, 124), INVALID), (2, 8, (64, 1024), INVALID),
    (2, 8, (128, 252), INVALID), (1, 8, (0, 124), INVALID), (2, 1, (124, 0), INVALID),
    (2, 8, (2**60, 2**60), INVALID),
    # apart: the call goes on to its unaligned query
    (2, 8, (1024, 128), ALIGNMENT), (2, 8, (2**60, 128), ALIGNMENT), (2, 8, (128, 256), ALIGNMENT),
    (2, 8, (128, 2**60), ALIGNMENT), (1, 8, (0, 128), ALIGNMENT), (1, 8, (2**60, 132), ALIGNMENT),
    (2, 1, (128, 0), ALIGNMENT), (1, 1, (0, 0), ALIGNMENT),
])
def test_decode_refuses_outputs_that_overlap(lib, B, Hq, strides, code):
    """Rows of out that share elements would be written by several heads at
    once; a broadcast q is read, and stays allowed."""
    p = _plan(batch=B, kv_heads=1, q_heads=Hq)
    two = ctypes.c_int64 * 2
    assert lib.deltakv_kv_decode_attention(p.handle, ctypes.byref(_view()), FAKE + 2, two(0, 0), FAKE, two(*strides),
                                           None, None, 0, 1.0, FAKE, 1 << 40, None) == code
    rows = sorted(b * strides[0] + h * strides[1] for b in range(B) for h in range(Hq))
    assert (code == ALIGNMENT) == all(y - x >= 128 for x, y in zip(rows, rows[1:]))


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


@pytest.mark.parametrize("terms", [3, 2, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_the_counted_bounds_tell_a_missing_weight_term(terms, d):
    """A weight of three bfloat16 terms stays inside few_bounds, one that lost
    its third or its second does not."""
    c = KvCase([[2] * 6] * 8, 6, d=d)
    q = few_queries(c).double().numpy()
    g = torch.Generator().manual_seed(11)
    worst = 0.0
    for b in range(c.B):
        for h in range(c.H):
            K, V = (torch.randn(2, d, generator=g).bfloat16().double().numpy() for _ in range(2))
            qh = q[b, h:h + 1]
            ref, _, p = attend64(qh, K, V)
            x = (qh @ K.T / math.sqrt(d))[0]
            w = np.exp(x - x.max()).astype(np.float32)
            rest, got = w.copy(), np.zeros(d)
            for _ in range(terms):
                t = _bf16(rest)
                got += t.astype(np.float64) @ V
                rest = rest - t
            tol, _, _ = few_bounds(qh, K, V, p, unit_rows(c))
            worst = max(worst, float((np.abs(got / w.astype(np.float64).sum() - ref[0]) / tol[0]).max()))
    assert worst < 0.5 if terms == 3 else worst > 1.5
