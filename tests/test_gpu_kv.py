"""Plain paged cache on the GPU: append, decode attention and eviction against
plain implementations in 64 bits (kv_util)."""
import dataclasses

import numpy as np
import pytest
import torch

from decode_attention_strided_b200 import deltakv as dkv
from kv_util import KvCase, Setup, attend64, attend_bounds, evict64, few_bounds, few_queries, unit_rows

pytestmark = pytest.mark.gpu

BOUNDS = 7  # ERR_DEVICE_BOUNDS


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from decode_attention_strided_b200 import build
    build.build()


# ---- attention

def _attend(s: Setup, weights=True, decay=1.0, lse=True, max_len=None):
    c = s.c
    out = torch.full((c.B, c.Hq, c.d), float("nan"), device="cuda")
    ls = torch.full((c.B, c.Hq), float("nan"), device="cuda") if lse else None
    w = s.w.cuda() if weights else None
    dkv.kv_decode_attention(s.p, s.cache, max_len or c.n, s.q.cuda(), out, s.ws, weights=w, decay=decay, lse=ls)
    return out, ls, w


def _check_attend(s: Setup, out, lse, w, decay=1.0, pairs=None):
    c = s.c
    out = out.cpu().double().numpy()
    w0 = s.w.double().numpy()
    for b in range(c.B):
        for h in range(c.H):
            if pairs is not None and (b, h) not in pairs:
                continue
            n, g0 = c.lens[b][h], h * c.G
            q = s.q[b, g0:g0 + c.G].double().numpy()
            K, V = s.K[b, h].double().numpy(), s.V[b, h].double().numpy()
            ref, ref_lse, p = attend64(q, K, V)
            got = out[b, g0:g0 + c.G]
            if n == 0:
                assert (got == 0).all()
                if lse is not None:
                    assert (lse[b, g0:g0 + c.G] == -np.inf).all()
                if w is not None:
                    assert torch.equal(w[b, h].cpu(), s.w[b, h])
                continue
            tol, tol_lse, rel = attend_bounds(q, K, V, p)
            err = np.abs(got - ref)
            assert (err <= tol).all(), (b, h, n, float((err / tol).max()))
            if lse is not None:
                e = np.abs(lse[b, g0:g0 + c.G].cpu().double().numpy() - ref_lse)
                assert (e <= tol_lse).all(), (b, h, n, float((e / tol_lse).max()))
            if w is not None:
                want = decay * w0[b, h, :n] + p.sum(axis=0)
                e = np.abs(w[b, h, :n].cpu().double().numpy() - want)
                lim = (rel[:, None] * p).sum(axis=0) + 2.0 ** -22 * want
                assert (e <= lim).all(), (b, h, n, float((e / lim).max()))
                assert torch.equal(w[b, h, n:].cpu(), s.w[b, h, n:])  # rows behind the last


ATTEND = [
    ("one_row", KvCase([[1]], 1)),
    ("sixteen", KvCase([[16, 15, 17]], 3, page=16)),
    ("g8_d64", KvCase([[1000, 3], [64, 129]], 16, d=64, page=32)),
    ("g8_d128", KvCase([[1000, 31], [255, 257]], 16, page=256)),
    ("g3", KvCase([[700, 1, 0]], 9, page=128)),
    ("g5_d64", KvCase([[333], [2047]], 5, d=64, page=16)),
    ("g7", KvCase([[130, 64]], 14)),
    ("empty_between", KvCase([[0, 200], [0, 0], [77, 0]], 8)),
    ("all_empty", KvCase([[0, 0]], 4, max_len=40)),
    ("long", KvCase([[20011, 5]], 8)),
    ("many_pairs", KvCase([[(37 * i + 11 * h) % 300 for h in range(8)] for i in range(40)], 32)),
    ("peaked", KvCase([[3001, 900]], 8, scale=6.0)),
    ("mostly_empty", KvCase([[300 if h in (3, 290, 580, 599) else 0 for h in range(600)]], 600, d=64, page=32)),
    ("full_clusters", KvCase([[500, 33, 90, 1, 0, 256, 255, 511]] * 4, 32, page=32)),
    ("f32", KvCase([[1000, 3], [64, 129]], 16, dtype=dkv.F32)),
    ("f32_d64_g1", KvCase([[2049, 16, 0]], 3, d=64, page=16, dtype=dkv.F32)),
    ("f32_g3", KvCase([[5003, 100]], 6, page=32, dtype=dkv.F32, scale=3.0)),
    ("code4_plan", KvCase([[100, 300]], 8, dtype=dkv.BF16_CODE4)),
]


@pytest.mark.parametrize("name,case", ATTEND, ids=[n for n, _ in ATTEND])
@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("form", ["as_is", "cut"])
def test_attend(name, case, weights, form):
    """Short rows take a cluster per pair; a bound far above the lengths
    (form "cut") makes the same rows go through the cut over the whole GPU."""
    if form == "cut":
        if case.B * case.H > 32:
            pytest.skip("goes through the cut as it is")
        case = dataclasses.replace(case, max_len=40000)
    s = Setup(case)
    decay = 0.75 if case.seed == 0 and case.G % 2 else 1.0
    out, lse, w = _attend(s, weights, decay)
    assert dkv.device_status(s.p, s.ws) == 0
    _check_attend(s, out, lse, w, decay)


@pytest.mark.parametrize("longest", [9001, 901], ids=["cut", "cluster"])
def test_attend_is_deterministic_and_optional_outputs_change_nothing(longest):
    s = Setup(KvCase([[longest, 40], [300, 700]], 8))
    first = _attend(s)
    for _ in range(3):
        again = _attend(s)
        for a, b in zip(first, again):
            assert torch.equal(a, b)
    out, _, _ = _attend(s, weights=False, lse=False)
    assert torch.equal(out, first[0])


def test_attend_max_len_above_the_lengths():
    """max_len bounds the lengths; it need not be the longest."""
    s = Setup(KvCase([[50, 300]], 4, max_len=4000))
    out, lse, w = _attend(s)
    assert dkv.device_status(s.p, s.ws) == 0
    _check_attend(s, out, lse, w)


def test_attend_strided_queries_and_outputs():
    c = KvCase([[500, 17], [64, 900]], 8)
    s = Setup(c)
    q = torch.zeros(c.Hq, c.B, 2 * c.d, dtype=c.torch_dtype(), device="cuda")
    q[:, :, :c.d] = s.q.cuda().transpose(0, 1)
    buf = torch.full((c.Hq, c.B, c.d + 4), 7.0, device="cuda")
    out = buf[:, :, :c.d].transpose(0, 1)
    dkv.kv_decode_attention(s.p, s.cache, c.n, q[:, :, :c.d].transpose(0, 1), out, s.ws)
    assert dkv.device_status(s.p, s.ws) == 0
    _check_attend(s, out, None, None)
    assert (buf[:, :, c.d:] == 7.0).all()


@pytest.mark.parametrize("max_len", [0, 40000], ids=["cluster", "cut"])
@pytest.mark.parametrize("Hq,dtype", [(4, dkv.BF16), (8, dkv.BF16), (16, dkv.BF16), (4, dkv.F32)])
def test_attend_infinities_and_nan_in_valid_rows_stay_in_their_pair(max_len, Hq, dtype):
    c = KvCase([[100, 100], [90, 30]], Hq, max_len=max_len, dtype=dtype)
    s = Setup(c)
    ids = s.table_host
    s.pool[0, ids[0, 0, 1], 3, 5] = float("nan")
    s.pool[1, ids[1, 1, 0], 2, 7] = float("inf")
    out, lse, w = _attend(s)
    assert dkv.device_status(s.p, s.ws) == 0
    _check_attend(s, out, lse, w, pairs=[(0, 1), (1, 0)])
    G = Hq // 2
    assert torch.isnan(out[0, :G]).all()
    got = out[1, G:]
    assert torch.isinf(got[:, 7]).all() and torch.isfinite(got[:, :7]).all() and torch.isfinite(got[:, 8:]).all()


@pytest.mark.parametrize("max_len", [0, 40000], ids=["cluster", "cut"])
@pytest.mark.parametrize("Hq,dtype", [(4, dkv.BF16), (6, dkv.BF16), (16, dkv.BF16), (4, dkv.F32)])
def test_attend_logits_of_minus_infinity_and_nothing_but_nan(max_len, Hq, dtype):
    """A pair whose logits are all -inf counts as one without rows, one where
    some are is its other rows, and one that holds only NaN gives NaN."""
    c = KvCase([[100, 100], [40, 1]], Hq, max_len=max_len, dtype=dtype)
    s = Setup(c)
    G = c.G
    s.q.abs_()
    dead = torch.zeros(100, dtype=torch.bool)
    dead[::3] = dead[64:90] = True
    for pair, rows in (((0, 0), torch.ones(100, dtype=torch.bool)), ((0, 1), dead)):
        at = rows.nonzero()[:, 0]
        s.pool[0, s.table_host[pair][at // c.page].long(), at % c.page] = float("-inf")
    s.pool[0, s.table_host[1, 1, 0], 0] = float("nan")
    out, lse, w = _attend(s, decay=0.5)
    assert dkv.device_status(s.p, s.ws) == 0
    _check_attend(s, out, lse, w, 0.5, pairs=[(1, 0)])
    assert (out[0, :G] == 0).all() and (lse[0, :G] == float("-inf")).all()
    assert torch.equal(w[0, 0].cpu()[:100], 0.5 * s.w[0, 0, :100])
    for x in (out[1, G:], lse[1, G:], w[1, 1, :1]):
        assert torch.isnan(x).all()
    q, K, V = (x.double().numpy() for x in (s.q[0, G:], s.K[0, 1][~dead], s.V[0, 1][~dead]))
    ref, ref_lse, p = attend64(q, K, V)
    tol, tol_lse, rel = attend_bounds(q, K, V, p)
    assert (np.abs(out[0, G:].cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse[0, G:].cpu().numpy() - ref_lse) <= tol_lse).all()
    want = torch.zeros(100, dtype=torch.float64)
    want[~dead] = torch.from_numpy(p.sum(axis=0))
    want += 0.5 * s.w[0, 1, :100].double()
    assert ((w[0, 1].cpu()[:100].double() - want).abs() <= float(rel.max()) * want + 2.0 ** -22 * want).all()


@pytest.mark.parametrize("max_len,page", [(300, 64), (40000, 64), (40000, 16), (300, 16)])
def test_attend_bad_page_is_skipped_and_reported(max_len, page):
    c = KvCase([[300, 200], [300, 64]], 8, max_len=max_len, page=page)
    s = Setup(c)
    first, last = (64, 128) if page == 64 else (16, 32)  # the rows that are lost
    gone = last - first
    for bad in (-1, s.pool.shape[1]):
        t = s.table_host.clone()
        t[0, 0, 1] = bad
        s.table.copy_(t)
        out, lse, w = _attend(s)
        assert dkv.device_status(s.p, s.ws) == BOUNDS
        assert dkv.device_status(s.p, s.ws) == 0
        # the skipped rows get no weight; the check below has the others in order
        assert torch.equal(w[0, 0, first:last].cpu(), s.w[0, 0, first:last])
        r = Setup.__new__(Setup)
        r.__dict__.update(s.__dict__)
        r.c = dataclasses.replace(c, lens=[[300 - gone, 200], [300, 64]], max_len=c.n)

        def without(x):
            return torch.cat([x[:first], x[last:300]])

        r.K, r.V, r.w = dict(s.K), dict(s.V), s.w.clone()
        r.K[0, 0], r.V[0, 0] = without(s.K[0, 0]), without(s.V[0, 0])
        r.w[0, 0, :300 - gone] = without(s.w[0, 0])
        wr = w.clone()
        wr[0, 0, :300 - gone] = without(w[0, 0])
        wr[0, 0, 300 - gone:] = r.w[0, 0, 300 - gone:].cuda()
        _check_attend(r, out, lse, wr)


@pytest.mark.parametrize("max_len", [0, 40000], ids=["cluster", "cut"])
def test_attend_all_pages_bad_gives_an_empty_row(max_len):
    s = Setup(KvCase([[40, 50]], 2, max_len=max_len))
    s.table[0, 0] = -5
    out, lse, w = _attend(s)
    assert dkv.device_status(s.p, s.ws) == BOUNDS
    assert (out[0, 0] == 0).all() and lse[0, 0] == -float("inf")
    assert torch.equal(w[0, 0].cpu(), s.w[0, 0])
    _check_attend(s, out, lse, w, pairs=[(0, 1)])


@pytest.mark.parametrize("max_len", [300, 40000], ids=["cluster", "cut"])
@pytest.mark.parametrize("bad", [-1, 40001, 2**31 - 1])
def test_attend_bad_length_is_an_empty_row_and_reported(bad, max_len):
    c = KvCase([[300, 200], [299, 64]], 8, max_len=max_len)
    s = Setup(c)
    s.lens[1, 0] = bad
    out, lse, w = _attend(s)
    assert dkv.device_status(s.p, s.ws) == BOUNDS
    assert (out[1, :4] == 0).all() and (lse[1, :4] == -float("inf")).all()
    assert torch.equal(w[1, 0].cpu(), s.w[1, 0])
    _check_attend(s, out, lse, w, pairs=[(0, 0), (0, 1), (1, 1)])


def test_attend_on_another_stream_and_in_two_graphs():
    """Captured and replayed with lengths that change between replays; two
    graphs, each with a workspace of its own, replayed on two streams."""
    cases = [KvCase([[3000, 120]], 8, seed=1), KvCase([[77, 2500]], 8, seed=2)]
    ss = [Setup(c) for c in cases]
    qs = [s.q.cuda() for s in ss]
    outs = [torch.empty(1, 8, 128, device="cuda") for _ in ss]
    ws = [s.w.cuda() for s in ss]
    graphs = []
    streams = [torch.cuda.Stream() for _ in ss]
    torch.cuda.synchronize()
    for i, s in enumerate(ss):
        with torch.cuda.stream(streams[i]):
            dkv.kv_decode_attention(s.p, s.cache, s.c.n, qs[i], outs[i], s.ws, weights=ws[i])
            torch.cuda.synchronize()
            _check_attend(s, outs[i], None, ws[i])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=streams[i]):
                dkv.kv_decode_attention(s.p, s.cache, s.c.n, qs[i], outs[i], s.ws, weights=ws[i])
            graphs.append(g)
    for lens in ([[3000, 120], [77, 2500]], [[1, 0], [60, 1999]], [[2999, 64], [0, 2500]]):
        for i, s in enumerate(ss):
            s.lens.copy_(torch.tensor([lens[i]], dtype=torch.int32))
            ws[i].copy_(s.w)
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i, s in enumerate(ss):
            assert dkv.device_status(s.p, s.ws) == 0
            t = Setup.__new__(Setup)
            t.__dict__.update(s.__dict__)
            t.c = KvCase([lens[i]], 8, max_len=s.c.n)
            t.K = {k: v[:lens[i][k[1]]] for k, v in s.K.items()}
            t.V = {k: v[:lens[i][k[1]]] for k, v in s.V.items()}
            _check_attend(t, outs[i], None, None)
            total = float((ws[i] - s.w.cuda()).sum())
            heads = sum(4 for n in lens[i] if n)
            assert abs(total - 3 * heads) < 1e-3 * max(1, heads)


# ---- append

def _append_ref(s, K, V, counts, first_pos, tok_w, w, pos, pool):
    c = s.c
    pool, w, pos = pool.clone(), w.clone(), pos.clone()
    for b in range(c.B):
        n = counts[b]
        for h in range(c.H):
            for t in range(n):
                r = c.lens[b][h] - n + t
                pg = int(s.table_host[b, h, r // c.page])
                pool[0, pg, r % c.page] = K[b, h, t]
                pool[1, pg, r % c.page] = V[b, h, t]
                w[b, h, r] = 0.0 if tok_w is None else tok_w[b, h, t]
                pos[b, h, r] = first_pos[b] + t
    return pool, w, pos


def _same(a, b):
    """Bit for bit (NaN included)."""
    v = torch.int32 if a.dtype == torch.float32 else torch.int16 if a.dtype == torch.bfloat16 else a.dtype
    return torch.equal(a.cpu().view(v), b.cpu().view(v))


APPEND = [
    ("one_token", KvCase([[1, 64], [65, 300]], 2), 1, None),
    ("block", KvCase([[40, 100], [90, 40], [200, 128]], 2, page=16), 40, [40, 0, 17]),
    ("f32", KvCase([[33, 47]], 2, page=32, dtype=dkv.F32), 33, None),
    ("f32_d64", KvCase([[33, 47], [9, 8]], 2, d=64, page=16, dtype=dkv.F32), 33, [30, 8]),
    ("d64", KvCase([[130, 131]], 2, d=64, page=256), 129, None),
]


@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("name,case,n_new,counts", APPEND, ids=[a[0] for a in APPEND])
def test_append(name, case, n_new, counts, layout):
    s = Setup(case)
    c = case
    g = torch.Generator().manual_seed(5)
    shape = (c.B, c.H, n_new, c.d) if layout == "bhtd" else (c.B, n_new, c.H, c.d)
    K, V = (torch.randn(*shape, generator=g).to(c.torch_dtype()) for _ in range(2))
    if layout == "bthd":
        K, V = K.transpose(1, 2), V.transpose(1, 2)
    cnt = counts or [n_new] * c.B
    first = [1000 * b + 3 for b in range(c.B)]
    tok_w = torch.rand(c.B, c.H, n_new, generator=g)
    cap = c.n + 5
    w0 = torch.rand(c.B, c.H, cap, generator=g)
    pos0 = torch.full((c.B, c.H, cap), -9, dtype=torch.int32)
    pool0 = s.pool.cpu()
    for tw in (tok_w, None):
        s.pool.copy_(pool0)
        w, pos = w0.cuda(), pos0.cuda()
        # .cuda() keeps the strides of a transposed view
        dkv.kv_append(s.p, s.cache, c.n, K.cuda(), V.cuda(), s.ws,
                      n_tokens=None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda"),
                      first_pos=torch.tensor(first, dtype=torch.int32, device="cuda"), weights=w, pos=pos,
                      token_weights=None if tw is None else tw.cuda())
        assert dkv.device_status(s.p, s.ws) == 0
        pool, wr, pr = _append_ref(s, K, V, cnt, first, tw, w0, pos0, pool0)
        assert _same(s.pool, pool) and _same(w, wr) and _same(pos, pr)
    # without the optional arrays only the rows change
    s.pool.copy_(pool0)
    dkv.kv_append(s.p, s.cache, c.n, K.cuda(), V.cuda(), s.ws,
                  n_tokens=None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda"))
    assert _same(s.pool, _append_ref(s, K, V, cnt, first, None, w0, pos0, pool0)[0])


def test_append_reports_bad_counts_lengths_and_pages():
    c = KvCase([[40, 100], [90, 70], [30, 20], [64, 65]], 2, page=16)
    s = Setup(c)
    K = torch.zeros(4, 2, 25, 128, dtype=torch.bfloat16, device="cuda")
    pool0 = s.pool.cpu()
    # sequence 0: negative; 1: above n_new; 2: above the second head's length only; 3: fine
    s.lens.copy_(s.lens_host)
    cnt = torch.tensor([-1, 26, 25, 2], dtype=torch.int32, device="cuda")
    dkv.kv_append(s.p, s.cache, c.n, K, K, s.ws, n_tokens=cnt)
    assert dkv.device_status(s.p, s.ws) == BOUNDS
    want = pool0.clone()
    for b, h, r0, n in ((2, 0, 5, 25), (3, 0, 62, 2), (3, 1, 63, 2)):
        for r in range(r0, r0 + n):
            want[:, s.table_host[b, h, r // 16], r % 16] = 0
    assert _same(s.pool, want)
    # a length out of range and a page out of range write nothing there
    s.pool.copy_(pool0)
    s.lens[0, 0] = c.n + 1
    s.table[3, 1, 4] = s.pool.shape[1]  # row 64
    cnt = torch.tensor([1, 0, 0, 2], dtype=torch.int32, device="cuda")
    dkv.kv_append(s.p, s.cache, c.n, K, K, s.ws, n_tokens=cnt)
    assert dkv.device_status(s.p, s.ws) == BOUNDS
    want = pool0.clone()
    for b, h, r in ((0, 1, 99), (3, 0, 62), (3, 0, 63), (3, 1, 63)):
        want[:, s.table_host[b, h, r // 16], r % 16] = 0
    assert _same(s.pool, want)


# ---- evict

def _evict_check(s, budget, n_first, n_recent, w, pos, in_place, whole=()):
    """Run an eviction and compare every byte with the definition."""
    c = s.c
    cap = w.shape[2]
    pool0 = s.pool.cpu()
    wd, pd = w.cuda(), pos.cuda()
    bud = torch.tensor(budget, dtype=torch.int32, device="cuda")
    if in_place:
        wo, po, lo = wd, pd, s.lens
        w_want, p_want = w.clone(), pos.clone()
    else:
        wo, po = torch.full_like(wd, -3.0), torch.full_like(pd, -4)
        lo = torch.full_like(s.lens, -5)
        w_want, p_want = wo.cpu(), po.cpu()
    dkv.kv_evict(s.p, s.cache, c.n, bud, wd, pd, s.ws, n_first=n_first, n_recent=n_recent, lens_out=lo,
                 weights_out=wo, pos_out=po)
    st = dkv.device_status(s.p, s.ws)
    pool_want = pool0.clone()
    l_want = torch.zeros(c.B, c.H, dtype=torch.int32)
    for b in range(c.B):
        for h in range(c.H):
            n = c.lens[b][h]
            if (b, h) in whole:
                m, src = n, np.arange(n)
            else:
                m, src = evict64(n, budget[b][h], n_first, n_recent, w[b, h, :n].numpy(), pos[b, h, :n].numpy())
            l_want[b, h] = m
            src = torch.from_numpy(src).long()
            w_want[b, h, :m] = w[b, h][src]
            p_want[b, h, :m] = pos[b, h][src]
            for r in range(m):
                q = int(src[r])
                if q != r:
                    pool_want[:, s.table_host[b, h, r // c.page], r % c.page] = \
                        pool0[:, s.table_host[b, h, q // c.page], q % c.page]
    assert torch.equal(lo.cpu(), l_want)
    assert _same(po, p_want)
    assert _same(wo, w_want)
    assert _same(s.pool, pool_want)
    if not in_place:
        assert _same(wd, w) and _same(pd, pos)
    return st


def _meta(c, seed, kind, cap=None):
    g = torch.Generator().manual_seed(seed)
    cap = cap or c.n
    if kind == "random":
        w = torch.exp(torch.randn(c.B, c.H, cap, generator=g) * 3)
    elif kind == "equal":
        w = torch.full((c.B, c.H, cap), 0.25)
    elif kind == "few":      # many ties at every threshold
        w = torch.randint(0, 4, (c.B, c.H, cap), generator=g).float() * 0.5
    elif kind == "close":    # differ in the last bits only
        w = (torch.randint(0, 50, (c.B, c.H, cap), generator=g) + 0x3f800000).to(torch.int32).view(torch.float32)
    else:                    # zeros of both signs, infinities, NaN of both signs, subnormals, negatives
        pick = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), -float("nan"), 1e-42, -1e-42,
                             3.4e38, -1.0, 1.0])
        w = pick[torch.randint(0, len(pick), (c.B, c.H, cap), generator=g)]
    pos = torch.stack([torch.randperm(3 * cap, generator=g)[:cap] for _ in range(c.B * c.H)])
    return w.contiguous(), pos.view(c.B, c.H, cap).to(torch.int32).contiguous()


EVICT = [
    ("one_out", KvCase([[101, 64, 17]], 3, page=16), 1, 0, 4),
    ("half", KvCase([[1000, 999], [3, 2500]], 2), 2, 2, 10),
    ("guard_only", KvCase([[500, 20]], 2, page=32), 8, 5, 30),
    ("long", KvCase([[20000, 30011]], 2, d=64, page=128), 5, 4, 100),
    # a CTA per pair, whose rows do not fit its registers
    ("chunks", KvCase([[17 + i, 17003 if i == 5 else 40] for i in range(19)] * 2 + [[33000, 1]], 2, d=64, page=256), 3, 4, 50),
    ("f32", KvCase([[300, 700, 0]], 3, dtype=dkv.F32), 2, 1, 0),
    ("f32_d64", KvCase([[1, 2, 130]], 3, d=64, page=16, dtype=dkv.F32), 2, 0, 0),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("kind", ["random", "equal", "few", "close", "special"])
@pytest.mark.parametrize("name,case,div,first,recent", EVICT, ids=[e[0] for e in EVICT])
def test_evict(name, case, div, first, recent, kind, in_place):
    c = case
    s = Setup(c)
    w, pos = _meta(c, 3, kind, c.n + 3)
    budget = [[(n - 1 if div == 1 else n // div) for n in row] for row in c.lens]
    assert _evict_check(s, budget, first, recent, w, pos, in_place) == 0


def _few_long(n, pairs):
    """`pairs` pairs, one of n rows and one of n - 1, the others short."""
    return [[n if b == 1 else n - 1 if b == 3 else 3 + b % 60] for b in range(pairs)]


# rows per thread of the selection (4, 8, 16) and row sizes; who makes the moves
EVICT_FORMS = [
    ("4_bf16", KvCase([[17000], [30011]], 1, page=128)),
    ("4_f32", KvCase([[17003, 2]], 2, page=256, dtype=dkv.F32)),
    ("8_bf16_d64", KvCase(_few_long(7001, 100), 1, d=64)),
    ("8_bf16", KvCase(_few_long(13001, 60), 1)),
    ("8_f32", KvCase(_few_long(6001, 100), 1, dtype=dkv.F32)),
    ("16_bf16", KvCase([[70003], [65000]], 1, page=256)),
    ("16_f32", KvCase([[66001]], 1, page=256, dtype=dkv.F32)),
]


@pytest.mark.parametrize("kind", ["random", "equal", "special"])
@pytest.mark.parametrize("drop", ["two", "half"])
@pytest.mark.parametrize("name,case", EVICT_FORMS, ids=[e[0] for e in EVICT_FORMS])
def test_evict_forms(name, case, drop, kind):
    s = Setup(case)
    w, pos = _meta(case, 5, kind, case.n)
    budget = [[max(0, n - 2) if drop == "two" else n // 2 for n in row] for row in case.lens]
    assert _evict_check(s, budget, 2, 30, w, pos, True) == 0


def test_evict_budgets_of_nothing_everything_and_out_of_range():
    c = KvCase([[300, 301, 302, 303]], 4)
    s = Setup(c)
    w, pos = _meta(c, 4, "random")
    assert _evict_check(s, [[0, 303, 2**31 - 1, 1]], 0, 0, w, pos, False) == 0
    s = Setup(c)
    assert _evict_check(s, [[-1, 303, 4, -2**31]], 0, 0, w, pos, False, whole=[(0, 0), (0, 3)]) == BOUNDS


def test_evict_bad_pages_and_lengths_leave_the_pair_whole():
    c = KvCase([[300, 200, 129]], 3)
    s = Setup(c)
    w, pos = _meta(c, 4, "random")
    s.table[0, 1, 3] = -7  # only rows 192 .. 199
    assert _evict_check(s, [[100, 100, 100]], 0, 0, w, pos, False, whole=[(0, 1)]) == BOUNDS
    s = Setup(c)
    s.lens[0, 2] = 301
    s.c = KvCase([[300, 200, 0]], 3)
    assert _evict_check(s, [[100, 100, 100]], 0, 0, w, pos, False) == BOUNDS


def test_evict_one_array_in_place_and_the_other_apart():
    c = KvCase([[700, 90]], 2)
    for which in (0, 1):
        s = Setup(c)
        w, pos = _meta(c, 4, "random")
        wd, pd = w.cuda(), pos.cuda()
        wo, po = (wd, torch.zeros_like(pd)) if which else (torch.zeros_like(wd), pd)
        lo = torch.zeros_like(s.lens)
        dkv.kv_evict(s.p, s.cache, c.n, torch.tensor([[300, 80]], dtype=torch.int32, device="cuda"), wd, pd, s.ws,
                     n_first=1, n_recent=20, lens_out=lo, weights_out=wo, pos_out=po)
        assert dkv.device_status(s.p, s.ws) == 0
        for h, (n, b) in enumerate(((700, 300), (90, 80))):
            m, src = evict64(n, b, 1, 20, w[0, h, :n].numpy(), pos[0, h, :n].numpy())
            assert _same(wo[0, h, :m], w[0, h][src]) and _same(po[0, h, :m], pos[0, h][src]) and int(lo[0, h]) == m


def test_evict_negative_positions_are_not_the_first():
    c = KvCase([[300, 299]], 2)
    for n_first, n_recent in ((0, 0), (5, 0), (0, 7), (5, 7)):
        s = Setup(c)
        w, pos = _meta(c, 4, "random")
        pos -= 450
        assert _evict_check(s, [[120, 296]], n_first, n_recent, w, pos, False) == 0


def test_evict_repeated_positions_stay_in_bounds():
    """Positions that repeat guard more rows than the budget holds: the guarded
    rows rank first, the lowest rows of them are kept."""
    c = KvCase([[500, 400]], 2)
    s = Setup(c)
    w, pos = _meta(c, 4, "random")
    pos[:] = 7
    assert _evict_check(s, [[50, 60]], 4, 10, w, pos, False) == 0


# ---- together

@pytest.mark.parametrize("dtype", [dkv.BF16, dkv.F32], ids=["bf16", "f32"])
def test_serving_steps_under_a_budget(dtype):
    """Prompts appended, then steps of append, decode with weights and evict
    back to the budget: every step's attention against 64 bits over the rows
    the definition keeps, ranked by the weights the GPU had."""
    B, H, Hq, d, page, budget, steps = 2, 2, 8, 128, 16, 96, 14
    prompt = [90, 41]
    cap = 256
    dt = torch.float32 if dtype == dkv.F32 else torch.bfloat16
    g = torch.Generator().manual_seed(9)
    p = dkv.plan(dkv.Config(batch=B, kv_heads=H, q_heads=Hq, d_h=d, max_T=cap, stride_s=8, k=2, d_c=16, hidden=128,
                            dtype=dtype))
    per = cap // page
    pool = dkv.alloc_kv_pool(p, B * H * per, page)
    table = torch.randperm(B * H * per, generator=g).to(torch.int32).view(B, H, per).cuda()
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")[:, None].repeat(1, H)
    cache = dkv.KVCache(p, pool, table, lens)
    ws = dkv.alloc_kv_workspace(p, cap, weights=True)
    w = torch.zeros(B, H, cap, device="cuda")
    pos = torch.zeros(B, H, cap, dtype=torch.int32, device="cuda")
    bud = torch.full((B, H), budget, dtype=torch.int32, device="cuda")
    next_pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    cnt = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    toks = {}
    K = torch.randn(B, H, max(prompt), d, generator=g).to(dt)
    V = torch.randn(B, H, max(prompt), d, generator=g).to(dt)
    dkv.kv_append(p, cache, cap, K.cuda(), V.cuda(), ws, n_tokens=cnt, first_pos=next_pos, weights=w, pos=pos)
    next_pos += cnt
    model = {}
    for b in range(B):
        for h in range(H):
            for t in range(prompt[b]):
                toks[b, h, t] = (K[b, h, t], V[b, h, t])
            model[b, h] = list(range(prompt[b]))
    for step in range(steps):
        lens += 1
        K = torch.randn(B, H, 1, d, generator=g).to(dt)
        V = torch.randn(B, H, 1, d, generator=g).to(dt)
        dkv.kv_append(p, cache, cap, K.cuda(), V.cuda(), ws, first_pos=next_pos, weights=w, pos=pos)
        q = torch.randn(B, Hq, d, generator=g).to(dt)
        out = torch.empty(B, Hq, d, device="cuda")
        w_before = w.clone()
        dkv.kv_decode_attention(p, cache, cap, q.cuda(), out, ws, weights=w, decay=0.9)
        w_mid, pos_mid = w.cpu(), pos.cpu()
        dkv.kv_evict(p, cache, cap, bud, w, pos, ws, n_first=2, n_recent=8)
        assert dkv.device_status(p, ws) == 0
        for b in range(B):
            for h in range(H):
                now = prompt[b] + step
                toks[b, h, now] = (K[b, h, 0], V[b, h, 0])
                rows = model[b, h] + [now]
                assert pos_mid[b, h, :len(rows)].tolist() == rows
                Kr = torch.stack([toks[b, h, t][0] for t in rows]).double().numpy()
                Vr = torch.stack([toks[b, h, t][1] for t in rows]).double().numpy()
                qh = q[b, h * 4:h * 4 + 4].double().numpy()
                ref, _, pr = attend64(qh, Kr, Vr)
                tol, _, rel = attend_bounds(qh, Kr, Vr, pr)
                assert (np.abs(out[b, h * 4:h * 4 + 4].cpu().double().numpy() - ref) <= tol).all()
                want = 0.9 * w_before[b, h, :len(rows)].cpu().double().numpy() + pr.sum(axis=0)
                lim = (rel[:, None] * pr).sum(axis=0) + 2.0 ** -22 * want
                assert (np.abs(w_mid[b, h, :len(rows)].double().numpy() - want) <= lim).all()
                m, src = evict64(len(rows), budget, 2, 8, w_mid[b, h, :len(rows)].numpy(),
                                 pos_mid[b, h, :len(rows)].numpy())
                model[b, h] = [rows[i] for i in src]
                assert int(lens[b, h]) == m
                assert torch.equal(w[b, h, :m].cpu(), w_mid[b, h][torch.from_numpy(src).long()])
        next_pos += 1


@pytest.mark.parametrize("budget,prompt", [(96, 90), (3000, 2999)], ids=["short", "long"])
def test_captured_serving_step_replays_like_eager_calls(budget, prompt):
    """One append, attention with weights and eviction captured in a graph on a
    side stream (passed explicitly), replayed for steps; the same steps eagerly
    give the same bytes, the error word included."""
    B, H, Hq, d, page = 2, 4, 16, 64, 32
    cap = 6000 if budget > 1000 else 160
    g = torch.Generator(device="cuda").manual_seed(4)
    p = dkv.plan(dkv.Config(batch=B, kv_heads=H, q_heads=Hq, d_h=d, max_T=cap, stride_s=8, k=2, d_c=16, hidden=128))
    per = -(-cap // page)
    prompt_kv = torch.randn(2, B, H, prompt, d, generator=g, device="cuda").bfloat16()
    steps = torch.randn(6, 3, B, max(H, Hq), 1, d, generator=g, device="cuda").bfloat16()
    ends = []
    for captured in (False, True):
        pool = dkv.alloc_kv_pool(p, B * H * per, page)
        table = torch.randperm(B * H * per, generator=torch.Generator().manual_seed(3)).to(torch.int32)
        lens = torch.full((B, H), prompt, dtype=torch.int32, device="cuda")
        cache = dkv.KVCache(p, pool, table.view(B, H, per).cuda(), lens)
        ws = dkv.alloc_kv_workspace(p, cap, weights=True)
        w = torch.zeros(B, H, cap, device="cuda")
        pos = torch.zeros(B, H, cap, dtype=torch.int32, device="cuda")
        bud = torch.full((B, H), budget, dtype=torch.int32, device="cuda")
        at = torch.zeros(B, dtype=torch.int32, device="cuda")
        dkv.kv_append(p, cache, cap, prompt_kv[0], prompt_kv[1], ws, first_pos=at, weights=w, pos=pos)
        at += prompt
        K, V, q = (torch.empty(B, n, 1, d, dtype=torch.bfloat16, device="cuda") for n in (H, H, Hq))
        out, lse = torch.empty(B, Hq, d, device="cuda"), torch.empty(B, Hq, device="cuda")

        def step(stream):
            lens.add_(1)
            dkv.kv_append(p, cache, cap, K, V, ws, first_pos=at, weights=w, pos=pos, stream=stream)
            dkv.kv_decode_attention(p, cache, cap, q[:, :, 0], out, ws, weights=w, decay=0.95, lse=lse, stream=stream)
            dkv.kv_evict(p, cache, cap, bud, w, pos, ws, n_first=1, n_recent=16, stream=stream)
            at.add_(1)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = None
        outs = []
        with torch.cuda.stream(side):
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step(side)
            for i in range(len(steps)):
                K.copy_(steps[i, 0, :, :H])
                V.copy_(steps[i, 1, :, :H])
                q.copy_(steps[i, 2, :, :Hq])
                graph.replay() if captured else step(side)
                outs.append((out.clone(), lse.clone()))
        side.synchronize()
        assert dkv.device_status(p, ws) == 0
        assert (lens == min(budget, prompt + len(steps))).all()
        ends.append([pool, w, pos, lens, at] + [x for o in outs for x in o])
    for a, b in zip(*ends):
        assert _same(a, b)


def test_calls_on_another_device_than_the_current_one_are_refused():
    s = Setup(KvCase([[10]], 1))
    out = torch.empty(1, 1, 128, device="cuda")
    s.cache.dev += 1  # as if the cache lived on another GPU
    with pytest.raises(ValueError):
        dkv.kv_decode_attention(s.p, s.cache, 10, s.q.cuda(), out, s.ws)


def test_offsets_past_32_bits():
    """The same append, attention and eviction with every array's used part
    past 2^32 bytes (weights, positions, dot products: past 2^31 elements) as
    with small ones: the same bytes."""
    H, G, d, page = 9, 4, 128, 256
    lens_host = torch.tensor([[0, 5000, 64, 1, 300, 17, 900, 33, 2000]], dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(6)
    n = int(lens_host.max())
    K, V = torch.randn(2, 1, H, n, d, generator=g, device="cuda").bfloat16()
    q = torch.randn(1, H * G, d, generator=g, device="cuda").bfloat16()
    tok_w = torch.rand(1, H, n, generator=g, device="cuda")
    per = -(-n // page)
    ends = []
    for max_len, cap, n_pages, apart in ((40000, 40000, H * per, n * d), (1 << 26, 1 << 28, 66000, 1 << 28)):
        p = dkv.plan(dkv.Config(batch=1, kv_heads=H, q_heads=H * G, d_h=d, max_T=1 << 26, stride_s=8, k=2, d_c=16,
                                hidden=128))
        pool = torch.empty(2, n_pages, page, d, dtype=torch.bfloat16, device="cuda")
        table = torch.full((1, H, -(-max_len // page)), -1, dtype=torch.int32)
        table[:, :, :per] = n_pages - 1 - torch.arange(H * per).view(1, H, per)
        lens = lens_host.cuda()
        cache = dkv.KVCache(p, pool, table.cuda(), lens)
        ws = dkv.alloc_kv_workspace(p, max_len, weights=True)
        w = torch.empty(1, H, cap, device="cuda")
        pos = torch.empty(1, H, cap, dtype=torch.int32, device="cuda")
        src = torch.empty(H * apart, dtype=torch.bfloat16, device="cuda")
        Ks = src.as_strided((1, H, n, d), (0, apart, d, 1))
        at = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = torch.empty(1, H * G, d, device="cuda"), torch.empty(1, H * G, device="cuda")
        # a call per pair: the last lens rows of the others would be written too, so their counts are theirs
        Ks.copy_(K)
        for h in range(H):
            m = int(lens_host[0, h])
            only = torch.zeros_like(lens)
            only[0, h] = m
            one = dkv.KVCache(p, pool, cache.page_table, only)
            count = torch.full((1,), m, dtype=torch.int32, device="cuda")
            dkv.kv_append(p, one, max_len, Ks, Ks, ws, n_tokens=count, first_pos=at, weights=w, pos=pos,
                          token_weights=tok_w)
            dkv.device_status(p, ws)  # (the other pairs have no room for m tokens: reported, not written)
        for h in range(H):
            ids = table[0, h, :per].long().cuda()
            rows = pool[:, ids].view(2, -1, d)
            m = int(lens_host[0, h])
            assert torch.equal(rows[0, :m], K[0, h, :m]) and torch.equal(rows[1, :m], K[0, h, :m])
        pool[1, table[:, :, :per].reshape(-1).long().cuda()] = V.new_tensor(0.5)
        dkv.kv_decode_attention(p, cache, max_len, q, out, ws, weights=w, decay=0.9, lse=lse)
        used = [w[0, h, :int(lens_host[0, h])].clone() for h in range(H)]
        budget = (lens_host // 2).cuda()
        dkv.kv_evict(p, cache, max_len, budget, w, pos, ws, n_first=1, n_recent=2)
        assert dkv.device_status(p, ws) == 0
        kept = []
        for h in range(H):
            m = int(lens[0, h])
            assert m == min(int(lens_host[0, h]), max(int(lens_host[0, h]) // 2, 3))
            ids = table[0, h, :per].long().cuda()
            kept += [pool[0, ids].view(-1, d)[:m].clone(), w[0, h, :m].clone(), pos[0, h, :m].clone()]
            assert torch.equal(kept[-3], K[0, h][kept[-1].long()])
        ends.append([out, lse] + used + kept)
        del pool, w, pos, src, Ks, ws, cache, one
    for a, b in zip(*ends):
        assert _same(a, b)


def test_two_threads_share_a_cache():
    """Two host threads, each with a stream, a workspace and a max_len (so a
    form of the attention) of its own, read one cache at once."""
    import threading

    s = Setup(KvCase([[500, 17], [64, 900]], 8, max_len=40000))
    q = s.q.cuda()
    bounds = (900, 40000)
    outs = [[torch.full((2, 8, 128), float("nan"), device="cuda") for _ in range(40)] for _ in bounds]
    wss = [dkv.alloc_kv_workspace(s.p, n) for n in bounds]
    want = []
    for n, ws in zip(bounds, wss):
        out = torch.empty(2, 8, 128, device="cuda")
        dkv.kv_decode_attention(s.p, s.cache, n, q, out, ws)
        want.append(out)
    torch.cuda.synchronize()
    failed = []

    def calls(i):
        try:
            stream = torch.cuda.Stream()
            for out in outs[i]:
                dkv.kv_decode_attention(s.p, s.cache, bounds[i], q, out, wss[i], stream=stream)
            stream.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for o, ref, ws in zip(outs, want, wss):
        assert dkv.device_status(s.p, ws) == 0
        assert all(torch.equal(x, ref) for x in o)


FIRST_CALLS = """
import sys
import torch
from decode_attention_strided_b200 import deltakv as dkv
n, B, H, Hq, d = int(sys.argv[1]), 1, 4, 8, 128
per = -(-n // 64)
p = dkv.plan(dkv.Config(batch=B, kv_heads=H, q_heads=Hq, d_h=d, max_T=n, stride_s=8, k=2, d_c=16, hidden=128))
pool = dkv.alloc_kv_pool(p, H * per, 64)
table = torch.arange(H * per, dtype=torch.int32, device="cuda").view(B, H, per)
lens = torch.full((B, H), n, dtype=torch.int32, device="cuda")
cache = dkv.KVCache(p, pool, table, lens)
ws = dkv.alloc_kv_workspace(p, n, weights=True)
w, at = torch.zeros(B, H, n, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
pos = torch.zeros(B, H, n, dtype=torch.int32, device="cuda")
K = torch.randn(B, H, n, d, device="cuda").bfloat16()
q, out = torch.randn(B, Hq, d, device="cuda").bfloat16(), torch.zeros(B, Hq, d, device="cuda")
budget = torch.full((B, H), n // 2, dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dkv.kv_append(p, cache, n, K, K, ws, first_pos=at, weights=w, pos=pos)
    dkv.kv_decode_attention(p, cache, n, q, out, ws, weights=w)
    dkv.kv_evict(p, cache, n, budget, w, pos, ws, n_recent=4)
g.replay()
torch.cuda.synchronize()
x = (q.float().view(B, H, 2, d) @ K.float().transpose(-1, -2)) / d ** 0.5
ref = (x.softmax(-1) @ K.float()).reshape(B, Hq, d)
# (float32 on both sides: 2^-8 of rows near 1 is far above their rounding, far below a wrong row)
assert (out - ref).abs().max() < 2 ** -8, (out - ref).abs().max()
assert (lens == n // 2).all() and dkv.device_status(p, ws) == 0
"""


@pytest.mark.parametrize("n", [300, 70001], ids=["short", "long"])
def test_first_calls_of_a_process_may_be_captured(n):
    import pathlib
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, str(n)], cwd=pathlib.Path(__file__).parent.parent,
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_assigned_tensors_are_the_ones_that_are_read_and_written():
    """Lengths, pages and pool assigned to a cache are what the next calls
    use; eviction in place writes the lengths that it read."""
    c = KvCase([[300, 200], [40, 129]], 8)
    s = Setup(c)
    fresh = Setup(dataclasses.replace(c, seed=1))
    other = dkv.KVCache(s.p, fresh.pool, fresh.table, fresh.lens)
    first_lens, first_table, first_pool = other.lens, other.page_table, other.pool  # (kept: none is freed)
    other.pool, other.page_table, other.lens = s.pool, s.table, s.lens - 0
    out, lse, w = _attend(s)
    s.cache = other
    for a, b in zip((out, lse, w), _attend(s)):
        assert _same(a, b)
    other.lens = less = s.lens // 2
    half = Setup.__new__(Setup)
    half.__dict__.update(s.__dict__)
    half.c = dataclasses.replace(c, lens=less.tolist(), max_len=c.n)
    half.K = {k: v[:half.c.lens[k[0]][k[1]]] for k, v in s.K.items()}
    half.V = {k: v[:half.c.lens[k[0]][k[1]]] for k, v in s.V.items()}
    _check_attend(half, *_attend(s))
    wd, pos = s.w.cuda(), torch.arange(c.n, dtype=torch.int32, device="cuda").expand(2, 2, c.n).contiguous()
    dkv.kv_evict(s.p, other, c.n, torch.full((2, 2), 11, dtype=torch.int32, device="cuda"), wd, pos, s.ws)
    assert dkv.device_status(s.p, s.ws) == 0
    assert (less == 11).all() and other.lens is less
    assert torch.equal(s.lens.cpu(), s.lens_host) and torch.equal(first_lens.cpu(), fresh.lens_host)
    assert _same(first_pool, Setup(dataclasses.replace(c, seed=1)).pool) and first_table is fresh.table


@pytest.mark.parametrize("bad", [-1, 301, 2**31 - 1])
@pytest.mark.parametrize("n", [300, 5000], ids=["block", "cluster"])
def test_evict_in_place_leaves_a_length_out_of_range_as_it_is(n, bad):
    """The pair's rows, weights, positions and length are all as before; the
    other pairs are evicted, and a second call with the length put right too."""
    c = KvCase([[n, 200, 129]], 3, max_len=n)
    s = Setup(c)
    w, pos = _meta(c, 4, "random")
    wrong = n + 1 if bad == 301 else bad
    s.lens[0, 0] = wrong
    pool0, wd, pd = s.pool.cpu(), w.cuda(), pos.cuda()
    budget = torch.full((1, 3), 100, dtype=torch.int32, device="cuda")
    dkv.kv_evict(s.p, s.cache, n, budget, wd, pd, s.ws)
    assert dkv.device_status(s.p, s.ws) == BOUNDS
    assert s.lens.tolist() == [[wrong, 100, 100]]
    ids = s.table_host[0, 0, :-(-n // c.page)].long()
    assert _same(s.pool[:, ids.cuda()], pool0[:, ids]) and _same(wd[0, 0], w[0, 0]) and _same(pd[0, 0], pos[0, 0])
    s.lens[0, 0] = n
    s.c = KvCase([[n, 100, 100]], 3, max_len=n)
    s.lens_host = torch.tensor(s.c.lens, dtype=torch.int32)
    assert _evict_check(s, [[100, 100, 100]], 0, 0, wd.cpu(), pd.cpu(), True) == 0


# ---- every kernel that the dispatch can choose

def _ran(p, call):
    """Names of the kernels that a call launched."""
    dkv.profile_collect(p)
    dkv.set_profiling(p, True)
    try:
        got = call()
        return got, set(dkv.profile_collect(p))
    finally:
        dkv.set_profiling(p, False)


SHORT, CUT, WEIGHTS = {"kv_attend_short"}, {"kv_attend", "kv_join"}, {"kv_attend", "kv_join", "kv_weights"}


@pytest.mark.parametrize("form", ["cluster", "cut"])
@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [dkv.BF16, dkv.F32], ids=["bf16", "f32"])
def test_attend_few_rows_closely(dtype, d, G, form):
    """Both types and head sizes, one to eight heads a kv-head and both forms
    of the split, with weights, on pairs of few rows and almost exact logits:
    within bounds that a weight of two bfloat16 terms does not meet
    (test_the_counted_bounds_tell_a_missing_weight_term)."""
    H = 6
    pattern = (2, 3, 2, 17, 2, 100, 2, 0, 2, 33, 1, 16)
    c = KvCase([[pattern[(b * H + h) % 12] for h in range(H)] for b in range(8)], H * G, d=d, page=32, dtype=dtype,
               max_len=2200 if form == "cut" else 0, seed=G)
    s = Setup(c)
    s.q = few_queries(c)
    (out, lse, w), ran = _ran(s.p, lambda: _attend(s, decay=0.5))
    assert dkv.device_status(s.p, s.ws) == 0
    assert ran == (WEIGHTS if form == "cut" else SHORT)
    out, lse, w = (x.cpu().double().numpy() for x in (out, lse, w))
    w0 = s.w.double().numpy()
    for b in range(c.B):
        for h in range(H):
            n, g = c.lens[b][h], slice(h * G, h * G + G)
            if n == 0:
                assert (out[b, g] == 0).all() and (lse[b, g] == -np.inf).all() and (w[b, h] == w0[b, h]).all()
                continue
            q, K, V = (x.double().numpy() for x in (s.q[b, g], s.K[b, h], s.V[b, h]))
            ref, ref_lse, p = attend64(q, K, V)
            tol, tol_lse, rel = few_bounds(q, K, V, p, unit_rows(c))
            err = np.abs(out[b, g] - ref) / tol
            assert err.max() <= 1, (b, h, n, float(err.max()))
            err = np.abs(lse[b, g] - ref_lse) / tol_lse
            assert err.max() <= 1, (b, h, n, float(err.max()))
            want = 0.5 * w0[b, h, :n] + p.sum(axis=0)
            # the heads' sum and the old weight's product: G + 1 roundings
            err = np.abs(w[b, h, :n] - want) / (rel @ p + (G + 1) * 2.0 ** -24 * want)
            assert err.max() <= 1, (b, h, n, float(err.max()))
            assert (w[b, h, n:] == w0[b, h, n:]).all()


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("name,case", ATTEND, ids=[n for n, _ in ATTEND])
def test_attend_cases_take_the_form_they_name(name, case, weights):
    cut = WEIGHTS if weights else CUT
    _, ran = _ran((s := Setup(case)).p, lambda: _attend(s, weights))
    # as they are: a cluster per pair up to 128 pairs, but for rows of more than 16 units a CTA ("long": 20011 rows are
    # 626 units, "f32_g3": 5003 are 313, both for clusters of eight)
    assert ran == (cut if name in ("long", "f32_g3", "many_pairs", "mostly_empty") else SHORT)
    if case.B * case.H <= 32:
        _, ran = _ran((s := Setup(dataclasses.replace(case, max_len=40000))).p, lambda: _attend(s, weights))
        assert ran == cut


@pytest.mark.parametrize("name,case", EVICT_FORMS, ids=[e[0] for e in EVICT_FORMS])
def test_evict_cases_take_the_form_they_name(name, case):
    """The clusters make the moves up to eight rows a thread, the second kernel
    from there on."""
    s = Setup(case)
    w, pos = _meta(case, 5, "random", case.n)
    budget = torch.tensor([[n // 2 for n in row] for row in case.lens], dtype=torch.int32, device="cuda")
    _, ran = _ran(s.p, lambda: dkv.kv_evict(s.p, s.cache, case.n, budget, w.cuda(), pos.cuda(), s.ws))
    assert dkv.device_status(s.p, s.ws) == 0
    assert ran == ({"kv_select", "kv_move"} if name.startswith("16") else {"kv_select"})


@pytest.mark.parametrize("kind", ["random", "equal", "few", "special"])
@pytest.mark.parametrize("drop", ["two", "half"])
def test_evict_short_rows_of_d64(drop, kind):
    """Two rows a thread at most, rows of 128 bytes, moved by the block."""
    case = KvCase([[900, 1, 33], [0, 1999, 2000]], 3, d=64, page=16)
    s = Setup(case)
    w, pos = _meta(case, 5, kind, case.n + 1)
    budget = [[max(0, n - 2) if drop == "two" else n // 2 for n in row] for row in case.lens]
    assert _evict_check(s, budget, 1, 9, w, pos, True) == 0
