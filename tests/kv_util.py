"""Plain implementations, in 64 bits, of the plain paged cache's operators
(append, decode attention, eviction), and the cases' inputs."""
import dataclasses
import math

import numpy as np
import torch

from decode_attention_strided_b200 import deltakv as dkv


@dataclasses.dataclass
class KvCase:
    lens: list                 # [B][H]
    Hq: int
    d: int = 128
    page: int = 64
    dtype: int = dkv.BF16
    max_len: int = 0           # 0: the longest of lens
    seed: int = 0
    scale: float = 1.0         # of K: how peaked the softmax is

    @property
    def B(self):
        return len(self.lens)

    @property
    def H(self):
        return len(self.lens[0])

    @property
    def G(self):
        return self.Hq // self.H

    @property
    def n(self):
        return self.max_len or max(1, max(max(r) for r in self.lens))

    def torch_dtype(self):
        return torch.float32 if self.dtype == dkv.F32 else torch.bfloat16


class Setup:
    """Inputs of a case on the GPU.  Every row that is not valid holds NaN, and
    page-table entries that must not be read are out of range, so reading
    either shows up in the results or in the error word."""

    def __init__(self, c: KvCase, spare=2):
        g = torch.Generator().manual_seed(c.seed + 17)
        self.c = c
        B, H, d = c.B, c.H, c.d
        dt = c.torch_dtype()
        self.lens_host = torch.tensor(c.lens, dtype=torch.int32)
        need = (self.lens_host.long() + c.page - 1) // c.page
        per_pair = -(-c.n // c.page)
        n_pages = int(need.sum()) + spare
        perm = torch.randperm(n_pages, generator=g)[:int(need.sum())].to(torch.int32)
        table = torch.full((B, H, per_pair), 2**31 - 1, dtype=torch.int32)
        used = torch.arange(per_pair)[None, None] < need[..., None]
        table[used] = perm
        pool = torch.full((2, n_pages, c.page, d), float("nan"), dtype=dt)
        self.K, self.V = {}, {}
        for b in range(B):
            for h in range(H):
                n = c.lens[b][h]
                k = (torch.randn(n, d, generator=g) * c.scale).to(dt)
                v = torch.randn(n, d, generator=g).to(dt)
                self.K[b, h], self.V[b, h] = k, v
                for i, x in ((0, k), (1, v)):
                    for l in range(-(-n // c.page)):
                        part = x[l * c.page:(l + 1) * c.page]
                        pool[i, table[b, h, l], :len(part)] = part
        self.q = torch.randn(B, c.Hq, d, generator=g).to(dt)
        self.w = torch.rand(B, H, c.n, generator=g)
        self.p = dkv.plan(dkv.Config(batch=B, kv_heads=H, q_heads=c.Hq, d_h=d, max_T=c.n, stride_s=8, k=2, d_c=16,
                                     hidden=128, dtype=c.dtype))
        self.table_host = table
        self.pool, self.table, self.lens = pool.cuda(), table.cuda(), self.lens_host.cuda()
        self.cache = dkv.KVCache(self.p, self.pool, self.table, self.lens)
        self.ws = dkv.alloc_kv_workspace(self.p, c.n, weights=True)
        # everything after the error word NaN: a region read before it is written shows up
        self.ws[256:].fill_(0xFF)

    def rows(self, plane, b, h, n):
        """Rows 0 .. n-1 of a pair as the pool holds them now."""
        x = self.pool[plane].cpu()
        ids = self.table_host[b, h, :-(-n // self.c.page)].long()
        return x[ids].reshape(-1, self.c.d)[:n]


def attend64(q, K, V):
    """out [G, d], lse [G], p [G, n] in float64."""
    G, d = q.shape
    if K.shape[0] == 0:
        return np.zeros((G, d)), np.full(G, -np.inf), np.zeros((G, 0))
    s = q @ K.T / math.sqrt(d)
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(axis=1, keepdims=True)
    p = e / z
    return p @ V, (m + np.log(z))[:, 0], p


def attend_bounds(q, K, V, p):
    """How far float32 results may be off: (out [G, d], lse [G], relative
    error of p [G]).

    A logit is a dot product of d exact products summed in float32 (an
    addition on the tensor cores may truncate: one step, 2^-23, each), then
    scaled and multiplied by log2(e) rounded to float32: |dx| <= (d + 4) 2^-23
    sum |q||k| / sqrt(d).  2^x by the special-function unit is within 2 steps
    (2^-22) and its argument, x minus the maximum, is rounded once more
    (2^-24 |x - m| log2 e, at most 2^-23 (|x| + |m|)).  A sum of n terms runs
    through at most n / 8 + 400 additions (eight warps at least share a
    pair's rows; then the join of warps and of up to 296 parts), each within
    2^-23.  Numerator and denominator both carry the sum's error."""
    n, d = K.shape
    u = 2.0 ** -23
    mag = (np.abs(q) @ np.abs(K).T).max(axis=1) / math.sqrt(d)       # [G]
    dx = (d + 4) * u * mag + 2 * u * mag * 1.5
    rel = 2 * dx + 4 * u + 2 * (n / 8 + 400) * u
    return rel[:, None] * (p @ np.abs(V)) + 1e-37, dx + (n / 8 + 404) * u + u * mag, rel


def evict64(n, budget, n_first, n_recent, w, pos):
    """Rows kept, by the definition: (m, source row of each of the rows 0 ..
    m-1 afterwards).  w float32 and pos int arrays of n rows."""
    m = min(n, max(budget, n_first + n_recent))
    if m == n:
        return m, np.arange(n)
    pos = pos.astype(np.int64)
    guarded = ((pos >= 0) & (pos < n_first)) | (pos > pos.max() - n_recent)
    with np.errstate(invalid="ignore"):  # signalling NaN
        w = w.astype(np.float64)
    # ascending sort of (class, -weight, row): guarded, then numbers by weight, then NaN
    cls = np.where(guarded, 0, np.where(np.isnan(w), 2, 1))
    neg = np.where(cls == 1, -np.nan_to_num(w, nan=0.0, posinf=np.inf, neginf=-np.inf), 0.0)
    kept = np.zeros(n, dtype=bool)
    kept[np.lexsort((np.arange(n), neg, cls))[:m]] = True
    src = np.arange(m)
    src[~kept[:m]] = np.arange(m, n)[kept[m:]]
    return m, src


def few_queries(c: KvCase):
    """Queries of two non-zero elements each, at places that differ by head:
    logits come out almost exact, and within about one of each other, so that
    what is left of an error is the softmax weights' and the sums'."""
    q = torch.zeros(c.B * c.Hq, c.d)
    i = torch.arange(c.B * c.Hq)
    at = 7 * i + 3
    v = 4.0 if c.d == 128 else 3.0
    q[i, at % c.d] = v
    q[i, (at + 1 + 5 * (i % 11)) % c.d] = -v
    return q.view(c.B, c.Hq, c.d).to(c.torch_dtype())


def unit_rows(c: KvCase):
    """Rows of one step of a warp: 8 KB of K."""
    return 8192 // (c.d * (4 if c.dtype == dkv.F32 else 2))


def few_bounds(q, K, V, p, unit):
    """attend_bounds for queries of few non-zero elements and pairs of at most
    eight units of rows, counted term by term: (out, lse, relative error of a
    weight).  u = 2^-24.

    A logit: one rounding or truncation (2 u) per non-zero product.  Its
    exponent, one fused multiply-add: u of its distance from the maximum, plus
    3 u of that distance for the scale's roundings; the maximum's own rounding
    is common to all rows.  2^x: 4 u.  Where the rows are several units (a warp
    each), a part is scaled twice, by 2^x of a difference of maxima each time.
    Additions of the sum of p V, 2 u each: a unit's rows (a product's terms
    come smallest first; with several 16-row groups each of the three terms is
    added to a full sum), the running sum, two for the columns of a head, the
    warps, the parts; of the sum of p, u each, no more of them.  What three
    bfloat16 terms leave of a weight is below u / 4; 1 / l and its product two
    u."""
    n, d = K.shape
    u = 2.0 ** -24
    units = -(-n // unit)
    assert units <= 8
    x = q @ K.T / math.sqrt(d)
    span = x.max(axis=1) - x.min(axis=1)
    mag = (np.abs(q) @ np.abs(K).T).max(axis=1) / math.sqrt(d)
    dx = 2 * u * np.count_nonzero(q, axis=1) * mag
    stages = 0 if units == 1 else 2
    ep = 2 * dx + 4 * u * span + 4 * u + stages * (4 * u + 1.5 * u * span)
    rows = min(n, unit)
    adds = (rows if rows <= 16 else 3 * rows) + 4 + 2 * (units - 1)
    rel = 2 * ep + 3 * u * adds + 3 * u
    top = x.max(axis=1)
    lse = top + np.log(np.exp(x - top[:, None]).sum(axis=1))
    tol_lse = dx + 4 * u * np.abs(top) + ep + u * adds + 4 * u * (1 + np.abs(lse) + math.log(n))
    return rel[:, None] * (p @ np.abs(V)), tol_lse, rel + 4 * u
