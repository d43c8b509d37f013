"""Measured cases of the plain paged key-value cache: writing tokens into its
pages, decode attention over them, and eviction by accumulated attention
weight.

Shapes: B sequences, H kv-heads, Hq query heads (G = Hq / H consecutive query
heads share a kv-head), head size d.  The pool holds K and V as
[2, pages, page, d]; a page is `page` consecutive rows of one (sequence,
kv-head), named by a page table [B, H, pages per pair] whose unused entries
are -1.  Row r of pair (b, h) is valid for r < lens[b, h].

  attend  out[b, hq] = sum_r p_r V_r, p = softmax_r(q . K_r / sqrt(d)) over the
          valid rows (0 and lse -inf for an empty row); with `weights`, also
          w[b, h, r] <- decay w[b, h, r] + sum over the pair's heads of p_r.
  append  the n_b new tokens of sequence b become the rows
          lens - n_b .. lens - 1 of each of its pairs, with their position
          and their first weight.
  evict   of n rows keep m = min(n, max(budget, first + recent)): the rows
          with position < first or within the last `recent` positions, then
          the largest weights (ties to the lower row); kept rows >= m move, in
          order, into the evicted rows < m.  Positions and weights of the kept
          rows go to arrays of their own.
"""
import math

import torch

own = False

DEV = "cuda"


def _attend(name, B, H, Hq, d, page, max_len, dtype="bf16", lens="ragged", weights=False, decay=1.0):
    return dict(name=name, op="attend", B=B, H=H, Hq=Hq, d=d, page=page, max_len=max_len, dtype=dtype, lens=lens,
                weights=weights, decay=decay)


def _append(name, B, H, d, page, max_len, n_new, dtype="bf16"):
    return dict(name=name, op="append", B=B, H=H, Hq=H, d=d, page=page, max_len=max_len, n_new=n_new, dtype=dtype)


def _evict(name, B, H, d, page, max_len, budget, first, recent, dtype="bf16", lens="ragged"):
    return dict(name=name, op="evict", B=B, H=H, Hq=H, d=d, page=page, max_len=max_len, budget=budget, first=first,
                recent=recent, dtype=dtype, lens=lens)


def listed():
    return [
        # one short conversation: the call's latency
        _attend("attend_short", 1, 8, 32, 128, 64, 513, lens="full"),
        # an ordinary batch of conversations of different lengths
        _attend("attend_batch", 8, 8, 32, 128, 64, 4097),
        # the batch-8, 128k-token decode of the compressed cache's benchmark, uncompressed
        _attend("attend_128k", 8, 8, 32, 128, 128, 131072, lens="full"),
        # the same heads while weights are gathered for eviction; lengths differ by head, as eviction leaves them
        _attend("attend_weights", 8, 8, 32, 128, 64, 16384, lens="heads", weights=True, decay=1.0),
        # many short-to-medium sequences, small heads, eight query heads a kv-head, small pages, one sequence empty
        _attend("attend_d64_many", 16, 4, 32, 64, 32, 20011, lens="heads", weights=False),
        # float32 caches, three query heads a kv-head, decayed weights
        _attend("attend_f32", 2, 4, 12, 64, 16, 5003, dtype="f32", weights=True, decay=0.875),
        # one decoded token of each sequence
        _append("append_token", 8, 8, 128, 64, 4097, 1),
        # prompts of different lengths written at once
        _append("append_prompts", 4, 8, 128, 64, 8191, 8191),
        # a cache held at its budget: one row out for each token in
        _evict("evict_one", 8, 8, 128, 64, 2049, 2048, 4, 256, lens="full"),
        # one long prompt cut down after prefill
        _evict("evict_128k", 1, 8, 128, 128, 131072, 16384, 4, 1024, lens="full"),
        # a batch cut down, lengths below and above the budget
        _evict("evict_batch", 8, 8, 128, 64, 32768, 8192, 4, 512),
        # float32 rows, odd sizes, lengths by head
        _evict("evict_f32", 3, 5, 64, 16, 7001, 2503, 1, 100, dtype="f32", lens="heads"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    es = 4 if dtype == "f32" else 2
    most = 8 * 8 * 131072 * 128 * 2 // (d * es)  # rows: no more bytes than the largest listed case
    B, H = _log_int(rng, 1, 16), rng.choice([1, 2, 3, 5, 8])
    if op == "attend":
        G = rng.randint(1, 8)
        max_len = min(_log_int(rng, 1, 131072), most // (B * H))
        weights = rng.random() < 0.5
        return dict(op=op, B=B, H=H, Hq=H * G, d=d, page=page, max_len=max_len, dtype=dtype,
                    lens=rng.choice(["full", "ragged", "heads"]), weights=weights,
                    decay=rng.choice([1.0, 0.875]) if weights else 1.0)
    if op == "append":
        max_len = min(_log_int(rng, 1, 32768), most // (4 * B * H))
        return dict(op=op, B=B, H=H, Hq=H, d=d, page=page, max_len=max_len,
                    n_new=min(max_len, _log_int(rng, 1, 16384)), dtype=dtype)
    max_len = min(_log_int(rng, 2, 131072), most // (8 * B * H))
    budget = min(max_len, _log_int(rng, 1, max(1, max_len)))
    return dict(op=op, B=B, H=H, Hq=H, d=d, page=page, max_len=max_len, budget=budget, first=rng.choice([0, 1, 4]),
                recent=rng.choice([0, 1, budget // 8]), dtype=dtype, lens=rng.choice(["full", "ragged", "heads"]))


def _host_lens(case, seed):
    """Row counts [B, H] of a case, on the host: the first sequence is the
    longest; with lens "heads" they differ by head, and of a batch of more
    than eight the last sequence is empty."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    B, H, n = case["B"], case["H"], case["max_len"]
    if case.get("lens") == "full":
        return torch.full((B, H), n, dtype=torch.int32)
    # every length within a factor of eight of the longest, evenly over the logarithm
    lo = max(1, n // 8)
    shape = (B, H) if case.get("lens") == "heads" else (B, 1)
    u = torch.rand(shape, generator=g, dtype=torch.float64)
    lens = torch.exp(math.log(lo) + u * (math.log(n) - math.log(lo))).round().clamp(1, n).to(torch.int32)
    lens = lens.expand(B, H).contiguous()
    lens[0, 0] = n
    if case.get("lens") == "heads" and B > 8:
        lens[-1] = 0
    return lens


def _new_counts(case, seed):
    """Tokens that each sequence of an append case brings, on the host."""
    g = torch.Generator().manual_seed(seed * 7 + 2)
    n = case["n_new"]
    cnt = torch.randint(max(1, n // 4), n + 1, (case["B"],), generator=g).to(torch.int32)
    cnt[0] = n
    return cnt


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _tokens(g, n, d, dt, dev):
    """K or V rows of one pair: eight shared high-norm directions with N(0, 4)
    coefficients, plus N(0, 0.25) noise."""
    u = torch.randn(8, d, generator=g, device=dev)
    u *= math.sqrt(d) / u.norm(dim=1, keepdim=True)
    c = torch.randn(n, 8, generator=g, device=dev) * 2
    return (torch.randn(n, d, generator=g, device=dev) * 0.5).addmm_(c, u).to(dt)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, H, Hq, d, page, n = (case[k] for k in ("B", "H", "Hq", "d", "page", "max_len"))
    dt = _dtype(case)
    op = case["op"]
    if op == "append":
        cnt = _new_counts(case, seed)
        gh = torch.Generator().manual_seed(seed * 7 + 3)
        old = (torch.rand(B, H, generator=gh) * (n - cnt[:, None] + 1)).floor().to(torch.int32)
        lens = (old + cnt[:, None]).to(torch.int32)
    else:
        lens = _host_lens(case, seed)
    need = (lens.long() + page - 1) // page
    per_pair = max(1, -(-n // page))
    n_pages = B * H * per_pair + 1  # as many for every seed; a pool has pages that nobody holds
    perm = torch.randperm(n_pages, generator=g, device=DEV)[:int(need.sum())].to(torch.int32)
    table = torch.full((B, H, per_pair), -1, dtype=torch.int32, device=DEV)
    used = torch.arange(per_pair)[None, None, :] < need[:, :, None]
    table[used.to(DEV)] = perm
    pool = torch.zeros(2, n_pages, page, d, dtype=dt, device=DEV)
    for b in range(B):
        for h in range(H):
            k = int(need[b, h])
            if k and op != "append":
                ids = table[b, h, :k].long()
                for i in range(2):
                    pool[i].index_copy_(0, ids, _tokens(g, k * page, d, dt, DEV).view(k, page, d))
    st = dict(case=case, pool=pool, table=table, lens=lens.to(DEV), max_len=n)
    if op == "attend":
        st["q"] = torch.randn(B, Hq, d, generator=g, device=DEV).to(dt)
        st["out"] = torch.empty(B, Hq, d, device=DEV)
        st["lse"] = torch.empty(B, Hq, device=DEV)
        if case["weights"]:
            st["w"] = torch.rand(B, H, n, generator=g, device=DEV) * 1e-2
    elif op == "append":
        m = case["n_new"]
        # the projection's own layout: token-major, heads inside
        st["K"] = torch.randn(B, m, H, d, generator=g, device=DEV).to(dt).transpose(1, 2)
        st["V"] = torch.randn(B, m, H, d, generator=g, device=DEV).to(dt).transpose(1, 2)
        st["count"] = cnt.to(DEV)
        st["first_pos"] = st["lens"].amax(dim=1).contiguous() - st["count"]
        st["tok_w"] = torch.rand(B, H, m, generator=g, device=DEV)
        st["w"] = torch.zeros(B, H, n, device=DEV)
        st["pos"] = torch.zeros(B, H, n, dtype=torch.int32, device=DEV)
    else:
        # weights as sums of softmax rows are: heavy-tailed over tokens
        st["w"] = torch.exp(torch.randn(B, H, n, generator=g, device=DEV) * 2 - 6)
        # positions: increasing with gaps, the rows in the order earlier evictions left
        p = torch.randint(1, 4, (B, H, n), generator=g, device=DEV).cumsum(-1) - 1
        order = torch.rand(B, H, n, generator=g, device=DEV)
        order = order.masked_fill(torch.arange(n, device=DEV) >= st["lens"][..., None], 2.0).argsort(dim=-1)
        st["pos"] = p.gather(-1, order).to(torch.int32)
        st["budget"] = torch.full((B, H), case["budget"], dtype=torch.int32, device=DEV)
        st["lens_out"] = torch.zeros_like(st["lens"])
        st["w_out"] = torch.zeros_like(st["w"])
        st["pos_out"] = torch.zeros_like(st["pos"])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from decode_attention_strided_b200 import deltakv as dkv
        p = dkv.plan(dkv.Config(batch=case["B"], kv_heads=case["H"], q_heads=case["Hq"], d_h=case["d"],
                                max_T=case["max_len"], stride_s=16, k=4, d_c=32, hidden=256,
                                dtype=dkv.F32 if case["dtype"] == "f32" else dkv.BF16))
        st["plan"] = p
        st["cache"] = dkv.KVCache(p, st["pool"], st["table"], st["lens"])
        st["ws"] = dkv.alloc_kv_workspace(p, case["max_len"], weights=bool(case.get("weights")))
    return st


def run(st):
    case = st["case"]
    if own:
        from decode_attention_strided_b200 import deltakv as dkv
        if case["op"] == "attend":
            dkv.kv_decode_attention(st["plan"], st["cache"], st["max_len"], st["q"], st["out"], st["ws"],
                                    weights=st.get("w"), decay=case["decay"], lse=st["lse"])
            return _attended(st)
        if case["op"] == "append":
            dkv.kv_append(st["plan"], st["cache"], st["max_len"], st["K"], st["V"], st["ws"], n_tokens=st["count"],
                          first_pos=st["first_pos"], weights=st["w"], pos=st["pos"], token_weights=st["tok_w"])
            return {"pool": st["pool"], "weights": st["w"], "pos": st["pos"]}
        dkv.kv_evict(st["plan"], st["cache"], st["max_len"], st["budget"], st["w"], st["pos"], st["ws"],
                     n_first=case["first"], n_recent=case["recent"], lens_out=st["lens_out"],
                     weights_out=st["w_out"], pos_out=st["pos_out"])
        return _evicted(st)
    if case["op"] == "attend":
        return _plain_attend(st)
    if case["op"] == "append":
        return _plain_append(st)
    return _plain_evict(st)


def _attended(st):
    got = {"out": st["out"], "lse": st["lse"]}
    if "w" in st:
        got["weights"] = st["w"]
    return got


def _evicted(st):
    return {"pool": st["pool"], "lens": st["lens_out"], "weights": st["w_out"], "pos": st["pos_out"]}


def _plain_attend(st):
    case = st["case"]
    B, H, Hq, d, n = (case[k] for k in ("B", "H", "Hq", "d", "max_len"))
    table = st["table"].clamp(min=0).long()
    valid = torch.arange(n, device=DEV) < st["lens"][..., None]  # [B, H, n]
    K = st["pool"][0][table].view(B, H, -1, d)[:, :, :n].float()
    q = st["q"].float().view(B, H, Hq // H, d) / math.sqrt(d)
    s = torch.matmul(q, K.transpose(-1, -2)).masked_fill(~valid[:, :, None], -math.inf)
    del K
    m = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)  # an empty row has none
    e = torch.exp(s - m)
    del s
    total = e.sum(-1, keepdim=True)
    V = st["pool"][1][table].view(B, H, -1, d)[:, :, :n].float().masked_fill(~valid[..., None], 0.0)
    safe = torch.where(total > 0, total, 1.0)
    st["out"].copy_((torch.matmul(e, V) / safe).view(B, Hq, d))
    st["lse"].copy_((m + torch.log(total)).view(B, Hq))
    if "w" in st:
        w = st["w"]
        w.copy_(torch.where(valid, case["decay"] * w + (e / safe).sum(2), w))
    return _attended(st)


def _plain_append(st):
    case = st["case"]
    page, m = case["page"], case["n_new"]
    base = (st["lens"] - st["count"][:, None]).long()
    i = torch.arange(m, device=DEV)
    b, h, t = torch.nonzero((i < st["count"][:, None])[:, None].expand(-1, case["H"], -1), as_tuple=True)
    row = base[b, h] + t
    pg = st["table"][b, h, row // page].long()
    st["pool"][0][pg, row % page] = st["K"][b, h, t]
    st["pool"][1][pg, row % page] = st["V"][b, h, t]
    st["w"][b, h, row] = st["tok_w"][b, h, t]
    st["pos"][b, h, row] = st["first_pos"][b] + t.int()
    return {"pool": st["pool"], "weights": st["w"], "pos": st["pos"]}


def _plain_evict(st):
    case = st["case"]
    page, n = case["page"], case["max_len"]
    lens = st["lens"].long()[..., None]
    m = torch.minimum(lens, st["budget"].long()[..., None].clamp(min=case["first"] + case["recent"]))
    row = torch.arange(n, device=DEV)
    valid = row < lens
    pos = st["pos"].long()
    last = pos.masked_fill(~valid, -(1 << 40)).amax(-1, keepdim=True)
    guarded = (pos < case["first"]) | (pos > last - case["recent"])
    key = torch.where(guarded, math.inf, st["w"]).masked_fill(~valid, -1.0)
    rank = torch.empty_like(pos).scatter_(-1, key.argsort(dim=-1, descending=True, stable=True), row.expand_as(pos))
    keep = valid & (rank < m)
    hole = torch.nonzero((row < m) & ~keep, as_tuple=True)  # as many of each pair's as
    move = torch.nonzero((row >= m) & keep, as_tuple=True)  # these, both in order
    hb, hh, hr = hole
    mb, mh, mr = move
    dst = st["table"][hb, hh, hr // page].long()
    src = st["table"][mb, mh, mr // page].long()
    for i in range(2):
        st["pool"][i][dst, hr % page] = st["pool"][i][src, mr % page]
    inside = row < m
    st["w_out"].copy_(torch.where(inside, st["w"], st["w_out"]))
    st["pos_out"].copy_(torch.where(inside, st["pos"], st["pos_out"]))
    st["w_out"][hole] = st["w"][move]
    st["pos_out"][hole] = st["pos"][move]
    st["lens_out"].copy_(m[..., 0])
    return _evicted(st)


def _rows(case):
    """Mean number of valid rows over all pairs of a case (lengths are spread
    evenly over the logarithm of [max_len / 8, max_len])."""
    n = case["max_len"]
    pairs = case["B"] * case["H"]
    if case["lens"] == "full" or n < 16:
        return pairs * n
    empty = case["H"] if case["lens"] == "heads" and case["B"] > 8 else 0
    return n + (pairs - 1 - empty) * n * (1 - 1 / 8) / math.log(8)


def work(case):
    """Bytes and operations that a pass cannot do without: every valid K and V
    row once for attend (and the weights read and written), the new rows read
    and written for append; for evict the weights and positions read, those of
    the kept rows written, and the rows that move read and written."""
    d, es = case["d"], 4 if case["dtype"] == "f32" else 2
    pairs = case["B"] * case["H"]
    if case["op"] == "attend":
        rows = _rows(case)
        heads = case["B"] * case["Hq"]
        return {"bytes": rows * (2 * d * es + (8 if case["weights"] else 0)) + heads * (d * es + d * 4 + 4),
                "flops": rows * (case["Hq"] // case["H"]) * 4 * d}
    if case["op"] == "append":
        some = case["n_new"] if case["n_new"] < 4 else case["n_new"] * 5 / 8  # the mean of _new_counts
        rows = case["H"] * (case["n_new"] + (case["B"] - 1) * some)
        return {"bytes": rows * (2 * 2 * d * es + 4 + 4 + 4), "flops": 0}
    rows = _rows(case)
    each = rows / pairs
    kept = min(each, max(case["budget"], case["first"] + case["recent"]))
    # of the kept rows, the share above row `kept` moves down
    moved = kept * max(0.0, each - kept) / each
    return {"bytes": rows * 8 + pairs * (kept * 8 + moved * 2 * 2 * d * es), "flops": 0}


def exact(case, seed):
    """What run() returns, from the definitions, one (sequence, kv-head) at a
    time in 64 bits."""
    st = _inputs(case, seed)
    B, H, Hq, d, page = (case[k] for k in ("B", "H", "Hq", "d", "page"))
    lens = st["lens"].tolist()

    def rows_of(i, b, h, count):
        ids = st["table"][b, h, :-(-count // page)].long()
        return st["pool"][i].index_select(0, ids).reshape(-1, d)[:count].double()

    if case["op"] == "attend":
        G = Hq // H
        out = torch.zeros(B, Hq, d, dtype=torch.float64)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
        w = st["w"].double().cpu() if "w" in st else None
        for b in range(B):
            for h in range(H):
                n = lens[b][h]
                if n == 0:
                    continue
                q = st["q"][b, h * G:(h + 1) * G].double()
                logit = (rows_of(0, b, h, n) @ q.T) * d ** -0.5  # [n, G]
                top = logit.max(dim=0).values
                p = (logit - top).exp()
                z = p.sum(dim=0)
                p /= z
                out[b, h * G:(h + 1) * G] = (p.T @ rows_of(1, b, h, n)).cpu()
                lse[b, h * G:(h + 1) * G] = (top + z.log()).cpu()
                if w is not None:
                    w[b, h, :n] = w[b, h, :n] * case["decay"] + p.sum(dim=1).cpu()
        got = {"out": out, "lse": lse}
        if w is not None:
            got["weights"] = w
        return got
    if case["op"] == "append":
        w = st["w"].double().cpu()
        for b in range(B):
            n = int(st["count"][b])
            for h in range(H):
                w[b, h, lens[b][h] - n:lens[b][h]] = st["tok_w"][b, h, :n].double().cpu()
        return {"pool": None, "weights": w, "pos": None}
    w_all, p_all = st["w"].cpu(), st["pos"].cpu()
    w_out = torch.zeros(w_all.shape, dtype=torch.float64)
    for b in range(B):
        for h in range(H):
            n = lens[b][h]
            m = min(n, max(case["budget"], case["first"] + case["recent"]))
            w, p = w_all[b, h, :n].double(), p_all[b, h, :n].long()
            if n == 0:
                continue
            must = (p < case["first"]) | (p > int(p.max()) - case["recent"])
            score = [(0 if g else 1, -x) for g, x in zip(must.tolist(), w.tolist())]
            kept = set(sorted(range(n), key=score.__getitem__)[:m])
            late = iter(r for r in range(m, n) if r in kept)
            take = [r if r in kept else next(late) for r in range(m)]
            w_out[b, h, :m] = w[torch.tensor(take, dtype=torch.long)]
    return {"pool": None, "lens": None, "weights": w_out, "pos": None}
