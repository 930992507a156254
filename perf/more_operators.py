"""Cases and plain forms of the operators between the products of a decoding step.

A decoding or verification step runs matrix products over W12 records; between them stand three
operators, each here in its plain form (elementary torch operations in 32 bits, 64 where a border
between tokens needs them) and, with ``own`` set, through the package's entry points:

  append     rows of the stacked q/k/v product: q and k rotated by position, k and v into the pages
             of a cache (bfloat16, or 8-bit e4m3 with a scale per head)
  attention  the new tokens of each sequence (one, a chain or a tree of drafts) over that cache
  sample     a token per row of logits: temperature, top-k, top-p, min-p and a given uniform number

Row j of a sequence's T new tokens has place lens - T + j in the cache.  It sees the places before
lens - T and, of the new ones, those up to its own, or those whose bit its tree mask has.
"""
import math

import torch

own = False

VOCAB = 152064
PHI, PHI2 = 0.6180339887498949, 0.7548776662466927


def listed():
    """The listed cases (sizes: the stacked q/k/v projection and the LM head of a 27B-class model)."""
    return [
        # plain decoding of one request: a call's latency
        dict(name="append_token", op="append", seqs=1, lo=700, hi=700, new=1, hq=48, hkv=8, d=128, page=64, rot=128,
             inter=False, f32=False, e4m3=False, nhd=False),
        # drafts of a batch of requests into an 8-bit cache, from the products' float outputs
        dict(name="append_drafts_e4m3", op="append", seqs=64, lo=20, hi=120, new=16, hq=24, hkv=4, d=256, page=64,
             rot=64, inter=False, f32=True, e4m3=True, nhd=False),
        # prompts taken in whole: a stream of rows
        dict(name="append_prompts", op="append", seqs=5, lo=1024, hi=4096, new=-1, hq=48, hkv=8, d=128, page=16,
             rot=128, inter=True, f32=True, e4m3=False, nhd=True),
        # one request early in its answer: latency
        dict(name="attention_token_short", op="attention", seqs=1, lo=517, hi=517, new=1, tree=False, hq=48, hkv=8,
             d=128, page=64, e4m3=False, nhd=False),
        # one request over a long document: one cache read by the whole chip
        dict(name="attention_token_long", op="attention", seqs=1, lo=131071, hi=131071, new=1, tree=False, hq=48,
             hkv=8, d=128, page=64, e4m3=False, nhd=False),
        # a batch of requests of uneven lengths
        dict(name="attention_batch_64", op="attention", seqs=64, lo=60, hi=8192, new=1, tree=False, hq=48, hkv=8,
             d=128, page=64, e4m3=False, nhd=False),
        # verification of draft trees of up to 16 nodes over an 8-bit cache
        dict(name="attention_trees_e4m3", op="attention", seqs=16, lo=1000, hi=16384, new=16, tree=True, hq=24,
             hkv=4, d=256, page=64, e4m3=True, nhd=False),
        # a full server: many requests, small pages, rows of all heads side by side
        dict(name="attention_batch_256", op="attention", seqs=256, lo=400, hi=4096, new=1, tree=False, hq=48, hkv=8,
             d=128, page=16, e4m3=False, nhd=True),
        # one request's next token
        dict(name="sample_1", op="sample", m=1, n=VOCAB, pad=0, bf16=False, temp=0.7, k=20, p=0.8, minp=0.0,
             mixed=False, masked=0.0),
        # the nodes of a draft tree, nucleus sampling
        dict(name="sample_tree_64", op="sample", m=64, n=VOCAB, pad=0, bf16=False, temp=1.0, k=0, p=0.95, minp=0.0,
             mixed=False, masked=0.0),
        # a full server: every request with parameters of its own
        dict(name="sample_mixed_256_bf16", op="sample", m=256, n=VOCAB, pad=0, bf16=True, temp=1.0, k=0, p=1.0,
             minp=0.0, mixed=True, masked=0.0),
        # a ragged vocabulary cut out of padded rows, most of it masked (a grammar), some rows wholly
        dict(name="sample_ragged_masked", op="sample", m=33, n=32001, pad=63, bf16=False, temp=1.5, k=0, p=0.9,
             minp=0.02, mixed=False, masked=0.97),
    ]


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    def between(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append", "attention", "attention", "sample"])
    if op == "sample":
        n = between(1000, 200000)
        m = between(1, min(256, max(1, (256 * 152064) // n)))
        return dict(op=op, m=m, n=n, pad=rng.choice([0, 0, 1, 17, 64]), bf16=rng.random() < 0.5,
                    temp=rng.choice([0.0, 0.3, 0.7, 1.0, 1.5]), k=rng.choice([0, 0, 1, 20, 50, 1000]),
                    p=rng.choice([1.0, 0.99, 0.95, 0.8, 0.3]), minp=rng.choice([0.0, 0.0, 0.02, 0.1]),
                    mixed=rng.random() < 0.25, masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 6, 8, 16])
    page = rng.choice([16, 32, 48, 64, 128])
    e4m3, nhd = rng.random() < 0.4, rng.random() < 0.5
    if op == "append":
        seqs = between(1, 256)
        new = rng.choice([1, 1, between(1, 16), -1])
        hi = between(16, max(17, min(4096, 80_000_000 // ((hq + 2 * hkv) * d * seqs))))
        new = min(new, hi)
        return dict(op=op, seqs=seqs, lo=max(1, hi // 5), hi=hi, new=new, hq=hq, hkv=hkv, d=d, page=page,
                    rot=rng.choice([d, d // 2, d // 4]), inter=rng.random() < 0.5, f32=rng.random() < 0.5, e4m3=e4m3,
                    nhd=nhd)
    seqs = between(1, 256)
    new = rng.choice([1, 1, 1, between(1, 32)])
    hi = between(16, max(17, min(131072, 500_000_000 // (seqs * hkv * max(d, new * hq // hkv)))))
    return dict(op=op, seqs=seqs, lo=max(1, hi // rng.choice([1, 3, 100])), hi=hi, new=new,
                tree=new > 1 and rng.random() < 0.5, hq=hq, hkv=hkv, d=d, page=page, e4m3=e4m3, nhd=nhd)


def _lengths(case):
    """(lengths of the cache, numbers of new tokens) of the case's sequences."""
    lo, hi, new = case["lo"], case["hi"], case["new"]
    lens, news = [], []
    for i in range(case["seqs"]):
        n = int(round(lo * (hi / lo) ** ((0.5 + (i + 1) * PHI) % 1.0))) if hi > lo else hi
        lens.append(n)
        t = 1 if new == 1 else n if new < 0 else 1 + int(((i + 1) * PHI2 % 1.0) * new)
        news.append(min(t, n))
    return lens, news


def _cast(x, scale, e4m3):
    """x [.., heads, ..] as the cache holds it; scale broadcasts over x."""
    if not e4m3:
        return x.to(torch.bfloat16)
    return torch.clamp(x / scale, -448.0, 448.0).to(torch.float8_e4m3fn)


def prepare(case, seed):
    """What a caller holds before the call: the cache and its tables, the product's rows, the logits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "sample":
        m, n = case["m"], case["n"]
        full = torch.randn(m, n + case["pad"], generator=gen, device="cuda") * 2.0
        # a trained head raises some tokens far above the rest, on some rows one of them alone
        hot = torch.randint(0, n, (m, 1), generator=gen, device="cuda")
        hot = (hot + torch.arange(48, device="cuda") * (n // 48)) % n
        full.scatter_add_(1, hot, torch.rand(m, 48, generator=gen, device="cuda") ** 2 * 16.0)
        full.scatter_add_(1, hot[:, :1], torch.rand(m, 1, generator=gen, device="cuda") * 14.0)
        if case["masked"] > 0:
            u = torch.rand(m, n + case["pad"], generator=gen, device="cuda")
            full = full.masked_fill(u < case["masked"], -math.inf)
            full[::16] = -math.inf          # a row that its mask leaves nothing
        if case["bf16"]:
            full = full.to(torch.bfloat16)
        st["y"] = full[:, :n]
        st["u"] = torch.rand(m, generator=gen, device="cuda")
        if case["mixed"]:
            sets = [(0.7, 20, 0.8, 0.0), (1.0, 0, 1.0, 0.0), (1.2, 0, 0.98, 0.0), (0.0, 0, 1.0, 0.0),
                    (1.0, 0, 1.0, 0.05), (0.6, 50, 0.95, 0.01)]
        else:
            sets = [(case["temp"], case["k"], case["p"], case["minp"])]
        rows = [sets[i % len(sets)] for i in range(m)]
        st["temp"] = torch.tensor([r[0] for r in rows], device="cuda")
        st["k"] = torch.tensor([r[1] for r in rows], dtype=torch.int32, device="cuda")
        st["p"] = torch.tensor([r[2] for r in rows], device="cuda")
        st["minp"] = torch.tensor([r[3] for r in rows], device="cuda")
        return st
    lens, news = _lengths(case)
    hq, hkv, d, page, seqs = case["hq"], case["hkv"], case["d"], case["page"], case["seqs"]
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((seqs, max(need)), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(max(need), device="cuda")
    nd = torch.tensor(need, device="cuda")
    table[col < nd[:, None]] = order[:sum(need)]
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = [0]
    for t in news:
        starts.append(starts[-1] + t)
    m = starts[-1]
    st["starts"] = None if case["new"] == 1 else torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["scales"] = (None, None)
    if case["e4m3"]:
        st["scales"] = tuple((0.5 + torch.rand(hkv, generator=gen, device="cuda")) * (6.0 / 448.0) for _ in range(2))
    # pages as [pages, heads, page, dim], in memory in this order or with the heads of a token side by side
    kv = []
    for sc in st["scales"]:
        shape = (pages, page, hkv, d) if case["nhd"] else (pages, hkv, page, d)
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        if sc is not None:
            sc = sc[None, None, :, None] if case["nhd"] else sc[None, :, None, None]
        x = _cast(x, sc, case["e4m3"])
        kv.append(x.transpose(1, 2) if case["nhd"] else x)
    st["cache"] = tuple(kv)
    st["tree"] = None
    if case["op"] == "append":
        y = torch.randn(m, (hq + 2 * hkv) * d, generator=gen, device="cuda")
        st["y"] = y if case["f32"] else y.to(torch.bfloat16)
        # the rotation's table: cos and sin of position * 10000^(-2 i / rot), from 64 bits
        half = case["rot"] // 2
        ang = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            10000.0, -torch.arange(half, device="cuda", dtype=torch.float64) / half)
        st["rope"] = torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()
    else:
        st["q"] = (torch.randn(m, hq * d, generator=gen, device="cuda") * 2.0).to(torch.bfloat16)
        if case["tree"]:
            # a node sees itself and its ancestors
            r = torch.rand(m, generator=gen, device="cuda").tolist()
            masks = []
            for s in range(seqs):
                for j in range(news[s]):
                    up = masks[starts[s] + int(r[starts[s] + j] * j)] if j else 0
                    masks.append(up | 1 << j)
            st["tree"] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in masks], dtype=torch.int64,
                                      device="cuda")
    if own:
        from lossless_bit_weight_02_amd import w12
        st["kv"] = w12.KVCache(*st["cache"], *st["scales"])
        st["batch"] = w12.KVBatch(table, st["lens"], q_start=st["starts"], tree=st["tree"])
    return st


def _places(state, m):
    """Per row its sequence, its place in the cache, the place of its sequence's first new token."""
    lens = state["lens"].long()
    row = torch.arange(m, device="cuda")
    if state["starts"] is None:
        return row, lens - 1, lens - 1
    starts = state["starts"].long()
    seq = (row[:, None] >= starts[None, 1:]).sum(1)
    base = (lens - (starts[1:] - starts[:-1]))[seq]
    return seq, base + row - starts[seq], base


def _rotate(x, cos, sin, rot, inter):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, s = cos[:, None, :], sin[:, None, :]
    r = (a * c - b * s, b * c + a * s)
    head = torch.stack(r, -1).flatten(-2) if inter else torch.cat(r, -1)
    return torch.cat([head, x[..., rot:]], -1)


def _append(state):
    case = state["case"]
    hq, hkv, d, page, rot = case["hq"], case["hkv"], case["d"], case["page"], case["rot"]
    y = state["y"].float()
    m = y.shape[0]
    seq, place, _ = _places(state, m)
    x = y.view(m, hq + 2 * hkv, d)
    cs = state["rope"][place]
    qk = _rotate(x[:, :hq + hkv], cs[:, :rot // 2], cs[:, rot // 2:], rot, case["inter"])
    pg = state["table"][seq, place // page].long()
    off = place % page
    for i, (vals, sc) in enumerate(zip((qk[:, hq:], x[:, hq + hkv:]), state["scales"])):
        c = state["cache"][i]
        v = _cast(vals, None if sc is None else sc[None, :, None], case["e4m3"])
        raw = torch.uint8 if case["e4m3"] else torch.bfloat16
        c.view(raw)[pg, :, off] = v.view(raw)
    return (qk[:, :hq].reshape(m, hq * d).to(torch.bfloat16), *state["cache"])


def _attention(state):
    case = state["case"]
    hq, hkv, d, page, seqs = case["hq"], case["hkv"], case["d"], case["page"], case["seqs"]
    q = state["q"].float()
    m, g = q.shape[0], hq // hkv
    lens = state["lens"].long()
    big = state["table"].shape[1] * page
    t = torch.arange(big, device="cuda")
    pg = state["table"][:, t // page].long().clamp(min=0)          # [seqs, big]
    h = torch.arange(hkv, device="cuda")
    raw = torch.uint8 if case["e4m3"] else torch.bfloat16
    kk, vv = (c.view(raw)[pg[:, None, :], h[None, :, None], (t % page)[None, None, :]].view(c.dtype).float()
              for c in state["cache"])                             # [seqs, hkv, big, d]
    if case["e4m3"]:
        kk = kk * state["scales"][0][None, :, None, None]
        vv = vv * state["scales"][1][None, :, None, None]
    seq, place, base = _places(state, m)
    j = place - base
    width = 1 if state["starts"] is None else min(case["new"], case["hi"])
    full = torch.zeros(seqs, width, hq, d, device="cuda")
    full[seq, j] = q.view(m, hq, d)
    rows = full.view(seqs, width, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, width * g, d)
    s = torch.matmul(rows, kk.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    bit = t[None, :] - base[:, None]                               # [m, big]
    if state["tree"] is None:
        new = bit <= j[:, None]
    else:
        new = ((state["tree"][:, None] >> bit.clamp(0, 63)) & 1 == 1) & (bit < 64)
    sees = ((bit < 0) | new) & (t[None, :] < lens[seq][:, None])
    mask = torch.zeros(seqs, width, big, dtype=torch.bool, device="cuda")
    mask[seq, j] = sees
    mask = mask[:, None, :, None, :].expand(seqs, 1, width, g, big).reshape(seqs, 1, width * g, big)
    s = torch.where(mask, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    tot = e.sum(-1, keepdim=True)
    o = torch.matmul(e, vv) / torch.where(tot > 0, tot, torch.ones_like(tot))
    o = o.view(seqs, hkv, width, g, d).permute(0, 2, 1, 3, 4).reshape(seqs, width, hq * d)
    return o[seq, j].to(torch.bfloat16)


def _sample(state):
    """Token, log probability among the kept ones, number kept; -1, -Inf and 0 for a row without any."""
    x = state["y"].double()
    m, n = x.shape
    temp = state["temp"].double()[:, None]
    best = x.amax(1, keepdim=True)
    some = best > -math.inf
    diff = x - torch.where(some, best, torch.zeros_like(best))
    hard = temp <= 0.0
    z = torch.where(diff == 0, diff, torch.where(hard, -math.inf, diff / torch.where(hard, torch.ones_like(temp), temp)))
    order = torch.sort(state["y"].float(), dim=1, descending=True, stable=True).indices
    zs = z.gather(1, order)
    w = torch.exp(zs)
    at = torch.arange(n, device="cuda")[None, :]
    k = state["k"].long()[:, None]
    keep = (zs > -math.inf) & torch.where(hard, at < 1, (k <= 0) | (at < k))
    mass = torch.cumsum(torch.where(keep, w, 0.0), 1)
    p = state["p"].double()[:, None]
    first = at == 0
    keep &= first | (p >= 1.0) | (mass - w < p * mass[:, -1:])
    keep &= first | (w >= state["minp"].double()[:, None])
    keep &= some
    wk = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    cum = torch.cumsum(wk, 1)
    tot = cum[:, -1:]
    tok = (cum <= state["u"].double()[:, None] * tot).sum(1, keepdim=True).clamp(max=n - 1)
    logp = torch.where(some, z.gather(1, tok) - torch.log(torch.where(some, tot, 1.0)), -math.inf)
    tok = torch.where(some, tok, -1)
    return tok[:, 0].to(torch.int32), logp[:, 0].float(), keep.sum(1).to(torch.int32)


def run(state):
    """One pass through the operator, and its outputs."""
    case = state["case"]
    op = case["op"]
    if own:
        from lossless_bit_weight_02_amd import w12
        if op == "append":
            q = w12.kv_append(state["y"], state["kv"], state["batch"], rope=state["rope"],
                              interleaved=case["inter"])
            return (q, *state["cache"])
        if op == "attention":
            return w12.attention(state["q"], state["kv"], state["batch"])
        r = w12.sample(state["y"], state["u"], temperature=state["temp"], top_k=state["k"], top_p=state["p"],
                       min_p=state["minp"])
        return r.token, r.logp, r.kept
    if op == "append":
        return _append(state)
    return _attention(state) if op == "attention" else _sample(state)


def work(case):
    """Bytes and operations of one pass that it cannot do without."""
    if case["op"] == "sample":
        m, n = case["m"], case["n"]
        # a difference, a product, an exponential and a sum a logit
        return dict(bytes=m * n * (2 if case["bf16"] else 4) + 32 * m, flops=4 * m * n)
    lens, news = _lengths(case)
    hq, hkv, d, size = case["hq"], case["hkv"], case["d"], 1 if case["e4m3"] else 2
    m = sum(news)
    if case["op"] == "append":
        src = (hq + 2 * hkv) * d * (4 if case["f32"] else 2)
        return dict(bytes=m * (src + 2 * hq * d + 2 * hkv * d * size + 4 * case["rot"]) + 8 * case["seqs"],
                    flops=m * (hq + hkv) * case["rot"] * 3)
    seen = sum(t * (n - t) + t * (t + 1) // 2 for n, t in zip(lens, news))
    return dict(bytes=sum(lens) * 2 * hkv * d * size + 4 * m * hq * d, flops=4 * seen * hq * d)


def exact(case, seed):
    """run's outputs in 64 bits from the operator's definition, one sequence or row at a time."""
    st = prepare(case, seed)
    if case["op"] == "sample":
        x = st["y"].double()
        m, n = x.shape
        # (whole numbers are compared with the plain form's)
        lp = torch.full((m,), -math.inf, dtype=torch.float64, device="cuda")
        temps, ks, ps, mps, us = (st[a].tolist() for a in ("temp", "k", "p", "minp", "u"))
        for r in range(m):
            row = x[r]
            top = float(row.max())
            if top == -math.inf:
                continue
            live = torch.nonzero(row > -math.inf)[:, 0]
            if temps[r] <= 0:
                lp[r] = 0.0
                continue
            e = (row[live] - top) / temps[r]
            by = torch.sort(e, descending=True, stable=True)
            live, e = live[by.indices], by.values
            if ks[r] > 0:
                live, e = live[:ks[r]], e[:ks[r]]
            prob = torch.softmax(e, 0)
            if ps[r] < 1.0:
                before = torch.cumsum(prob, 0) - prob
                cut = max(1, int((before < ps[r]).sum()))
                live, e, prob = live[:cut], e[:cut], prob[:cut]
            if mps[r] > 0:
                cut = max(1, int((prob >= mps[r] * prob[0]).sum()))
                live, e = live[:cut], e[:cut]
            cols = torch.sort(live)
            le = torch.log_softmax(e, 0)[cols.indices]
            cdf = torch.cumsum(torch.exp(le), 0)
            pick = min(int((cdf <= us[r]).sum()), len(cdf) - 1)
            lp[r] = le[pick]
        return None, lp, None
    lens, news = _lengths(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    kc, vc = (c.double() for c in st["cache"])
    ks, vs = (torch.ones(hkv, dtype=torch.float64, device="cuda") if s is None else s.double() for s in st["scales"])
    first = 0
    if case["op"] == "append":
        y = st["y"].double()
        rot, half = case["rot"], case["rot"] // 2
        # each column's partner and the sign of its sine, columns past rot with the angle 0
        c = torch.arange(d, device="cuda")
        if case["inter"]:
            other, pair = c ^ 1, c // 2
            sign = torch.where(c % 2 == 0, -1.0, 1.0).double()
        else:
            other, pair = (c + half) % rot, c % half
            sign = torch.where(c < half, -1.0, 1.0).double()
        inside = c < rot
        other, pair = torch.where(inside, other, c), torch.where(inside, pair, 0)
        out = torch.empty(y.shape[0], hq, d, dtype=torch.float64, device="cuda")
        for s, (n, t) in enumerate(zip(lens, news)):
            at = torch.arange(n - t, n, device="cuda")
            x = y[first:first + t].view(t, hq + 2 * hkv, d)
            co = torch.where(inside, st["rope"].double()[at][:, pair], 1.0)[:, None, :]
            si = torch.where(inside, st["rope"].double()[at][:, half + pair] * sign, 0.0)[:, None, :]
            r = x * co + x[..., other] * si
            out[first:first + t] = r[:, :hq]
            pg = st["table"][s].long()[at // page]
            kc[pg, :, at % page] = r[:, hq:hq + hkv] / ks[None, :, None]
            vc[pg, :, at % page] = x[:, hq + hkv:] / vs[None, :, None]
            first += t
        if case["e4m3"]:
            kc, vc = kc.clamp(-448.0, 448.0), vc.clamp(-448.0, 448.0)
        return out.view(-1, hq * d), kc, vc
    q = st["q"].double()
    out = torch.empty(q.shape[0], hq, d, dtype=torch.float64, device="cuda")
    tree = None if st["tree"] is None else st["tree"].tolist()
    for s, (n, t) in enumerate(zip(lens, news)):
        pg = st["table"][s, :(n + page - 1) // page].long()
        k = kc[pg].transpose(0, 1).reshape(hkv, -1, d)[:, :n] * ks[:, None, None]
        v = vc[pg].transpose(0, 1).reshape(hkv, -1, d)[:, :n] * vs[:, None, None]
        for j in range(t):
            seen = list(range(n - t, n - t + j + 1)) if tree is None else \
                [n - t + b for b in range(t) if tree[first + j] >> b & 1]
            hide = torch.zeros(n, dtype=torch.bool, device="cuda")
            hide[n - t:] = True
            hide[seen] = False
            x = q[first + j].view(hkv, hq // hkv, d) / math.sqrt(d)
            a = torch.softmax(torch.matmul(x, k.transpose(1, 2).contiguous()).masked_fill(hide, -math.inf), -1)
            out[first + j] = torch.matmul(a, v).view(hq, d)
        first += t
    return out.view(-1, hq * d)
