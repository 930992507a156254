"""Cases and plain forms of the operators at the vocabulary end of a decoding step.

A decoding or verification step starts with token ids and ends with a distribution over the
vocabulary.  Four operators, each in its plain form (elementary torch operations, float32) and, with
``own`` set, through the package's entry points:

  embed      rows of a weight matrix by token id, scaled (the matrix held as a W12 record)
  mx4_copy   the microscaled 4-bit copy of a weight matrix for the Q pass, built and read back
  mx4_gemm   the Q pass on that copy: y = x Wq^T
  logprobs   log probabilities of given tokens, entropy and top alternatives of rows of logits

The 4-bit copy keeps the record's escapes exact: per row, the 16-binade exponent window that holds
the most weights (ties to the smallest base); weights outside it (zeros, Inf and NaN always) stay
as they are.  In-window weights are quantised in blocks of 32 columns: block scale 2^(e - 2) with e
the exponent of the block's largest in-window magnitude, each weight divided by it and rounded to
the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} (ties to the even code, magnitudes above 6 to 6).
"""
import math

import torch

own = False

ATTN = (5120, 5120)
GATE_UP = (34816, 5120)
DOWN = (5120, 17408)
VOCAB = (152064, 5120)


def listed():
    """The listed cases (sizes: the projections and the LM head of a 27B-class model)."""
    return [
        # the ids of a 16-node draft tree
        dict(name="embed_tree_16", op="embed", n=VOCAB[0], k=VOCAB[1], m=16, scale=1.0),
        # a long prompt, with the square root of the width as the scale some models apply
        dict(name="embed_prompt_4096", op="embed", n=VOCAB[0], k=VOCAB[1], m=4096, scale=math.sqrt(VOCAB[1])),
        # one layer's projections converted for the Q pass
        dict(name="mx4_copy_attn", op="mx4_copy", n=ATTN[0], k=ATTN[1]),
        dict(name="mx4_copy_gate_up", op="mx4_copy", n=GATE_UP[0], k=GATE_UP[1]),
        # a single token through a square projection: latency and a 14 MB stream
        dict(name="mx4_gemm_attn_m1", op="mx4_gemm", n=ATTN[0], k=ATTN[1], m=1, bf16=False),
        # the Q pass of a 16-node tree over the LM head
        dict(name="mx4_gemm_lm_head_m16", op="mx4_gemm", n=VOCAB[0], k=VOCAB[1], m=16, bf16=False),
        # a batch of trees through the MLP's first product
        dict(name="mx4_gemm_gate_up_m64", op="mx4_gemm", n=GATE_UP[0], k=GATE_UP[1], m=64, bf16=False),
        # long rows, an odd number of tokens, bfloat16 outputs
        dict(name="mx4_gemm_down_m7_bf16", op="mx4_gemm", n=DOWN[0], k=DOWN[1], m=7, bf16=True),
        # plain decoding: one row, its sampled token, eight alternatives
        dict(name="logprobs_m1", op="logprobs", m=1, n=VOCAB[0], pad=0, bf16=False, tokens=1, top=8, masked=0.0),
        # a verification step over 64 nodes, four candidates a node, alternatives for the next tree
        dict(name="logprobs_tree_64", op="logprobs", m=64, n=VOCAB[0], pad=0, bf16=False, tokens=4, top=16, masked=0.0),
        # scoring a given text: many rows, bfloat16 logits
        dict(name="logprobs_score_1024_bf16", op="logprobs", m=1024, n=VOCAB[0], pad=0, bf16=True, tokens=1, top=1,
             masked=0.0),
        # a ragged vocabulary cut out of padded rows, most of it masked, some rows wholly
        dict(name="logprobs_ragged_masked", op="logprobs", m=33, n=32001, pad=63, bf16=False, tokens=2, top=5,
             masked=0.97),
    ]


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    def between(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["embed", "mx4_copy", "mx4_gemm", "logprobs"])
    if op == "logprobs":
        n = between(1000, 200000)
        m = between(1, min(1024, max(1, (1024 * 152064) // n)))
        top = rng.choice([0, 1, 3, 8, 20, 32])
        return dict(op=op, m=m, n=n, pad=rng.choice([0, 0, 1, 17, 64]), bf16=rng.random() < 0.5,
                    tokens=rng.choice([1, 2, 5]), top=top, masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
    k = 128 * between(4, 136)
    n = between(64, min(152064, (34816 * 5120) // k))
    if op == "embed":
        return dict(op=op, n=n, k=k, m=between(1, 4096), scale=rng.choice([1.0, 0.5, math.sqrt(k)]))
    if op == "mx4_copy":
        return dict(op=op, n=n, k=k)
    return dict(op=op, n=n, k=k, m=between(1, 64), bf16=rng.random() < 0.3)


def _weight(gen, n, k):
    """Synthetic bfloat16 weights: a scale per row, rare outliers, a few exact zeros."""
    s = 0.02 * torch.exp(0.5 * torch.randn(n, 1, generator=gen, device="cuda"))
    w = torch.randn(n, k, generator=gen, device="cuda") * s
    u = torch.rand(n, k, generator=gen, device="cuda")
    w = torch.where(u < 7.3e-5, w * 64.0, w)
    w = torch.where(u > 1.0 - 1e-3, torch.zeros_like(w), w)
    return w.to(torch.bfloat16)


def prepare(case, seed):
    """What a caller holds before the call: the weights (own: their W12 record and 4-bit copy), x,
    token ids, logits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "logprobs":
        m, n = case["m"], case["n"]
        full = torch.randn(m, n + case["pad"], generator=gen, device="cuda") * 3.0
        # a trained head is confident on many rows: one token raised by 0 to 20
        hot = torch.randint(0, n, (m, 1), generator=gen, device="cuda")
        full.scatter_add_(1, hot, torch.rand(m, 1, generator=gen, device="cuda") * 20.0)
        if case["masked"] > 0:
            u = torch.rand(m, n + case["pad"], generator=gen, device="cuda")
            full = full.masked_fill(u < case["masked"], -math.inf)
            full[::16] = -math.inf          # a row that its mask leaves nothing
        if case["bf16"]:
            full = full.to(torch.bfloat16)
        st["y"] = full[:, :n]
        tok = torch.randint(0, n, (m, case["tokens"]), generator=gen, device="cuda")
        tok[:, :1] = torch.where(torch.rand(m, 1, generator=gen, device="cuda") < 0.7, hot, tok[:, :1])
        st["tokens"] = tok
        return st
    n, k = case["n"], case["k"]
    w = _weight(gen, n, k)
    if op == "embed":
        st["ids"] = torch.randint(0, n, (case["m"],), generator=gen, device="cuda")
    if op == "mx4_gemm":
        st["x"] = torch.randn(case["m"], k, generator=gen, device="cuda").to(torch.bfloat16)
    if own:
        from lossless_bit_weight_02_amd import w12
        st["rec"] = w12.encode(w)
        if op == "mx4_gemm":
            st["copy"] = w12.mx4_build(st["rec"])
        return st
    if op == "mx4_gemm":
        # the copy as a caller without the package would keep it: codes (twice the value), block
        # exponents, and the exact weights outside the windows
        codes, exps, rows, cols, vals = [], [], [], [], []
        for r0 in range(0, n, 16384):
            c, e, esc = _quantise(w[r0:r0 + 16384])
            codes.append(c)
            exps.append(e)
            r, col = esc.nonzero(as_tuple=True)
            rows.append(r + r0)
            cols.append(col)
            vals.append(w[r0:r0 + 16384][r, col])
        st.update(codes=torch.cat(codes), exps=torch.cat(exps), rows=torch.cat(rows), cols=torch.cat(cols),
                  vals=torch.cat(vals))
        return st
    st["w"] = w
    return st


def _windows(w):
    """True where a weight lies outside its row's exponent window."""
    e = (w.view(torch.int16).to(torch.int64) >> 7) & 0xFF
    hist = torch.zeros(w.shape[0], 256, dtype=torch.int64, device=w.device)
    hist.scatter_add_(1, e, torch.ones_like(e))
    hist[:, 0] = 0
    hist[:, 255] = 0
    cs = torch.cumsum(hist, 1)
    cover = cs[:, 16:255] - cs[:, 0:239]                     # bases 1 .. 239
    # the largest cover, ties to the smallest base
    base = 1 + (cover * 256 - torch.arange(239, device=w.device)).argmax(1, keepdim=True)
    return (e < base) | (e > base + 15) | (e == 0) | (e == 255)


def _power(e):
    """Two to the integers e (int32), exactly."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(w):
    """(int8 codes holding twice the value, int16 exponent of each 32-column block's scale, escapes)."""
    n, k = w.shape
    esc = _windows(w)
    v = torch.where(esc, torch.zeros_like(w), w).float().view(n, k // 32, 32)
    big = v.abs().amax(2, keepdim=True)
    ebits = (big.view(torch.int32) >> 23) & 0xFF
    ex = torch.where(big > 0, ebits - 129, torch.zeros_like(ebits))
    mag = v.abs() * _power(-ex)
    step = torch.where(mag < 2.0, 0.5, torch.where(mag < 4.0, 1.0, 2.0))
    q = torch.clamp(torch.round(mag / step) * step, max=6.0)
    q = torch.where(v < 0, -q, q)
    return (2.0 * q).to(torch.int8).view(n, k), ex.view(n, k // 32).to(torch.int16), esc


def _values(codes, exps):
    """float32 values of codes (twice the value) under their block exponents."""
    n, k = codes.shape
    v = codes.float().view(n, k // 32, 32) * _power(exps.to(torch.int32) - 1).unsqueeze(2)
    return v.view(n, k)


def _logprobs(y, tokens, top):
    """Plain form: log probabilities of `tokens`, entropy, and the `top` largest with their indices.
    A row without any finite logit gives -Inf and entropy 0; equal logits go by the lower index."""
    x = y.float()
    big = x.amax(1, keepdim=True)
    big = torch.where(torch.isinf(big), torch.zeros_like(big), big)
    d = x - big
    e = torch.exp(d)
    # sums over a whole vocabulary: 64 bits
    s = e.sum(1, keepdim=True, dtype=torch.float64)
    t = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, keepdim=True, dtype=torch.float64)
    some = s > 0
    safe = torch.where(some, s, torch.ones_like(s))
    lse = torch.log(safe)
    logp = torch.where(some, d.gather(1, tokens).double() - lse, -math.inf)
    ent = torch.where(some, lse - t / safe, 0.0)[:, 0]
    if top == 0:
        return logp.float(), ent.float()
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    val, idx = val[:, :top], idx[:, :top]
    tl = torch.where(some, (val - big).double() - lse, -math.inf)
    return logp.float(), ent.float(), idx.to(torch.int32), tl.float()


def run(state):
    """One pass through the operator, and its outputs."""
    case = state["case"]
    op = case["op"]
    if own:
        from lossless_bit_weight_02_amd import w12
        if op == "embed":
            return w12.embed(state["ids"], state["rec"], scale=case["scale"])
        if op == "mx4_copy":
            return w12.mx4_decode(w12.mx4_build(state["rec"]))
        if op == "mx4_gemm":
            return w12.mx4_gemm(state["x"], state["copy"], out_bf16=case["bf16"])
        r = w12.logprobs(state["y"], state["tokens"], top=case["top"])
        if case["top"] == 0:
            return r.logp, r.entropy
        return r.logp, r.entropy, r.top_index, r.top_logp
    if op == "embed":
        return (state["w"][state["ids"]].float() * case["scale"]).to(torch.bfloat16)
    if op == "mx4_copy":
        w = state["w"]
        codes, exps, esc = _quantise(w)
        return torch.where(esc, w.float(), _values(codes, exps)).to(torch.bfloat16)
    if op == "mx4_gemm":
        wq = _values(state["codes"], state["exps"])
        wq[state["rows"], state["cols"]] = state["vals"].float()
        y = state["x"].float() @ wq.t()
        return y.to(torch.bfloat16) if case["bf16"] else y
    return _logprobs(state["y"], state["tokens"], case["top"])


def work(case):
    """Bytes and operations of one pass that it cannot do without."""
    op = case["op"]
    if op == "logprobs":
        m, n = case["m"], case["n"]
        out = m * (case["tokens"] * 4 + 4 + case["top"] * 8)
        # a subtraction, an exponential and two multiply-adds a logit
        return dict(bytes=m * n * (2 if case["bf16"] else 4) + m * case["tokens"] * 8 + out, flops=6 * m * n)
    n, k = case["n"], case["k"]
    if op == "embed":
        # 12 bits a weight read, bfloat16 written
        m = case["m"]
        return dict(bytes=m * (k * 3 // 2 + k * 2 + 8), flops=m * k)
    copy = n * k * 17 // 32                                  # 4 bits a weight and a byte a block
    if op == "mx4_copy":
        # the record read, the copy written and read back, its values written
        return dict(bytes=n * k * 3 // 2 + 2 * copy + 2 * n * k, flops=4 * n * k)
    m = case["m"]
    return dict(bytes=copy + 2 * m * k + m * n * (2 if case["bf16"] else 4), flops=2 * m * n * k)


def _exact_copy(w):
    """float64 values the Q pass sees, from the definition: windows by counting, codes by the
    thresholds between neighbouring values."""
    n, k = w.shape
    raw = w.view(torch.int16).to(torch.int64) & 0xFFFF
    e = (raw // 128) % 256
    rows = torch.arange(n, device=w.device).unsqueeze(1)
    counts = torch.bincount((rows * 256 + e).flatten(), minlength=n * 256).view(n, 256)
    best = torch.full((n,), -1, dtype=torch.int64, device=w.device)
    base = torch.zeros(n, dtype=torch.int64, device=w.device)
    for b in range(1, 240):
        c = counts[:, b:b + 16].sum(1) if b + 16 <= 255 else counts[:, b:255].sum(1)
        better = c > best
        best = torch.where(better, c, best)
        base = torch.where(better, torch.full_like(base, b), base)
    inside = (e >= base.unsqueeze(1)) & (e < base.unsqueeze(1) + 16) & (e > 0) & (e < 255)
    v = w.double()
    q = torch.where(inside, v, torch.zeros_like(v)).view(n, k // 32, 32)
    top = torch.where(inside, e, torch.zeros_like(e)).view(n, k // 32, 32).amax(2, keepdim=True)
    scale = ((top - 129 + 1023) << 52).view(torch.float64)      # 2^(top - 129)
    mag = q.abs() / scale
    # from one value to the next: past the midpoint, or at it where the next code is even
    grid = 0.5 * ((mag > 0.25).double() + (mag >= 0.75).double() + (mag > 1.25).double() + (mag >= 1.75).double())
    grid += (mag > 2.5).double() + (mag >= 3.5).double() + 2.0 * (mag > 5.0).double()
    out = (torch.sign(q) * grid * scale).view(n, k)
    return torch.where(inside, out, v)


def exact(case, seed):
    """run's outputs in 64 bits from the operator's definition."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "logprobs":
        # the logits and ids of prepare; its bfloat16 rounding is part of the input
        st = prepare(case, seed)
        x, tok, top = st["y"].double(), st["tokens"], case["top"]
        m = x.shape[0]
        logp = torch.empty(m, case["tokens"], dtype=torch.float64, device="cuda")
        ent = torch.empty(m, dtype=torch.float64, device="cuda")
        idx = torch.empty(m, max(top, 1), dtype=torch.int32, device="cuda")
        tlp = torch.empty(m, max(top, 1), dtype=torch.float64, device="cuda")
        for r in range(m):
            row = x[r]
            if not bool(torch.isfinite(row).any()):
                logp[r], ent[r], tlp[r] = -math.inf, 0.0, -math.inf
                idx[r] = torch.arange(max(top, 1), device="cuda")
                continue
            z = torch.logsumexp(row, 0)
            lp = row - z
            logp[r] = lp[tok[r]]
            live = lp[torch.isfinite(lp)]
            ent[r] = -(live.exp() * live).sum()
            order = torch.sort(row, descending=True, stable=True).indices[:max(top, 1)]
            idx[r], tlp[r] = order.to(torch.int32), lp[order]
        return (logp, ent) if top == 0 else (logp, ent, idx, tlp)
    n, k = case["n"], case["k"]
    w = _weight(gen, n, k)
    if op == "embed":
        ids = torch.randint(0, n, (case["m"],), generator=gen, device="cuda")
        return w[ids].double() * case["scale"]
    if op == "mx4_copy":
        return torch.cat([_exact_copy(w[r0:r0 + 8192]) for r0 in range(0, n, 8192)])
    x = torch.randn(case["m"], k, generator=gen, device="cuda").to(torch.bfloat16).double()
    return torch.cat([x @ _exact_copy(w[r0:r0 + 8192]).t() for r0 in range(0, n, 8192)], 1)
