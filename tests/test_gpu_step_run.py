"""A decoding step's operators together: a small model's prompt, single tokens and a tree of drafts through the
package's calls, each stage against the float64 oracle on what it was given (tolerances as in
test_gpu_step); the same step captured and replayed, calls on several streams, scratch.
"""
import numpy as np
import pytest

from lossless_bit_weight_02_amd import synth
from tests.gpu_util import say, to_dev
from tests.test_gpu_step import Step, check_append, check_attention, check_sample, f64, params, queries, rope_table

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

VOCAB, HIDDEN, INNER, HQ, HEADS, DIM, LAYERS = 2003, 512, 640, 8, 2, 64, 2


@pytest.fixture(scope="module")
def w12():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lossless_bit_weight_02_amd import w12 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def model(w12):
    rng = np.random.default_rng(12)

    def rec(n, k):
        return w12.encode(to_dev(synth.f32_to_bf16_bits((rng.standard_normal((n, k)) * k ** -0.5).astype(np.float32))))

    layers = [dict(qkv=rec((HQ + 2 * HEADS) * DIM, HIDDEN), o=rec(HIDDEN, HQ * DIM),
                   gu=w12.interleave_rows(rec(INNER, HIDDEN), rec(INNER, HIDDEN)), down=rec(HIDDEN, INNER))
              for _ in range(LAYERS)]
    return dict(layers=layers, emb=rec(VOCAB, HIDDEN), rope=torch.tensor(rope_table(256, DIM)).cuda())


def norm(x):
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def forward(w12, model, ids, caches, batch, seen=None):
    """Logits of every row; seen(layer, qkv, caches before, q, y): looks each layer's stages over."""
    x = w12.embed(ids, model["emb"], scale=HIDDEN ** 0.5, out_f32=True)
    for i, (la, kv) in enumerate(zip(model["layers"], caches)):
        qkv = w12.gemm(norm(x), la["qkv"], out_bf16=i % 2 == 1)
        before = (kv.k.clone(), kv.v.clone()) if seen else None
        q = w12.kv_append(qkv, kv, batch, rope=model["rope"], interleaved=i % 2 == 1)
        y = w12.attention(q, kv, batch)
        if seen:
            seen(i, qkv, before, q, y)
        x = x + w12.gemm(y, la["o"])
        x = x + w12.gemm(w12.gemm_silu_mul(norm(x), la["gu"], out_bf16=True), la["down"])
    return w12.gemm(norm(x), model["emb"])


def fresh(w12, lens, e4m3, page=16):
    """The layers' caches of the same tables, long enough for `lens`."""
    return [Step(w12, lens, None, HEADS, DIM, page, e4m3, nhd=i == 1, seed=4) for i in range(LAYERS)]


def move(sts, w12, lens, news=None, tree=None):
    """The step's batch; the caches' bookkeeping with it."""
    for st in sts:
        st.lens = np.array(lens, np.int32)
        st.start = None if news is None else np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        st.tree = tree
        st.make()
    return sts[0].batch


@pytest.mark.parametrize("e4m3", [False, True])
def test_model(w12, model, e4m3):
    say(f"decoding run e4m3={e4m3}")
    prompts, steps, drafts = [5, 70, 1, 16], 4, 6
    rng = np.random.default_rng(5)

    def run():
        sts = fresh(w12, [p + steps + drafts for p in prompts], e4m3)
        look = True

        def seen(i, qkv, before, q, y):
            st = sts[i]
            check_append(st, qkv, HQ, f64(model["rope"]), i % 2 == 1, q, before, qkv.shape[0])
            check_attention(st, q, HQ, y)

        out = []
        ids = torch.tensor(rng.integers(0, VOCAB, sum(prompts)), dtype=torch.int32).cuda()
        lens, news = list(prompts), list(prompts)
        for t in range(steps + 1):
            batch = move(sts, w12, lens, news)
            y = forward(w12, model, ids, [s.kv for s in sts], batch, seen if look else None)
            if news is not None:
                y = y[torch.tensor(np.cumsum(news) - 1).cuda()]
            u = rng.random(len(prompts)).astype(np.float32)
            kw = params(len(prompts), t)
            r = check_sample(w12, y, u, kw)
            assert w12.logprobs(y, r.token).logp.isfinite().all()
            out += [y, r.token, r.logp, r.kept]
            ids, news, lens = r.token, None, [n + 1 for n in lens]
        # a tree of drafts behind each sequence: node b hangs on node (b - 1) // 2
        n = [n - 1 + drafts for n in lens]
        mask = [0] * drafts
        for b in range(drafts):
            mask[b] = 1 << b | (mask[(b - 1) // 2] if b else 0)
        batch = move(sts, w12, n, [drafts] * len(n), np.array(mask * len(n), np.int64))
        ids = torch.tensor(rng.integers(0, VOCAB, drafts * len(n)), dtype=torch.int32).cuda()
        y = forward(w12, model, ids, [s.kv for s in sts], batch, seen)
        m = y.shape[0]
        r = check_sample(w12, y, rng.random(m).astype(np.float32), params(m, 9))
        return out + [y, r.token, *(t.view(torch.uint8) if e4m3 else t for s in sts for t in (s.k, s.v))]

    a = run()
    rng = np.random.default_rng(5)
    assert all(torch.equal(x, y) for x, y in zip(a, run()))     # and the same bits again


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured(w12, model, e4m3):
    """A whole step captured, the lengths counted and the tokens fed back inside it, replayed among eager work."""
    say(f"captured step e4m3={e4m3}")
    seqs, replays = 3, 6
    lens0 = [9, 60, 31]

    def setup():
        sts = fresh(w12, [n + replays for n in lens0], e4m3)
        batch = move(sts, w12, lens0)
        st = dict(ids=torch.tensor([3, 5, 7], dtype=torch.int32).cuda(), u=torch.tensor([0.1, 0.5, 0.9]).cuda(),
                  k=torch.tensor([0, 40, 2], dtype=torch.int32).cuda(), p=torch.tensor([0.9, 0.8, 1.0]).cuda())
        return sts, batch, st

    def step(sts, batch, st):
        batch.lens.add_(1)
        y = forward(w12, model, st["ids"], [s.kv for s in sts], batch)
        r = w12.sample(y, st["u"], top_k=st["k"], top_p=st["p"])
        st["ids"].copy_(r.token)
        return y, r

    sts, batch, st = setup()
    want = []
    for _ in range(replays):
        y, r = step(sts, batch, st)
        want.append((y, r.token, r.logp, r.kept))
        st["u"].copy_((st["u"] + 0.37) % 1.0)
    cache = [t.clone() for s in sts for t in (s.k, s.v)]
    torch.cuda.synchronize()

    sts, batch, st = setup()
    keep = [t.clone() for s in sts for t in (s.k, s.v)] + [batch.lens.clone(), st["ids"].clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(sts, batch, st)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, r = step(sts, batch, st)
    for dst, src in zip([t for s in sts for t in (s.k, s.v)] + [batch.lens, st["ids"]], keep):
        dst.copy_(src)
    other = Step(w12, [300, 7], None, 2, 128, 32)
    q = queries(other, 8)
    eager = w12.attention(q, other.kv, other.batch)
    for t in range(replays):
        g.replay()
        st["u"].copy_((st["u"] + 0.37) % 1.0)
        assert torch.equal(w12.attention(q, other.kv, other.batch), eager)
        torch.cuda.synchronize()
        for a, b in zip((y, r.token, r.logp, r.kept), want[t]):
            assert torch.equal(a, b), t
    for a, b in zip((t for s in sts for t in (s.k, s.v)), cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert batch.lens.tolist() == [n + replays for n in lens0] and seqs == len(lens0)


def test_streams_and_two_graphs(w12):
    """Calls in flight on two streams, and two graphs captured on one stream replayed on two at once: each as alone."""
    say("two streams, two graphs")
    sets = []
    for seed, lens in ((1, [9000, 40, 3]), (2, [5, 7000, 800])):
        st = Step(w12, lens, None, 2, 128, 64, seed=seed)
        g = torch.Generator().manual_seed(seed)
        y = (torch.randn(3, 60011, generator=g) * 2).cuda()
        kw = dict(temperature=torch.tensor([1.0, 0.7, 1.3]).cuda(), top_p=torch.tensor([0.97, 0.9, 0.99]).cuda())
        sets.append((st, queries(st, 16, seed), y, torch.rand(3, generator=g).cuda(), kw))

    def call(s):
        st, q, y, u, kw = s
        return (w12.attention(q, st.kv, st.batch), *w12.sample(y, u, **kw))

    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, on in zip(sets, streams):
            with torch.cuda.stream(on):
                got.append(call(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, z in zip(got, want) for a, b in zip(x, z))
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(s))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, on in zip(graphs, streams):
            with torch.cuda.stream(on):
                g.replay()
        now = call(sets[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, z in zip(outs, want) for a, b in zip(x, z))
        assert all(torch.equal(a, b) for a, b in zip(now, want[0]))


def test_scratch(w12):
    """Scratch grows with the calls, is given back by release_workspace, and no call minds what another left in it."""
    say("scratch")
    side = torch.cuda.Stream()
    small, big = Step(w12, [40], None, 1, 64, 16), Step(w12, [20000, 3], None, 4, 128, 64)
    data = [(s, queries(s, 4 * s.heads), torch.randn(m, n, generator=torch.Generator().manual_seed(n)).cuda())
            for s, m, n in ((small, 2, 300), (big, 40, 50021), (small, 3, 9001))]
    u = torch.full((64,), 0.6).cuda()
    p = torch.full((64,), 0.8).cuda()

    def call(st, q, y):
        m = y.shape[0]
        return (w12.attention(q, st.kv, st.batch), *w12.sample(y, u[:m], top_p=p[:m]))

    want = [call(*d) for d in data]
    for s, q, _ in data:
        check_attention(s, q, 4 * s.heads, w12.attention(q, s.kv, s.batch))
    torch.cuda.synchronize()
    w12.release_workspace(side)
    before = torch.cuda.memory_allocated()
    for _ in range(2):
        for d, w in zip(data, want):
            with torch.cuda.stream(side):
                r = call(*d)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(r, w))
            del r
        w12.release_workspace(side)
        assert torch.cuda.memory_allocated() == before
    torch.cuda.synchronize()


def test_kv_cache(w12):
    """A cache from kv_cache, filled by prompts of two steps and read."""
    say("kv_cache")
    kv = w12.kv_cache(6, 2, 64, page=32)
    assert kv.k.shape == (6, 2, 32, 64) and kv.nbytes() == 2 * 6 * 2 * 32 * 64 * 2 and not kv.k.any()
    st = Step(w12, [60, 33], [60, 33], 2, 64, 32, spare=2)
    st.k, st.v, st.pages = kv.k, kv.v, 6
    st.make()
    qkv = torch.randn(93, 8 * 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    before = (st.k.clone(), st.v.clone())
    q = w12.kv_append(qkv, st.kv, st.batch)
    check_append(st, qkv, 4, None, False, q, before, 93)
    check_attention(st, q, 4, w12.attention(q, st.kv, st.batch))


# ---- sampling's ways ----
@pytest.mark.parametrize("m,n,bf16,sigma,temp,k,p,mp", [
    (4, 20011, False, 3.0, 0.05, 50, 0.9, 0.0),      # most of the k below 2^-32 of the largest weight
    (4, 20011, True, 3.0, 0.05, 50, 1.0, 0.0),
    (4, 20011, False, 3.0, 0.02, 700, 0.999, 0.01),
    (4, 60013, False, 1.0, 1.0, 5003, 0.93, 0.0),    # a cut by mass among thousands of top-k
    (4, 60013, False, 1.0, 1.0, 5003, 1.0, 0.02),
    (4, 60013, True, 0.02, 1.0, 0, 0.873, 0.0),      # tens of thousands in a few bins
    (4, 60013, False, 0.0, 1.0, 0, 0.31337, 0.0),    # and all equal
    (4, 60013, False, 0.004, 1.0, 40001, 0.77, 0.0),
    (4, 60013, True, 2.0, 1.2, 0, 0.98, 0.0),
    (4, 60013, True, 2.0, 1.2, 20000, 1.0, 0.0),
    (4, 60013, False, 2.0, 1.0, 0, 1.0, 1e-5),       # thousands by min-p alone
    (3, 300007, False, 2.0, 1.0, 0, 0.95, 0.0),
    (3, 300007, True, 2.0, 0.8, 30, 0.95, 0.0),
    (3, 300007, True, 2.0, 1.0, 0, 1.0, 0.0),
    (1, 1 << 20, False, 2.0, 1.0, 0, 0.9, 0.0),
    (2, 1 << 20, True, 2.0, 0.7, 100, 1.0, 0.1)])
def test_sample_ways(w12, m, n, bf16, sigma, temp, k, p, mp):
    g = torch.Generator().manual_seed(n + k)
    y = torch.randn(m, n, generator=g) * sigma
    y = (y.to(torch.bfloat16) if bf16 else y).cuda()
    rng = np.random.default_rng(n + k)
    say(f"sample n={n} bf16={bf16} sigma={sigma} temp={temp} k={k} p={p} mp={mp}")
    kw = dict(temperature=np.full(m, temp, np.float32), top_k=np.full(m, k, np.int32), top_p=np.full(m, p, np.float32),
              min_p=np.full(m, mp, np.float32))
    for _ in range(2):
        check_sample(w12, y, rng.random(m).astype(np.float32), kw)


@pytest.mark.parametrize("base,step", [(3e7, 2.0), (-3e7, 2.0), (1e9, 64.0), (-1e12, 65536.0), (0.0, 2.0)])
def test_sample_large_logits(w12, base, step):
    """Logits whose own steps are coarse: the filters' ends fall as they do near zero."""
    m, n = 12, 9001
    rng = np.random.default_rng(int(abs(base)) % 1000 + 1)
    y = torch.tensor(base - step * np.floor(rng.random((m, n)) ** 3 * 400), dtype=torch.float32).cuda()
    say(f"sample logits about {base}")
    for kw in (dict(min_p=0.3), dict(min_p=0.011), dict(top_k=700, min_p=0.05), dict(top_k=700, top_p=0.937), dict(top_p=0.937),
               dict(top_p=0.937, min_p=0.1)):
        kw = {k: np.full(m, v, np.int32 if k == "top_k" else np.float32) for k, v in kw.items()}
        for temp in (2.0 * step, 0.25 * step, 0.01 * step):
            check_sample(w12, y, rng.random(m).astype(np.float32), dict(kw, temperature=np.full(m, temp, np.float32)))


def test_sample_more_rows_than_a_launch(w12):
    m, n = 9001, 67
    y = torch.randn(m, n, generator=torch.Generator().manual_seed(2)).cuda() * 3
    say("sample rows")
    check_sample(w12, y, np.random.default_rng(1).random(m).astype(np.float32), params(m, 3))


def test_rows_that_overlap(w12):
    """A q_start that falls back gives more rows than there are: attention writes nothing, and the next call is right."""
    say("overlapping rows")
    for seqs in (2, 90):
        st = Step(w12, [40] * (2 * seqs), [3] * (2 * seqs), 2, 64, 16)
        q = queries(st, 8)
        good = st.batch
        start = np.tile([0, st.rows], seqs + 1)[:2 * seqs + 1].astype(np.int32)
        bad = w12.KVBatch(good.table, good.lens, q_start=torch.tensor(start).cuda())
        y = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        w12.attention(q, st.kv, bad, out=y)
        assert (y == 7.0).all()
        check_attention(st, q, 8, w12.attention(q, st.kv, good))


def test_batch_too_large(w12):
    """Lengths that the table allows are refused where their work could not be counted."""
    say("batch too large")
    kv = w12.kv_cache(1, 128, 64, page=16)
    batch = w12.KVBatch(torch.zeros((1, 1 << 26), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(w12.W12Error) as e:
        w12.attention(torch.zeros((1, 128 * 64), dtype=torch.bfloat16, device="cuda"), kv, batch)
    assert e.value.status == w12.W12_ERR_RANGE
