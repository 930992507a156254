"""Edges of cache append, attention and sampling: calls with some of the settings absent, random numbers at
the ends of their range, non-finite values that some rows see, rows past the step's.  Tolerances as in
test_gpu_step.
"""
import ctypes
import threading

import numpy as np
import pytest

import oracle
from tests.gpu_util import say
from tests.test_gpu_step import H, U, Step, attend, check_append, check_attention, f64, queries, rope_table

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w12():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lossless_bit_weight_02_amd import w12 as mod
    mod.lib()
    return mod


# ---- sampling ----
POISON = -77


def raw_sample(w12, y, u, **kw):
    """w12_sample into outputs that hold POISON, as numpy arrays; settings that are not in kw are NULL."""
    m, n = y.shape
    flags = w12.LOGITS_BF16 if y.dtype == torch.bfloat16 else 0
    out = [torch.full((m,), POISON, dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.int32)]
    dev = {a: torch.tensor(b).cuda() for a, b in kw.items()}
    need = ctypes.c_uint64(0)
    assert w12.lib().w12_sample_scratch(m, n, flags, ctypes.byref(need)) == 0
    scratch = torch.full((need.value,), 0x5A, dtype=torch.uint8, device="cuda")
    ud = torch.tensor(u).cuda()
    ptr = [None if a not in dev else dev[a].data_ptr() for a in ("temperature", "top_k", "top_p", "min_p")]
    assert w12.lib().w12_sample(y.data_ptr(), m, n, y.stride(0) if m > 1 else n, *ptr, ud.data_ptr(), *(t.data_ptr() for t in out),
                                scratch.data_ptr(), need.value, flags, torch.cuda.current_stream().cuda_stream) == 0
    return tuple(t.cpu().numpy() for t in out)


def check_raw(w12, y, u, **kw):
    got = raw_sample(w12, y, u, **kw)
    tok, logp, kept = oracle.sample64(f64(y), u.astype(np.float64),
                                      **{a: b.astype(np.float64) if b.dtype != np.int32 else b for a, b in kw.items()})
    assert np.array_equal(got[2], kept), (np.argwhere(got[2] != kept)[:5], got[2][got[2] != kept][:5])
    assert np.array_equal(got[0], tok), (np.argwhere(got[0] != tok)[:5], got[0][got[0] != tok][:5], tok[got[0] != tok][:5])
    fin = np.isfinite(logp)
    lp = got[1].astype(np.float64)
    assert np.array_equal(np.isnan(lp), np.isnan(logp)) and np.array_equal(np.isneginf(lp), np.isneginf(logp))
    assert np.all(np.abs(lp[fin] - logp[fin]) <= U * np.abs(logp[fin]) + 1e-9)
    return got


def greedy_rows(m, n, seed):
    """Rows whose largest logit is one of thousands alike, of few, or of magnitudes where steps are coarse."""
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(m, n, generator=g)
    y[0] = 0.0
    y[1] = -0.0
    y[1, n // 2:] = 0.0
    y[2] *= 0.01
    y[3] = y[3].round()
    y[4] = torch.where(torch.rand(n, generator=g) < 0.5, 3e38, -3e38)
    y[5] = y[5] * 1e6 + 3e9
    y[6] = -1e30
    y[7] = -float("inf")
    y[8] = -float("inf")
    y[8, n - 1] = -3e38
    y[9, n // 3] = float("nan")
    y[10, n - 1] = float("inf")
    y[11, n - 1] = 50.0
    return y


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [1, 2, 200, 20011, 152064, 262145, 300007])
def test_greedy_alone(w12, n, bf16):
    """Temperatures of 0 and below with no other setting given; some rows are drawn."""
    m = 14
    y = greedy_rows(m, n, n)
    y = (y.to(torch.bfloat16) if bf16 else y).cuda()
    u = np.random.default_rng(n).random(m).astype(np.float32)
    say(f"greedy n={n} bf16={bf16}")
    for temps in ([0.0], [-1.0, 0.0, -float("inf")]):
        check_raw(w12, y, u, temperature=np.resize(np.array(temps, np.float32), m))
    mixed = np.zeros(m, np.float32)
    mixed[[0, 2, 11, 13]] = [1.0, 1.5, 0.7, float("nan")]
    check_raw(w12, y, u, temperature=mixed)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [1, 63, 5003, 65537, 300007])
def test_one_token_kept(w12, n, bf16):
    """The settings that keep the first token alone, each given by itself, as greedy rows."""
    m = 14
    y = greedy_rows(m, n, n + 1)
    y = (y.to(torch.bfloat16) if bf16 else y).cuda()
    u = np.random.default_rng(n).random(m).astype(np.float32)
    say(f"one token kept n={n} bf16={bf16}")
    a = check_raw(w12, y, u, temperature=np.zeros(m, np.float32))
    for kw in (dict(top_k=np.ones(m, np.int32)), dict(top_p=np.zeros(m, np.float32)), dict(min_p=np.full(m, 1.5, np.float32)),
               dict(top_k=np.ones(m, np.int32), top_p=np.full(m, 0.5, np.float32), min_p=np.full(m, 0.5, np.float32))):
        b = check_raw(w12, y, u, **kw)
        assert all(np.array_equal(s, t, equal_nan=True) for s, t in zip(a, b))


def test_greedy_batch(w12):
    """A server's batch of greedy rows, and greedy ones among filtered ones."""
    m, n = 256, 32001
    y = (torch.randn(m, n, generator=torch.Generator().manual_seed(3)) * 3).to(torch.bfloat16).cuda()
    rng = np.random.default_rng(4)
    u = rng.random(m).astype(np.float32)
    say("greedy batch")
    check_raw(w12, y, u, temperature=np.zeros(m, np.float32))
    check_raw(w12, y, u, temperature=np.where(np.arange(m) % 3 == 0, 0.0, 0.8).astype(np.float32),
              top_k=rng.choice([0, 1, 40], m).astype(np.int32))


@pytest.mark.parametrize("kw", [dict(top_k=1500), dict(top_k=9000), dict(top_p=0.9), dict(min_p=0.05), dict(min_p=0.4),
                                dict(top_k=2000, top_p=0.95, min_p=0.01), dict(top_k=20000, top_p=0.8), {}])
@pytest.mark.parametrize("sigma", [0.5, 2.0])
def test_sample_last_of_many(w12, kw, sigma):
    """u of 1 and more over kept tokens that every wave of a row's join holds some of, again and again alike."""
    m, n = 40, 33001
    y = (torch.randn(m, n, generator=torch.Generator().manual_seed(8)) * sigma).cuda()
    kw = {a: np.full(m, b, np.int32 if a == "top_k" else np.float32) for a, b in kw.items()}
    say(f"sample last of many sigma={sigma} {list(kw)}")
    u = np.resize(np.array([1.0, 1.5, np.inf], np.float32), m)
    a = check_raw(w12, y, u, **kw)
    for _ in range(4):
        assert all(np.array_equal(s, t) for s, t in zip(a, raw_sample(w12, y, u, **kw)))


def lonely_rows(n, bf16):
    """Rows whose first and last columns weigh 10^-18 to 10^-300 of the best, or nothing, with a few heavy ones between."""
    y = torch.randn(6, n, generator=torch.Generator().manual_seed(n))
    y[0, : n // 3] = -60.0
    y[0, -(n // 3):] = -70.0
    y[1, : n // 3] = -300.0
    y[1, -5:] = -250.0
    y[2, :7] = -1e30
    y[2, 7] = -45.0
    y[2, -9:] = -1e30
    y[2, -10] = -400.0
    y[3] = -50.0
    y[3, n // 2] = 9.0
    y[4] = -float("inf")
    y[4, n // 2] = 2.0
    y[4, n // 4] = -90.0
    y[4, n - n // 4] = -90.0
    y[5, ::2] = -80.0
    return (y.to(torch.bfloat16) if bf16 else y).cuda()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [40, 5003, 70001, 300007])
def test_sample_ends_of_u(w12, n, bf16):
    """u of 0 and below takes the first kept column of any mass, of 1 and above the last, a tiny one the column
    that its mass reaches; kept by no filter, and by ones that leave all but few."""
    y = lonely_rows(n, bf16)
    m = y.shape[0]
    say(f"sample ends of u n={n} bf16={bf16}")
    for u in (0.0, -3.0, float("nan"), 1.0, 2.0, float("inf"), 1e-28, 1e-20, 3e-9, 1.0 - 2.0 ** -24):
        uu = np.full(m, u, np.float32)
        for kw in ({}, dict(top_k=np.full(m, n - n // 8 + 1, np.int32)), dict(min_p=np.full(m, 1e-37, np.float32)),
                   dict(top_p=np.full(m, 0.99, np.float32)), dict(top_k=np.full(m, 17, np.int32), top_p=np.full(m, 0.8, np.float32))):
            a = check_raw(w12, y, uu, **kw)
            b = raw_sample(w12, y, uu, **kw)
            assert all(np.array_equal(s, t, equal_nan=True) for s, t in zip(a, b))


@pytest.mark.parametrize("n,kw", [(1000, dict(top_k=600)), (4000, dict(top_p=0.7)), (4000, {}), (2000, dict(min_p=0.2))])
def test_sample_on_the_border(w12, n, kw):
    """Rows of two equal halves and u = 1/2, so the number drawn for is a border up to the rounding of the sums: the
    token is the last of the one half that is kept or the first of the other."""
    m = 64
    half = torch.randn(m, n // 2, generator=torch.Generator().manual_seed(n))
    y = torch.cat([half, half], 1).cuda()
    kw = {a: np.full(m, b, np.int32 if a == "top_k" else np.float32) for a, b in kw.items()}
    say(f"sample on the border n={n}")
    got = raw_sample(w12, y, np.full(m, 0.5, np.float32), **kw)
    for r in range(m):
        x = f64(half[r])
        order = np.argsort(-x, kind="stable")
        w = np.exp(x - x.max())
        # (each logit twice: k / 2 of a half; the same share, the same least weight)
        k = len(order)
        if "top_k" in kw:
            k = kw["top_k"][0] // 2
        if "top_p" in kw:
            k = None
        if "min_p" in kw:
            k = int((w >= kw["min_p"][0]).sum())
        if k is None:
            tok, _, kept = oracle.sample64(f64(y[r:r + 1]), [0.5], top_p=[float(np.float32(0.7))])
            assert got[2][r] == kept[0]
            if kept[0] % 2:
                assert got[0][r] == tok[0]
                continue
            k = int(kept[0]) // 2
        cols = np.sort(order[:k])
        assert got[2][r] == 2 * k and got[0][r] in (cols[-1], n // 2 + cols[0]), r


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [3000, 60013, 152064, 300007])
@pytest.mark.parametrize("kw", [{}, dict(min_p=1e-13), dict(top_k=2900), dict(top_p=0.99999), dict(top_k=100000, top_p=0.999999)])
def test_sample_long_tails(w12, kw, n, bf16):
    """One logit far above a row of ties and near ties, which weigh 2^-26 to 2^-40 of it and come first: what is kept and
    drawn among them is decided to a part of one of them."""
    g = torch.Generator().manual_seed(n)
    y = torch.randn(12, n, generator=g)
    y[0] = -22.5
    y[1] = -18.3
    y[2] = -27.1
    y[3] = (y[3] * 8).round() / 8 - 20.0
    y[4:8] = y[4:8] * 0.5 - 21.0
    y[8:] = y[8:] * 2.0 - 24.0
    y[:, -1] = 0.4
    y = (y.to(torch.bfloat16) if bf16 else y).cuda()
    rng = np.random.default_rng(n)
    tail = np.exp(f64(y)[:, :-1] - f64(y)[:, -1:]).sum(axis=1)
    m = y.shape[0]
    kw = {a: np.full(m, min(b, n - 1) if a == "top_k" else b, np.int32 if a == "top_k" else np.float32) for a, b in kw.items()}
    say(f"sample long tails n={n} bf16={bf16} {list(kw)}")
    for _ in range(4):
        check_raw(w12, y, (rng.random(m) * tail).astype(np.float32), **kw)


@pytest.mark.parametrize("temp", [1e-38, 1e-30, 1e-3, 1e6, 1e30, float("inf")])
@pytest.mark.parametrize("n", [77, 9001, 70001])
def test_sample_extreme_temperatures(w12, n, temp):
    """Temperatures that leave one token or make all alike, with each filter."""
    m = 6
    y = torch.randn(m, n, generator=torch.Generator().manual_seed(n)) * 3
    y[1] = (y[1] * 4).round() / 4
    y[2, ::3] = -float("inf")
    y[3] *= 1e30
    y = y.cuda()
    rng = np.random.default_rng(n)
    say(f"sample n={n} temperature={temp}")
    for kw in (dict(top_k=5), dict(top_k=3000), dict(top_p=0.8713), dict(min_p=0.3), dict(top_k=60, top_p=0.7171, min_p=0.01)):
        kw = {a: np.full(m, b, np.int32 if a == "top_k" else np.float32) for a, b in kw.items()}
        check_raw(w12, y, rng.random(m).astype(np.float32), temperature=np.full(m, temp, np.float32), **kw)


# ---- attention ----
def bad_place(st, s, c, col, val):
    st.v[int(st.table[s, c // st.page]), :, c % st.page, col] = val


@pytest.mark.parametrize("dim,e4m3,group,t", [
    (64, False, 4, 1), (128, False, 6, 1), (256, False, 6, 1), (64, True, 4, 1), (128, True, 6, 1), (256, True, 6, 1),
    (128, False, 6, 2), (256, True, 6, 2), (64, False, 6, 4), (128, True, 6, 4), (128, False, 6, 4), (256, False, 6, 4),
    (128, False, 6, 9)])
def test_attention_seen_value(w12, dim, e4m3, group, t):
    """A NaN or an infinity in one column of a new token reaches that column of the rows that see the token, and
    no other: what stands behind the sequences is NaN, too.  (Up to 16, up to 32 and more rows a sequence.)"""
    lens = [t, t + 1, 17 + t, 31, 33, 47, 64, 129, 300, 530]
    st = Step(w12, lens, [t] * len(lens), 2, dim, 16, e4m3)
    hq = 2 * group
    q = queries(st, hq)
    bad = float("nan") if e4m3 else float("inf")
    for s, n in enumerate(lens):                                  # stale places of the last page
        for c in range(n, (n + 15) // 16 * 16):
            for x in (st.k, st.v):
                x[int(st.table[s, c // 16]), :, c % 16] = float("nan")
    say(f"attention seen value dim={dim} e4m3={e4m3} group={group} t={t}")
    for j in range(0, t, 3):
        for col in (0, 5, dim - 1):
            keep = st.v.clone()
            for s, n in enumerate(lens):
                bad_place(st, s, n - t + j, col, 0.0)
            zeroed = st.v.clone()
            for s, n in enumerate(lens):
                bad_place(st, s, n - t + j, col, bad)
            y = attend(w12, st, q)
            got = f64(y).reshape(-1, t, hq, dim)
            hit = ~np.isfinite(got)
            want = np.zeros_like(hit)
            want[:, j:, :, col] = True
            assert np.array_equal(hit, want), np.argwhere(hit != want)[:5]
            # the other columns, and the rows before, are what they are without it
            st.v.copy_(zeroed)
            y2 = torch.where(torch.tensor(want).cuda().reshape(y.shape), attend(w12, st, q), y)
            check_attention(st, q, hq, y2)
            st.v.copy_(keep)


@pytest.mark.parametrize("dim,e4m3,t,group", [(128, False, 3, 4), (64, True, 5, 3), (256, False, 4, 3), (128, True, 5, 6), (128, False, 8, 6)])
def test_attention_seen_value_in_a_tree(w12, dim, e4m3, t, group):
    """The same with masks: rows whose mask has the token's bit have the value, the others' are as if it were zero."""
    lens = [t, 19 + t, 32 + t, 61, 200]
    m = t * len(lens)
    rng = np.random.default_rng(dim + t)
    masks = rng.integers(0, 1 << t, m, dtype=np.int64)
    st = Step(w12, lens, [t] * len(lens), 1, dim, 16, e4m3, tree=masks)
    q = queries(st, group)
    bad = float("nan") if e4m3 else float("-inf")
    say(f"attention seen value in a tree dim={dim} e4m3={e4m3} t={t}")
    for j in range(t):
        col = int(rng.integers(dim))
        keep = st.v.clone()
        for s, n in enumerate(lens):
            bad_place(st, s, n - t + j, col, 0.0)
        zeroed = st.v.clone()
        for s, n in enumerate(lens):
            bad_place(st, s, n - t + j, col, bad)
        y = attend(w12, st, q)
        want = np.zeros((m, group, dim), bool)
        want[(masks >> j & 1) == 1, :, col] = True
        hit = ~np.isfinite(f64(y).reshape(want.shape))
        assert np.array_equal(hit, want), np.argwhere(hit != want)[:5]
        st.v.copy_(zeroed)
        check_attention(st, q, group, torch.where(torch.tensor(want).cuda().reshape(y.shape), attend(w12, st, q), y))
        st.v.copy_(keep)


@pytest.mark.parametrize("dim,e4m3,t,group", [(128, False, 1, 6), (64, True, 1, 6), (128, True, 1, 6), (256, True, 1, 6),
                                              (128, True, 4, 6), (128, False, 4, 6), (64, False, 20, 6), (256, True, 20, 6)])
def test_attention_differences(w12, dim, e4m3, t, group):
    """Pairs of places with nearly equal scores and opposite values, whose difference is left: it keeps the bits that the
    probabilities that meet the values have (16; over e4m3 22, in many rows 11; half a unit each), and float's of
    their sums and scores (as in test_gpu_step: scores are at most 1 here)."""
    st = Step(w12, [64 + t] * 3, [t] * 3, 1, dim, 16, e4m3, scales=False)
    rng = np.random.default_rng(dim + t)
    k, v = np.zeros((st.pages, 1, 16, dim)), np.zeros((st.pages, 1, 16, dim))
    for s in range(3):
        for c in range(0, 64, 2):
            val = rng.choice([1.0, 16.0, 448.0], dim) * rng.choice([-1, 1], dim)
            for at, sign in ((c, 1.0), (c + 1, -1.0)):
                p, o = int(st.table[s, at // 16]), at % 16
                v[p, 0, o] = sign * val
                k[p, 0, o, 0] = 0.5 * sign * 2.0 ** -int(rng.integers(3, 7))
    st.k.copy_(torch.tensor(k).to(st.k.dtype))
    st.v.copy_(torch.tensor(v).to(st.v.dtype))
    assert np.array_equal(st.values(0), k) and np.array_equal(st.values(1), v)
    q = torch.zeros((st.rows, group * dim), dtype=torch.bfloat16, device="cuda")
    q.view(st.rows, group, dim)[:, :, 0] = torch.tensor(rng.uniform(0.2, 1.0, (st.rows, group))).to(torch.bfloat16).cuda()
    say(f"attention differences dim={dim} e4m3={e4m3} t={t}")
    y = f64(attend(w12, st, q, scale=1.0)).reshape(st.rows, group, dim)
    want, mag, big = oracle.attention64(f64(q).reshape(st.rows, group, dim), k, v, st.table, st.lens, st.start, None, 1.0)
    bits = (2.0 ** -11 if t * group > 32 else 2.0 ** -22) if e4m3 else 2.0 ** -16
    rel = bits + 2 * (dim + 8) * U * big[:, :, None] + 4 * U + (64 + t + 8) * U
    bad = ~(np.abs(y - want) <= H * np.abs(want) + (1 + H) * rel * mag)
    assert not bad.any(), np.argwhere(bad)[:5]


# ---- rows past the step's ----
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("group,news,rows", [(3, [2, 5, 9], 11), (3, [1, 1, 1], 2), (8, [30, 40, 50], 75), (2, [4, 6, 3], 10)])
def test_sequence_past_the_rows(w12, e4m3, group, news, rows):
    """A q_start that passes the step's rows: the rows that exist keep their places, the others do nothing."""
    lens = [n + 40 * i for i, n in enumerate(news)]
    for tree in (False, True):
        masks = np.random.default_rng(rows).integers(0, 2 ** 63, rows, dtype=np.int64) if tree else None
        st = Step(w12, lens, news, 2, 64, 16, e4m3, tree=masks)
        hq = 2 * group
        g = torch.Generator().manual_seed(1)
        qkv = torch.randn(rows, (hq + 4) * 64, generator=g).cuda()
        before = (st.k.clone(), st.v.clone())
        rope = rope_table(max(lens) + 1, 64)
        out = torch.full((rows, hq * 64), 7.0, dtype=torch.bfloat16, device="cuda")
        say(f"sequence past the rows news={news} rows={rows} e4m3={e4m3} tree={tree}")
        w12.kv_append(qkv, st.kv, st.batch, rope=torch.tensor(rope).cuda(), out=out)
        check_append(st, qkv, hq, rope, False, out, before, rows)
        st.rows = rows
        q = queries(st, hq)
        check_attention(st, q, hq, attend(w12, st, q))


def test_sequence_far_past_the_rows(w12):
    """The same by 2^31 rows, where nothing but the last places' bounds holds them."""
    st = Step(w12, [70, 40, 30], [1, 2, 3], 2, 64, 16)
    st.start = np.array([0, 1, 2, 2 ** 31 - 1], np.int32)
    st.make()
    say("sequence far past the rows")
    before = (st.k.clone(), st.v.clone())
    qkv = torch.randn(5, 8 * 64, generator=torch.Generator().manual_seed(1)).cuda()
    q = w12.kv_append(qkv, st.kv, st.batch)
    y = attend(w12, st, q)
    # the last sequence's new tokens have places far below 0 .. 29, so they see nothing and put nothing
    assert (y[2:] == 0).all()
    touched = ((st.k != before[0]).any(dim=(1, 3)), (st.v != before[1]).any(dim=(1, 3)))
    for x in touched:
        assert x.sum() == 2 and x[int(st.table[0, 4]), 5] and x[int(st.table[1, 2]), 7]


def test_e4m3_cache(w12):
    """An e4m3 cache from kv_cache, appended to and read."""
    say("e4m3 cache")
    scale = torch.tensor([0.02, 0.05]).cuda()
    kv = w12.kv_cache(4, 2, 64, page=16, dtype=torch.float8_e4m3fn, k_scale=scale, v_scale=scale)
    assert kv.k.dtype == torch.float8_e4m3fn and kv.nbytes() == 2 * 4 * 2 * 16 * 64 and not kv.k.view(torch.uint8).any()
    st = Step(w12, [20, 9], [20, 9], 2, 64, 16, e4m3=True, spare=1)
    st.k, st.v, st.sc, st.pages = kv.k, kv.v, (scale, scale), 4
    st.make()
    qkv = torch.randn(29, 8 * 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    before = (st.k.clone(), st.v.clone())
    q = w12.kv_append(qkv, kv, st.batch)
    check_append(st, qkv, 4, None, False, q, before, 29)
    check_attention(st, q, 4, w12.attention(q, kv, st.batch))


# ---- outputs over inputs ----
def test_in_place(w12):
    """Rotation and attention into the rows of q themselves, of whole and split sequences, few rows and many; other
    overlaps are refused."""
    for lens, news, dim in (([5000, 40, 3], [1, 1, 1], 128), ([300, 40], [20, 40], 64), ([700, 9000], [2, 30], 256)):
        st = Step(w12, lens, news, 2, dim, 16)
        q = queries(st, 12)
        say(f"in place lens={lens} news={news}")
        want = w12.attention(q, st.kv, st.batch)
        y = q.clone()
        assert w12.attention(y, st.kv, st.batch, out=y) is y and torch.equal(y, want)
        k, v = queries(st, 2, seed=5), queries(st, 2, seed=6)
        rope = torch.tensor(rope_table(max(lens) + 1, dim)).cuda()
        for pairs in (False, True):
            r = w12.kv_append((q, k, v), st.kv, st.batch, rope=rope, interleaved=pairs)
            z = q.clone()
            w12.kv_append((z, k, v), st.kv, st.batch, rope=rope, interleaved=pairs, out=z)
            assert torch.equal(z, r)
    wide = torch.zeros((st.rows + 1) * 16 * dim, dtype=torch.bfloat16, device="cuda")
    qkv = wide[:st.rows * 16 * dim].view(st.rows, 16 * dim)
    for out in (wide[:st.rows * 12 * dim], wide[8:8 + st.rows * 12 * dim], wide[-st.rows * 12 * dim:]):
        with pytest.raises(ValueError):
            w12.kv_append(qkv, st.kv, st.batch, out=out.view(st.rows, 12 * dim))
        with pytest.raises(ValueError):
            w12.attention(qkv[:, :12 * dim], st.kv, st.batch, out=out.view(st.rows, 12 * dim))


# ---- threads ----
def test_two_threads_on_one_stream(w12):
    """Attention that ends in a join and sampling of several kernels, called from two threads on the same stream: each
    call's results are as alone."""
    say("two threads on one stream")
    sets = []
    for seed, lens in ((1, [9000, 40, 3]), (2, [5, 7000, 800])):
        st = Step(w12, lens, None, 2, 128, 64, seed=seed)
        g = torch.Generator().manual_seed(seed)
        y = (torch.randn(3, 60011, generator=g) * 2).cuda()
        sets.append((st, queries(st, 16, seed), y, torch.rand(3, generator=g).cuda(), torch.full((3,), 0.97).cuda()))

    def call(s):
        st, q, y, u, p = s
        return (w12.attention(q, st.kv, st.batch), *w12.sample(y, u, top_p=p))

    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(100):
            got[i].append(call(sets[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for mine, w in zip(got, want):
        assert len(mine) == 100 and all(torch.equal(a, b) for r in mine for a, b in zip(r, w))
