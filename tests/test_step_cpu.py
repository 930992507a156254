"""Cache append, attention and sampling without a GPU: what the C ABI refuses before it touches one, and
the oracle on cases small enough to be done by hand."""
import ctypes
import math
import os

import numpy as np
import pytest

import oracle
from lossless_bit_weight_02_amd import w12


def _lib():
    if not os.path.exists(w12.LIB_PATH):
        pytest.skip("libw12.so not built")
    return w12.lib()


def _kv(**over):
    s = w12._W12KV(10, 4, 64, 128, 0x10000, 0x20000, 4 * 64 * 128, 64 * 128, 128, None, None, 0)
    for k, v in over.items():
        setattr(s, k, v)
    return s


def _batch(**over):
    s = w12._W12KVBatch(3, 0x1000, 5, 5, 0x2000, None, None, None)
    for k, v in over.items():
        setattr(s, k, v)
    return s


E = dict(ARG=w12.W12_ERR_ARG, SHAPE=w12.W12_ERR_SHAPE, ALIGN=w12.W12_ERR_ALIGN, RANGE=w12.W12_ERR_RANGE)

BAD_KV = [("ARG", dict(k=None)), ("ARG", dict(v=None)), ("ARG", dict(flags=2)), ("ARG", dict(pages=0)),
          ("ARG", dict(heads=-1)), ("ARG", dict(page=0)), ("RANGE", dict(pages=1 << 31)), ("RANGE", dict(heads=65537)),
          ("RANGE", dict(page=65552)), ("SHAPE", dict(dim=96)), ("SHAPE", dict(page=24)), ("ARG", dict(head_stride=-8)),
          ("ALIGN", dict(token_stride=132)), ("ALIGN", dict(flags=1, token_stride=136)), ("RANGE", dict(token_stride=1 << 25)),
          ("ALIGN", dict(k=0x10008)), ("ARG", dict(k_scale=0x3000)), ("ALIGN", dict(flags=1, v_scale=0x3002))]
BAD_BATCH = [("ARG", dict(seqs=0)), ("RANGE", dict(seqs=1 << 20)), ("ARG", dict(table=None)), ("ARG", dict(lens=None)),
             ("ARG", dict(table_cols=0)), ("RANGE", dict(table_cols=1 << 26)), ("ARG", dict(table_stride=4)),
             ("ALIGN", dict(lens=0x2002)), ("ALIGN", dict(tree=0x2004)), ("ALIGN", dict(q_start=0x2001))]


def _append(L, kv, b, q=0x100000, ldq=8192, k=0x100000, ldk=8192, v=0x100000, ldv=8192, m=3, hq=8, rope=0x200000,
            rows=100, rot=128, out=0x300000, flags=0):
    return L.w12_kv_append(q, ldq, k, ldk, v, ldv, m, hq, rope, rows, rot, ctypes.byref(kv), ctypes.byref(b), out,
                           flags, None)


def _attention(L, kv, b, q=0x100000, ldq=8192, m=3, hq=8, y=0x300000, flags=0):
    return L.w12_attention(q, ldq, m, hq, ctypes.byref(kv), ctypes.byref(b), 0.1, y, None, 0, flags, None)


@pytest.mark.parametrize("want,over", BAD_KV)
def test_cache_refused(want, over):
    L = _lib()
    n = ctypes.c_uint64(0)
    assert _append(L, _kv(**over), _batch()) == E[want] and L.w12_last_error()
    assert _attention(L, _kv(**over), _batch()) == E[want]
    assert L.w12_attention_scratch(3, 8, ctypes.byref(_kv(**over)), ctypes.byref(_batch()), ctypes.byref(n)) == E[want]


@pytest.mark.parametrize("want,over", BAD_BATCH)
def test_batch_refused(want, over):
    L = _lib()
    assert _append(L, _kv(), _batch(**over)) == E[want]
    assert _attention(L, _kv(), _batch(**over)) == E[want]


@pytest.mark.parametrize("want,over", [
    ("ARG", dict(m=0)), ("RANGE", dict(m=1 << 31)), ("ARG", dict(flags=1)), ("SHAPE", dict(hq=6)), ("SHAPE", dict(hq=-4)),
    ("RANGE", dict(hq=65540)), ("ARG", dict(k=None)), ("ARG", dict(q=None)), ("ARG", dict(out=None)), ("ARG", dict(hq=0)),
    ("ALIGN", dict(v=0x100008)), ("ALIGN", dict(ldk=8196)), ("ALIGN", dict(ldk=8194, flags=w12.IN_F32)),
    ("ARG", dict(ldv=256)), ("RANGE", dict(ldq=1 << 32)), ("SHAPE", dict(rot=8)), ("SHAPE", dict(rot=144)),
    ("ARG", dict(rope=None)), ("ARG", dict(rot=0)), ("RANGE", dict(rows=0)), ("ALIGN", dict(rope=0x200004))])
def test_append_refused(want, over):
    assert _append(_lib(), _kv(), _batch(), **over) == E[want]


@pytest.mark.parametrize("want,over", [
    ("ARG", dict(m=0)), ("ARG", dict(flags=1)), ("SHAPE", dict(hq=0)), ("SHAPE", dict(hq=7)), ("ARG", dict(q=None)),
    ("ARG", dict(y=None)), ("ALIGN", dict(q=0x100004)), ("ALIGN", dict(ldq=8196)), ("ARG", dict(ldq=512)),
    ("RANGE", dict(ldq=1 << 32))])
def test_attention_refused(want, over):
    assert _attention(_lib(), _kv(), _batch(), **over) == E[want]


def test_null_structs_refused():
    L = _lib()
    b = ctypes.byref
    assert L.w12_attention(0x1000, 512, 3, 4, None, b(_batch()), 0.1, 0x1000, None, 0, 0, None) == w12.W12_ERR_ARG
    assert L.w12_attention(0x1000, 512, 3, 4, b(_kv()), None, 0.1, 0x1000, None, 0, 0, None) == w12.W12_ERR_ARG
    assert L.w12_attention_scratch(3, 4, b(_kv()), b(_batch()), None) == w12.W12_ERR_ARG
    assert L.w12_sample_scratch(3, 4, 0, None) == w12.W12_ERR_ARG


@pytest.mark.parametrize("want,over", [
    ("ARG", dict(y=None)), ("ARG", dict(u=None)), ("ARG", dict(m=0)), ("ARG", dict(n=-1)), ("RANGE", dict(m=1 << 31)),
    ("RANGE", dict(n=1 << 31)), ("ARG", dict(ldy=99)), ("RANGE", dict(ldy=(1 << 40) + 1)), ("ARG", dict(flags=1)),
    ("ALIGN", dict(y=0x1002)), ("ALIGN", dict(y=0x1001, flags=w12.LOGITS_BF16)), ("ALIGN", dict(t=0x1001)),
    ("ALIGN", dict(token=0x1001)), ("ALIGN", dict(u=0x1002))])
def test_sample_refused(want, over):
    a = dict(y=0x1000, m=2, n=100, ldy=100, t=None, u=0x2000, token=0x3000, flags=0)
    a.update(over)
    assert _lib().w12_sample(a["y"], a["m"], a["n"], a["ldy"], a["t"], None, None, None, a["u"], a["token"], None, None,
                             None, 0, a["flags"], None) == E[want]


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros(2, 4, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w12.KVCache(k, k.clone())
    with pytest.raises(ValueError):
        w12.KVBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        w12.sample(torch.zeros(2, 10), torch.zeros(2))


# ---- the oracle ----
def test_rotation_by_hand():
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    c, s = np.array([0.0, 1.0]), np.array([1.0, 0.0])     # a quarter turn, none
    assert np.array_equal(oracle.rotate64(x, c, s, False), [-3.0, 2.0, 1.0, 4.0, 5.0])
    assert np.array_equal(oracle.rotate64(x, c, s, True), [-2.0, 1.0, 3.0, 4.0, 5.0])


def test_rotation_keeps_relative_position():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 32))
    f = 10000.0 ** (-np.arange(16) / 16)

    def at(x, p, pairs):
        return oracle.rotate64(x, np.cos(p * f), np.sin(p * f), pairs)

    for pairs in (False, True):
        a = at(q, 7, pairs) @ at(k, 3, pairs)
        b = at(q, 1007, pairs) @ at(k, 1003, pairs)
        assert abs(a - b) < 1e-9


def test_append_places():
    k = np.arange(4 * 1 * 2, dtype=np.float64).reshape(4, 1, 2)
    table = np.array([[5, 2], [-1, 9]])
    # sequence 0: two new of 17 (places 15, 16), sequence 1: one new of 20 (place 19, page 9), a row of no sequence
    _, put = oracle.append64(None, k, -k, None, False, table, [17, 20], [0, 2, 3], None, 16, 10)
    assert sorted(put) == [(2, 0), (5, 15), (9, 3)]
    assert np.array_equal(put[9, 3][0], k[2]) and np.array_equal(put[9, 3][1], -k[2])
    # no page, no place
    assert not oracle.append64(None, k, k, None, False, table, [0, 3], [0, 0, 3], None, 16, 2)[1]


def test_attention_by_hand():
    k = np.zeros((2, 1, 16, 4))
    v = np.zeros((2, 1, 16, 4))
    v[1, 0, 0], v[1, 0, 1], v[1, 0, 2] = 1.0, 5.0, np.nan
    k[1, 0, 1, 0] = math.log(3.0)
    q = np.array([[[1.0, 0, 0, 0]], [[1.0, 0, 0, 0]]])
    table = np.array([[1]])
    y, mag, _ = oracle.attention64(q, k, v, table, [2], [0, 2], None, 1.0)
    assert np.allclose(y[0], 1.0) and np.allclose(y[1], (1 + 3 * 5) / 4) and np.allclose(mag, y)
    # the second token's mask leaves it only itself, the first one's nothing
    y, _, _ = oracle.attention64(q, k, v, table, [2], [0, 2], np.array([0, 2]), 1.0)
    assert np.array_equal(y[0, 0], np.zeros(4)) and np.allclose(y[1], 5.0)
    y, _, _ = oracle.attention64(q, k, v, table, [0], [0, 1], None, 1.0)
    assert np.array_equal(y[0, 0], np.zeros(4)) and np.isnan(y[1]).all()


def test_sampling_by_hand():
    # probabilities .5, .3, .1, .1 in the columns 3, 0, 1, 4 and a masked one
    y = np.log(np.array([[0.3, 0.1, 0.0 + 1e-300, 0.5, 0.1]]))
    y[0, 2] = -np.inf

    def draw(u, **kw):
        t, lp, k = oracle.sample64(y, [u], **{a: [b] for a, b in kw.items()})
        return int(t[0]), round(float(np.exp(lp[0])), 6), int(k[0])

    assert draw(0.0) == (0, 0.3, 4)
    assert draw(0.35) == (1, 0.1, 4)
    assert draw(0.95) == (4, 0.1, 4)
    assert draw(1.0) == (4, 0.1, 4)
    assert draw(0.99, top_k=3) == (3, round(5 / 9, 6), 3)       # of the equal ones the lower column
    assert draw(0.99, top_p=0.75) == (3, 0.625, 2)
    assert draw(0.0, top_k=2, top_p=0.6) == (3, 1.0, 1)          # .5 of .8 is enough
    assert draw(0.2, min_p=0.5) == (0, 0.375, 2)
    assert draw(0.2, min_p=7.0) == (3, 1.0, 1)
    assert draw(0.2, top_p=0.0) == (3, 1.0, 1)
    assert draw(0.2, temperature=0.0) == (3, 1.0, 1)
    assert oracle.sample64(np.full((1, 3), -np.inf), [0.5])[0][0] == -1
    assert np.isnan(oracle.sample64(np.array([[0.0, np.inf]]), [0.5])[1][0])


def test_sampling_frequencies():
    rng = np.random.default_rng(1)
    y = rng.standard_normal(20) * 2
    u = (np.arange(4000) + 0.5) / 4000
    t, lp, k = oracle.sample64(np.tile(y, (4000, 1)), u, temperature=np.full(4000, 1.3), top_k=np.full(4000, 7))
    e = np.exp(y / 1.3)
    e[np.argsort(-y)[7:]] = 0.0
    p = e / e.sum()
    assert np.abs(np.bincount(t, minlength=20) / 4000 - p).max() <= 1 / 4000 and np.all(k == 7)
    assert np.allclose(np.exp(lp), p[t])
