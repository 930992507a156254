"""Host-only checks of w12_embed and w12_logprobs: refusals before any launch, and the oracle's
conventions."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import oracle
from lossless_bit_weight_02_amd import w12
from tests.test_abi_cpu import HEADER, _lib, _rec


def test_flag_values_match_header():
    text = open(HEADER).read()
    for name in ("IDS_I64", "LOGITS_BF16"):
        assert int(re.search(rf"#define W12_{name} (0x[0-9a-fA-F]+)u", text).group(1), 16) == getattr(w12, name)


def _embed(ids=0x1000, count=3, rec=None, scale=1.0, out=0x2000, flags=0):
    return _lib().w12_embed(ids, count, ctypes.byref(rec or _rec()), scale, out, flags, None)


def test_embed_refusals():
    assert _embed(ids=None) == w12.W12_ERR_ARG
    assert _embed(out=None) == w12.W12_ERR_ARG
    assert _embed(count=0) == w12.W12_ERR_ARG
    assert _embed(count=-1) == w12.W12_ERR_ARG
    assert _embed(count=1 << 31) == w12.W12_ERR_RANGE
    assert _embed(rec=_rec(lo=None)) == w12.W12_ERR_ARG
    assert _embed(rec=_rec(k=130)) == w12.W12_ERR_SHAPE
    assert _embed(rec=_rec(esc_cap=(1 << 32) - 255)) == w12.W12_ERR_RANGE
    assert _embed(ids=0x1002) == w12.W12_ERR_ALIGN
    assert _embed(ids=0x1004, flags=w12.IDS_I64) == w12.W12_ERR_ALIGN
    assert _embed(out=0x2008) == w12.W12_ERR_ALIGN
    for bad in (1, w12.Q8_MIDPOINT, w12.LOGITS_BF16):
        assert _embed(flags=bad) == w12.W12_ERR_ARG


def _lp(y=0x1000, m=2, n=100, ldy=100, tokens=0x2000, nt=1, top=4, logp=0x3000, ent=0x4000, ti=0x5000, tl=0x6000,
        scratch=0x7000, nbytes=1 << 30, flags=0):
    return _lib().w12_logprobs(y, m, n, ldy, tokens, nt, top, logp, ent, ti, tl, scratch, nbytes, flags, None)


def test_logprobs_refusals():
    assert _lp(y=None) == w12.W12_ERR_ARG
    assert _lp(ent=None) == w12.W12_ERR_ARG
    assert _lp(m=0) == w12.W12_ERR_ARG
    assert _lp(n=0) == w12.W12_ERR_ARG
    assert _lp(m=1 << 31) == w12.W12_ERR_RANGE
    assert _lp(n=1 << 31, ldy=1 << 31) == w12.W12_ERR_RANGE
    assert _lp(ldy=99) == w12.W12_ERR_ARG
    assert _lp(ldy=1 << 41) == w12.W12_ERR_RANGE
    assert _lp(nt=-1) == w12.W12_ERR_ARG
    assert _lp(nt=1 << 31) == w12.W12_ERR_RANGE
    assert _lp(tokens=None) == w12.W12_ERR_ARG
    assert _lp(logp=None) == w12.W12_ERR_ARG
    assert _lp(ti=None) == w12.W12_ERR_ARG
    assert _lp(tl=None) == w12.W12_ERR_ARG
    assert _lp(top=65, n=1000, ldy=1000) == w12.W12_ERR_RANGE
    assert _lp(top=-1) == w12.W12_ERR_RANGE
    assert _lp(top=5, n=4, ldy=4) == w12.W12_ERR_RANGE
    assert _lp(y=0x1002) == w12.W12_ERR_ALIGN
    assert _lp(y=0x1001, flags=w12.LOGITS_BF16) == w12.W12_ERR_ALIGN
    assert _lp(tokens=0x2004, flags=w12.IDS_I64) == w12.W12_ERR_ALIGN
    assert _lp(tokens=0x2002) == w12.W12_ERR_ALIGN
    assert _lp(logp=0x3001) == w12.W12_ERR_ALIGN
    assert _lp(ent=0x4002) == w12.W12_ERR_ALIGN
    assert _lp(ti=0x5002) == w12.W12_ERR_ALIGN
    for bad in (1, w12.OUT_BF16, w12.Q8_MIDPOINT):
        assert _lp(flags=bad) == w12.W12_ERR_ARG
    need = ctypes.c_uint64(0)
    assert _lib().w12_logprobs_scratch(1, 100, 4, 0, None) == w12.W12_ERR_ARG
    assert _lib().w12_logprobs_scratch(1, 100, 101, 0, ctypes.byref(need)) == w12.W12_ERR_RANGE
    assert _lib().w12_logprobs_scratch(0, 100, 1, 0, ctypes.byref(need)) == w12.W12_ERR_ARG


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    rec = w12.W12Weight(16, 128, *([torch.zeros(16, dtype=torch.uint8)] * 3), *([torch.zeros(17, dtype=torch.int32)] * 3))
    with pytest.raises(TypeError):
        w12.embed(torch.zeros(3), rec)
    with pytest.raises(TypeError):
        w12.embed([1, 2], rec)
    with pytest.raises(ValueError):
        w12.embed(torch.zeros(3, dtype=torch.int32), rec, out=torch.zeros(3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        w12.logprobs(torch.zeros(3, 4))            # not on the GPU
    with pytest.raises(ValueError):
        w12.logprobs("logits")


def test_oracle_logprobs_conventions():
    inf, nan = math.inf, math.nan
    y = np.array([[0.0, 0.0, -inf, 0.0], [-inf] * 4, [1.0, inf, 0.0, 2.0], [nan, 1.0, 2.0, 2.0], [100.0, 0.0, -0.0, 50.0]])
    tok = np.array([[1, 2], [0, 9], [0, -1], [1, 4], [0, 1]])
    logp, ent, idx, tlp = oracle.logprobs64(y, tok, 3)
    assert np.allclose(logp[0], [-math.log(3), -inf]) and np.isclose(ent[0], math.log(3))
    assert idx[0].tolist() == [0, 1, 3]
    assert np.all(logp[1] == -inf) and ent[1] == 0 and idx[1].tolist() == [0, 1, 2] and np.all(tlp[1] == -inf)
    assert np.isnan(logp[2, 0]) and logp[2, 1] == -inf and np.isnan(ent[2]) and idx[2].tolist() == [1, 3, 0]
    assert idx[3].tolist() == [0, 2, 3]
    # a confident row keeps its small probability mass
    assert np.isclose(logp[4, 0], -math.exp(-50), rtol=1e-12) and idx[4].tolist() == [0, 3, 1]
