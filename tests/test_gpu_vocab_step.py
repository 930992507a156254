"""One verification step's vocabulary ends together: ids -> embedding rows of a W12 record -> logits over
the same record (exact pass, and the Q pass on its 4-bit copy) -> log probabilities, entropy and
alternatives; eagerly, and as one captured graph replayed on new ids.

The logits carry the products' documented bound B = 1e-3 sum |x w| (bfloat16 logits half an ulp
more); a log probability moves by at most twice the largest error of its row's logits, plus its own
float bounds.
"""
import numpy as np
import pytest

import oracle
from lossless_bit_weight_02_amd import synth
from tests.gpu_util import say, to_dev, to_host_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

N, K = 5003, 640


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lossless_bit_weight_02_amd import w12
    w12.lib()
    rng = np.random.default_rng(8)
    w = synth.f32_to_bf16_bits((rng.standard_normal((N, K)) * 0.05).astype(np.float32))
    w[rng.random((N, K)) < 2e-3] = 0
    w[rng.random((N, K)) < 2e-4] = 0x4080
    rec = w12.encode(to_dev(w))
    ref = oracle.encode(w)
    return w12, w, rec, w12.mx4_build(rec), oracle.mx4_weights64(ref, oracle.mx4_copy(ref))


def _check(r, y64, bound, tok, what):
    """r: LogProbs; y64 the oracle's logits, bound their error."""
    lp, ent, idx, tlp = oracle.logprobs64(y64, tok, r.top_index.shape[1])
    ls, etol = oracle.logprobs_tol(y64)
    slack = 2 * bound.max(axis=1)
    u = 2.0 ** -24
    got = r.logp.double().cpu().numpy()
    assert np.all(np.abs(got - lp) <= (slack + ls)[:, None] + 4 * u * np.abs(lp)), what
    # the entropy: d H = -sum p (log p + H) d y, at most (H + max |log p|) times the logits' error
    full = y64 - y64.max(axis=1, keepdims=True)
    spread = np.abs(full).max(axis=1) + ent + np.log(y64.shape[1])
    assert np.all(np.abs(r.entropy.double().cpu().numpy() - ent) <= slack * (spread + 1) + etol + 4 * u * ent), what
    # the alternatives are the largest up to the logits' error, in descending order
    gi = r.top_index.cpu().numpy()
    for j in range(y64.shape[0]):
        assert len(set(gi[j].tolist())) == gi.shape[1]
        kth = np.sort(y64[j])[::-1][gi.shape[1] - 1]
        assert np.all(y64[j, gi[j]] >= kth - 2 * bound[j].max()), what
    assert torch.all(r.top_logp[:, :-1] >= r.top_logp[:, 1:])


@pytest.mark.parametrize("m", [1, 2, 7, 16, 33, 64, 70])
def test_step(step, m):
    w12, w, rec, cp, wq = step
    rng = np.random.default_rng(m)
    ids, nxt = rng.integers(0, N, m), rng.integers(0, N, (m, 2))
    say(f"vocabulary step m={m}")
    x = w12.embed(torch.tensor(ids, device="cuda"), rec, scale=8.0)
    want_x = torch.from_numpy(synth.bf16_bits_to_f32(w[ids]) * np.float32(8.0)).to(torch.bfloat16)
    assert torch.equal(x.cpu(), want_x)
    xb = to_host_bits(x)
    t = torch.tensor(nxt, device="cuda")
    for name, y, w64 in (("exact", w12.gemm(x, rec), oracle.bf16_to_f64(w)), ("Q pass", w12.mx4_gemm(x, cp), wq)):
        y64, bound = oracle.gemm64_f(xb, w64), 1e-3 * oracle.abs_bound64_f(xb, w64)
        r = w12.logprobs(y, t, top=6)
        _check(r, y64, bound, nxt, f"{name} m={m}")
        # bfloat16 logits: half an ulp, 2^-9 of the larger neighbour, more
        y16 = w12.gemm(x, rec, out_bf16=True) if name == "exact" else w12.mx4_gemm(x, cp, out_bf16=True)
        _check(w12.logprobs(y16, t, top=6), y64, bound + 2.0 ** -8 * (np.abs(y64) + bound), nxt, f"{name} bf16 m={m}")
    # top-1 of the Q pass is the first alternative, up to the error of the two passes
    idx, _ = w12.mx4_top1(x, cp)
    y64, bound = oracle.gemm64_f(xb, wq), 1e-3 * oracle.abs_bound64_f(xb, wq)
    a, b = idx.cpu().numpy(), w12.logprobs(w12.mx4_gemm(x, cp), top=1).top_index[:, 0].cpu().numpy()
    j = np.arange(m)
    assert np.all(np.abs(y64[j, a] - y64[j, b]) <= 4 * bound.max(axis=1))


def test_step_captured(step):
    """The whole step as one graph, replayed on other ids among eager steps of the same shapes."""
    w12, w, rec, cp, wq = step
    m = 12
    g = torch.Generator().manual_seed(4)
    ids = [torch.randint(0, N, (m,), generator=g).cuda() for _ in range(3)]
    nxt = torch.randint(0, N, (m, 3), generator=g).cuda()

    def run(i):
        return w12.logprobs(w12.mx4_gemm(w12.embed(i, rec, scale=8.0), cp), nxt, top=4)

    say("vocabulary step captured")
    want = [run(i) for i in ids]
    st = ids[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(st)
    for j in (1, 2, 0, 2):
        st.copy_(ids[j])
        graph.replay()
        eager = run(ids[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[j]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
