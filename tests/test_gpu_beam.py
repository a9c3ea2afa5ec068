"""m2_beam_select against a plain 64-bit implementation: every request's k
best of beams x vocabulary by score + log_softmax(logits), ties to the lower
beam * vocab + token.

Bound: the log of a sum of f32 exponentials (each within 2^-22 relative, its
argument rounded twice, at most 45 additions deep) is within 2^-18 of exact,
and the score is rounded to f32 once.  Orders are compared exactly where the
exact values of neighbours lie further apart than twice that; where they do
not, the returned continuation's exact value has to be within it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

LSE = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _values(x, scores, done=None, eos=None):
    """Exact values [batch, beams, vocab] (64 bits; -inf: no continuation)."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        inf = np.isposinf(m)
        p = np.where(inf, np.where(np.isposinf(x), 1.0, 0.0), np.exp(x - np.where(np.isfinite(m), m, 0.0)))
        lse = np.log(p.sum(-1, keepdims=True)) + np.where(np.isfinite(m), m, 0.0)
        logp = np.where(inf, np.where(np.isposinf(x), -lse, -np.inf), np.where(np.isneginf(x), -np.inf, x - lse))
    val = np.where(np.isfinite(scores)[..., None], np.asarray(scores, np.float64)[..., None] + logp, -np.inf)
    if done is not None:
        for i, b in np.argwhere(done):
            val[i, b] = -np.inf
            if np.isfinite(scores[i, b]):
                val[i, b, eos] = scores[i, b]
    return val


def _check(step, x, scores, k, done=None, eos=None):
    val = _values(x, scores, done, eos)
    nb, kb, v = val.shape
    tok, par, sc = (t.cpu().numpy() for t in step[:3])
    dn = None if step.done is None else step.done.cpu().numpy()
    assert tok.shape == par.shape == sc.shape == (nb, k)
    for i in range(nb):
        flat = val[i].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:k + 1]
        order = order[flat[order] > -np.inf]
        n = min(k, len(order))
        got = par[i, :n].astype(np.int64) * v + tok[i, :n]
        assert len(set(got.tolist())) == n and (got >= 0).all() and (got < kb * v).all()
        best = flat[order]
        assert np.all(np.abs(flat[got] - best[:n]) <= 2 * LSE)
        apart = np.concatenate([[np.inf], -np.diff(best), [np.inf]])
        clear = (apart[:-1][:n] > 4 * LSE) | (apart[:-1][:n] == 0)
        clear &= (apart[1:][:n] > 4 * LSE) | (apart[1:][:n] == 0)
        assert np.array_equal(got[clear], order[:n][clear]), (i, got, order, best)
        assert np.all(np.abs(sc[i, :n] - flat[got]) <= LSE + 2.0 ** -24 * np.abs(flat[got]))
        assert np.all(tok[i, n:] == -1) and np.all(par[i, n:] == -1) and np.all(np.isneginf(sc[i, n:]))
        if dn is not None:
            was = np.zeros(kb, bool) if done is None else done[i]
            assert np.array_equal(dn[i, :n], was[par[i, :n]] | (tok[i, :n] == eos)) and not dn[i, n:].any()


def _case(nb, kb, v, dtype, seed, pad=0, std=2.5):
    rng = np.random.default_rng(seed)
    wide = torch.from_numpy((rng.standard_normal((nb * kb, v + pad)) * std).astype(np.float32)).to(dtype).cuda()
    scores = (-10.0 - 4.0 * rng.random((nb, kb))).astype(np.float32)
    x = wide[:, :v].float().cpu().numpy().reshape(nb, kb, v)
    return wide[:, :v], x, scores


def _go(logits, scores, k=None, **kw):
    done = kw.pop("done", None)
    step = m2.m2_beam_select(logits, torch.from_numpy(scores).cuda(), k,
                             done=None if done is None else torch.from_numpy(done).cuda(), **kw)
    torch.cuda.synchronize()
    return step


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("nb,kb,v,k,dtype,pad", [
    (1, 1, 1, 1, F32, 0), (1, 1, 7, 10, BF, 0), (1, 4, 32000, 4, BF, 0), (2, 3, 1001, 6, BF, 0), (2, 3, 1001, 6, F32, 3),
    (3, 5, 2048, 5, BF, 1), (1, 32, 2049, 64, BF, 0), (2, 32, 8193, 32, F32, 1), (5, 2, 50021, 4, BF, 7),
    (64, 8, 4099, 8, BF, 0), (128, 8, 1000, 16, F32, 0), (40, 8, 16411, 8, BF, 2), (1, 2, 131072, 64, F32, 0),
    (300, 1, 9000, 1, BF, 8), (1, 1, 300001, 33, BF, 0), (2, 4, 100, 64, F32, 0)])
def test_matches_the_formula(nb, kb, v, k, dtype, pad):
    logits, x, scores = _case(nb, kb, v, dtype, nb * 31 + v, pad)
    _check(_go(logits, scores, k), x, scores, k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [0, 1])
def test_finished_beams_go_on_as_themselves(dtype, pad):
    logits, x, scores = _case(6, 5, 3001, dtype, 5, pad)
    rng = np.random.default_rng(0)
    done = rng.random((6, 5)) < 0.4
    done[0], done[1] = True, False
    logits[torch.from_numpy(done.reshape(-1)).cuda()] = float("nan")      # what a finished beam's row holds is not read
    scores[2, 0], done[2, 0] = -np.inf, True
    step = _go(logits, scores, 10, done=done, eos_token=17)
    _check(step, x, scores, 10, done, 17)


def test_end_token_without_finished_beams():
    logits, x, scores = _case(3, 2, 11, F32, 8)
    _check(_go(logits, scores, 20, eos_token=3), x, scores, 20, None, 3)


@pytest.mark.parametrize("v", [500, 20000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks(v, dtype):
    """-inf, NaN, +inf, the type's lowest value, rows with nothing left and
    beams without a score."""
    logits, x, scores = _case(9, 3, v, dtype, 3 + v)
    low = float(torch.finfo(dtype).min)
    L = logits.view(9, 3, v)
    L[0, :, 5:] = float("-inf")                 # five tokens a beam
    L[1] = float("-inf")                        # nothing at all
    L[2, 1] = float("-inf")                     # one beam has nothing
    L[3, :, ::2] = float("nan")
    L[4] = float("nan")
    L[5, 0, 7] = float("inf")
    L[5, 1, 3:9] = float("inf")
    L[6] = low                                  # uniform, at the lowest value
    L[7, :, 2:] = low                           # two tokens, the rest at the lowest value
    scores[8, 0], scores[8, 1] = -np.inf, np.nan
    x = logits.float().cpu().numpy().reshape(9, 3, v)
    _check(_go(logits, scores, 12), x, scores, 12)


@pytest.mark.parametrize("v,pad", [(3000, 0), (3001, 0), (8192, 5), (40000, 1)])
@pytest.mark.parametrize("k", [3, 40])
def test_ties_go_to_the_lowest_index(v, pad, k):
    """All logits equal (more survivors than fit), equal rows at different
    alignments, +0 and -0, and equal scores: ties stay ties."""
    kb = 4
    rng = np.random.default_rng(v)
    wide = torch.zeros((3 * kb, v + pad), dtype=BF, device="cuda")
    logits = wide[:, :v]
    row = torch.from_numpy(rng.integers(-20, 20, v).astype(np.float32) / 8).cuda().to(BF)
    logits[kb:2 * kb] = row                     # four equal rows, many equal logits
    logits[2 * kb:, ::3] = -0.0
    scores = np.full((3, kb), -3.0, np.float32)
    step = _go(logits, scores, k)
    x = logits.float().cpu().numpy().reshape(3, kb, v)
    val = _values(x, scores)
    for i in range(3):
        flat = np.repeat(x[i, :1], kb, 0).reshape(-1) + 0.0       # equal rows: the logits decide
        want = np.argsort(-flat, kind="stable")[:k]
        assert np.array_equal(step.parents[i].cpu().numpy() * v + step.tokens[i].cpu().numpy(), want)
        assert np.allclose(step.scores[i].cpu().numpy(), val[i].reshape(-1)[want], rtol=2.0 ** -23, atol=LSE)


def test_many_equal_values_across_chunks_and_beams():
    """32 beams of equal rows: more equal candidates in the merge than it ranks by counting."""
    v = 70000
    logits = torch.zeros((32, v), dtype=F32, device="cuda")
    scores = np.zeros((1, 32), np.float32)
    step = _go(logits, scores, 64)
    assert step.parents.eq(0).all() and torch.equal(step.tokens[0].cpu(), torch.arange(64, dtype=torch.int32))


def test_large_logits_and_scores():
    logits, x, scores = _case(2, 4, 5000, F32, 21, std=3000.0)
    scores *= 100.0
    val = _values(x, scores)
    step = _go(logits, scores, 8)
    for i in range(2):
        want = np.argsort(-val[i].reshape(-1), kind="stable")[:8]
        assert np.array_equal(step.parents[i].cpu().numpy() * 5000 + step.tokens[i].cpu().numpy(), want)
        assert np.allclose(step.scores[i].cpu().numpy(), val[i].reshape(-1)[want], rtol=2.0 ** -24, atol=2.0 ** -11)


def test_values_past_f32():
    """Logits at the type's lowest next to scores at the top of f32: the sums
    the merge bounds its candidates with overflow, the values do not."""
    low = float(torch.finfo(F32).min)
    logits = torch.full((4, 700), low, device="cuda")
    logits[1, :5] = -1.0e38
    logits[3] = 0.0
    scores = np.array([[3.3e38, 3.2e38, 3.0e38, 3.25e38]], np.float32)
    step = _go(logits, scores, 12)
    val = _values(logits.cpu().numpy().reshape(1, 4, 700), scores)[0].reshape(-1)
    want = np.argsort(-val, kind="stable")[:12]
    assert np.array_equal(step.parents[0].cpu().numpy() * 700 + step.tokens[0].cpu().numpy(), want)
    assert np.allclose(step.scores[0].cpu().numpy(), val[want], rtol=2.0 ** -23, atol=0)


def test_rows_past_32_bit_offsets():
    """Rows a gigabyte apart: offsets above 2^31 elements."""
    v, stride = 1000, 1 << 29
    if torch.cuda.mem_get_info()[0] < 14 * (1 << 30):
        pytest.skip("needs 14 GB free")
    buf = torch.empty(5 * stride + v, dtype=BF, device="cuda")
    logits = buf.as_strided((6, v), (stride, 1))
    small, x, scores = _case(2, 3, v, BF, 77)
    logits.copy_(small)
    _check(_go(logits, scores, 6), x, scores, 6)


def test_in_place_scores_and_flags():
    logits, x, scores = _case(4, 4, 2500, BF, 9)
    done = np.zeros((4, 4), bool)
    done[1, 2] = True
    want = _go(logits, scores.copy(), 4, done=done, eos_token=1)
    sd, dd = torch.from_numpy(scores).cuda(), torch.from_numpy(done).cuda()
    out = m2.BeamStep(torch.empty((4, 4), dtype=torch.int32, device="cuda"),
                      torch.empty((4, 4), dtype=torch.int32, device="cuda"), sd, dd)
    got = m2.m2_beam_select(logits, sd, 4, eos_token=1, done=dd, out=out)
    torch.cuda.synchronize()
    assert got is out and all(torch.equal(a, b) for a, b in zip(got, want))


def test_repeats_on_streams_and_in_a_graph():
    logits, x, scores = _case(5, 4, 33001, BF, 4)
    want = _go(logits, scores, 8)
    sd = torch.from_numpy(scores).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [m2.m2_beam_select(logits, sd, 8, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o[:3], want[:3]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = m2.m2_beam_select(logits, sd, 8)
    logits.neg_()
    want2 = m2.m2_beam_select(logits, sd, 8)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out[:3], want2[:3])) and not torch.equal(out[0], want[0])


def test_no_requests():
    step = m2.m2_beam_select(torch.empty((0, 50), dtype=BF, device="cuda"), torch.empty((0, 4), device="cuda"))
    assert step.tokens.shape == (0, 4)


# ---- logits of any finite size.  A shift of a row by a constant leaves its
# values: they are taken here as scores + ((x - max) - log sum exp(x - max)),
# which keeps log sum exp where x - log sum exp(x) in 64 bits has no room for
# it.  The bound is the one above: the exponent is (x - max) log2 e, x - max
# rounded once at most, however large the row's maximum is.


def _shifted(x, scores):
    x = np.asarray(x, np.float64)
    m = x.max(-1, keepdims=True)
    d = x - m
    with np.errstate(under="ignore"):
        logp = d - np.log(np.exp(d).sum(-1, keepdims=True))
    return np.asarray(scores, np.float64)[..., None] + logp


def _check_values(step, val, k):
    """Every request has its k best (finite logits: there are that many), in
    order, and their scores."""
    nb, kb, v = val.shape
    tok, par, sc = (t.cpu().numpy() for t in step[:3])
    for i in range(nb):
        flat = val[i].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:k + 1]
        best = flat[order]
        assert (tok[i] >= 0).all() and (par[i] >= 0).all(), (i, "continuations lost", tok[i], par[i])
        got = par[i].astype(np.int64) * v + tok[i]
        assert len(set(got.tolist())) == k
        bound = LSE + 2.0 ** -24 * np.abs(flat[got])
        assert np.all(np.abs(sc[i] - flat[got]) <= bound), (i, sc[i], flat[got])
        assert np.all(np.abs(flat[got] - best[:k]) <= 2 * LSE)
        apart = np.concatenate([[np.inf], -np.diff(best), [np.inf]])
        clear = ((apart > 4 * LSE) | (apart == 0))
        clear = clear[:k] & clear[1:k + 1]
        assert np.array_equal(got[clear], order[:k][clear]), (i, got, order)


SIZES = [5e3, 1.1e4, 2e4, 1e5, 1e6, 1e7, 1e8, 1e9, 1e12, 1e30, 1e38]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v,pad", [(257, 0), (9001, 3), (70000, 0)])
@pytest.mark.parametrize("size", [s * c for c in SIZES for s in (1, -1)])
def test_large_finite_logits(size, v, pad, dtype):
    """Rows uniform at a large value (all beams, or one beside live ones), a
    few or most tokens masked with it, one token forced with it, and rows
    shifted by it."""
    nb, kb = 6, 3
    logits, _, scores = _case(nb, kb, v, dtype, 91 + v, pad)
    L = logits.view(nb, kb, v) if not pad else logits.as_strided((nb, kb, v), (kb * logits.stride(0), logits.stride(0), 1))
    L[0] = size
    L[1, 1] = size
    L[2, :, ::2] = size
    L[3, :, 12:] = size
    L[4, 0, v // 3] = size
    L[5] += size
    x = logits.float().cpu().numpy().reshape(nb, kb, v)
    _check_values(_go(logits, scores, 7), _shifted(x, scores), 7)
