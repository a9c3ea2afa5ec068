"""m2_token_logprobs against a plain 64-bit implementation.

Bound: with m the row's largest logit, log S is summed in f32 over at most 2^24
tokens: an exponential is within 2^-22 relative (its argument, at most 2^5 in
size where it counts, is rounded once: 2^-19 at most, less where the weight
is), a thread adds at most a few hundred terms one after another with errors of
either sign, and threads are joined in a tree: 2^-19 in all.  The result is
rounded to f32 once.  The entropy's mean is a quotient of two such sums, the
spread |x - m| under the weights at most 2^5: 2^-16.  (Both sides of a
comparison are rounded to f32: half a step each.)  Ranks and tokens are
compared exactly: they depend on the logits' order alone."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

LSE, ENT = 2.0 ** -19, 2.0 ** -16
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def reference(x, tokens, top):
    """(logprobs, ranks, entropy, top tokens, top logprobs) of float64 logits."""
    rows, v = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        inf = np.isposinf(m)
        d = np.where(inf, np.where(np.isposinf(x), 0.0, -np.inf), np.where(np.isneginf(x), -np.inf, x - m))
        p = np.exp(d)
        z = np.log(p.sum(1, keepdims=True))
        logp = np.where(np.isneginf(d), -np.inf, d - z)
        h = -np.where(p > 0, p / p.sum(1, keepdims=True) * np.where(p > 0, logp, 0.0), 0.0).sum(1)
    h = np.where(np.isneginf(m[:, 0]), 0.0, h)
    order = np.argsort(-x, axis=1, kind="stable")
    lp, rk = np.zeros(rows), np.zeros(rows, np.int64)
    tt, tl = np.full((rows, top), -1), np.full((rows, top), -np.inf)
    for r in range(rows):
        if tokens is not None and 0 <= tokens[r] < v:
            t = tokens[r]
            lp[r] = logp[r, t]
            rk[r] = 1 + (np.isfinite(x[r]) | np.isposinf(x[r])).sum() if np.isneginf(x[r, t]) else \
                1 + int(np.argmax(order[r] == t))
        best = [t for t in order[r][:top] if not np.isneginf(logp[r, t])]
        tt[r, :len(best)], tl[r, :len(best)] = best, logp[r, best]
    return lp, rk, h, tt, tl


def close(got, want, tol):
    got = got.cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)      # (differences past f32's range are -inf)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), (got, want)
    ok = ~np.isneginf(want)
    with np.errstate(invalid="ignore"):
        err = np.abs(got[ok] - want[ok])
        assert (err <= tol + 2.0 ** -23 * np.abs(want[ok])).all(), float(np.max(err, initial=0.0))


def check(logits, tokens, top, out=None):
    x = logits.float().cpu().numpy().astype(np.float64)
    t = None if tokens is None else torch.from_numpy(np.asarray(tokens, np.int32)).cuda()
    o = m2.m2_token_logprobs(logits, t, top, out=out)
    torch.cuda.synchronize()
    lp, rk, h, tt, tl = reference(x, tokens, top)
    if tokens is None:
        assert o.logprobs is None and o.ranks is None
    else:
        close(o.logprobs, lp, LSE)
        assert np.array_equal(o.ranks.cpu().numpy(), rk)
    close(o.entropy, h, ENT)
    if top:
        assert np.array_equal(o.top_tokens.cpu().numpy(), tt)
        close(o.top_logprobs, tl, LSE)
    return o


def make(rows, v, dtype, seed, pad=0, std=2.5):
    rng = np.random.default_rng(seed)
    wide = torch.from_numpy((rng.standard_normal((rows, v + pad)) * std).astype(np.float32)).to(dtype).cuda()
    return wide[:, :v], rng.integers(0, v, rows).astype(np.int32)


@pytest.mark.parametrize("rows,v,top,dtype,pad", [
    (1, 1, 1, F32, 0), (1, 1, 0, BF, 0), (3, 2, 5, BF, 0), (1, 7, 10, BF, 1), (5, 31, 3, F32, 0), (2, 255, 64, BF, 0),
    (2, 257, 64, F32, 1), (4, 1000, 20, BF, 0), (3, 1001, 20, BF, 1), (7, 2049, 33, F32, 3), (9, 8191, 64, BF, 0),
    (1, 16384, 20, BF, 0), (2, 32000, 5, BF, 0), (1, 32001, 5, F32, 0), (6, 50021, 10, F32, 3), (5, 50021, 20, BF, 5),
    (1, 131072, 20, BF, 0), (2, 131072, 64, F32, 0), (75, 9000, 8, BF, 8), (153, 5001, 1, F32, 0), (310, 3001, 4, BF, 0),
    (700, 1100, 2, F32, 1), (1, 300001, 33, BF, 0), (2, 1000003, 5, F32, 0)])
def test_matches_the_formula(rows, v, top, dtype, pad):
    logits, tokens = make(rows, v, dtype, rows * 31 + v, pad)
    check(logits, tokens, top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_that_are_not_asked_for(dtype):
    logits, tokens = make(5, 3001, dtype, 1)
    check(logits, None, 0)
    check(logits, None, 7)
    check(logits, tokens, 0)
    out = m2.TokenLogprobs(*[torch.full(s, -7, dtype=d, device="cuda") for s, d in
                             (((5,), F32), ((5,), torch.int32), ((5,), F32), ((5, 3), torch.int32), ((5, 3), F32))])
    assert check(logits, tokens, 3, out=out) is out


def test_rows_without_a_token_and_tokens_out_of_range():
    logits, tokens = make(6, 700, BF, 2)
    tokens[1] = tokens[4] = -1
    o = check(logits, tokens, 2)
    assert o.logprobs[1] == 0 and o.ranks[4] == 0
    m2.check_standalone()
    tokens[0], tokens[5] = 700, -2
    o = check(logits, tokens, 2)
    assert o.logprobs[0] == 0 and o.ranks[0] == 0 and o.ranks[5] == 0
    with pytest.raises(m2.M2Error) as e:
        m2.check_standalone()
    assert e.value.status == m2.M2_EINVAL and "token" in str(e.value)
    m2.check_standalone()


@pytest.mark.parametrize("v", [40, 700, 20000, 70001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks(v, dtype):
    """-inf, NaN, +inf, the type's lowest and largest values, rows with nothing
    left, and a masked token to score."""
    L, tokens = make(14, v, dtype, v)
    low, high = float(torch.finfo(dtype).min), float(torch.finfo(dtype).max)
    L[0, 5:] = float("-inf")                    # five tokens
    L[1] = float("-inf")                        # nothing
    L[2] = float("nan")                         # nothing
    L[3, ::2] = float("nan")
    L[4, 7] = float("inf")
    L[5, 3:9] = float("inf")
    L[6] = low                                  # uniform, at the lowest value
    L[7, 2:] = low                              # two tokens, the rest at the lowest value
    L[8] = high                                 # uniform, at the largest value
    L[9, 1:] = low
    L[9, 0] = high
    L[10, : v // 2] = float("-inf")
    L[11, v // 2:] = float("-inf")
    L[12] = -1e9                                # finite masks
    L[12, v // 3] = 4.0
    L[13, 9] = float("nan")
    tokens[:] = [3, 0, 1, 1, 7, 4, v - 1, 1, 5, 0, v - 1, 0, v // 3, 9]
    check(L, tokens, 12)
    tokens[:] = [7, v - 1, 0, 2, 6, 0, 0, 5, v - 1, 7, 0, v - 1, 0, 8]
    check(L, tokens, 12)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [3e4, -3e4, 7e4, -7e4, 1e6, -1e6, 1e30, -1e30, 2e38, -2e38])
def test_large_logits(dtype, shift):
    """Logits of any size: the logarithm is relative to the row's largest."""
    L, tokens = make(4, 3001, F32, 9)
    L = (L + shift).to(dtype)
    check(L, tokens, 9)
    L[:, 100:200] = 0.0 if shift < 0 else -shift      # values far from the rest
    check(L, tokens, 9)


@pytest.mark.parametrize("v", [100, 3000, 8192, 40001, 131072])
@pytest.mark.parametrize("top", [3, 40, 64])
def test_ties_go_to_the_lowest_token(v, top):
    """More equal logits than candidates fit, +0 and -0, few distinct values,
    ascending and descending rows."""
    rng = np.random.default_rng(v)
    rows = [np.zeros(v), np.where(rng.random(v) < 0.5, 0.0, -0.0), rng.integers(-20, 20, v) / 8.0,
            np.arange(v) / 1000.0, -np.arange(v) / 1000.0, np.where(np.arange(v) == v - 1, 1.0, -1e9),
            np.where(np.arange(v) % 7 == 3, 2.0, 1.0)]
    tokens = np.array([v - 1, v // 2, 5, v // 3, v // 3, 17, 3], np.int32)
    for dtype in (BF, F32):
        wide = torch.from_numpy(np.stack(rows).astype(np.float32)).to(dtype).cuda()
        check(wide, tokens, top)
        padded = torch.full((len(rows), v + 3), 9.0, dtype=dtype, device="cuda")
        padded[:, 1:v + 1] = wide
        check(padded[:, 1:v + 1], tokens, top)


def test_a_likely_token():
    """Probabilities near 1 and their rank; entropy near 0."""
    for dtype in (BF, F32):
        L, tokens = make(6, 20011, dtype, 4)
        for r in range(6):
            L[r, tokens[r]] = 10.0 + 8 * r
        o = check(L, tokens, 3)
        assert (o.ranks == 1).all() and (o.entropy >= 0).all()


def test_equal_ranks_and_alternatives():
    """The token at place i of the alternatives has rank i + 1 and the same log
    probability."""
    L, _ = make(4, 30011, BF, 6)
    top = m2.m2_token_logprobs(L, None, 32)
    for i in (0, 1, 17, 31):
        o = m2.m2_token_logprobs(L, top.top_tokens[:, i].contiguous())
        assert (o.ranks == i + 1).all() and torch.equal(o.logprobs, top.top_logprobs[:, i])


def test_no_rows():
    o = m2.m2_token_logprobs(torch.empty(0, 10, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert o.logprobs.shape == (0,) and o.top_tokens.shape == (0, 3)


@pytest.mark.parametrize("rows,v", [(2, 40000), (400, 1500)])
def test_captured_graphs_and_another_stream(rows, v):
    cases = [make(rows, v, BF, i) for i in range(4)]
    toks = [torch.from_numpy(t).cuda() for _, t in cases]
    want = [m2.m2_token_logprobs(L, t, 9) for (L, _), t in zip(cases, toks)]
    bufs = [(torch.empty_like(cases[0][0]), torch.empty_like(toks[0])) for _ in range(2)]
    graphs = []
    for L, t in bufs:
        L.zero_(), t.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = m2.m2_token_logprobs(L, t, 9)
        graphs.append((graph, o))
    for i in range(4):
        bufs[i % 2][0].copy_(cases[i][0])
        bufs[i % 2][1].copy_(toks[i])
        graphs[i % 2][0].replay()
        assert all(torch.equal(a, b) for a, b in zip(graphs[i % 2][1], want[i]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [m2.m2_token_logprobs(L, t, 9, stream=side) for (L, _), t in zip(cases, toks)]
    side.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_python_refuses_what_does_not_fit():
    L, tokens = make(4, 100, BF, 0)
    t = torch.from_numpy(tokens).cuda()
    for call in (lambda: m2.m2_token_logprobs(L, t.long()), lambda: m2.m2_token_logprobs(L, t[:3]),
                 lambda: m2.m2_token_logprobs(L.half(), t), lambda: m2.m2_token_logprobs(L.t(), None, 1),
                 lambda: m2.m2_token_logprobs(L, t, -1), lambda: m2.m2_token_logprobs(L[0], None, 1),
                 lambda: m2.m2_token_logprobs(L.expand(3, 4, 100)[:, 0], None, 1)):
        with pytest.raises(ValueError):
            call()
    full = m2.m2_token_logprobs(L, t, 5)
    for call in (lambda: m2.m2_token_logprobs(L, None, 5, out=full), lambda: m2.m2_token_logprobs(L, t, 0, out=full),
                 lambda: m2.m2_token_logprobs(L, t, 6, out=full), lambda: m2.m2_token_logprobs(L[:3], t[:3], 5, out=full),
                 lambda: m2.m2_token_logprobs(L, t, 5, out=full._replace(ranks=None))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m2.M2Error) as e:
        m2.m2_token_logprobs(L, t, 65)
    assert e.value.status == m2.M2_ESHAPE


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,v", [(3, 700), (40, 140001)])
def test_values_below_the_normal_range(rows, v, dtype):
    """Logits whose differences only subnormal numbers and the signs of zeros
    show: all equally likely, ordered by their values (-0 and +0 are equal)."""
    rng = np.random.default_rng(v)
    tiny = 2.0 ** (-149 if dtype == F32 else -133)
    x = rng.integers(-3, 4, (rows, v)) * tiny
    x = np.where(x == 0, np.where(rng.random((rows, v)) < 0.5, -0.0, 0.0), x)
    logits = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    check(logits, rng.integers(0, v, rows).astype(np.int32), 7)


@pytest.mark.parametrize("rows,v", [(3, 1000), (20, 140000)])
def test_offsets_past_32_bits(rows, v):
    """Rows so far apart that the last lie past 2^32 elements."""
    step = (1 << 32) // (rows - 1) + 17
    wide = torch.empty(step * (rows - 1) + v, dtype=BF, device="cuda").as_strided((rows, v), (step, 1))
    near, tokens = make(rows, v, BF, v)
    wide.copy_(near)
    t = torch.from_numpy(tokens).cuda()
    for a, b in zip(m2.m2_token_logprobs(wide, t, 11), m2.m2_token_logprobs(near, t, 11)):
        assert torch.equal(a, b) if a.dtype == torch.int32 else torch.allclose(a, b, rtol=0, atol=2 * LSE + 2.0 ** -20)


def test_two_streams_at_once():
    cases = [(make(r, v, d, r), k) for r, v, d, k in ((1, 131072, BF, 20), (64, 131072, BF, 5), (900, 9000, F32, 64),
                                                      (20, 140001, F32, 9))]
    cases = [(L, torch.from_numpy(t).cuda(), k) for (L, t), k in cases]
    want = [m2.m2_token_logprobs(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(8):
        for s, side in enumerate(streams):
            got.append((m2.m2_token_logprobs(*cases[(i + 2 * s) % 4], stream=side), (i + 2 * s) % 4))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o, k in got for a, b in zip(o, want[k]))
    m2.check_standalone()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,v", [(20, 140001), (330, 17001)])
def test_ties_in_many_long_rows(rows, v, dtype):
    """Finite masks with fewer allowed tokens than asked for, equal and sorted
    rows, few distinct values, ties that begin late in a row."""
    rng = np.random.default_rng(v)
    at = np.arange(v)
    low = float(torch.finfo(dtype).min)
    allowed = np.full(v, low)
    allowed[rng.choice(v, 9, replace=False)] = rng.standard_normal(9)
    kinds = [allowed, np.where(at < v - 50, -np.inf, low), np.zeros(v), at / 64.0, -at / 64.0,
             rng.integers(-20, 20, v) / 8.0, np.where(at > v // 2, 2.0, np.where(at % 2, 1.0, -np.inf)),
             np.where(rng.random(v) < 0.01, np.inf, 0.0)]
    x = np.stack([kinds[i % len(kinds)] for i in range(rows)]).astype(np.float32)
    logits = torch.from_numpy(x).to(dtype).cuda()
    check(logits, rng.integers(0, v, rows).astype(np.int32), 20)
    check(logits[:, 1:], rng.integers(0, v - 1, rows).astype(np.int32), 64)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,v", [(3, 5000), (400, 20001)])
def test_masks_in_front(rows, v, dtype):
    """Long masked stretches before a row's first logits, below and above the
    size from which rows are summed as differences."""
    rng = np.random.default_rng(v)
    x = rng.standard_normal((rows, v)) * 2
    for r in range(rows):
        x[r] += (0.0, 60000.0, -60000.0, -70000.0, -200000.0, 300.0)[r % 6]
        x[r, :(0, v // 2, v - 3, v - 1)[r % 4]] = (-np.inf, np.nan)[r % 2]
    logits = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    check(logits, rng.integers(0, v, rows).astype(np.int32), 6)
