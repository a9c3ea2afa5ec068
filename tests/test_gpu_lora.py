"""m2_lora_add: low-rank adapters of many requests beside a shared projection,
against the formula in 64 bits.

Bound per element: the result is rounded to bf16 once (half a step, 2^-8
relative), and the unrounded value is off by at most
    e = s sum_j |b_nj| sum_k |a_jk| |x_k| (2^-16 + (K + rank + 4) 2^-24):
f32 sums over K and the rank in any order, and a rank-wide intermediate kept
to 2^-16 or better.  Integer operands whose sums stay below 2^24, with an
intermediate below 2^16, are exact up to the final rounding."""
import numpy as np
import pytest
import torch

from helpers import bf16_dev, f32_dev, to_np

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).float().numpy().astype(np.float64)


def _inputs(M, N, K, rank, na, seed, ids=None):
    rng = np.random.default_rng(seed)
    x, y = _bf16(rng.standard_normal((M, K))), _bf16(rng.standard_normal((M, N)))
    a = _bf16(rng.standard_normal((na, rank, K)) * K ** -0.5)
    b = _bf16(rng.standard_normal((na, N, rank)) * rank ** -0.5)
    scale = rng.uniform(0.5, 2.0, na).astype(np.float32).astype(np.float64)
    if ids is None:
        ids = rng.integers(-1, na, M)
    return x, y, a, b, scale, np.asarray(ids, np.int32)


def _ref(x, y, a, b, scale, ids):
    """(unrounded value, bound on its error) per element."""
    val, err = y.copy(), np.zeros_like(y)
    K, rank = x.shape[1], a.shape[1]
    for i in np.unique(ids[ids >= 0]):
        at = np.nonzero(ids == i)[0]
        val[at] += scale[i] * ((x[at] @ a[i].T) @ b[i].T)
        err[at] = scale[i] * ((np.abs(x[at]) @ np.abs(a[i]).T) @ np.abs(b[i]).T)
    return val, err * (2.0 ** -16 + (K + rank + 4) * 2.0 ** -24)


def _check(got, val, err, y, ids):
    got = np.asarray(got, np.float64)
    bound = err + (np.abs(val) + err) * 2.0 ** -8
    over = np.abs(got - val) > bound
    assert not over.any(), f"{int(over.sum())} of {over.size} beyond the bound, first at {np.argwhere(over)[0]}"
    bare = ids < 0
    assert np.array_equal(got[bare], y[bare])


def _run(x, y, a, b, scale, ids, out=None, **kw):
    yd = bf16_dev(y)
    r = m2.m2_lora_add(yd, bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.from_numpy(ids).cuda(),
                       scale=None if scale is None else f32_dev(scale), out=yd if out == "in place" else out, **kw)
    torch.cuda.synchronize()
    m2.check_standalone()
    return r


@pytest.mark.parametrize("M,N,K,rank,na", [
    (1, 10304, 2688, 16, 4), (1, 1, 16, 8, 1), (2, 2688, 4096, 8, 3), (3, 77, 48, 24, 2), (7, 203, 160, 40, 5),
    (37, 2688, 4096, 64, 9), (64, 10304, 2688, 16, 64), (65, 130, 2688, 128, 3), (128, 2688, 4096, 128, 17),
    (130, 64, 64, 8, 200), (255, 1000, 272, 32, 12), (257, 1001, 528, 56, 7), (300, 10304, 2688, 16, 3),
    (513, 2688, 4096, 32, 2), (1000, 264, 2688, 104, 40), (2049, 136, 112, 16, 1), (5000, 33, 32, 8, 4096),
    (400, 1003, 272, 16, 120), (512, 520, 160, 72, 300), (900, 777, 1024, 24, 11), (300, 515, 96, 128, 2),
    (700, 4099, 64, 64, 3), (320, 2688, 512, 32, 2), (321, 515, 96, 128, 2), (321, 515, 96, 32, 46), (1024, 264, 272, 16, 150),
    (1023, 1001, 96, 72, 256), (1024, 130, 528, 8, 146), (1025, 72, 528, 24, 700)])
def test_matches_the_formula(M, N, K, rank, na):
    args = _inputs(M, N, K, rank, na, M * 7 + N)
    x, y, a, b, scale, ids = args
    val, err = _ref(*args)
    _check(to_np(_run(*args)), val, err, y, ids)


# batches whose tiles take both products in one kernel: fewer 64-column steps
# than CTAs, a last step of 8 columns, ranks that end inside a 16-wide step, K
# that ends inside a block, as many tiles as it takes and one more
@pytest.mark.parametrize("M,N,K,rank,na", [
    (513, 8, 512, 8, 1), (520, 72, 528, 24, 3), (640, 1000, 1040, 8, 5), (1100, 200, 2688, 32, 2), (2100, 5128, 512, 16, 4),
    (4097, 128, 1552, 32, 9), (9536, 264, 528, 16, 2), (9537, 264, 528, 16, 2), (600, 520, 4096, 16, 60)])
@pytest.mark.parametrize("place", ["in place", None])
def test_middling_batches(M, N, K, rank, na, place):
    args = _inputs(M, N, K, rank, na, M + N)
    x, y, a, b, scale, ids = args
    val, err = _ref(*args)
    _check(to_np(_run(*args, out=place)), val, err, y, ids)


@pytest.mark.parametrize("N", [1000, 1001, 1002, 1004, 262, 260, 30])
@pytest.mark.parametrize("M,K,rank,na", [(700, 528, 24, 3), (700, 1040, 16, 5), (1300, 272, 56, 4), (600, 64, 8, 9)])
def test_widths(M, N, K, rank, na):
    """Rows of y and out that start on 16, 8, 4 and 2 bytes."""
    args = _inputs(M, N, K, rank, na, M + N + rank)
    x, y, a, b, scale, ids = args
    val, err = _ref(*args)
    _check(to_np(_run(*args)), val, err, y, ids)
    _check(to_np(_run(*args, out="in place")), val, err, y, ids)
    off = torch.empty(M * N + 1, dtype=torch.bfloat16, device="cuda")[1:].view(M, N)
    _check(to_np(_run(*args, out=off)), val, err, y, ids)


@pytest.mark.parametrize("M,N,K,rank,na", [(900, 136, 544, 24, 3), (600, 72, 512, 32, 12)])
def test_middling_batches_of_integers_are_exact(M, N, K, rank, na):
    """|t| <= 12 K <= 2^13 and the sums stay below 2^24: only the final rounding."""
    rng = np.random.default_rng(M + N)
    x, y = rng.integers(-4, 5, (M, K)).astype(float), rng.integers(-64, 65, (M, N)).astype(float)
    a, b = rng.integers(-3, 4, (na, rank, K)).astype(float), rng.integers(-8, 9, (na, N, rank)).astype(float)
    scale = 2.0 ** rng.integers(-2, 3, na)
    ids = rng.integers(-1, na, M).astype(np.int32)
    val, _ = _ref(x, y, a, b, scale, ids)
    assert np.array_equal(to_np(_run(x, y, a, b, scale, ids)), _bf16(val))


@pytest.mark.parametrize("M", [5, 400])
def test_in_place_and_without_scale(M):
    x, y, a, b, scale, ids = _inputs(M, 2688, 4096, 16, 6, 11 + M)
    val, err = _ref(x, y, a, b, np.ones_like(scale), ids)
    _check(to_np(_run(x, y, a, b, None, ids, out="in place")), val, err, y, ids)


@pytest.mark.parametrize("M,N,K,rank,na", [(9, 500, 96, 16, 3), (200, 515, 160, 48, 5), (700, 520, 64, 128, 3),
                                           (1500, 96, 48, 8, 70)])
def test_integer_operands_are_exact(M, N, K, rank, na):
    """|t| <= 48 K <= 2^13 and the sums stay below 2^24: only the final rounding."""
    rng = np.random.default_rng(M + N)
    x, y = rng.integers(-8, 9, (M, K)).astype(float), rng.integers(-64, 65, (M, N)).astype(float)
    a, b = rng.integers(-6, 7, (na, rank, K)).astype(float), rng.integers(-8, 9, (na, N, rank)).astype(float)
    scale = 2.0 ** rng.integers(-2, 3, na)
    ids = rng.integers(-1, na, M).astype(np.int32)
    val, _ = _ref(x, y, a, b, scale, ids)
    assert np.array_equal(to_np(_run(x, y, a, b, scale, ids)), _bf16(val))


@pytest.mark.parametrize("M", [4, 90, 600])
def test_rows_without_an_adapter_keep_their_bits(M):
    """Every row bare: y's bits, NaN payload-free infinities and -0 included,
    whatever x holds; and an all-one-adapter call next to it."""
    x, y, a, b, scale, _ = _inputs(M, 300, 64, 16, 2, M)
    x[:] = np.nan
    y[0, :4] = [np.inf, -np.inf, -0.0, 3.0e38]
    ids = np.full(M, -1, np.int32)
    yd = bf16_dev(y)
    got = m2.m2_lora_add(yd, bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.from_numpy(ids).cuda())
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), yd.view(torch.int16))


@pytest.mark.parametrize("M", [6, 100, 500])
def test_a_row_does_not_reach_another(M):
    """One row of NaN and one of infinity in x: only those rows of out are not finite."""
    args = list(_inputs(M, 264, 160, 16, 3, M + 1, ids=np.arange(M) % 3))
    args[0][1] = np.nan
    args[0][M - 1, 5] = np.inf
    got = to_np(_run(*args))
    bad = np.zeros(M, bool)
    bad[[1, M - 1]] = True
    assert np.all(np.isfinite(got[~bad])) and not np.any(np.isfinite(got[bad]))
    clean = [v.copy() for v in args]
    clean[0][bad] = 0.0
    val, err = _ref(*clean)
    keep = ~bad
    _check(got[keep], val[keep], err[keep], args[1][keep], args[5][keep])


@pytest.mark.parametrize("M", [8, 300, 700])
def test_an_unknown_adapter_is_reported_and_taken_as_none(M):
    x, y, a, b, scale, ids = _inputs(M, 128, 64, 8, 3, M + 2)
    ids[:] = np.arange(M) % 3
    ids[2], ids[5] = 3, -2
    got = m2.m2_lora_add(bf16_dev(y), bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.from_numpy(ids).cuda(),
                         scale=f32_dev(scale))
    torch.cuda.synchronize()
    with pytest.raises(m2.M2Error) as e:
        m2.check_standalone()
    assert e.value.status == m2.M2_EINVAL and "adapter" in str(e.value)
    m2.check_standalone()                       # read once, then cleared
    ids[[2, 5]] = -1
    val, err = _ref(x, y, a, b, scale, ids)
    _check(to_np(got), val, err, y, ids)


def test_unaligned_rows_of_y():
    """y and out at an odd element offset of their buffers, in place and with
    an out of another alignment."""
    for M in (5, 300):
        x, y, a, b, scale, ids = _inputs(M, 264, 64, 16, 3, M + 9)
        src, dst = (torch.zeros(M * 264 + 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        yd, od = src[3:3 + M * 264].view(M, 264), dst[1:1 + M * 264].view(M, 264)
        yd.copy_(bf16_dev(y))
        m2.m2_lora_add(yd, bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.from_numpy(ids).cuda(), scale=f32_dev(scale),
                       out=od)
        val, err = _ref(x, y, a, b, scale, ids)
        _check(to_np(od), val, err, y, ids)
        assert not dst[:1].any() and not dst[1 + M * 264:].any() and torch.equal(yd, bf16_dev(y))
    for M in (5, 300):
        x, y, a, b, scale, ids = _inputs(M, 264, 64, 16, 3, M)
        buf = torch.zeros(M * 264 + 1, dtype=torch.bfloat16, device="cuda")
        yd = buf[1:].view(M, 264)
        yd.copy_(bf16_dev(y))
        got = m2.m2_lora_add(yd, bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.from_numpy(ids).cuda(),
                             scale=f32_dev(scale), out=yd)
        val, err = _ref(x, y, a, b, scale, ids)
        _check(to_np(got), val, err, y, ids)
        assert float(buf[0]) == 0.0


def test_empty_call():
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((1, 64, 8), dtype=torch.bfloat16, device="cuda")
    assert m2.m2_lora_add(z, z, w, b, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 64)


@pytest.mark.parametrize("M", [64, 700])
def test_repeats_bit_for_bit_on_streams_and_in_a_graph(M):
    """Two calls on two streams at once, and a captured call replayed on new
    inputs, give the bits of a plain call."""
    x, y, a, b, scale, ids = _inputs(M, 2688, 512, 16, 5, M)
    d = [bf16_dev(y), bf16_dev(x), bf16_dev(a), bf16_dev(b), torch.from_numpy(ids).cuda()]
    sc = f32_dev(scale)
    want = m2.m2_lora_add(*d, scale=sc)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [m2.m2_lora_add(*d, scale=sc, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m2.m2_lora_add(*d, scale=sc, out=out)
    d[1].neg_()
    d[4].copy_(torch.roll(d[4], 1))
    want2 = m2.m2_lora_add(*d, scale=sc)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2) and not torch.equal(out, want)
    m2.check_standalone()


@pytest.mark.parametrize("M,N,K,rank,na", [
    (64, 264, 160, 16, 5), (9, 515, 96, 40, 3), (300, 200, 64, 128, 2), (130, 96, 2688, 24, 40),   # few rows
    (640, 1000, 1040, 8, 5), (700, 1004, 528, 24, 3), (1100, 202, 1040, 32, 2),                     # both products in one
    (700, 1000, 272, 56, 4), (700, 1001, 528, 24, 3), (400, 264, 64, 128, 2), (1300, 261, 96, 72, 3)])
@pytest.mark.parametrize("whole", [False, True])
def test_infinite_weights(M, N, K, rank, na, whole):
    """Infinities and a NaN in b: the columns they reach are the formula's
    infinities or NaN, every other one is as without them.  whole: integers,
    an intermediate that bf16 holds exactly."""
    x, y, a, b, scale, ids = _inputs(M, N, K, rank, na, M + 3 * N)
    if whole:
        rng = np.random.default_rng(M + N)
        x[:], a[:] = 0.0, 0.0
        x[:, :2], a[:, :, :2] = rng.integers(1, 8, (M, 2)), rng.integers(-7, 8, (na, rank, 2)) * 2.0 + 1.0
        scale[:] = 0.5
    b[0, 3, 1] = np.inf
    b[0, N - 1, rank - 1] = -np.inf
    b[1, 5, :2] = np.inf                        # two: an infinity or, of both signs, NaN
    b[1, N // 2, 0] = np.nan
    b[1, 7] = np.inf
    with np.errstate(invalid="ignore"):
        val, err = _ref(x, y, a, b, scale, ids)
    got = to_np(_run(x, y, a, b, scale, ids)).astype(np.float64)
    odd = ~np.isfinite(val)
    assert odd.any() and np.array_equal(got[odd], val[odd], equal_nan=True)
    b[~np.isfinite(b)] = 0.0
    val, err = _ref(x, y, a, b, scale, ids)
    over = np.abs(got - val) > err + (np.abs(val) + err) * 2.0 ** -8
    assert not (over & ~odd).any()
