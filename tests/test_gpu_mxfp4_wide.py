"""The products' kernels where a CTA or a pair of them goes through several
tiles, each of several stages of K, against sums in 64 bits: units of 256 + 192
columns (the widths that large products take), and the persistent walk over the
weights of up to 64 rows.  The bound is that of test_gpu_mxfp4.py: operands are
exact, an MMA of 64 values of K adds with an error of at most 2^-22 of the sum of
magnitudes, and the result is rounded once."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def operand(rng, rows, K, spread=4):
    """A random Mxfp4 and its values, scales within 2^-spread .. 2^spread."""
    code = rng.integers(0, 16, (rows, K), dtype=np.uint8)
    scale = rng.integers(127 - spread, 128 + spread, (rows, K // 32)).astype(np.uint8)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
    v = grid[code] * np.repeat(np.exp2(scale.astype(np.float64) - 127), 32, axis=1)
    q = m2.mxfp4_pack(torch.from_numpy(code[:, 0::2] | code[:, 1::2] << 4).cuda(), torch.from_numpy(scale).cuda())
    return q, v


def check(y, want, size, K):
    """y against the exact sums `want` of products whose magnitudes sum up to `size`."""
    got = y.double().cpu().numpy()
    step = 2.0 ** -8 if y.dtype == BF else 2.0 ** -24
    bound = step * (1 + 2.0 ** -7) * np.abs(want) + (-(-K // 64) + 8) * 2.0 ** -22 * size + 2.0 ** -140
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


def waves(M, N, span):
    """Turns that the device's CTA pairs take over 256-row tiles of span columns."""
    tiles = -(-M // 256) * -(-N // span)
    return -(-tiles // (torch.cuda.get_device_properties(0).multi_processor_count // 2))


def takes_wide_units(M, N):
    """Whether units of 256 + 192 columns have the shortest turns (a stage brings
    68, 31, 26 and 22 KB into an SM)."""
    wide, *others = (waves(M, N, s) * kb for s, kb in ((448, 68), (192, 31), (128, 26), (64, 22)))
    return wide < min(others)


# (one unit a pair and up to a dozen; columns that end with a unit, inside its
# second tile, inside its first, with its first; rows on no 16-byte boundary; K
# that ends after 32, 64, 128, 160 and all of a stage's 256 values)
@pytest.mark.parametrize("M,N,K", [(700, 10304, 2688), (5669, 2688, 4000), (5669, 2687, 1312), (1000, 33000, 1056),
                                   (600, 40001, 288), (4096, 10304, 2560), (517, 131072, 320)])
def test_units_of_two_widths(M, N, K):
    assert takes_wide_units(M, N)
    rng = np.random.default_rng(M + N + K)
    (qa, a), (qw, w) = operand(rng, M, K), operand(rng, N, K)
    want, size = a @ w.T, np.abs(a) @ np.abs(w).T
    for dtype in (BF, F32):
        y = torch.full((M * N + 8,), float("nan"), dtype=dtype, device="cuda")
        m2.mxfp4_linear(qa, qw, y=y[:M * N].view(M, N))
        m2.check_standalone()
        check(y[:M * N].view(M, N), want, size, K)
        assert torch.isnan(y[M * N:]).all()
    # quantised inside: a's values are MXFP4 already, the sums are these
    check(m2.mxfp4_linear_bf16(m2.mxfp4_dequant(qa), qw, dtype=F32), want, size, K)


@pytest.mark.parametrize("M,N,K", [(700, 10304, 2688), (5669, 2687, 2688)])
def test_units_of_two_widths_sum_exactly(M, N, K):
    """Equal scales and 36 K / 4 within f32's 24 bits: nothing is rounded."""
    assert takes_wide_units(M, N)
    rng = np.random.default_rng(K)
    (qa, a), (qw, w) = operand(rng, M, K, 0), operand(rng, N, K, 0)
    y = m2.mxfp4_linear(qa, qw, dtype=F32)
    assert np.array_equal(y.double().cpu().numpy(), a @ w.T)


@pytest.mark.parametrize("M", [3, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(40000, 2688), (40001, 1312)])
def test_few_rows_walk_over_many_weights(M, N, K):
    rng = np.random.default_rng(M + N)
    (qa, a), (qw, w) = operand(rng, M, K), operand(rng, N, K)
    want, size = a @ w.T, np.abs(a) @ np.abs(w).T
    for dtype in (BF, F32):
        check(m2.mxfp4_linear(qa, qw, dtype=dtype), want, size, K)
        m2.check_standalone()


@pytest.mark.parametrize("N", [131072, 131071])
def test_sums_at_offsets_past_32_bits(N):
    """The first and the last rows of an output of more than 2^31 elements."""
    M, K = 16500, 544
    rng = np.random.default_rng(N)
    (qa, a), (qw, w) = operand(rng, M, K), operand(rng, N, K)
    y = m2.mxfp4_linear(qa, qw)
    for rows in (slice(0, 3), slice(16300, 16303), slice(M - 61, M)):
        check(y[rows], a[rows] @ w.T, np.abs(a[rows]) @ np.abs(w).T, K)
