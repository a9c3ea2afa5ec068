"""MXFP4: mxfp4_quant, mxfp4_dequant and mxfp4_pack bit for bit against the
format's definition in 64 bits, and the products against exact sums.

Bound of a product: the operands are exact, an MMA of 64 values of K adds to
the f32 accumulator with an error of at most 2^-22 of the sum of magnitudes so
far (alignment and truncation below the largest term), there are ceil(K / 64)
of them and at most 8 partial sums are added, and the result is rounded once:
|y - exact| <= half a step + (ceil(K / 64) + 8) 2^-22 sum |a w|."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def np64(t):
    return t.float().cpu().numpy().astype(np.float64)


def quantise(x):
    """(codes [rows, K], scale codes [rows, K / 32]) of float64 values."""
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(2)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 2, -127)
    e = np.maximum(e, -127)
    a = np.abs(b) / np.exp2(e)[..., None]
    d = np.abs(a[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    even = np.arange(8) % 2 == 0
    code = np.where(near.sum(-1) > 1, np.argmax(near & even, -1), np.argmax(near, -1))
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.int64)


def values(code, scale):
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(code.shape[0], -1, 32) * s[..., None]).reshape(code.shape)


def unpack(q):
    """(codes [rows, K], row-major scale codes, the tiles' other bytes) of an Mxfp4."""
    c = q.codes.cpu().numpy().astype(np.int64)
    rows, K = q.shape
    code = np.stack([c & 15, c >> 4], 2).reshape(rows, K)
    t = q.scales.cpu().numpy().astype(np.int64)
    # [row block, K block, r % 32, r / 32, b] -> rows x blocks
    t = t.reshape(t.shape[0], t.shape[1], 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, t.shape[1] * 4)
    rest = np.concatenate([t[rows:].ravel(), t[:rows, K // 32:].ravel()])
    return code, t[:rows, :K // 32], rest


def check_quant(x, q):
    code, scale, rest = unpack(q)
    want, want_scale = quantise(np64(x))
    assert np.array_equal(scale, want_scale)
    assert np.array_equal(code, want)
    assert not rest.any()


@pytest.mark.parametrize("rows,K", [(1, 32), (1, 2688), (2, 64), (3, 96), (127, 160), (128, 128), (129, 4096), (300, 1056),
                                    (1000, 2688), (5, 8192)])
def test_quant_is_the_definition(rows, K):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + K)
    x = (torch.randn(rows, K, generator=g, device="cuda") *
         torch.exp(2 * torch.randn(rows, K, generator=g, device="cuda"))).to(BF)
    q = m2.mxfp4_quant(x)
    check_quant(x, q)
    assert torch.equal(m2.mxfp4_dequant(q), torch.from_numpy(values(*unpack(q)[:2])).to(BF).cuda())


def test_quant_at_the_edges_of_the_types():
    """Zeros of both signs, subnormals, ties, the largest values, and blocks
    with infinities and NaN, which become NaN and leave their neighbours."""
    x = torch.zeros(10, 128, dtype=BF)
    x[0, 1] = -0.0
    x[1, :32] = torch.tensor([2.0 ** -133 * i for i in range(32)])             # subnormals alone
    x[1, 32:64] = torch.tensor([2.0 ** -126 * i / 16 for i in range(32)])
    x[2, :32] = torch.tensor([6.0 * i / 31 for i in range(32)])
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 6.5, 7.5, 0.2490234375])
    x[3, :12], x[3, 32:44], x[3, 64:76] = ties, -ties, ties * 2.0 ** 100
    x[4, :32] = torch.finfo(BF).max
    x[4, 32:64] = torch.finfo(BF).min
    x[5, 3], x[5, 40], x[5, 100] = float("inf"), float("-inf"), float("nan")
    x[5, 70] = 3.0
    x[6, :] = float("nan")
    x[7, 127], x[7, 0] = 1.0, 2.0 ** -30
    x[8, 5] = 2.0 ** -125
    x[9, 64:96] = torch.tensor([(-1.0) ** i * 2.0 ** (i - 140) for i in range(32)])
    x = x.cuda()
    q = m2.mxfp4_quant(x)
    check_quant(x, q)
    v = m2.mxfp4_dequant(q)
    nan = torch.isnan(v)
    assert nan[5].tolist() == [True] * 64 + [False] * 32 + [True] * 32 and nan[6].all() and nan.sum() == 96 + 128
    assert v[5, 70] == 3.0


def test_quant_of_slices_and_into_buffers():
    """Rows that are a slice of wider ones, an odd number of them; outputs
    given; what is behind them stays."""
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(77, 10304, generator=g, device="cuda").to(BF)
    for c0, K in ((0, 4096), (4096, 6144), (8, 32), (10240, 64)):
        x = wide[:, c0:c0 + K]
        whole = torch.full((77 * K // 2 + 64,), 171, dtype=torch.uint8, device="cuda")
        scales = torch.full((((K + 127) // 128) * 512 + 64,), 171, dtype=torch.uint8, device="cuda")
        out = m2.Mxfp4(whole[:77 * K // 2].view(77, K // 2), scales[:-64].view(1, -1, 512))
        q = m2.mxfp4_quant(x, out=out)
        assert q is out
        check_quant(x, q)
        assert (whole[77 * K // 2:] == 171).all() and (scales[-64:] == 171).all()
    with pytest.raises(ValueError):
        m2.mxfp4_quant(wide[:, :4100])
    with pytest.raises(ValueError):
        m2.mxfp4_quant(wide.t()[:64])
    with pytest.raises(ValueError):
        m2.mxfp4_quant(torch.zeros(4, 68, dtype=BF, device="cuda")[:, :64])     # rows on no 16-byte boundary
    with pytest.raises(ValueError):
        m2.mxfp4_quant(wide[:, :64].float())
    with pytest.raises(m2.M2Error):
        m2.mxfp4_quant(wide[:, 4:36])                                          # starts on no 16-byte boundary


def test_dequant_and_pack_of_every_code():
    """All 16 codes under all 256 scale codes; bf16 of the exact value."""
    code = np.tile(np.arange(16), 2)[None].repeat(256, 0).reshape(2, 128 * 32)
    scale = np.arange(256).reshape(2, 128)
    packed = (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)
    q = m2.mxfp4_pack(torch.from_numpy(packed).cuda(), torch.from_numpy(scale.astype(np.uint8)).cuda())
    assert np.array_equal(unpack(q)[1], scale) and not unpack(q)[2].any()
    want = torch.from_numpy(values(code, scale)).to(F32).to(BF)
    got = m2.mxfp4_dequant(q).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (129, 160), (300, 2688)])
def test_pack(rows, K):
    rng = np.random.default_rng(K)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)).cuda()
    scale = rng.integers(0, 256, (rows, K // 32)).astype(np.uint8)
    wide = torch.zeros(rows * (K // 32) + 1, dtype=torch.uint8, device="cuda")
    s = wide[1:].view(rows, K // 32)                                          # any alignment
    s.copy_(torch.from_numpy(scale))
    q = m2.mxfp4_pack(codes, s)
    assert q.codes is codes and np.array_equal(unpack(q)[1], scale) and not unpack(q)[2].any()


def operand(rng, rows, K, spread=4):
    code = rng.integers(0, 16, (rows, K))
    scale = rng.integers(127 - spread, 128 + spread, (rows, K // 32))
    packed = (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)
    q = m2.mxfp4_pack(torch.from_numpy(packed).cuda(), torch.from_numpy(scale.astype(np.uint8)).cuda())
    return q, values(code, scale)


def check_product(y, a, w):
    K = a.shape[1]
    want = a @ w.T
    got = y.double().cpu().numpy()
    half = (2.0 ** -8 if y.dtype == BF else 2.0 ** -24) * np.abs(want)
    bound = half * (1 + 2.0 ** -7) + (-(-K // 64) + 8) * 2.0 ** -22 * (np.abs(a) @ np.abs(w).T) + 2.0 ** -140
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 517])
@pytest.mark.parametrize("N,K", [(1, 32), (64, 64), (127, 96), (129, 128), (200, 160), (1000, 288), (333, 1056)])
def test_product(M, N, K):
    rng = np.random.default_rng(M * 1000 + N + K)
    (qa, a), (qw, w) = operand(rng, M, K), operand(rng, N, K)
    for dtype in (BF, F32):
        y = m2.mxfp4_linear(qa, qw, dtype=dtype)
        torch.cuda.synchronize()
        m2.check_standalone()
        check_product(y, a, w)


@pytest.mark.parametrize("M,N,K", [(1, 10304, 2688), (64, 2688, 4096), (96, 10304, 2688), (3, 50021, 512), (700, 2688, 4096),
                                   (300, 5003, 2688), (2500, 1999, 160), (40, 8, 8192), (130, 1, 8192)])
def test_product_of_larger_sizes(M, N, K):
    rng = np.random.default_rng(M + N + K)
    (qa, a), (qw, w) = operand(rng, M, K), operand(rng, N, K)
    y = torch.full((M * N + 8,), float("nan"), dtype=F32, device="cuda")
    m2.mxfp4_linear(qa, qw, y=y[:M * N].view(M, N))
    check_product(y[:M * N].view(M, N), a, w)
    assert torch.isnan(y[M * N:]).all()
    check_product(m2.mxfp4_linear(qa, qw), a, w)


@pytest.mark.parametrize("M,N", [(5, 40), (70, 300), (200, 193), (300, 520)])
def test_sums_of_small_whole_numbers_are_exact(M, N):
    """Equal scales and 36 K / 4 within f32's 24 bits: nothing is rounded."""
    rng = np.random.default_rng(N)
    (qa, a), (qw, w) = operand(rng, M, 2688, 0), operand(rng, N, 2688, 0)
    y = m2.mxfp4_linear(qa, qw, dtype=F32)
    assert np.array_equal(y.double().cpu().numpy(), a @ w.T)


@pytest.mark.parametrize("M", [20, 300])
def test_nan_blocks_stay_in_their_row_and_column(M):
    rng = np.random.default_rng(M)
    (qa, a), (qw, w) = operand(rng, M, 416), operand(rng, 140, 416)
    clean = m2.mxfp4_linear(qa, qw, dtype=F32)
    x = m2.mxfp4_dequant(qa)
    x[7, 33] = float("nan")
    x[11, 415] = float("inf")
    qa2 = m2.mxfp4_quant(x)
    wv = m2.mxfp4_dequant(qw)
    wv[139, 0] = float("nan")
    qw2 = m2.mxfp4_quant(wv)
    y = m2.mxfp4_linear(qa2, qw2, dtype=F32)
    bad = torch.zeros(M, 140, dtype=torch.bool, device="cuda")
    bad[7] = bad[11] = True
    bad[:, 139] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], m2.mxfp4_linear(m2.mxfp4_quant(m2.mxfp4_dequant(qa)),
                                                m2.mxfp4_quant(m2.mxfp4_dequant(qw)), dtype=F32)[~bad])
    check_product(clean, a, w)


@pytest.mark.parametrize("M", [3, 260])
def test_scales_far_apart(M):
    """Scales from 2^-60 to 2^60: each product's bound is that of its own sum."""
    rng = np.random.default_rng(M)
    (qa, a), (qw, w) = operand(rng, M, 288, 30), operand(rng, 130, 288, 30)
    check_product(m2.mxfp4_linear(qa, qw, dtype=F32), a, w)


@pytest.mark.parametrize("M,N,K", [(1, 300, 2688), (2, 10304, 2688), (16, 129, 160), (7, 2000, 5000 // 32 * 32), (17, 777, 1056),
                                   (33, 2688, 32), (64, 2688, 4096), (50, 1000, 288), (64, 10304, 2688), (130, 333, 160),
                                   (500, 1000, 96)])
def test_quantise_inside(M, N, K):
    """The values of mxfp4_quant, products within the bound, and where it takes
    a workspace (the same kernels on the same operands) the same bits."""
    g = torch.Generator(device="cuda").manual_seed(M)
    wide = torch.randn(M, K + 40, generator=g, device="cuda").to(BF)
    qw, w = operand(np.random.default_rng(K), N, K)
    x = wide[:, 8:8 + K]
    x[M // 2, 5] = 0.0
    q = m2.mxfp4_quant(x)
    a = values(*unpack(q)[:2])
    need = m2.mxfp4_linear_bf16_workspace_size(M, N, K)
    for dtype in (BF, F32):
        got = m2.mxfp4_linear_bf16(x, qw, dtype=dtype)
        torch.cuda.synchronize()
        m2.check_standalone()
        check_product(got, a, w)
        if need:
            assert torch.equal(got, m2.mxfp4_linear(q, qw, dtype=dtype))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        buf = torch.full((M * N + 8,), float("nan"), dtype=dtype, device="cuda")
        y = buf[:M * N].view(M, N)
        assert m2.mxfp4_linear_bf16(x, qw, y=y, workspace=ws) is y and torch.equal(y, got)
        assert torch.isnan(buf[M * N:]).all()


@pytest.mark.parametrize("M", [3, 20, 60])
def test_quantise_inside_of_small_whole_numbers_is_exact(M):
    """Sums within f32's 24 bits: the quantised values and places have to be
    right to the bit, blocks that become NaN too."""
    rng = np.random.default_rng(M)
    (qa, a), (qw, w) = operand(rng, M, 800, 0), operand(rng, 640, 800, 0)
    x = m2.mxfp4_dequant(qa)
    x[:, 3::32] = 6.0                                          # every block's scale stays 1
    y = m2.mxfp4_linear_bf16(x, qw, dtype=F32)
    assert np.array_equal(y.double().cpu().numpy(), np64(x) @ w.T)
    x[1, 70], x[2, 799] = float("nan"), float("inf")
    z = m2.mxfp4_linear_bf16(x, qw, dtype=F32)
    bad = torch.zeros(M, 640, dtype=torch.bool, device="cuda")
    bad[1] = bad[2] = True
    assert torch.equal(torch.isnan(z), bad) and torch.equal(z[~bad], y[~bad])


@pytest.mark.parametrize("M", [12, 300])
def test_outputs_on_any_element_boundary(M):
    rng = np.random.default_rng(1)
    (qa, a), (qw, w) = operand(rng, M, 64), operand(rng, 72, 64)
    for dtype in (BF, F32):
        buf = torch.full((M * 72 + 2,), float("nan"), dtype=dtype, device="cuda")
        y = buf[1:-1].view(M, 72)
        m2.mxfp4_linear(qa, qw, y=y)
        assert torch.equal(y, m2.mxfp4_linear(qa, qw, dtype=dtype))
        assert torch.isnan(buf[0]) and torch.isnan(buf[-1])


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(0)
    (qa, _), (qw, _) = operand(rng, 48, 2688), operand(rng, 2688, 2688)
    first = m2.mxfp4_linear(qa, qw, dtype=F32)
    for _ in range(5):
        assert torch.equal(m2.mxfp4_linear(qa, qw, dtype=F32), first)


def test_no_rows():
    qw, _ = operand(np.random.default_rng(0), 10, 64)
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    q = m2.mxfp4_quant(x)
    assert q.shape == (0, 64) and m2.mxfp4_dequant(q).shape == (0, 64)
    assert m2.mxfp4_linear(q, qw).shape == (0, 10) and m2.mxfp4_linear_bf16(x, qw).shape == (0, 10)


@pytest.mark.parametrize("M", [9, 400])
def test_captured_graphs_and_another_stream(M):
    """Two graphs with workspaces of their own, replayed in turn with new
    inputs, and eager calls on another stream."""
    g = torch.Generator(device="cuda").manual_seed(M)
    qw, _ = operand(np.random.default_rng(2), 500, 352)
    xs = [torch.randn(M, 352, generator=g, device="cuda").to(BF) for _ in range(4)]
    want = [m2.mxfp4_linear_bf16(x, qw) for x in xs]
    bufs = [torch.empty_like(xs[0]) for _ in range(2)]
    ys = [torch.empty((M, 500), dtype=BF, device="cuda") for _ in range(2)]
    wss = [torch.empty(m2.mxfp4_linear_bf16_workspace_size(M, 500, 352), dtype=torch.uint8, device="cuda")
           for _ in range(2)]
    graphs = []
    for b, y, ws in zip(bufs, ys, wss):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m2.mxfp4_linear_bf16(b, qw, y=y, workspace=ws)
        graphs.append(graph)
    for i, x in enumerate(xs):
        bufs[i % 2].copy_(x)
        graphs[i % 2].replay()
        assert torch.equal(ys[i % 2], want[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [m2.mxfp4_linear_bf16(x, qw, stream=side) for x in xs]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_python_refuses_what_does_not_fit():
    qw, _ = operand(np.random.default_rng(0), 10, 64)
    qa, _ = operand(np.random.default_rng(0), 3, 96)
    with pytest.raises(ValueError):
        m2.mxfp4_linear(qa, qw)                                                # another K
    with pytest.raises(ValueError):
        m2.mxfp4_linear(m2.Mxfp4(qa.codes, qw.scales.view(-1)), qw)
    with pytest.raises(ValueError):
        m2.mxfp4_linear(qw, qw, dtype=torch.float16)
    with pytest.raises(ValueError):
        m2.mxfp4_linear(qw, qw, y=torch.empty(10, 11, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        m2.mxfp4_pack(qw.codes, qw.scales)
    with pytest.raises(m2.M2Error) as e:
        m2.mxfp4_linear_bf16(torch.zeros(100, 64, dtype=BF, device="cuda"), qw,
                             workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == m2.M2_ENOMEM


def test_one_matrix_on_both_sides():
    q, v = operand(np.random.default_rng(3), 130, 160)
    exact = v @ v.T
    y = np64(m2.mxfp4_linear(q, q, dtype=F32))
    assert (np.abs(y - exact) <= 2.0 ** -24 * np.abs(exact) + (3 + 8) * 2.0 ** -22 * (np.abs(v) @ np.abs(v).T)).all()


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 values and outputs of more than 2^31: the rows
    at the end are those of a small call."""
    rows, K = (1 << 32) // 2688 + 200, 2688
    x = torch.zeros(rows, K, dtype=BF, device="cuda")
    x[-200:] = torch.randn(200, K, device="cuda").to(BF)
    q = m2.mxfp4_quant(x)
    small = m2.mxfp4_quant(x[-200:])
    assert torch.equal(q.codes[-200:], small.codes) and not q.codes[:-200].any()
    back = m2.mxfp4_dequant(q)
    assert torch.equal(back[-200:], m2.mxfp4_dequant(small)) and not back[:-200].any()
    # (a row block on its own: its tiles of scales start on a multiple of 128)
    r0 = rows // 128 * 128 - 128
    end = m2.Mxfp4(q.codes[r0:], q.scales[r0 // 128:])
    qw, _ = operand(np.random.default_rng(0), 96, K)
    assert torch.equal(m2.mxfp4_linear(q, qw)[r0:], m2.mxfp4_linear(end, qw))
    far = x.view(-1).as_strided((3, 64), ((rows // 3) * K // 8 * 8, 1))
    assert torch.equal(m2.mxfp4_quant(far).codes, m2.mxfp4_quant(far.contiguous()).codes)


@pytest.mark.parametrize("N", [131072, 131071])
def test_outputs_past_32_bits(N):
    M, K = 16500, 32
    (qa, _), (qw, _) = operand(np.random.default_rng(1), M, K), operand(np.random.default_rng(2), N, K)
    y = m2.mxfp4_linear(qa, qw)
    r0 = M // 256 * 256
    end = m2.Mxfp4(qa.codes[r0:], qa.scales[r0 // 128:])
    assert torch.equal(y[r0:], m2.mxfp4_linear(end, qw))
    assert torch.equal(y[:100], m2.mxfp4_linear(m2.Mxfp4(qa.codes[:100], qa.scales[:1]), qw))


def test_two_streams_at_once():
    """Products of all kinds on two streams at the same time give what they give
    one after another."""
    rng = np.random.default_rng(4)
    qw, _ = operand(rng, 4000, 1056)
    xs = [torch.randn(M, 1056, device="cuda").to(BF) for M in (1, 20, 64, 70, 600)]
    want = [m2.mxfp4_linear_bf16(x, qw) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for i in range(12):
        for s, side in enumerate(streams):
            got[s].append((m2.mxfp4_linear_bf16(xs[(i + 2 * s) % 5], qw, stream=side), (i + 2 * s) % 5))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for g in got for y, k in g)
    m2.check_standalone()
