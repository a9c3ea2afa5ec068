"""m2_token_logprobs on long rows whose logits are nearly all equal: every
addition to a sum within a binade then errs by the same amount in the same
direction, so that errors add up instead of averaging out.

Rows are a constant a, or that with one token at a + d; then log S, the
entropy, ranks and alternatives have closed forms.  Bound of log S in units of
2^-24, every error of one sign:
 - an exponential is within 2^-22 (4); its argument is rounded once, |u| <= 16
   where a thread's reference lies below its largest logit (6);
 - n terms one after another err by (n + 1) / 2 of a sum that grows evenly: a
   chunk's 8 and 32 chunks' sums, its 16 and 17 sums, or 32 terms (21 at most);
 - the halves of a pair and what was put by are added (2);
 - lanes, warps and slices are joined in at most 5 + 3 + 3 levels (11);
 - what a reference in base 2 leaves out of a spread of d <= 17 (4), the
   logarithm and its parts (2).
50 together.  Logits beyond +-2^16 are summed as x - m, which is exact (they are
multiples of 2^-8 at least, and close): an exponential within an ulp (2), 8 terms
of a vector (5), lanes and warps (5 + 8): less.  The entropy is log S less the
mean of x - m: with a share w of the weight d away from the rest, d w (1 - w) <=
17 / 4 times the bound more: 250 units, 300 here.  Results are rounded to f32
once."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

UNIT = 2.0 ** -24
LSE, ENT = 50 * UNIT, 300 * UNIT
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check_rows(base, d, v, dtype, where):
    """Rows of v tokens at base[r], the one at where[r] at base[r] + d[r] (d >= 0;
    0: all equal); scored: that token in even rows, the last one in odd rows."""
    rows = len(base)
    high = base + d
    logits = torch.empty(rows, v, dtype=dtype, device="cuda")
    logits.copy_(torch.from_numpy(base).to(dtype).cuda()[:, None].expand(rows, v))
    at = torch.from_numpy(where).cuda()
    logits[torch.arange(rows, device="cuda"), at] = torch.from_numpy(high).to(dtype).cuda()
    assert np.array_equal(logits[:, -1].double().cpu().numpy(), base)   # (the values are the type's)
    assert np.array_equal(logits[torch.arange(rows, device="cuda"), at].double().cpu().numpy(), high)
    tokens = np.where(np.arange(rows) % 2 == 0, where, v - 1).astype(np.int32)
    o = m2.m2_token_logprobs(logits, torch.from_numpy(tokens).cuda(), 3)
    z = np.log1p((v - 1) * np.exp(-d))                                  # log S relative to the largest
    w = (v - 1) / ((v - 1) + np.exp(d))                                 # the others' weight
    lone = d > 0
    is_high = tokens == where
    lp = np.where(is_high, -z, -d - z)
    rank = np.where(lone, np.where(is_high, 1, tokens + 1 + (tokens < where)), tokens + 1)
    first = np.array([[q, *[t for t in (0, 1, 2) if t != q][:2]] if l else [0, 1, 2] for q, l in zip(where, lone)])
    top = np.stack([-z, -d - z, -d - z], 1)

    def err(got, want):
        e = np.abs(got.double().cpu().numpy() - want) - UNIT * (1 + 2 ** -20) * np.abs(want)
        return float(e.max()) / UNIT

    worst = dict(logprobs=err(o.logprobs, lp), top=err(o.top_logprobs, top), entropy=err(o.entropy, z + w * d))
    assert np.array_equal(o.ranks.cpu().numpy(), rank)
    assert np.array_equal(o.top_tokens.cpu().numpy(), first)
    assert worst["logprobs"] <= LSE / UNIT and worst["top"] <= LSE / UNIT and worst["entropy"] <= ENT / UNIT, worst


# (more rows than a cluster's slices serve at once, rows in slices, the longest)
SUMS = [(160, 131071, F32), (160, 400003, F32), (160, 1 << 20, F32), (160, 1 << 20, BF), (2, (1 << 23) + 5, F32),
        (1, 1 << 24, BF), (2, 1 << 24, F32)]


@pytest.mark.parametrize("rows,v,dtype", SUMS)
def test_equal_logits(rows, v, dtype):
    r = np.arange(rows, dtype=np.float64)
    base = (r + 1) * 0.125 - 9.9375 if dtype == F32 else (r % 31 + 1) * 0.0625
    check_rows(base, np.zeros(rows), v, dtype, (r * 7919 % v).astype(np.int64))


@pytest.mark.parametrize("rows,v,dtype", SUMS)
def test_one_likely_token_among_equal_ones(rows, v, dtype):
    r = np.arange(rows, dtype=np.float64)
    base = (r + 1) * 0.125 - 9.9375 if dtype == F32 else (r % 31 + 1) * 0.0625
    d = (r % 17) + 0.5 if dtype == F32 else np.where(r % 2, 1.0, 2.0) - base + np.where(r % 3, 2.0, 12.0)
    check_rows(base, d, v, dtype, (r * 7919 % v).astype(np.int64))


@pytest.mark.parametrize("around", [70000.0, -70000.0, 1000000.0])
@pytest.mark.parametrize("rows,v", [(3, 131071), (3, 60000), (200, 131072), (160, 1 << 20), (2, 1 << 23), (1, 1 << 24)])
def test_large_logits(rows, v, around):
    r = np.arange(rows, dtype=np.float64)
    d = (r * 5 % 150 + 2) / 16
    check_rows(around + r - d, d, v, F32, (r * 7919 % v).astype(np.int64))


def patterns(v, dtype):
    """Rows of v tokens: random, masked in front, behind and nearly everywhere (by
    -inf, NaN, finite values), in order, of +inf, of nothing."""
    g = torch.Generator(device="cuda").manual_seed(v)
    lowest = torch.finfo(dtype).min

    def random():
        return torch.randn(v, generator=g, device="cuda") * 2.5

    rows = [random() for _ in range(10)]
    rows[1][:v * 9 // 10] = float("-inf")
    rows[2][v // 10:] = float("nan")
    rows[3] = torch.linspace(-60000, 60000, v, device="cuda")
    rows[4] = torch.linspace(60000, -60000, v, device="cuda")
    few = torch.tensor([v // 7, v // 2, v - 2], device="cuda")
    rows[5][:] = float("-inf")
    rows[5][few] = torch.tensor([1.0, 3.0, 2.0], device="cuda")
    rows[6][:] = lowest
    rows[6][few] = torch.tensor([-1.0, 0.5, 0.25], device="cuda")
    rows[7][:] = float("-inf")
    rows[8][few] = float("inf")
    rows[9][:] = lowest
    return torch.stack(rows).to(dtype)


# (slices of 2^17 tokens and more; whole rows)
@pytest.mark.parametrize("rows,v,dtype", [(10, 4000003, F32), (10, 4000003, BF), (160, 600001, F32), (160, 600001, BF)])
def test_masks_and_order_in_long_rows(rows, v, dtype):
    """Against 64 bits, where terms differ and any of n additions may err by half a
    step of the whole sum: 40 units for 21 in the bound above, 70 together; the
    entropy's mean is of |x - m| up to 17 under the weights, half of it apart."""
    from test_gpu_token_logprobs import close, reference
    some = patterns(v, dtype)
    logits = some.repeat(rows // 10, 1)
    tokens = torch.tensor([v // 2, v - 2, 5, v - 1, 0, v // 7, v - 2, 3, v // 2, v // 3], dtype=torch.int32, device="cuda")
    o = m2.m2_token_logprobs(logits, tokens.repeat(rows // 10), 20)
    torch.cuda.synchronize()
    m2.check_standalone()
    lp, rk, h, tt, tl = reference(some.float().cpu().numpy().astype(np.float64), tokens.cpu().numpy(), 20)
    for at in (slice(0, 10), slice(rows - 10, rows)):
        close(o.logprobs[at], lp, 70 * UNIT)
        close(o.entropy[at], h, 70 * 9.5 * UNIT)
        close(o.top_logprobs[at], tl, 70 * UNIT)
        assert np.array_equal(o.ranks[at].cpu().numpy(), rk)
        assert np.array_equal(o.top_tokens[at].cpu().numpy(), tt)
