"""The head on a stack: prompts scored by Mamba2Stack.score, and decode rows
through the 4-bit head into a beam step.  The stages are checked where they
meet: the 4-bit form of the final norm's bf16 rows, exact products of it, and
the log probabilities of the device's own logits."""
import numpy as np
import pytest
import torch

import synth
from helpers import device_weights

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

VOCAB = 5003
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def stack():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    blocks = [m2.Mamba2Mixer(device_weights(synth.make_weights(s))) for s in (0, 1)]
    ws = [torch.ones(2688, dtype=BF, device="cuda") for _ in blocks]
    yield m2.Mamba2Stack(blocks, ws)
    for b in blocks:
        b.close()


@pytest.fixture(scope="module")
def head():
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(VOCAB, 2688, generator=g, device="cuda").mul_(2688 ** -0.5 * 2).to(BF)
    norm_w = (1 + 0.1 * torch.randn(2688, generator=g, device="cuda")).to(BF)
    return m2.Mxfp4Head(norm_w, m2.mxfp4_quant(w)), norm_w


def _states(n):
    return ([torch.zeros((n, 6144, 3), dtype=BF, device="cuda") for _ in range(2)],
            [torch.zeros((n, 64, 64, 128), device="cuda") for _ in range(2)])


def _exact_logits(h, head, norm_w):
    a = m2.mxfp4_dequant(m2.mxfp4_quant(m2.m2_rmsnorm_residual(h, None, norm_w, 1e-5))).double()
    w = m2.mxfp4_dequant(head.weight).double()
    return a @ w.T, a.abs() @ w.abs().T


@pytest.mark.parametrize("seqlens", [[1], [5, 1, 33], [100, 61, 7]])
def test_score_of_prompts(stack, head, seqlens):
    head, norm_w = head
    T = sum(seqlens)
    hidden = torch.from_numpy(synth.make_hidden(3, T)).to(BF).cuda()
    tokens = np.random.default_rng(T).integers(0, VOCAB, T).astype(np.int32)
    tokens[np.cumsum(seqlens) - 1] = -1                     # nothing follows a sequence's last row
    t = torch.from_numpy(tokens).cuda()
    o = stack.score(hidden, seqlens, *_states(len(seqlens)), head, t, top=4)
    h = stack.prefill(hidden, seqlens, *_states(len(seqlens)))
    before = h.clone()
    logits = head.logits(h)
    assert torch.equal(h, before) and logits.dtype == F32
    exact, size = _exact_logits(h, head, norm_w)
    assert ((logits.double() - exact).abs() <= 2.0 ** -24 * exact.abs() + (42 + 8) * 2.0 ** -22 * size).all()
    same = m2.m2_token_logprobs(logits, t, 4)
    assert all(torch.equal(a, b) for a, b in zip(o, same))
    logp = torch.log_softmax(exact, 1)
    # an error e of every logit moves a log probability by 2 e at most
    e = (2.0 ** -24 * exact.abs() + 50 * 2.0 ** -22 * size).amax(1)
    want = torch.where(t < 0, 0.0, logp.gather(1, t.long().clamp(min=0)[:, None])[:, 0])
    assert ((o.logprobs.double() - want).abs() <= 2 * e + 2.0 ** -18).all()
    assert (o.ranks[t < 0] == 0).all() and (o.ranks[t >= 0] >= 1).all()
    # in pieces of a few rows, and with bf16 logits
    parts = head.logprobs(h, t, 4, max_rows=40)
    assert torch.allclose(parts.logprobs, o.logprobs, rtol=0, atol=float(4 * e.max()) + 2.0 ** -17)
    assert parts.top_tokens.shape == (T, 4)
    half = m2.Mxfp4Head(norm_w, head.weight, dtype=BF)
    assert torch.equal(half.logits(h), m2.mxfp4_linear_bf16(m2.m2_rmsnorm_residual(h, None, norm_w, 1e-5), head.weight))
    m2.check_standalone()


def test_decode_rows_into_a_beam_step(stack, head):
    head, _ = head
    conv, ssm = _states(8)
    slots = torch.randperm(8, device="cuda").int()[:6].view(2, 3)
    x = torch.from_numpy(synth.make_hidden(4, 6)).to(BF).cuda()
    scores = torch.tensor([[0.0, -1.0, -2.0]] * 2, device="cuda")
    h = stack.decode(x, conv, ssm, slots.view(-1))
    logits = head.logits(h)
    step, slots = stack.beam_step(logits, scores, conv, ssm, slots)
    # each selected token's score is its beam's plus its log probability
    for i in range(2):
        rows = (3 * i + step.parents[i]).long()
        o = m2.m2_token_logprobs(logits[rows].contiguous(), step.tokens[i])
        assert torch.allclose(step.scores[i], scores[i][step.parents[i].long()] + o.logprobs, rtol=0, atol=2.0 ** -17)
    m2.check_standalone()


def test_head_refuses_what_does_not_fit(head):
    head, norm_w = head
    with pytest.raises(ValueError):
        m2.Mxfp4Head(norm_w[:-8], head.weight)
    with pytest.raises(ValueError):
        m2.Mxfp4Head(norm_w, head.weight, dtype=torch.float16)
    h = torch.zeros(3, 2688, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        head.logprobs(h, torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        head.logprobs(h, max_rows=0)
