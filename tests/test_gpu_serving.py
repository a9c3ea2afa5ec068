"""Many requests on one block and on a stack: adapters inside m2_prefill_lora,
m2_decode_lora and m2_mixed_lora, and a beam search over a paged stack.

Adapters inside the block are checked at three joints: the in_proj rows are
m2_lora_add of the plain call's rows, bit for bit; everything between the
projections is the oracle's on those rows (the block tolerances); and the
output is m2_lora_add of out_proj of the block's own codes (or bf16 rows),
bit for bit.  m2_lora_add itself is checked against its formula elsewhere."""
import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import (assert_state, bf16_dev, device_weights, f32_dev, rel_l2, to_np, u8_dev)

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module", params=["w8a8", "w8a16"])
def block(request):
    Wt = synth.make_weights(0)
    blk = m2.Mamba2Mixer(device_weights(Wt), arm=m2.M2_ARM_W8A16 if request.param == "w8a16" else m2.M2_ARM_W8A8)
    yield Wt, blk, request.param
    blk.close()


def _adapters(n=3, rank=16, seed=0, which="both", scale=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def t(*shape, std):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)

    i = (t(n, rank, 2688, std=2688 ** -0.5), t(n, 10304, rank, std=0.3 * rank ** -0.5))
    o = (t(n, rank, 4096, std=4096 ** -0.5), t(n, 2688, rank, std=0.3 * rank ** -0.5))
    sc = torch.rand(n, generator=g, device="cuda") + 0.5 if scale else None
    return m2.LoraAdapters(*(i if which != "out" else (None, None)), *(o if which != "in" else (None, None)), scale=sc), i, o, sc


def _taps(T):
    return dict(zx=torch.zeros((T, 10304), dtype=torch.bfloat16, device="cuda"),
                y=torch.zeros((T, 4096), dtype=torch.bfloat16, device="cuda"),
                o=torch.zeros((T, 4096), dtype=torch.bfloat16, device="cuda"),
                q2=torch.zeros((T, 4096), dtype=torch.uint8, device="cuda"))


def _middle(Wt, zx, seqlens, conv, ssm):
    """The oracle's conv, scan and gated norm on given in_proj rows."""
    g = Wt["geo"]
    z, xbc, dt_raw = oracle.split_zxbcdt(zx, g.d_inner, g.conv_dim, g.nheads)
    A = -np.exp(np.asarray(Wt["A_log"], np.float64))
    dt = oracle.softplus(dt_raw + np.asarray(Wt["dt_bias"], np.float64)[None, :])
    y, S, W = np.empty((len(zx), g.d_inner)), [], []
    t = 0
    for s, T in enumerate(seqlens):
        sl = slice(t, t + T)
        u, w = oracle.causal_conv1d_silu(xbc[sl], Wt["conv_w"], Wt["conv_b"], conv[s])
        x, B, C = oracle.split_xbc(u, g.d_inner, g.n_groups, g.d_state)
        ys, Sn = oracle.ssd_sequential(x.reshape(T, g.nheads, g.headdim), dt[sl], A, B.reshape(T, g.n_groups, g.d_state),
                                       C.reshape(T, g.n_groups, g.d_state), Wt["D"], ssm[s])
        y[sl] = oracle.bf16_round(ys.reshape(T, g.d_inner))
        S.append(Sn), W.append(w)
        t += T
    return y, oracle.bf16_round(oracle.gated_rmsnorm_group(y, z, Wt["norm_w"], g.n_groups, Wt["eps"])), S, W


def _check_joints(Wt, arm, taps, zx0, hidden, ids, i, o, sc, out, which="both"):
    want = m2.m2_lora_add(zx0, hidden, *i, ids, scale=sc) if which != "out" else zx0
    assert torch.equal(taps["zx"], want)
    if arm == "w8a8":
        base = m2.fp8_linear(taps["q2"], Wt["s_y"], u8_dev(Wt["out_proj"]), Wt["s_w2"])
    else:
        base = m2.bf16_linear(taps["o"], m2.fp8_dequant(u8_dev(Wt["out_proj"]), Wt["s_w2"]), 1.0)
    if which != "in":
        base = m2.m2_lora_add(base, taps["o"], *o, ids, scale=sc)
    assert torch.equal(out, base)
    m2.check_standalone()


@pytest.mark.parametrize("which", ["both", "in", "out"])
def test_decode(block, which):
    Wt, blk, arm = block
    lora, i, o, sc = _adapters(which=which, scale=which != "in")
    Bt, n_slots = 9, 16
    conv0, ssm0 = synth.make_conv_state(2, n_slots), synth.make_ssm_state(2, n_slots)
    h = bf16_dev(synth.make_hidden(2, Bt))
    slots = np.array([4, 9, -1, 0, 15, 7, 3, -1, 8])
    ids = torch.tensor([0, 2, 1, -1, 1, 0, 0, -1, 2], dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots.astype(np.int32)).cuda()
    taps = _taps(Bt)
    blk.set_taps(**taps)
    plain = blk.decode(h, bf16_dev(conv0), f32_dev(ssm0), sl)
    zx0 = taps["zx"].clone()
    conv, ssm = bf16_dev(conv0), f32_dev(ssm0)
    out = blk.decode_lora(h, conv, ssm, sl, lora, ids)
    torch.cuda.synchronize()
    blk.set_taps()
    blk.check()
    _check_joints(Wt, arm, taps, zx0, h, ids, i, o, sc, out, which)
    assert torch.equal(out[3], plain[3]) and not out[[2, 7]].any()      # no adapter; padding rows
    live = slots >= 0
    y, on, S, W = _middle(Wt, to_np(taps["zx"])[live], [1] * int(live.sum()), conv0[slots[live]], ssm0[slots[live]])
    assert rel_l2(to_np(taps["o"])[live], on) < 1e-2
    assert_state(ssm.cpu().numpy()[slots[live]], np.stack(S))
    assert np.array_equal(to_np(conv)[slots[live]], np.stack(W))
    rest = np.setdiff1d(np.arange(n_slots), slots[live])
    assert np.array_equal(ssm.cpu().numpy()[rest], ssm0[rest])


@pytest.mark.parametrize("lens,ids", [([300, 37, 5], [1, -1, 0]), ([20, 9, 1], [2, 2, -1]), ([1], [0]),
                                      ([64] * 5, [0, 1, 2, 1, -1])])
def test_prefill(block, lens, ids):
    Wt, blk, arm = block
    lora, i, o, sc = _adapters(seed=1)
    T, n = sum(lens), len(lens)
    h = bf16_dev(synth.make_hidden(5, T))
    conv0, ssm0 = synth.make_conv_state(5, n), synth.make_ssm_state(5, n)
    has = [k % 2 for k in range(n)]
    taps = _taps(T)
    blk.set_taps(**taps)
    blk.prefill(h, lens, bf16_dev(conv0), f32_dev(ssm0), has_initial=has)
    zx0 = taps["zx"].clone()
    conv, ssm = bf16_dev(conv0), f32_dev(ssm0)
    out = blk.prefill_lora(h, lens, conv, ssm, lora, ids, has_initial=has)
    torch.cuda.synchronize()
    blk.set_taps()
    blk.check()
    row = torch.tensor(np.repeat(ids, lens), dtype=torch.int32, device="cuda")
    _check_joints(Wt, arm, taps, zx0, h, row, i, o, sc, out)
    mask = np.array(has, np.float64)
    y, on, S, W = _middle(Wt, to_np(taps["zx"]), lens, conv0 * mask[:, None, None], ssm0 * mask[:, None, None, None])
    assert rel_l2(to_np(taps["o"]), on) < 1e-2
    assert_state(ssm.cpu().numpy(), np.stack(S))
    assert np.array_equal(to_np(conv), np.stack(W))


@pytest.mark.parametrize("Bt,lens", [(3, [40, 300]), (70, [20, 9]), (5, []), (0, [17, 70])])
def test_mixed(block, Bt, lens):
    Wt, blk, arm = block
    if arm == "w8a16":
        with pytest.raises(m2.M2Error):
            blk.mixed_lora_workspace_size(2, [3], _adapters()[0])
        return
    lora, i, o, sc = _adapters(seed=2, n=4)
    T, n, n_slots = sum(lens), len(lens), 128
    h = bf16_dev(synth.make_hidden(6, Bt + T))
    pool0, ssmp0 = synth.make_conv_state(2, n_slots), synth.make_ssm_state(2, n_slots)
    slots = np.random.default_rng(1).permutation(n_slots)[:max(Bt, 1)].astype(np.int32)
    if Bt > 4:
        slots[2] = -1
    rid = torch.tensor(np.arange(max(Bt, 1)) % 5 - 1, dtype=torch.int32, device="cuda")
    sid = [k % 4 for k in range(n)]
    sl = torch.from_numpy(slots).cuda()
    dec = (lambda: (bf16_dev(pool0), f32_dev(ssmp0))) if Bt else (lambda: (None, None))
    conv_s, ssm_s = synth.make_conv_state(6, max(n, 1)), synth.make_ssm_state(6, max(n, 1))
    pre = (lambda: (bf16_dev(conv_s), f32_dev(ssm_s))) if n else (lambda: (None, None))
    taps = _taps(Bt + T)
    blk.set_taps(**taps)
    blk.mixed(h, Bt, *dec(), sl if Bt else None, lens, *pre())
    zx0 = taps["zx"].clone()
    cp, sp = dec()
    cs, ss = pre()
    out = blk.mixed_lora(h, Bt, cp, sp, sl if Bt else None, rid if Bt else None, lens, cs, ss, lora, sid)
    torch.cuda.synchronize()
    blk.set_taps()
    blk.check()
    row = np.concatenate([rid.cpu().numpy()[:Bt], np.repeat(sid, lens).astype(np.int32)]).astype(np.int32)
    _check_joints(Wt, arm, taps, zx0, h, torch.from_numpy(row).cuda(), i, o, sc, out)
    zx = to_np(taps["zx"])
    if Bt:
        live = slots >= 0
        _, on, S, _ = _middle(Wt, zx[:Bt][live], [1] * int(live.sum()), pool0[slots[live]], ssmp0[slots[live]])
        assert rel_l2(to_np(taps["o"])[:Bt][live], on) < 1e-2 and not out[:Bt][torch.from_numpy(~live).cuda()].any()
        assert_state(sp.cpu().numpy()[slots[live]], np.stack(S))
    if n:
        _, on, S, _ = _middle(Wt, zx[Bt:], lens, np.zeros_like(conv_s), np.zeros_like(ssm_s))
        assert rel_l2(to_np(taps["o"])[Bt:], on) < 1e-2
        assert_state(ss.cpu().numpy(), np.stack(S))


def test_no_request_names_an_adapter(block):
    """All -1: the plain calls' bits, states included."""
    _, blk, _ = block
    lora = _adapters()[0]
    conv0, ssm0 = synth.make_conv_state(2, 4), synth.make_ssm_state(2, 4)
    h = bf16_dev(synth.make_hidden(2, 304))
    sl = torch.arange(4, dtype=torch.int32, device="cuda")
    a, b = [(bf16_dev(conv0), f32_dev(ssm0)) for _ in range(2)]
    assert torch.equal(blk.decode(h[:4], *a, sl), blk.decode_lora(h[:4], *b, sl, lora, -torch.ones_like(sl)))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    lens = [200, 104]
    a, b = [(bf16_dev(conv0[:2]), f32_dev(ssm0[:2])) for _ in range(2)]
    assert torch.equal(blk.prefill(h, lens, *a), blk.prefill_lora(h, lens, *b, lora, [-1, -1]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    blk.check()


def test_unknown_row_adapter_is_reported_by_the_block(block):
    _, blk, _ = block
    lora = _adapters()[0]
    conv0, ssm0 = synth.make_conv_state(2, 2), synth.make_ssm_state(2, 2)
    h = bf16_dev(synth.make_hidden(2, 2))
    sl = torch.arange(2, dtype=torch.int32, device="cuda")
    plain = blk.decode(h, bf16_dev(conv0), f32_dev(ssm0), sl)
    out = blk.decode_lora(h, bf16_dev(conv0), f32_dev(ssm0), sl, lora, torch.tensor([3, -1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    with pytest.raises(m2.M2Error) as e:
        blk.check()
    assert "adapter" in str(e.value) and torch.equal(out, plain)
    blk.check()


# ---------------------------------------------------------------- a beam search over a paged stack

LAYERS, BATCH, BEAMS, VOCAB, STEPS, EOS = 2, 3, 4, 1009, 6, 5


@pytest.fixture(scope="module")
def search():
    blocks, norm_ws, adapters = [], [], []
    for l in range(LAYERS):
        blocks.append(m2.Mamba2Mixer(device_weights(synth.make_weights(4, l))))
        norm_ws.append(bf16_dev(synth.make_stack_norm_w(4, l)))
        adapters.append(_adapters(n=2, rank=8, seed=10 + l)[0])
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    embed = torch.randn((VOCAB, 2688), generator=g, device="cuda").to(torch.bfloat16)
    head = torch.randn((VOCAB, 2688), generator=g, device="cuda").mul_(0.05).to(torch.bfloat16)
    head[EOS] += 0.02 * embed[:40].float().mean(0).to(torch.bfloat16)
    return blocks, norm_ws, adapters, embed, head


def _start(rows, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    conv = [torch.randn((rows, 6144, 3), generator=g, device="cuda").to(torch.bfloat16) for _ in range(LAYERS)]
    ssm = [torch.randn((rows, 64, 64, 128), generator=g, device="cuda").mul_(0.1) for _ in range(LAYERS)]
    return conv, ssm


@pytest.mark.parametrize("fused", [False, True])
def test_beam_search_over_a_stack(search, fused):
    """Prefill-free search from given states with an adapter per request,
    against the same search with every row's state gathered whole."""
    blocks, norm_ws, adapters, embed, head = search
    stk = m2.Mamba2Stack(blocks, norm_ws, fused=fused)
    rows = BATCH * BEAMS
    row_adapter = torch.tensor([0, -1, 1], dtype=torch.int32, device="cuda").repeat_interleave(BEAMS)
    conv, ssm = _start(rows + 5)
    slots = torch.randperm(rows + 5, generator=torch.Generator().manual_seed(2))[:rows].int().view(BATCH, BEAMS).cuda()
    rconv, rssm = [c[slots.view(-1).long()].clone() for c in conv], [s[slots.view(-1).long()].clone() for s in ssm]
    ident = torch.arange(rows, dtype=torch.int32, device="cuda")
    scores = torch.full((BATCH, BEAMS), float("-inf"), device="cuda")
    scores[:, 0] = 0.0                                  # the beams of a request start equal: one of them counts
    done = torch.zeros((BATCH, BEAMS), dtype=torch.bool, device="cuda")
    tok = torch.zeros(rows, dtype=torch.long, device="cuda")
    rtok, rscores, rdone = tok.clone(), scores.clone(), done.clone()
    some_copied = False
    for _ in range(STEPS):
        h = stk.decode_lora(embed[tok], conv, ssm, slots.view(-1), adapters, row_adapter)
        step, slots = stk.beam_step(m2.bf16_linear(h, head), scores, conv, ssm, slots, eos_token=EOS, done=done)
        tok, scores, done = step.tokens.view(-1).clamp(min=0).long(), step.scores, step.done
        # the same with whole gathers (and the parents' rows of a plain pool)
        rh = stk.decode_lora(embed[rtok], rconv, rssm, ident, adapters, row_adapter)
        assert torch.equal(rh, h)
        rstep = m2.m2_beam_select(m2.bf16_linear(rh, head), rscores, eos_token=EOS, done=rdone)
        assert all(torch.equal(a, b) for a, b in zip(step, rstep))
        src = (rstep.parents + BEAMS * torch.arange(BATCH, device="cuda")[:, None]).view(-1).long()
        rconv, rssm = [c[src] for c in rconv], [s[src] for s in rssm]
        rtok, rscores, rdone = rstep.tokens.view(-1).clamp(min=0).long(), rstep.scores, rstep.done
        some_copied |= bool((rstep.parents != torch.arange(BEAMS, device="cuda")).any())
        at = slots.view(-1).long()
        for l in range(LAYERS):
            assert torch.equal(conv[l][at], rconv[l]) and torch.equal(ssm[l][at], rssm[l])
    assert some_copied and sorted(slots.view(-1).tolist()) == sorted(set(slots.view(-1).tolist()))
    for b in blocks:
        b.check()
    m2.check_standalone()


def test_stack_prefill_and_decode_compose_by_layer(search):
    blocks, norm_ws, adapters, embed, _ = search
    stk = m2.Mamba2Stack(blocks, norm_ws, fused=True)
    lens, ids = [70, 3], [1, -1]
    h = embed[:sum(lens)].contiguous()
    conv = [torch.zeros((2, 6144, 3), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
    ssm = [torch.zeros((2, 64, 64, 128), device="cuda") for _ in range(LAYERS)]
    c2, s2 = [c.clone() for c in conv], [s.clone() for s in ssm]
    out = stk.prefill_lora(h, lens, conv, ssm, adapters, ids, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    hr, prev = h.clone(), None
    for l in range(LAYERS):
        x = m2.m2_rmsnorm_residual(hr, prev, norm_ws[l], 1e-5)
        prev = blocks[l].prefill_lora(x, lens, c2[l], s2[l], adapters[l], ids)
    m2.m2_rmsnorm_residual(hr, prev, None, 1e-5, norm=False)
    torch.cuda.synchronize()
    assert torch.equal(hr, out)
    assert all(torch.equal(a, b) for a, b in zip(conv + ssm, c2 + s2))


def test_a_search_step_in_a_graph(search):
    """decode_lora, the head, beam_step captured together and replayed."""
    blocks, norm_ws, adapters, embed, head = search
    stk = m2.Mamba2Stack(blocks, norm_ws)
    rows = BATCH * BEAMS
    ids = torch.arange(rows, dtype=torch.int32, device="cuda") % 2
    scores0 = -torch.rand((BATCH, BEAMS), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    runs = []
    for captured in (False, True):
        conv, ssm = _start(rows, 7)
        slots = torch.arange(rows, dtype=torch.int32, device="cuda").view(BATCH, BEAMS)
        scores, tok = scores0.clone(), torch.arange(rows, device="cuda")

        def one():
            h = stk.decode_lora(embed[tok], conv, ssm, slots.view(-1), adapters, ids)
            step, new = stk.beam_step(m2.bf16_linear(h, head), scores, conv, ssm, slots)
            slots.copy_(new), scores.copy_(step.scores), tok.copy_(step.tokens.view(-1))

        if captured:
            keep = [t.clone() for t in (*conv, *ssm, slots, scores, tok)]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                one()                                   # warm-up outside the capture
            torch.cuda.current_stream().wait_stream(s)
            for t, k in zip((*conv, *ssm, slots, scores, tok), keep):
                t.copy_(k)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
            for _ in range(4):
                g.replay()
        else:
            for _ in range(4):
                one()
        torch.cuda.synchronize()
        runs.append((*conv, *ssm, slots, scores, tok))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    m2.check_standalone()


def test_prefill_takes_its_lengths_from_any_iterable(block):
    _, blk, _ = block
    lora, *_ = _adapters(seed=1)
    lens = [9, 4]
    h = bf16_dev(synth.make_hidden(6, sum(lens)))
    outs = [blk.prefill_lora(h, n, bf16_dev(synth.make_conv_state(6, 2)), f32_dev(synth.make_ssm_state(6, 2)), lora, [1, -1])
            for n in (lens, iter(lens))]
    torch.cuda.synchronize()
    assert torch.equal(*outs)
