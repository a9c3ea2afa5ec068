"""Host-side refusals of the head's entry points (mxfp4_*, m2_token_logprobs):
bad shapes, null and misaligned pointers, overlapping buffers and short
workspaces are refused before any device work.  No kernel is launched; the
pointers are never read."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m2():
    if not os.path.exists(os.path.join(ROOT, "mamba2_ssm_mixer_gb300", "libm2.so")):
        import __graft_entry__
        __graft_entry__.build()
    import mamba2_ssm_mixer_gb300 as pkg
    return pkg


BIG = 1 << 40   # a workspace size above every need


def at(i):
    return i << 32   # an address far from the others


def _quant(m2, **kw):
    a = dict(x=at(1), stride=128, rows=4, K=128, codes=at(2), scales=at(3))
    a.update(kw)
    return m2._lib.mxfp4_quant(a["x"], a["stride"], a["rows"], a["K"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("kw", [dict(K=0), dict(K=16), dict(K=33), dict(K=(1 << 24) + 32, stride=1 << 25), dict(rows=-1),
                                dict(rows=(1 << 24) + 1), dict(stride=120), dict(stride=132), dict(stride=(1 << 40) + 8)])
def test_quant_refuses_shapes(m2, kw):
    assert _quant(m2, **kw) == m2.M2_ESHAPE
    assert m2.last_error()


@pytest.mark.parametrize("kw", [dict(x=None), dict(codes=None), dict(scales=None), dict(x=at(1) + 8),
                                dict(codes=at(2) + 8), dict(scales=at(3) + 4), dict(codes=at(1) + 16),
                                dict(scales=at(1) + 512), dict(scales=at(2) + 128)])
def test_quant_refuses_pointers(m2, kw):
    assert _quant(m2, **kw) == m2.M2_EINVAL
    assert m2.last_error()


def _dequant(m2, **kw):
    a = dict(codes=at(1), scales=at(2), rows=4, K=128, out=at(3))
    a.update(kw)
    return m2._lib.mxfp4_dequant(a["codes"], a["scales"], a["rows"], a["K"], a["out"], None)


@pytest.mark.parametrize("kw,want", [(dict(K=48), "M2_ESHAPE"), (dict(rows=-1), "M2_ESHAPE"), (dict(codes=None), "M2_EINVAL"),
                                     (dict(scales=None), "M2_EINVAL"), (dict(out=None), "M2_EINVAL"),
                                     (dict(out=at(3) + 8), "M2_EINVAL"), (dict(codes=at(1) + 4), "M2_EINVAL"),
                                     (dict(scales=at(2) + 4), "M2_EINVAL"), (dict(out=at(1) + 64), "M2_EINVAL"),
                                     (dict(out=at(2) + 64), "M2_EINVAL")])
def test_dequant_refuses(m2, kw, want):
    assert _dequant(m2, **kw) == getattr(m2, want)
    assert m2.last_error()


def test_scale_bytes_and_pack(m2):
    n = ctypes.c_size_t()
    lib = m2._lib
    assert lib.mxfp4_scale_bytes(1, 128, None) == m2.M2_EINVAL
    assert lib.mxfp4_scale_bytes(1, 40, ctypes.byref(n)) == m2.M2_ESHAPE
    for rows, K, want in ((0, 32, 0), (1, 32, 512), (128, 128, 512), (129, 160, 2048), (10304, 2688, 81 * 21 * 512)):
        assert lib.mxfp4_scale_bytes(rows, K, ctypes.byref(n)) == m2.M2_OK and n.value == want
    assert lib.mxfp4_pack_scales(at(1), 4, 100, at(2), None) == m2.M2_ESHAPE
    assert lib.mxfp4_pack_scales(None, 4, 128, at(2), None) == m2.M2_EINVAL
    assert lib.mxfp4_pack_scales(at(1), 4, 128, None, None) == m2.M2_EINVAL
    assert lib.mxfp4_pack_scales(at(1), 4, 128, at(2) + 8, None) == m2.M2_EINVAL
    assert lib.mxfp4_pack_scales(at(1) + 100, 4, 128, at(1), None) == m2.M2_EINVAL


def _linear(m2, **kw):
    a = dict(ac=at(1), asc=at(2), wc=at(3), ws=at(4), y=at(5), dtype=1, M=4, N=64, K=128)
    a.update(kw)
    return m2._lib.mxfp4_linear(a["ac"], a["asc"], a["wc"], a["ws"], a["y"], a["dtype"], a["M"], a["N"], a["K"], None)


@pytest.mark.parametrize("kw", [dict(K=0), dict(K=80), dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0), dict(N=(1 << 24) + 1),
                                dict(M=1 << 24, N=(1 << 16) + 1)])
def test_linear_refuses_shapes(m2, kw):
    assert _linear(m2, **kw) == m2.M2_ESHAPE
    assert m2.last_error()


@pytest.mark.parametrize("kw", [dict(ac=None), dict(asc=None), dict(wc=None), dict(ws=None), dict(y=None), dict(dtype=2),
                                dict(ac=at(1) + 8), dict(asc=at(2) + 8), dict(wc=at(3) + 8), dict(ws=at(4) + 8),
                                dict(y=at(5) + 1), dict(y=at(5) + 2, dtype=0), dict(y=at(1) + 64), dict(y=at(2) + 64),
                                dict(y=at(3) + 64), dict(y=at(4) + 64)])
def test_linear_refuses_pointers(m2, kw):
    assert _linear(m2, **kw) == m2.M2_EINVAL
    assert m2.last_error()


def _linear_bf16(m2, **kw):
    a = dict(x=at(1), stride=128, wc=at(3), ws=at(4), y=at(5), dtype=1, M=100, N=64, K=128, work=at(6), n=BIG)
    a.update(kw)
    return m2._lib.mxfp4_linear_bf16(a["x"], a["stride"], a["wc"], a["ws"], a["y"], a["dtype"], a["M"], a["N"], a["K"],
                                     a["work"], a["n"], None)


def test_linear_bf16_refuses(m2):
    n = ctypes.c_size_t()
    assert m2._lib.mxfp4_linear_bf16_workspace_size(4, 64, 128, None) == m2.M2_EINVAL
    assert m2._lib.mxfp4_linear_bf16_workspace_size(4, 0, 128, ctypes.byref(n)) == m2.M2_ESHAPE
    assert m2._lib.mxfp4_linear_bf16_workspace_size(4, 64, 130, ctypes.byref(n)) == m2.M2_ESHAPE
    assert m2._lib.mxfp4_linear_bf16_workspace_size(100, 64, 128, ctypes.byref(n)) == m2.M2_OK and n.value > 0
    assert _linear_bf16(m2, n=n.value - 1) == m2.M2_ENOMEM
    assert _linear_bf16(m2, work=None) == m2.M2_ENOMEM
    for kw in (dict(work=at(6) + 128), dict(x=at(1) + 8), dict(x=None), dict(y=at(1) + 64), dict(work=at(1), n=n.value),
               dict(work=at(3), n=n.value), dict(work=at(4), n=n.value), dict(work=at(5), n=n.value), dict(dtype=7)):
        assert _linear_bf16(m2, **kw) == m2.M2_EINVAL, kw
        assert m2.last_error()
    for kw in (dict(stride=64), dict(stride=129), dict(K=100), dict(M=-2), dict(N=0)):
        assert _linear_bf16(m2, **kw) == m2.M2_ESHAPE, kw


def _logprobs(m2, **kw):
    a = dict(logits=at(1), dtype=0, stride=1000, rows=4, vocab=1000, tokens=at(2), top=5, lp=at(3), rk=at(4), en=at(5),
             tt=at(6), tl=at(7))
    a.update(kw)
    return m2._lib.m2_token_logprobs(a["logits"], a["dtype"], a["stride"], a["rows"], a["vocab"], a["tokens"], a["top"],
                                     a["lp"], a["rk"], a["en"], a["tt"], a["tl"], None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1),
                                dict(top=-1), dict(top=65), dict(stride=999), dict(stride=(1 << 40) + 1)])
def test_logprobs_refuses_shapes(m2, kw):
    assert _logprobs(m2, **kw) == m2.M2_ESHAPE
    assert m2.last_error()


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(logits=None), dict(logits=at(1) + 2), dict(logits=at(1) + 1, dtype=1),
                                dict(tokens=None), dict(lp=None), dict(rk=None), dict(tokens=at(2) + 2), dict(lp=at(3) + 2),
                                dict(rk=at(4) + 1), dict(en=at(5) + 2), dict(tt=None), dict(tl=None), dict(tt=at(6) + 2),
                                dict(tl=at(7) + 3), dict(lp=at(1) + 1024), dict(en=at(2)), dict(rk=at(3) + 8),
                                dict(tl=at(6) + 64), dict(tokens=None, lp=None, rk=None, en=None, top=0, tt=None, tl=None)])
def test_logprobs_refuses_pointers(m2, kw):
    assert _logprobs(m2, **kw) == m2.M2_EINVAL
    assert m2.last_error()


def test_python_refuses_host_tensors_and_shapes(m2):
    """Without a device every call of the binding stops at its own checks."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: m2.mxfp4_quant(x), lambda: m2.mxfp4_dequant((u8, u8)), lambda: m2.mxfp4_pack(u8, u8),
                 lambda: m2.mxfp4_linear_bf16(x, (u8, u8)), lambda: m2.m2_token_logprobs(x),
                 lambda: m2.mxfp4_linear(m2.Mxfp4(u8, u8), m2.Mxfp4(u8, u8)),
                 lambda: m2.Mxfp4Head(x[0], m2.Mxfp4(u8, u8))):
        with pytest.raises(ValueError):
            call()


def test_weights_past_the_largest_operand_are_refused(m2):
    n = ctypes.c_size_t()
    big = dict(M=100, N=1 << 24, K=1 << 15)
    assert _linear(m2, **big) == m2.M2_ESHAPE
    assert _linear_bf16(m2, stride=1 << 15, **big) == m2.M2_ESHAPE
    assert m2._lib.mxfp4_linear_bf16_workspace_size(100, 1 << 24, 1 << 15, ctypes.byref(n)) == m2.M2_ESHAPE


def test_products_ask_for_packed_weights(m2):
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="must be an Mxfp4"):
        m2._need_mx((u8, u8), "w", K=64)


def test_score_refuses_before_it_runs(m2, monkeypatch):
    """A call that the head cannot serve leaves the stack's states alone."""
    monkeypatch.setattr(m2, "_on_device", lambda ref, stream, others, call: call(None))
    ran = []

    class Stack(m2.Mamba2Stack):
        def __init__(self):
            pass

        def prefill(self, *a, **kw):
            ran.append(1)

    head = object.__new__(m2.Mxfp4Head)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    head.norm_w, head.weight = u8[0], m2.Mxfp4(u8, u8)
    hidden = torch.zeros(3, 64, dtype=torch.bfloat16)
    for kw in (dict(top=65), dict(top=-1), dict(max_rows=0), dict(tokens=torch.zeros(4, dtype=torch.int32)),
               dict(hidden=torch.zeros(3, 96, dtype=torch.bfloat16))):
        a = dict(hidden=hidden, tokens=None, top=1, max_rows=4)
        a.update(kw)
        with pytest.raises(ValueError):
            Stack().score(a["hidden"], [3], [], [], head, a["tokens"], top=a["top"], max_rows=a["max_rows"])
    assert not ran
