"""Host-side refusals of the many-requests entry points (m2_lora_add,
m2_beam_select, m2_state_reorder): bad shapes, null and misaligned pointers,
overlapping buffers and short workspaces are refused before any device work.
No kernel is launched; the pointers are never read."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m2():
    if not os.path.exists(os.path.join(ROOT, "mamba2_ssm_mixer_gb300", "libm2.so")):
        import __graft_entry__
        __graft_entry__.build()
    import mamba2_ssm_mixer_gb300 as pkg
    return pkg


BIG = 1 << 40   # a workspace size above every need


def _lora(m2, **kw):
    a = dict(y=1 << 20, x=2 << 20, a=3 << 20, b=4 << 20, scale=None, n=4, rank=16, ids=5 << 20, out=6 << 20, M=4, N=64,
             K=64, ws=7 << 20, wsn=BIG)
    a.update(kw)
    return m2._lib.m2_lora_add(a["y"], a["x"], a["a"], a["b"], a["scale"], a["n"], a["rank"], a["ids"], a["out"], a["M"],
                               a["N"], a["K"], a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw", [dict(rank=12), dict(rank=0), dict(rank=136), dict(K=24), dict(K=0), dict(N=0), dict(N=(1 << 24) + 1), dict(K=(1 << 24) + 16), dict(M=-1),
                                dict(M=(1 << 24) + 1), dict(n=0), dict(n=4097)])
def test_lora_add_refuses_shapes(m2, kw):
    assert _lora(m2, **kw) == m2.M2_ESHAPE
    assert m2.last_error()


@pytest.mark.parametrize("kw", [dict(y=None), dict(x=None), dict(a=None), dict(b=None), dict(ids=None), dict(out=None),
                                dict(x=(2 << 20) + 8), dict(a=(3 << 20) + 2), dict(b=(4 << 20) + 8),
                                dict(y=(1 << 20) + 1), dict(ids=(5 << 20) + 2), dict(scale=(8 << 20) + 2),
                                dict(out=(1 << 20) + 2), dict(out=(2 << 20) + 16)])
def test_lora_add_refuses_pointers(m2, kw):
    assert _lora(m2, **kw) == m2.M2_EINVAL
    assert m2.last_error()


def test_lora_add_workspace(m2):
    n = ctypes.c_size_t()
    assert m2._lib.m2_lora_add_workspace_size(5000, 64, 64, 16, 4, None) == m2.M2_EINVAL
    assert m2._lib.m2_lora_add_workspace_size(5000, 64, 64, 20, 4, ctypes.byref(n)) == m2.M2_ESHAPE
    assert m2._lib.m2_lora_add_workspace_size(5000, 64, 64, 16, 4, ctypes.byref(n)) == m2.M2_OK and n.value > 0
    assert _lora(m2, M=5000, y=1 << 30, x=2 << 30, out=3 << 30, wsn=n.value - 1) == m2.M2_ENOMEM
    assert _lora(m2, M=5000, y=1 << 30, x=2 << 30, out=3 << 30, ws=(7 << 20) + 16) == m2.M2_EINVAL


def _beam(m2, **kw):
    a = dict(logits=1 << 30, dtype=0, stride=1000, batch=2, beams=4, vocab=1000, scores=1 << 20, done=None, eos=-1, k=4,
             tokens=2 << 20, parents=3 << 20, oscores=4 << 20, odone=None, ws=5 << 20, wsn=BIG)
    a.update(kw)
    return m2._lib.m2_beam_select(a["logits"], a["dtype"], a["stride"], a["batch"], a["beams"], a["vocab"], a["scores"],
                                  a["done"], a["eos"], a["k"], a["tokens"], a["parents"], a["oscores"], a["odone"],
                                  a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw", [dict(beams=0), dict(beams=33), dict(batch=-1), dict(batch=1025), dict(vocab=0),
                                dict(vocab=(1 << 24) + 1), dict(k=0), dict(k=65), dict(stride=999)])
def test_beam_select_refuses_shapes(m2, kw):
    assert _beam(m2, **kw) == m2.M2_ESHAPE
    assert m2.last_error()


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(logits=None), dict(scores=None), dict(tokens=None),
                                dict(parents=None), dict(oscores=None), dict(logits=(1 << 30) + 2),
                                dict(dtype=1, logits=(1 << 30) + 1), dict(scores=(1 << 20) + 2),
                                dict(done=6 << 20, eos=-1), dict(done=6 << 20, eos=1000), dict(odone=6 << 20, eos=-1),
                                dict(oscores=1 << 20, k=8), dict(oscores=(1 << 20) + 4),
                                dict(done=6 << 20, odone=6 << 20, eos=1, k=3), dict(tokens=(1 << 30) + 64),
                                dict(parents=(2 << 20) + 8), dict(ws=(5 << 20) + 16)])
def test_beam_select_refuses_pointers(m2, kw):
    assert _beam(m2, **kw) == m2.M2_EINVAL
    assert m2.last_error()


def test_beam_select_workspace(m2):
    n = ctypes.c_size_t()
    assert m2._lib.m2_beam_select_workspace_size(2, 4, 1000, 4, None) == m2.M2_EINVAL
    assert m2._lib.m2_beam_select_workspace_size(2, 4, 1000, 65, ctypes.byref(n)) == m2.M2_ESHAPE
    assert m2._lib.m2_beam_select_workspace_size(2, 4, 1000, 4, ctypes.byref(n)) == m2.M2_OK and n.value > 0
    assert _beam(m2, wsn=n.value - 1) == m2.M2_ENOMEM


def _reorder(m2, **kw):
    a = dict(conv=[1 << 30], ssm=[2 << 30], layers=None, dtype=0, n_slots=8, slots=1 << 20, parents=2 << 20, out=3 << 20,
             batch=2, beams=4)
    a.update(kw)
    c, s = a["conv"], a["ssm"]
    conv = None if c is None else (ctypes.c_void_p * 65)(*c)
    ssm = None if s is None else (ctypes.c_void_p * 65)(*s)
    return m2._lib.m2_state_reorder(conv, ssm, a["layers"] if a["layers"] is not None else 1, a["dtype"], a["n_slots"],
                                    a["slots"], a["parents"], a["out"], a["batch"], a["beams"], None)


@pytest.mark.parametrize("kw", [dict(layers=0), dict(layers=65), dict(beams=0), dict(beams=33), dict(batch=-1),
                                dict(batch=1025)])
def test_state_reorder_refuses_shapes(m2, kw):
    assert _reorder(m2, **kw) == m2.M2_ESHAPE
    assert m2.last_error()


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(n_slots=0), dict(conv=None), dict(ssm=None), dict(conv=[None]),
                                dict(ssm=[None]), dict(ssm=[(2 << 30) + 8]), dict(layers=2), dict(slots=None),
                                dict(parents=None), dict(out=None), dict(out=1 << 20), dict(out=(2 << 20) + 28),
                                dict(slots=(1 << 20) + 2)])
def test_state_reorder_refuses_pointers(m2, kw):
    assert _reorder(m2, **kw) == m2.M2_EINVAL
    assert m2.last_error()


def test_binding_refuses_host_tensors_and_types(m2):
    """The Python wrappers refuse tensors that are not on the device, before
    any call into the library."""
    import torch
    bf = torch.zeros((4, 64), dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    w = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m2.m2_lora_add(bf, bf, w, w.transpose(1, 2).contiguous(), ids)
    with pytest.raises(ValueError):
        m2.m2_beam_select(torch.zeros((4, 10)), torch.zeros((1, 4)))
    with pytest.raises(ValueError):
        m2.m2_beam_select(torch.zeros((4, 10), dtype=torch.float16), torch.zeros((1, 4)))
    with pytest.raises(ValueError):
        m2.m2_beam_select(torch.zeros((5, 10)), torch.zeros((1, 4)))
    with pytest.raises(ValueError):
        m2.m2_state_reorder([], [], ids.reshape(1, 4), ids.reshape(1, 4))


def _adapters(m2, **kw):
    f = dict(n_adapters=2, rank=16, in_a=1 << 20, in_b=2 << 20, out_a=3 << 20, out_b=4 << 20, scale=None)
    f.update(kw)
    return m2.m2_lora(*[f[n] for n, _ in m2.m2_lora._fields_])


@pytest.mark.parametrize("kw,status", [(dict(rank=12), "M2_ESHAPE"), (dict(n_adapters=0), "M2_ESHAPE"),
                                       (dict(in_b=None), "M2_EINVAL"), (dict(out_a=None), "M2_EINVAL"),
                                       (dict(in_a=None, in_b=None, out_a=None, out_b=None), "M2_EINVAL"),
                                       (dict(out_b=(4 << 20) + 8), "M2_EINVAL"), (dict(scale=2), "M2_EINVAL")])
def test_block_adapters_refused(m2, kw, status):
    """A bad adapter set is refused by all three block calls and their
    workspace queries, before the handle is looked at."""
    ref = ctypes.byref(_adapters(m2, **kw))
    want = getattr(m2, status)
    lens, ids, p = (ctypes.c_int32 * 1)(4), (ctypes.c_int32 * 1)(0), 1 << 21
    L = m2._lib
    assert L.m2_prefill_lora(None, p, lens, 1, None, p, p, ref, ids, p, p, BIG, None) == want
    assert "m2_prefill_lora" in m2.last_error()
    assert L.m2_decode_lora(None, p, 1, p, p, 1, p, ref, p, p, p, BIG, None) == want
    assert "m2_decode_lora" in m2.last_error()
    assert L.m2_mixed_lora(None, p, 1, p, p, 1, p, p, lens, 1, None, p, p, ref, ids, p, p, BIG, None) == want
    assert "m2_mixed_lora" in m2.last_error()


def test_block_adapter_ids_refused(m2):
    ref, p = ctypes.byref(_adapters(m2)), 1 << 21
    lens = (ctypes.c_int32 * 2)(4, 4)
    L = m2._lib
    for bad in ((0, 2), (-2, 0)):
        ids = (ctypes.c_int32 * 2)(*bad)
        assert L.m2_prefill_lora(None, p, lens, 2, None, p, p, ref, ids, p, p, BIG, None) == m2.M2_EINVAL
        assert "seq_adapter" in m2.last_error()
        assert L.m2_mixed_lora(None, p, 0, None, None, 0, None, None, lens, 2, None, p, p, ref, ids, p, p, BIG,
                               None) == m2.M2_EINVAL
        assert "seq_adapter" in m2.last_error()
    assert L.m2_prefill_lora(None, p, lens, 257, None, p, p, ref, None, p, p, BIG, None) == m2.M2_ESHAPE
    assert L.m2_decode_lora(None, p, 1, p, p, 1, p, ref, None, p, p, BIG, None) == m2.M2_EINVAL
    assert L.m2_decode_lora(None, p, 1, p, p, 1, p, ref, p, p, p, BIG, None) == m2.M2_EINVAL      # null handle
    n = ctypes.c_size_t()
    assert L.m2_prefill_lora_workspace_size(None, lens, 2, ref, ctypes.byref(n)) == m2.M2_EINVAL
    assert L.m2_decode_lora_workspace_size(None, 1, ref, ctypes.byref(n)) == m2.M2_EINVAL
    assert L.m2_mixed_lora_workspace_size(None, 1, lens, 2, ref, ctypes.byref(n)) == m2.M2_EINVAL


def test_lora_struct_matches_the_header(m2):
    import re
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "m2.h")).read(), flags=re.S)
    body = re.search(r"typedef struct m2_lora \{(.*?)\} m2_lora;", src, flags=re.S).group(1)
    assert re.findall(r"(\w+)\s*;", body) == [n for n, _ in m2.m2_lora._fields_]
