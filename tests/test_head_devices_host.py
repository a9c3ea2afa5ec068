"""What the binding of the head keeps per device, checked without one: the size of
the products' workspace, which depends on the device's SMs and clusters."""
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


def test_workspace_sizes_are_the_current_devices(m2, monkeypatch):
    """A size found on one device is not given out for another."""
    here, asked = [0], []

    class Lib:
        @staticmethod
        def mxfp4_linear_bf16_workspace_size(M, N, K, out):
            asked.append(here[0])
            out._obj.value = 4096 * here[0]
            return m2.M2_OK

    monkeypatch.setattr(m2, "_lib", Lib)
    monkeypatch.setattr(m2, "_current_device", lambda: here[0])
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    shape = (24, 999, 1312)   # (asked for nowhere else)
    for device in (0, 1, 0, 1, 1):
        here[0] = device
        assert m2.mxfp4_linear_bf16_workspace_size(*shape) == 4096 * device
    assert asked == [0, 1]    # (and it is found once for each)


def test_workspace_sizes_without_a_device(m2):
    assert m2.mxfp4_linear_bf16_workspace_size(100, 64, 128) > 0


def test_heads_that_no_call_could_serve_are_refused(m2, monkeypatch):
    """What the kernels refuse of a head, whatever its rows, is refused when it is
    made, so that no call finds it after the states have moved."""
    monkeypatch.setattr(m2, "_need", lambda *a, **kw: None)   # (host tensors stand for the device's)
    monkeypatch.setattr(m2, "_need_mx", lambda *a, **kw: None)

    def cut(t, by):   # the same values off a 16-byte boundary
        wide = torch.zeros(t.numel() + 16, dtype=t.dtype)
        return wide[by:by + t.numel()].view(t.shape)

    norm_w, codes = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8)
    scales = torch.zeros(1, 1, 512, dtype=torch.uint8)
    assert not any(t.data_ptr() % 16 for t in (norm_w, codes, scales))
    m2.Mxfp4Head(norm_w, m2.Mxfp4(codes, scales))
    for eps in (0.0, -1e-5, float("nan"), 1e-60):   # (1e-60: 0 in f32)
        with pytest.raises(ValueError, match="eps"):
            m2.Mxfp4Head(norm_w, m2.Mxfp4(codes, scales), eps=eps)
    for head in ((cut(norm_w, 1), codes, scales), (norm_w, cut(codes, 8), scales), (norm_w, codes, cut(scales, 4))):
        with pytest.raises(ValueError, match="16-byte"):
            m2.Mxfp4Head(head[0], m2.Mxfp4(head[1], head[2]))
    for vocab, half in ((0, 32), ((1 << 24) + 1, 32), (1 << 24, (1 << 14) + 32)):
        big = torch.empty(1, dtype=torch.uint8).expand(vocab, half)
        with pytest.raises(ValueError, match="vocab"):
            m2.Mxfp4Head(norm_w, m2.Mxfp4(big, scales))
