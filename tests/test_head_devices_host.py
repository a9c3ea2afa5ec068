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
