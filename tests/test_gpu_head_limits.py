"""Sizes past the head's limits that 32 bits do not hold: the binding refuses
them; cut to 32 bits, each of these would pass as a small matrix."""
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

BF, U8 = torch.bfloat16, torch.uint8
K = (1 << 32) + 32   # 32 in 32 bits


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


def test_rows_past_32_bits():
    x = torch.empty(1, K, dtype=BF, device="cuda")
    for call in (lambda: m2.m2_token_logprobs(x, None, 1), lambda: m2.mxfp4_quant(x)):
        with pytest.raises(ValueError, match="2\\^24"):
            call()


def test_packed_rows_past_32_bits():
    codes = torch.empty(1, K // 2, dtype=U8, device="cuda")
    with pytest.raises(ValueError, match="2\\^24"):
        m2.mxfp4_pack(codes, torch.empty(1, K // 32, dtype=U8, device="cuda"))
    q = m2.Mxfp4(codes, torch.empty(1, (K + 127) // 128, 512, dtype=U8, device="cuda"))
    for call in (lambda: m2.mxfp4_dequant(q), lambda: m2.mxfp4_linear(q, q)):
        with pytest.raises(ValueError, match="2\\^24"):
            call()


def test_alternatives_and_sizes_past_32_bits():
    logits = torch.zeros(1, 100, device="cuda")
    with pytest.raises(ValueError, match="top"):
        m2.m2_token_logprobs(logits, None, (1 << 32) + 5)
    for shape in ((K, 64, 64), (64, K, 64), (64, 64, K)):
        with pytest.raises(ValueError, match="2\\^24"):
            m2.mxfp4_linear_bf16_workspace_size(*shape)
