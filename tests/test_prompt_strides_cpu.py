"""kvq_attend_prompt's binding refuses a token stride that its 32-bit field
cannot hold (it was cut to its low bits, another stride)."""
import pytest
import torch

from decode_attention_quantized_gb300 import kvq


def rows(stride, H=2, D=64):
    return torch.empty_strided((2, H, D), (stride, D, 1), dtype=torch.bfloat16, device="meta")


@pytest.mark.parametrize("stride", [128, 136, 2 ** 31 - 8])
def test_strides_that_fit(stride):
    assert kvq._rows("q", rows(stride), (2, 2, 64), rows(stride).get_device())[1] == stride


@pytest.mark.parametrize("stride", [64, 120, 2 ** 31, 2 ** 32 + 128, 2 ** 33])
def test_strides_that_do_not(stride):
    with pytest.raises(ValueError):
        kvq._rows("q", rows(stride), (2, 2, 64), rows(stride).get_device())
