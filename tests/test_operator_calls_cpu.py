"""Calls of the norm, grouped and few-row operators that a binding has to refuse
or to arrange on the host, without a GPU."""
import os

import pytest
import torch

import fp4_precision_gemms_amd as F


@pytest.fixture(autouse=True)
def built():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("lead_codes,lead_scales", [((3,), (3,)), ((1,), (1,)), ((2, 3), (2, 3)), ((3,), (2,))])
def test_decode_refuses_stacks_of_activations(lead_codes, lead_scales):
    """One operand a call: a stack would lose all but its first."""
    M, N, K = 40, 64, 96
    w = u8(*F.code_shape(N, K)), u8(*F.scale_shape(N, K))
    with pytest.raises(ValueError, match="a codes must have two .* or three"):
        F.fp4_gemm_decode(u8(*lead_codes, *F.code_shape(M, K)), u8(*lead_scales, *F.scale_shape(M, K)), *w)


def test_decode_refuses_activations_of_one_dimension():
    w = u8(*F.code_shape(64, 96)), u8(*F.scale_shape(64, 96))
    with pytest.raises(ValueError, match="a codes must have two .* or three"):
        F.fp4_gemm_decode(u8(96), u8(3), *w)
