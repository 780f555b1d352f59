"""Which blocks of few rows take the kernel whose products are exact: by the sizes,
as fp8q_gemm_swiglu_workspace tells, and each side with its own accuracy."""

import pytest
import torch

import fp8_fine_grained_quant_amd as fq

# (rows, width, inner), exact: of 256 compute units
SIZES = [((8, 4096, 128), True), ((8, 4224, 128), False), ((8, 8192, 128), False), ((1, 32768, 128), False),
         ((16, 6144, 1024), True), ((16, 6272, 1024), False), ((16, 8192, 1024), True), ((16, 8320, 1024), False),
         ((1, 22528, 7168), True), ((1, 22656, 7168), False), ((16, 32768, 7168), False),
         ((16, 53248, 16384), True), ((3, 65536, 16384), True), ((17, 2048, 7168), True), ((128, 2048, 7168), True),
         ((256, 2048, 7168), False)]


def units():
    return torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 256


@pytest.mark.parametrize("size, exact", SIZES, ids=str)
def test_rule(size, exact):
    if units() != 256:
        pytest.skip("the sizes are those of 256 compute units")
    m, f, _ = size
    assert fq.gemm_swiglu_workspace(*size, True) == (m * f * 4 if exact else 0)
    assert fq.gemm_swiglu_workspace(*size, False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(8, 4096, 128), (8, 4224, 128), (8, 8192, 128), (3, 16384, 256), (16, 6144, 1024),
                                  (16, 6272, 1024), (16, 8192, 1024), (9, 8320, 1024)], ids=str)
def test_accuracy_on_either_side(size):
    from test_gpu_swiglu import check_block, few, operands
    ops = operands(*size)
    check_block(*ops, *fq.gemm_swiglu_quant(*ops, with_output=True, with_gu=True), exact=few(*size))
