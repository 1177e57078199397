"""Rows at the edges of the forms that the quantiser and the gating choose by length:
one wave or several to a row, pieces held in registers, H held in LDS or not."""
import pytest

import test_gpu_int8 as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1008, 2048, 2064, 4096, 4112, 8192, 8208, 12288, 12304, 16368, 32768, 32784])
def test_rows(K):
    base.test_rows_from_bf16_are_exact(9, K)


@pytest.mark.parametrize("K", [16, 1024, 1040, 2064, 8208, 12304, 16400, 32784, 65536])
def test_rows_from_fp32(K):
    base.test_rows_from_fp32(5, K)


@pytest.mark.parametrize("I", [512, 576, 8192, 8256, 14336, 14400, 39936, 40064])
@pytest.mark.parametrize("save", [True, False])
def test_gating(I, save):
    base.test_gating_forward(4, I, save)
