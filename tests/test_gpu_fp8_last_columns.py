"""8-bit floating-point products whose last column tile has few columns, behind the last expert's weights."""

import pytest
import torch

import moe_expert_grouped_group_amd as mx
from test_gpu_ragged_fp8 import BF, HF, _case, _check, _ms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [8, 16, 24, 264, 272, 520, 1032])
@pytest.mark.parametrize("k", [144, 240, 1040])
def test_last_columns(n, k):
    """Tiles (more than 256 rows an expert) of 8, 16 and 24 columns, with a second stage and without."""
    for splits in ([300], [257, 0, 700]):
        case = _case(sum(splits), splits, k, n)
        for dtype in (BF, HF):
            _check(*case, splits, None, mx.ragged_gemm_fp8(*case, _ms(splits), out_dtype=dtype))
