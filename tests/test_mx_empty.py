"""Products of rows that name no row of x at all."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import weight_only_bit_gemv_b200 as q4

A = 1 << 20          # an aligned fake address; never dereferenced


def test_x_without_rows_may_be_null():
    """Every row index is outside an x of no rows: the rows are zeros, and there
    is no address.  (The call stops at misaligned offsets, checked after NULL.)"""
    f = q4.load().q4_gemm_experts
    assert f(A, A, None, A, A + 8, A, 0, 0, 80, 3, 64, 96, A, 1 << 40, None) == 3
    assert f(A, A, None, A, A, A, 0, 1, 80, 3, 64, 96, A, 1 << 40, None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 100])
def test_rows_of_no_x_are_zeros(T):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(T)
    codes = torch.from_numpy(rng.integers(0, 256, (2, 1, 2, 128, 64), dtype=np.uint8)).cuda()
    scales = torch.full((2, 1, 2, 512), 120, dtype=torch.uint8, device="cuda")
    x = torch.empty(0, 200, dtype=torch.bfloat16, device="cuda")
    rows = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    rows[T // 2] = 0
    offsets = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    y = torch.full((T, 100), float("nan"), device="cuda")
    q4.q4_gemm_experts(codes, scales, x, offsets, rows, y=y, N=100)
    assert not y.any() and not y.isnan().any()
