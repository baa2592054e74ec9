"""Row-major microscaled matrices, as checkpoints are published, into blocks: the
moves that README.md and include/q4.h give, against the reference's packing."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_reference as ref


def _row_major(w):
    """Codes [N, K / 2] and exponent bytes [N, K / 32] of w [N, K], byte by byte
    out of the reference's blocks."""
    N, K = w.shape
    codes, scales = ref.pack(w)
    rc, rs = np.zeros((N, K // 2), np.uint8), np.zeros((N, K // 32), np.uint8)
    for n in range(N):
        for kb in range(K // 128):
            rc[n, 64 * kb:64 * kb + 64] = codes[n // 128, kb, n % 128]
            for g in range(4):
                rs[n, 4 * kb + g] = scales[n // 128, kb, ref.scale_at(n % 128, g)]
    return rc, rs, codes, scales


@pytest.mark.parametrize("N,K", [(128, 128), (256, 640), (384, 256)])
def test_row_major_to_blocks(N, K):
    rng = np.random.default_rng(N + K)
    w = rng.standard_normal((N, K)) * 2.0 ** rng.integers(-6, 6, (N, 1))
    rc, rs, codes, scales = _row_major(w)
    # the row-major form is the published one: even k in the low nibble, one byte for 32 k
    k = np.arange(K)
    value = ref.GRID[(rc[:, k // 2] >> (4 * (k % 2))) & 7] * np.where((rc[:, k // 2] >> (4 * (k % 2))) & 8, -1.0, 1.0)
    assert np.array_equal(value * 2.0 ** (rs[:, k // 32].astype(float) - 127), ref.unpack(codes, scales, N, K))
    rc, rs = torch.from_numpy(rc), torch.from_numpy(rs)
    cm = rc.view(N // 128, 128, K // 128, 64).permute(0, 2, 1, 3).contiguous()
    sm = rs.view(N // 128, 4, 32, K // 128, 4).permute(0, 3, 2, 1, 4).reshape(N // 128, K // 128, 512)
    assert np.array_equal(cm.numpy(), codes) and np.array_equal(sm.numpy(), scales)
