"""The accuracy that include/q4.h states for the microscaled products: its
arithmetic redone on the host, and the products on the GPU, with x that stands
far out of its group where W is zero."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_reference as ref
import weight_only_bit_gemv_b200 as q4


def stated_bound(w, x, dtype):
    """include/q4.h: c * S + 2^-22 * D, then the rounding to bfloat16, for W
    [N, K] and x [M, K] in 64 bits, K up to 2^18.

    c counts, in 2^-24 S: 33 for each step of 32 k (32 exact products and the
    accumulator, aligned to the largest and cut below 2^-24 of it), 32 steps a
    reading for binary32 and 256 for bfloat16; one for each reading added in
    binary32, hi and lo once more, and one for each of at most 64 parts:
    33 * 32 + 2^18 / 1024 + 66 = 1378, or 8.3e-5 <= 1e-4, and
    33 * 256 + 2^18 / 8192 + 66 = 8546, or 5.1e-4 <= 5.2e-4."""
    absw, absx = np.abs(w), np.abs(x)
    K = w.shape[1]
    top = np.pad(absx, ((0, 0), (0, -K % 32))).reshape(len(x), -1, 32).max(-1)
    D = np.repeat(top, 32, axis=1)[:, :K] @ absw.T
    bound = (1e-4 if dtype == torch.float32 else 5.2e-4) * (absx @ absw.T) + 2.0 ** -22 * D + 2.0 ** -126
    if dtype == torch.bfloat16:
        bound = bound + torch.finfo(dtype).eps / 2 * (np.abs(x @ w.T) + bound)
    return bound


def _e4m3(v):
    return torch.from_numpy(np.clip(v, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()


def two_parts(x):
    """x [M, K] in 64 bits, K a multiple of 32, as s * hi + s / 32 * lo."""
    g = x.reshape(-1, 32)
    s = 2.0 ** (np.frexp(np.abs(g).max(1, keepdims=True))[1] - 1 - 7)
    hi = _e4m3(g / s)
    return (s * hi + s / 32 * _e4m3((g / s - hi) * 32)).reshape(x.shape)


def _spiky(rng, M, K, octaves):
    """x of ordinary size with one 2^octaves times as large in each 32, and
    where they are."""
    x = rng.uniform(1, 2, (M, K)) * rng.choice([-1.0, 1.0], (M, K))
    spike = np.arange(K) % 32 == rng.integers(0, 32, K // 32).repeat(32)
    x[:, spike] = 2.0 ** octaves
    return torch.from_numpy(x).to(torch.bfloat16), spike


@pytest.mark.parametrize("octaves", [0, 13, 14, 15, 16, 20, 24, 40])
def test_split_of_x(octaves):
    """Exact from 2^-14 of the group's largest on, else within 2^-22 of it; the
    bits that a neighbour of a spike keeps; and nothing lost by a row that is
    passed as two."""
    x, spike = _spiky(np.random.default_rng(octaves), 8, 256, octaves)
    x = x.double().numpy()
    err = np.abs(two_parts(x) - x)
    top = np.repeat(np.abs(x).reshape(8, -1, 32).max(-1), 32, axis=1)
    assert not err[np.abs(x) >= 2.0 ** -14 * top].any()
    assert np.all(err <= 2.0 ** -22 * top)
    worst = (err / np.abs(x)).max()
    for o, bits in ((15, 7), (20, 2)):
        if octaves == o:
            assert worst <= 2.0 ** -bits
    if octaves >= 24:
        assert not two_parts(x)[:, ~spike].any()
    for keep in (spike, ~spike):
        part = np.where(keep, x, 0.0)
        assert np.array_equal(two_parts(part), part)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 16, 40, 100])
@pytest.mark.parametrize("octaves", [3, 15, 18, 24])
def test_spikes_under_zero_codes(M, octaves):
    """W is zero at each group's spike: y within the stated bound, and within
    its first term for rows passed as two."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(M * 100 + octaves)
    N, K = 200, 1024
    x, spike = _spiky(rng, M, K, octaves)
    w = rng.choice([-1.5, -1.0, 0.5, 1.0, 3.0, 6.0], (N, K)) * 2.0 ** -7
    w[:, spike] = 0
    codes, scales = (torch.from_numpy(v).cuda() for v in ref.pack(w))
    w = ref.unpack(codes.cpu().numpy(), scales.cpu().numpy(), N, K)
    assert not w[:, spike].any()
    x64 = x.double().numpy()
    for dtype in (torch.float32, torch.bfloat16):
        y = q4.q4_gemm_mx(codes, scales, x.cuda(), N=N, dtype=dtype)
        assert np.all(np.abs(y.double().cpu().numpy() - x64 @ w.T) <= stated_bound(w, x64, dtype))
    here = torch.from_numpy(spike)
    two = torch.cat([torch.where(here, x, 0), torch.where(here, 0, x)]).to(torch.bfloat16)
    y = q4.q4_gemm_mx(codes, scales, two.cuda(), N=N)
    y = (y[:M] + y[M:]).double().cpu().numpy()
    # the sum of the two rounds once more, 2^-24 of it: within 1e-4 S with 8.3e-5 S counted
    assert np.all(np.abs(y - x64 @ w.T) <= 1e-4 * (np.abs(x64) @ np.abs(w).T) + 2.0 ** -126)
