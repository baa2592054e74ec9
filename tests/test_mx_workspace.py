"""Workspace sizes of the microscaled products, on the host: a workspace made
for the largest batch serves every smaller one."""
from __future__ import annotations

import numpy as np
import pytest

import weight_only_bit_gemv_b200 as q4

A = 1 << 20          # an aligned fake address; never dereferenced

MATRICES = [(1, 1), (128, 128), (128, 11008), (4096, 4096), (333, 2000), (4096, 14336), (28672, 8192), (57344, 8192),
            (128256, 4096), (130, 1500), (1 << 20, 100), (64, 1 << 20)]


@pytest.mark.parametrize("N,K", MATRICES)
def test_gemm_sizes_never_fall(N, K):
    last = 0
    for M in [*range(1, 500), *range(500, 5000, 37), 8192, 65536]:
        need = q4.q4_gemm_mx_workspace(M, N, K)
        if need == -1:                       # more units than the call takes
            break
        assert need >= last and need % 16 == 0, (M, need, last)
        last = need


@pytest.mark.parametrize("E", [2, 3, 8, 60, 64, 256, 1024])
@pytest.mark.parametrize("N,K", [(128, 128), (2048, 4096), (28672, 4096), (1408, 2048), (130, 28672), (40000, 128), (3000, 300)])
def test_expert_sizes_never_fall(E, N, K):
    if E * -(-N // 128) * -(-K // 128) > 16777215:
        pytest.skip("more blocks than a stack may have")
    rng = np.random.default_rng(E + N)
    counts = sorted({*range(1, 40), *(f * E + d for f in (1, 2, 8, 16, 64, 120) for d in (-1, 0, 1)), *rng.integers(1, 130 * E, 300).tolist()})
    last = 0
    for T in counts:
        need = q4.q4_gemm_experts_workspace(T, E, N, K)
        assert need >= last and need % 16 == 0, (T, need, last)
        last = need


def test_few_tokens_need_none():
    """Where every smaller batch runs in one launch, too."""
    for M, N, K in ((1, 4096, 4096), (8, 4096, 4096), (8, 28672, 4096), (1, 128256, 4096), (1, 28672, 8192)):
        assert q4.q4_gemm_mx_workspace(M, N, K) == 0
    assert q4.q4_gemm_experts_workspace(8, 8, 28672, 4096) == 0


def test_a_workspace_for_more_tokens_is_enough():
    """The calls check against the same sizes: with that of M they refuse no
    smaller batch for its workspace.  (They stop at a misaligned x, checked before.)"""
    lib = q4.load()
    for N, K in MATRICES[:10]:
        for M in (13, 121, 125, 250):
            need = lib.q4_gemm_mx_workspace(M, N, K)
            for m in (1, 4, 8, 12, 64, 120, 121):
                if m <= M:
                    assert lib.q4_gemm_mx_workspace(m, N, K) <= need
            if need:
                assert lib.q4_gemm_mx(A, A, A, A, 0, M, N, K, A, need - 1, None) == 6
                assert lib.q4_gemm_mx(A, A, A + 8, A, 0, M, N, K, A, need, None) == 3


@pytest.mark.gpu
def test_one_workspace_for_all_batches():
    """Batches of every tile size, one after the other in the workspace of the
    largest, give the bits that workspaces of their own give."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(0)
    N, K, E = 300, 1500, 5
    nb, kb = -(-N // 128), -(-K // 128)
    codes = torch.from_numpy(rng.integers(0, 256, (E, nb, kb, 128, 64), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(118, 125, (E, nb, kb, 512), dtype=np.uint8)).cuda()
    x = torch.from_numpy(rng.standard_normal((700, K))).to(torch.bfloat16).cuda()
    ws = torch.full((q4.q4_gemm_mx_workspace(300, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    for M in (300, 121, 120, 64, 13, 8, 1, 250, 9, 65):
        want = q4.q4_gemm_mx(codes[0], scales[0], x[:M], N=N)
        assert torch.equal(q4.q4_gemm_mx(codes[0], scales[0], x[:M], N=N, workspace=ws), want), M
    ws = torch.full((q4.q4_gemm_experts_workspace(700, E, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    for T in (700, 11, 10, 41, 40, 3, 81, 321, 80):
        ids = torch.from_numpy(rng.integers(0, E, (T, 1))).cuda()
        offsets, rows, _ = q4.q4_sort_experts(ids, E)
        want = q4.q4_gemm_experts(codes, scales, x[:T], offsets, rows, N=N)
        assert torch.equal(q4.q4_gemm_experts(codes, scales, x[:T], offsets, rows, N=N, workspace=ws), want), T
