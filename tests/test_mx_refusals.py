"""What the microscaled and expert-routing calls refuse, on the host: every
call here returns from argument checks before any CUDA call."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_reference as ref
import weight_only_bit_gemv_b200 as q4

OK, NULL, SHAPE, ALIGN, TOO_LARGE = 0, 1, 2, 3, 6
A = 1 << 20          # an aligned fake address; never dereferenced
MIS = A + 8
HALF = A + 16        # 16-byte aligned, not 32
BIG = 1 << 40        # a workspace size no call exceeds


@pytest.fixture(scope="module")
def lib():
    return q4.load()


@pytest.mark.parametrize("name", ["q4_pack_mx", "q4_dequant_mx"])
def test_pack_and_dequant(lib, name):
    def f(a, b, c, type_, E, N, K):
        args = (a, type_, b, c) if name == "q4_pack_mx" else (a, b, c, type_)
        return getattr(lib, name)(*args, E, N, K, None)
    assert f(A, A, A, 0, 1, 4, 0) == SHAPE
    assert f(A, A, A, 0, 1, 4, (1 << 20) + 1) == SHAPE
    assert f(A, A, A, 0, 1, -1, 64) == SHAPE
    assert f(A, A, A, 0, -1, 4, 64) == SHAPE
    assert f(A, A, A, 3, 1, 4, 64) == SHAPE                 # no such type
    assert f(A, A, A, -1, 1, 4, 64) == SHAPE
    assert f(A, A, A, 0, 1, 1 << 30, 1 << 20) == SHAPE      # more blocks than Q4_MX_MAX_BLOCKS
    assert f(A, A, A, 0, 1 << 30, 1, 1) == SHAPE
    assert f(None, None, None, 0, 1, 0, 64) == OK
    assert f(None, None, None, 0, 0, 5, 64) == OK
    for i in range(3):
        args = [A, A, A]
        args[i] = None
        assert f(*args, 0, 1, 4, 1) == NULL
        args[i] = MIS
        assert f(*args, 0, 1, 4, 1) == ALIGN


def test_gemm(lib):
    def f(codes=A, scales=A, x=A, y=A, type_=0, M=40, N=64, K=96, ws=A, bytes_=BIG):
        return lib.q4_gemm_mx(codes, scales, x, y, type_, M, N, K, ws, bytes_, None)
    assert f(M=-1) == SHAPE
    assert f(N=-1) == SHAPE
    assert f(K=0) == SHAPE
    assert f(K=(1 << 20) + 1) == SHAPE
    assert f(M=(1 << 30) + 1) == SHAPE
    assert f(type_=2) == SHAPE                               # y is never binary16
    assert f(M=0, codes=None, x=None, y=None, ws=None) == OK
    assert f(N=0, codes=None, x=None, y=None, ws=None) == OK
    for name in ("codes", "scales", "x", "y", "ws"):
        assert f(**{name: None}) == NULL
        assert f(**{name: MIS}) == ALIGN
    assert f(codes=HALF) == ALIGN
    need = lib.q4_gemm_mx_workspace(40, 64, 96)
    assert need > 0 and f(bytes_=need - 1) == TOO_LARGE
    assert lib.q4_gemm_mx_workspace(-1, 64, 96) == -1
    assert lib.q4_gemm_mx_workspace(4, 64, 0) == -1
    assert lib.q4_gemm_mx_workspace(0, 64, 96) == 0


def test_gemm_experts(lib):
    def f(codes=A, scales=A, x=A, rows=A, offsets=A, y=A, type_=1, Mx=4, T=80, E=3, N=64, K=96, ws=A, bytes_=BIG):
        return lib.q4_gemm_experts(codes, scales, x, rows, offsets, y, type_, Mx, T, E, N, K, ws, bytes_, None)
    assert f(E=0) == SHAPE
    assert f(E=1025) == SHAPE
    assert f(T=-1) == SHAPE
    assert f(Mx=-1) == SHAPE
    assert f(T=(1 << 30) + 1) == SHAPE
    assert f(rows=None) == SHAPE                             # then x has T rows
    assert f(rows=None, Mx=80, offsets=None) == NULL
    assert f(T=0, codes=None) == OK
    for name in ("codes", "scales", "x", "offsets", "y", "ws"):
        assert f(**{name: None}) == NULL
    for name in ("codes", "scales", "x", "rows", "offsets", "y", "ws"):
        assert f(**{name: MIS}) == ALIGN
    need = lib.q4_gemm_experts_workspace(80, 3, 64, 96)
    assert need > 0 and f(bytes_=need - 1) == TOO_LARGE
    assert lib.q4_gemm_experts_workspace(8, 1025, 64, 96) == -1


def test_sort(lib):
    def f(ids=A, offsets=A, rows=A, places=A, M=4, top=2, E=8):
        return lib.q4_sort_experts(ids, 0, offsets, rows, places, M, top, E, None)
    assert f(M=-1) == SHAPE
    assert f(top=0) == SHAPE
    assert f(E=0) == SHAPE
    assert f(E=1025) == SHAPE
    assert f(M=1 << 30, top=2) == SHAPE                      # T above 2^31 - 1
    assert f(offsets=None, M=0) == NULL
    for name in ("ids", "offsets", "rows", "places"):
        assert f(**{name: None}) == NULL
        assert f(**{name: MIS}) == ALIGN


def test_row_movement(lib):
    calls = {
        "q4_dispatch": lambda p, t, M, top, K: lib.q4_dispatch(*p[:3], t, M, top, K, None),
        "q4_combine": lambda p, t, M, top, K: lib.q4_combine(p[0], p[1], p[3], p[2], t, M, top, K, None),
        "q4_combine_grad": lambda p, t, M, top, K: lib.q4_combine_grad(*p[:6], t, M, top, K, None),
    }
    for name, f in calls.items():
        good = [A] * 6
        assert f(good, 3, 4, 2, 64) == SHAPE
        assert f(good, 0, -1, 2, 64) == SHAPE
        assert f(good, 0, 4, 0, 64) == SHAPE
        assert f(good, 0, 4, 2, 0) == SHAPE
        assert f(good, 0, 4, 2, (1 << 20) + 1) == SHAPE
        assert f(good, 0, 1 << 30, 4, 64) == SHAPE
        assert f([None] * 6, 0, 0, 2, 64) == OK
        for i in range({"q4_dispatch": 3, "q4_combine": 3, "q4_combine_grad": 6}[name]):
            bad = list(good)
            bad[i] = None
            assert f(bad, 0, 4, 2, 64) == NULL, (name, i)
            bad[i] = MIS
            assert f(bad, 0, 4, 2, 64) == ALIGN, (name, i)


def test_binding_refuses():
    codes, scales = torch.zeros(1, 1, 128, 64, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8)
    x = torch.zeros(2, 100, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                          # host tensors
        q4.q4_gemm_mx(codes, scales, x)
    with pytest.raises(ValueError):                          # K of another number of blocks
        q4.q4_gemm_mx(codes, scales, torch.zeros(2, 129, dtype=torch.bfloat16))
    with pytest.raises(ValueError):                          # N of another number of blocks
        q4.q4_gemm_mx(codes, scales, x, N=129)
    with pytest.raises(ValueError):                          # not blocks
        q4.q4_gemm_mx(codes[0, 0], scales, x)
    with pytest.raises(TypeError):
        q4.q4_pack_mx(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        q4.q4_pack_mx(torch.zeros(64))
    with pytest.raises(TypeError):                           # ids are whole numbers
        q4.q4_sort_experts(torch.zeros(4, 2), 8)
    with pytest.raises(ValueError):
        q4.q4_sort_experts(torch.zeros(4, dtype=torch.int32), 8)
    places = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):                          # x has another number of tokens
        q4.q4_dispatch(torch.zeros(3, 8), places)
    with pytest.raises(ValueError):                          # ys has not M * top rows
        q4.q4_combine(torch.zeros(7, 8), places)
    with pytest.raises(ValueError):                          # host tensors
        q4.q4_combine_grad(torch.zeros(4, 8), torch.zeros(8, 8), places, torch.zeros(4, 2))


def test_reference_round_trip():
    """The tests' own reference: values on the grid survive, and padding reads back as zeros."""
    rng = np.random.default_rng(0)
    w = ref.GRID[rng.integers(0, 8, (130, 70))] * rng.choice([-1.0, 1.0], (130, 70)) * 2.0 ** -9
    w[:, ::32] = 6 * 2.0 ** -9                               # every group's scale is 2^-9
    codes, scales = ref.pack(w)
    assert codes.shape == (2, 1, 128, 64) and scales.shape == (2, 1, 512)
    assert np.array_equal(ref.unpack(codes, scales, 130, 70), w)
    assert not ref.unpack(codes, scales, 256, 128)[130:].any()
