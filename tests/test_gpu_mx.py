"""Microscaled 4-bit matrices on the GPU against the 64-bit reference: pack and
dequant bit for bit, products within a bound counted from the arithmetic
(mx_reference.tolerance) and exactly where every sum is exact."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mx_reference as ref
import weight_only_bit_gemv_b200 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    q4.load()
    yield
    torch.cuda.synchronize()
    assert q4.timeout_flags() == 0


def _f64(t):
    return t.detach().double().cpu().numpy()


def _packed(rng, N, K, E=None):
    """Random packed matrices, on the GPU and as 64-bit values: every code, and
    a spread of scales."""
    nb, kb = -(-N // 128), -(-K // 128)
    codes = rng.integers(0, 256, (E or 1, nb, kb, 128, 64), dtype=np.uint8)
    scales = rng.integers(118, 125, (E or 1, nb, kb, 512), dtype=np.uint8)
    values = [ref.unpack(c, s, N, K) for c, s in zip(codes, scales)]
    codes, scales = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    return (codes[0], scales[0], values[0]) if E is None else (codes, scales, values)


def _x(rng, M, K, spread=1.0):
    x = torch.from_numpy(rng.standard_normal((M, K)) * spread * np.where(rng.random(K) < 0.01, 30, 1))
    return x.to(torch.bfloat16).cuda()


def _close(y, w, x):
    """y against x @ w.T within the counted bound."""
    want = _f64(x) @ w.T
    err = np.abs(_f64(y) - want)
    bound = ref.tolerance(w, _f64(x), y.dtype)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3g} of the bound"
    if y.dtype == torch.float32 and want.size >= 1024:
        # truncation takes up to 2^-23 of the accumulator a step, 2^-24 on average, for 32 steps
        assert np.linalg.norm(err) <= 32 * 2.0 ** -24 * np.linalg.norm(want)


# ---- pack and dequant ---------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 31), (128, 128), (129, 130), (257, 72), (40, 1000)])
def test_pack_bits(N, K, dtype):
    rng = np.random.default_rng(N * K)
    w = torch.from_numpy(rng.standard_normal((N, K)) * 2.0 ** rng.integers(-8, 8, (N, 1))).to(dtype)
    w[rng.random((N, K)) < 0.1] = 0
    codes, scales = q4.q4_pack_mx(w.cuda())
    want = ref.pack(_f64(w))
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])
    back = q4.q4_dequant_mx(codes, scales, N=N, K=K, dtype=dtype)
    assert back.dtype == dtype and np.array_equal(_f64(back), _f64(torch.from_numpy(ref.unpack(*want, N, K)).to(dtype)))


def test_pack_rounding_and_edges():
    """Every tie of the grid in either sign, saturation, zero and subnormal
    groups, the largest numbers, and groups with an infinity or NaN."""
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = np.concatenate([ties, np.nextafter(np.float32(ties), np.float32(0)), np.nextafter(np.float32(ties), np.float32(9))])
    for top in (4.0, 7.99):
        g = np.concatenate([[top], near, [0.0, -0.0]])
        rows.append(np.pad(np.concatenate([g, -near[:32 - len(g)]]), (0, 0)))
    rows.append(np.zeros(32))
    rows.append(np.full(32, -0.0))
    rows.append(np.linspace(0, 1.4e-44, 32))                   # subnormal
    rows.append(np.linspace(-2.0 ** -124, 2.0 ** -124, 32))    # scales at the lowest byte
    rows.append(np.linspace(-3.4e38, 3.4e38, 32))
    for odd in (np.inf, -np.inf, np.nan):
        r = np.linspace(-1, 1, 32)
        r[5] = odd
        rows.append(r)
    w = np.float32(np.stack([np.resize(r, 32) for r in rows]))
    codes, scales = q4.q4_pack_mx(torch.from_numpy(w).cuda())
    want = ref.pack(w)
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])
    back = _f64(q4.q4_dequant_mx(codes, scales, N=len(rows), K=32))
    np.testing.assert_array_equal(back, ref.unpack(*want, len(rows), 32))


def test_dequant_every_code_and_byte():
    """All 16 codes under all 256 exponent bytes, in the three types."""
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (2, 2, 128, 64), dtype=np.uint8)
    scales = np.arange(2 * 2 * 512, dtype=np.uint32).astype(np.uint8).reshape(2, 2, 512)
    want = torch.from_numpy(ref.unpack(codes, scales, 256, 256))
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        got = q4.q4_dequant_mx(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), dtype=dtype)
        torch.testing.assert_close(got.cpu(), want.float().to(dtype), rtol=0, atol=0, equal_nan=True)


def test_pack_stack_and_guards():
    """A stack of matrices packs as its members do, and nothing is written outside the outputs."""
    rng = np.random.default_rng(4)
    E, N, K = 3, 130, 200
    w = torch.from_numpy(rng.standard_normal((E, N, K))).float()
    codes = torch.full((E * 2 * 2 * 8192 + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((E * 2 * 2 * 512 + 512,), 0xCD, dtype=torch.uint8, device="cuda")
    c, s = codes[256:-256].view(E, 2, 2, 128, 64), scales[256:-256].view(E, 2, 2, 512)
    q4.q4_pack_mx(w.cuda(), c, s)
    for e in range(E):
        want = ref.pack(w[e].numpy())
        assert np.array_equal(c[e].cpu().numpy(), want[0]) and np.array_equal(s[e].cpu().numpy(), want[1])
    for buf, v in ((codes, 0xAB), (scales, 0xCD)):
        assert (buf[:256] == v).all() and (buf[-256:] == v).all()
    out = torch.full((E * N * K + 64,), 7.0, device="cuda")
    q4.q4_dequant_mx(c, s, out[32:-32].view(E, N, K), N=N, K=K)
    assert (out[:32] == 7).all() and (out[-32:] == 7).all()


# ---- one matrix -----------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 24, 25, 32, 33, 40, 49, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (200, 130), (384, 1024)])
def test_gemm(M, N, K):
    rng = np.random.default_rng(M * 1000 + N)
    codes, scales, w = _packed(rng, N, K)
    x = _x(rng, M, K)
    for dtype in (torch.float32, torch.bfloat16):
        y = q4.q4_gemm_mx(codes, scales, x, N=N, dtype=dtype)
        assert y.dtype == dtype and y.shape == (M, N)
        _close(y, w, x)


@pytest.mark.parametrize("M,N,K", [(1, 128, 28672), (3, 4096, 4096), (40, 130, 14336), (200, 1000, 8200), (1, 20000, 160)])
def test_gemm_long_and_wide(M, N, K):
    """K cut over many thread blocks, and many row blocks of W."""
    rng = np.random.default_rng(K + N)
    codes, scales, w = _packed(rng, N, K)
    x = _x(rng, M, K)
    _close(q4.q4_gemm_mx(codes, scales, x, N=N), w, x)
    _close(q4.q4_gemm_mx(codes, scales, x, N=N, dtype=torch.bfloat16), w, x)


@pytest.mark.parametrize("M", [1, 3, 8, 13])
@pytest.mark.parametrize("N,K", [(128, 3000), (130, 1500), (5000, 1408), (4096, 4096), (128, 11008), (20000, 2304), (18900, 4224)])
def test_gemm_few_tokens(M, N, K):
    """Every split of K over a tile's thread blocks, rings that go round many
    times, one tile and several for a block, and K of an odd number of blocks."""
    rng = np.random.default_rng(M + N + K)
    codes, scales, w = _packed(rng, N, K)
    for _ in range(3):
        x = _x(rng, M, K)
        _close(q4.q4_gemm_mx(codes, scales, x, N=N), w, x)


@pytest.mark.parametrize("M", [1, 5, 16, 31, 64, 130])
def test_gemm_exact_on_integers(M):
    """Whole-number x and scales of 1: every sum is a multiple of 1/2 below
    2^20, so y is exact, whatever the order."""
    rng = np.random.default_rng(M)
    N, K = 300, 1184
    codes = torch.from_numpy(rng.integers(0, 256, (3, 10, 128, 64), dtype=np.uint8)).cuda()
    scales = torch.full((3, 10, 512), 127, dtype=torch.uint8, device="cuda")
    x = torch.from_numpy(rng.integers(-128, 129, (M, K))).to(torch.bfloat16).cuda()
    w = ref.unpack(codes.cpu().numpy(), scales.cpu().numpy(), N, K)
    y = q4.q4_gemm_mx(codes, scales, x, N=N)
    assert np.array_equal(_f64(y), _f64(x) @ w.T)


def test_gemm_every_significant_bit_of_x():
    """One-hot W picks single x: the two parts of x give it back exactly where
    it is within 2^14 of its group's largest, else to 2^-22 of that: with the
    largest at 128 s or more, the low part's step is 2^-9 * s / 32, and half of
    it 2^-15 s <= 2^-22 of the largest."""
    K = 128
    rng = np.random.default_rng(3)
    w = np.zeros((K, K))
    np.fill_diagonal(w, 1.0)
    codes, scales = (torch.from_numpy(v).cuda() for v in ref.pack(w))
    x = torch.from_numpy(rng.uniform(1, 2, (64, K)) * 2.0 ** rng.integers(-24, 1, (64, K))
                         * rng.choice([-1.0, 1.0], (64, K))).to(torch.bfloat16)
    y = _f64(q4.q4_gemm_mx(codes, scales, x.cuda()))
    x = _f64(x)
    top = np.repeat(np.abs(x).reshape(64, 4, 32).max(-1), 32, axis=1)
    near = np.abs(x) >= top * 2.0 ** -14
    assert near.any() and (~near).any()
    assert np.array_equal(y[near], x[near])
    assert np.all(np.abs(y - x) <= top * 2.0 ** -22)


def test_gemm_extremes():
    """The smallest and largest exponents on either side, zero rows, and NaN scales or rows that stay where they are."""
    rng = np.random.default_rng(5)
    N, K = 256, 256
    codes = torch.from_numpy(rng.integers(0, 256, (2, 2, 128, 64), dtype=np.uint8))
    scales = torch.full((2, 2, 512), 127, dtype=torch.uint8)
    scales[1, 1, ref.scale_at(3, 2)] = 255                     # row 131 of W is NaN
    scales[0, :, ref.scale_at(9, 0)] = 0
    w = ref.unpack(codes.numpy(), scales.numpy(), N, K)
    x = _x(rng, 6, K)
    x[1] = 0
    x[2, 40] = float("nan")
    x[3, 40] = float("inf")
    x[4] *= 2.0 ** -120
    x[5] *= 2.0 ** 100
    y = _f64(q4.q4_gemm_mx(codes.cuda(), scales.cuda(), x))
    assert np.isnan(y[:, 131]).all() and np.isnan(y[2]).all() and np.isnan(y[3]).all()
    keep = np.ones(N, bool)
    keep[131] = False
    assert not y[1, keep].any()
    for m in (0, 4, 5):
        xm = _f64(x)[m:m + 1]
        assert np.all(np.abs(y[m:m + 1, keep] - xm @ w[keep].T) <= ref.tolerance(w[keep], xm, torch.float32))
    for b, factor in ((0, 2.0 ** 100), (254, 2.0 ** -60)):     # all scales at one end
        scales = torch.full((2, 2, 512), b, dtype=torch.uint8)
        w = ref.unpack(codes.numpy(), scales.numpy(), N, K)
        xb = (_x(rng, 3, K).double() * factor).to(torch.bfloat16)
        _close(q4.q4_gemm_mx(codes.cuda(), scales.cuda(), xb), w, xb)


@pytest.mark.parametrize("M", [1, 33, 150])
def test_gemm_outputs_workspace_and_stream(M):
    """A given y, workspace (of any contents) and stream; nothing written outside y; the same bits again."""
    rng = np.random.default_rng(M)
    N, K = 333, 2000
    codes, scales, w = _packed(rng, N, K)
    x = _x(rng, M, K)
    want = q4.q4_gemm_mx(codes, scales, x, N=N)
    need = q4.q4_gemm_mx_workspace(M, N, K)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    buf = torch.full((M * N + 64,), 3.5, device="cuda")
    y = buf[32:32 + M * N].view(M, N)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert q4.q4_gemm_mx(codes, scales, x, y=y, N=N, workspace=ws[256:-256], stream=side) is y
    side.synchronize()
    assert torch.equal(y, want)
    assert (buf[:32] == 3.5).all() and (buf[32 + M * N:] == 3.5).all()
    assert (ws[:256] == 0xFF).all() and (ws[-256:] == 0xFF).all()
    by_handle = q4.q4_gemm_mx(codes, scales, x, N=N, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(by_handle, want)
    if need > 0:                                               # few tokens need none
        with pytest.raises(q4.Q4Error) as e:
            q4.q4_gemm_mx(codes, scales, x, N=N, workspace=ws[:need - 16])
        assert e.value.status == 6


def test_gemm_in_graphs():
    """Two captured calls, each with the workspace of its own that the call
    allocated under capture, replayed on two streams at once on new inputs."""
    rng = np.random.default_rng(11)
    made, alive = [], []
    for M, N, K in ((4, 1000, 3000), (70, 500, 1500), (40, 300, 9000)):
        codes, scales, w = _packed(rng, N, K)
        x = _x(rng, M, K)
        q4.q4_gemm_mx(codes, scales, x, N=N)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = q4.q4_gemm_mx(codes, scales, x, N=N)
        made.append((g, x, y, w, torch.cuda.Stream()))
        alive.append((codes, scales))                          # the graph reads them
    for _ in range(3):
        for g, x, y, w, s in made:
            x.copy_(_x(rng, *x.shape))
            y.fill_(-1)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, x, y, w, s in made:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for g, x, y, w, s in made:
            _close(y, w, x)


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
import weight_only_bit_gemv_b200 as q4
from test_gpu_mx import _close, _packed, _x
torch.cuda.set_device(0)
rng = np.random.default_rng(1)
codes, scales, w = _packed(rng, 300, 700, 3)
x = [_x(rng, M, 700) for M in (2, 12, 30, 60, 150)]
ids = torch.from_numpy(rng.integers(0, 3, (2, 2))).cuda()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ys = [q4.q4_gemm_mx(codes[0], scales[0], v, N=300) for v in x]
    offsets, rows, places = q4.q4_sort_experts(ids, 3)
    out = q4.q4_combine(q4.q4_gemm_experts(codes, scales, x[0], offsets, rows, N=300), places)
g.replay()
torch.cuda.synchronize()
for v, y in zip(x, ys):
    _close(y, w[0], v)
print("captured")
"""


def test_first_calls_may_be_captured():
    """A process whose first calls of every kernel are made under capture."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "captured" in res.stdout, res.stdout + res.stderr


def test_gemm_empty():
    codes = torch.zeros(1, 1, 128, 64, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, 1, 512, dtype=torch.uint8, device="cuda")
    assert q4.q4_gemm_mx(codes, scales, torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")).shape == (0, 128)


def test_pack_then_gemm():
    """Weights packed on the GPU feed the product: y is x times the values they read back as."""
    rng = np.random.default_rng(8)
    wt = torch.from_numpy(rng.standard_normal((520, 777)) * 0.02).to(torch.bfloat16).cuda()
    codes, scales = q4.q4_pack_mx(wt)
    x = _x(rng, 12, 777)
    y = q4.q4_gemm_mx(codes, scales, x, N=520)
    _close(y, _f64(q4.q4_dequant_mx(codes, scales, N=520, K=777)), x)


# ---- rows grouped by expert ------------------------------------------------------

def _experts_close(y, w, x, offsets, rows):
    offsets = offsets.tolist()
    for e in range(len(w)):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            _close(y[a:b], w[e], x[rows[a:b].long()])
    assert not y[offsets[-1]:].any()


@pytest.mark.parametrize("M,top,E", [(1, 1, 1), (1, 2, 4), (5, 2, 8), (9, 4, 60), (40, 3, 7), (300, 2, 4), (130, 1, 1), (64, 8, 128)])
@pytest.mark.parametrize("N,K", [(130, 200), (384, 512)])
def test_experts(M, top, E, N, K):
    rng = np.random.default_rng(M * E + N)
    codes, scales, w = _packed(rng, N, K, E)
    x = _x(rng, M, K)
    ids = np.argsort(rng.random((M, E)) + 0.3 * rng.random(E), axis=1)[:, :top]
    offsets, rows, _ = q4.q4_sort_experts(torch.from_numpy(ids).cuda(), E)
    for dtype in (torch.float32, torch.bfloat16):
        _experts_close(q4.q4_gemm_experts(codes, scales, x, offsets, rows, N=N, dtype=dtype), w, x, offsets, rows)


@pytest.mark.parametrize("counts", [[0, 0, 0, 17], [33, 0, 0, 0], [0, 129, 0, 1], [0, 0, 0, 0], [1, 1, 1, 1], [0, 200, 5, 0]])
def test_experts_uneven(counts):
    """Experts without rows, all rows with one expert, and rows of no expert behind them."""
    rng = np.random.default_rng(sum(counts))
    N, K, E, behind = 200, 300, 4, 6
    codes, scales, w = _packed(rng, N, K, E)
    T = sum(counts) + behind
    x = _x(rng, T, K)
    offsets = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    y = torch.full((T, N), float("nan"), device="cuda")
    q4.q4_gemm_experts(codes, scales, x, offsets, y=y, N=N)
    _experts_close(y, w, x, offsets, torch.arange(T, device="cuda"))


def test_experts_bad_rows_and_offsets():
    """Row indexes outside x give zero rows; offsets out of order stay inside the arrays."""
    rng = np.random.default_rng(2)
    N, K, E = 130, 140, 3
    codes, scales, w = _packed(rng, N, K, E)
    x = _x(rng, 5, K)
    rows = torch.tensor([0, -1, 4, 5, 2, 1 << 30], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 3, 3, 6], dtype=torch.int32, device="cuda")
    y = q4.q4_gemm_experts(codes, scales, x, offsets, rows, N=N)
    for p, (e, r) in enumerate([(0, 0), (0, None), (0, 4), (2, None), (2, 2), (2, None)]):
        if r is None:
            assert not y[p].any()
        else:
            _close(y[p:p + 1], w[e], x[r:r + 1])
    for bad in ([0, 5, 2, 6], [0, 1 << 30, 3, 6], [0, -7, 4, 9], [4, 2, 1, 0]):
        buf = torch.full((6 * N + 64,), 2.0, device="cuda")
        q4.q4_gemm_experts(codes, scales, x, torch.tensor(bad, dtype=torch.int32, device="cuda"), rows.clamp(0, 4),
                           y=buf[32:-32].view(6, N), N=N)
        assert (buf[:32] == 2).all() and (buf[-32:] == 2).all()


def test_experts_many():
    """As many experts as there may be, most without rows."""
    rng = np.random.default_rng(6)
    E, N, K, T = 1024, 128, 128, 50
    codes, scales, w = _packed(rng, N, K, E)
    x = _x(rng, T, K)
    ids = torch.from_numpy(rng.integers(0, E, (T, 1))).cuda()
    ids[0], ids[1] = 0, E - 1
    offsets, rows, _ = q4.q4_sort_experts(ids, E)
    _experts_close(q4.q4_gemm_experts(codes, scales, x, offsets, rows, N=N), w, x, offsets, rows)
    with pytest.raises(ValueError):
        q4.q4_gemm_experts(codes[0], scales[0], x, offsets, rows)
    with pytest.raises(ValueError):
        q4.q4_gemm_mx(codes, scales, x)


def test_one_expert_is_the_plain_product():
    rng = np.random.default_rng(9)
    codes, scales, w = _packed(rng, 300, 640, 1)
    x = _x(rng, 50, 640)
    offsets = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    assert torch.equal(q4.q4_gemm_experts(codes, scales, x, offsets, N=300), q4.q4_gemm_mx(codes[0], scales[0], x, N=300))
