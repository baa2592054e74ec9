"""Paths of the microscaled calls that only larger matrices reach, at the
smallest sizes that do: several turns of a cluster, several tiles of a pair or
block, experts with more rows than a tile, and the pack and dequant kernels for
2-byte matrices of 1024 blocks and more.  References are computed on the GPU in
64 bits, from the formulas and by torch alone."""
from __future__ import annotations

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


def _values(codes, scales, N, K):
    """mx_reference.unpack on the GPU: W [N, K] in 64 bits."""
    nb, kb = codes.shape[:2]
    grid = torch.from_numpy(np.concatenate([ref.GRID, -ref.GRID])).cuda()
    powers = torch.from_numpy(np.append(ref.POWERS, np.nan)[:256]).cuda()
    spot = torch.tensor([[ref.scale_at(r, g) for g in range(4)] for r in range(128)], device="cuda")
    w = torch.empty(nb * 128, kb * 128, dtype=torch.float64, device="cuda")
    for b in range(nb):
        code = torch.stack([codes[b] & 15, codes[b] >> 4], -1).flatten(-2).long()
        factor = powers[scales[b][:, spot].long()]
        block = (grid[code].view(kb, 128, 4, 32) * factor[..., None]).view(kb, 128, 128)
        w[b * 128:(b + 1) * 128] = block.transpose(0, 1).reshape(128, -1)
    return w[:N, :K]


def _tolerance(w, x, out_dtype):
    """mx_reference.tolerance on the GPU, without its proof."""
    K = w.shape[1]
    absw, absx = w.abs(), x.abs()
    top = torch.nn.functional.pad(absx, (0, -K % 32)).unflatten(1, (-1, 32)).amax(2)
    split = top.repeat_interleave(32, 1)[:, :K] @ absw.T * 2.0 ** -22
    flush = 8 if out_dtype == torch.float32 else 64
    steps, rounds = min(-(-K // 32), 4 * flush), -(-K // (128 * flush)) + 64
    bound = absx @ absw.T * 2.0 ** -24 * (33 * steps + rounds) + split + 1e-37
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ((x @ w.T).abs() + bound)
    return bound


def _close(y, w, x):
    x = x.double()
    err = (y.double() - x @ w.T).abs()
    bound = _tolerance(w, x, y.dtype)
    assert torch.all(err <= bound), f"worst {(err / bound).max().item():.3g} of the bound"


def _packed(gen, N, K, E=None):
    nb, kb = -(-N // 128), -(-K // 128)
    lead = () if E is None else (E,)
    codes = torch.randint(0, 256, (*lead, nb, kb, 128, 64), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(118, 125, (*lead, nb, kb, 512), dtype=torch.uint8, device="cuda", generator=gen)
    return codes, scales


def _x(gen, M, K):
    x = torch.randn(M, K, device="cuda", generator=gen)
    return (x * (1 + 29 * (torch.rand(K, device="cuda", generator=gen) < 0.01))).bfloat16()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def test_reference_on_the_gpu():
    """_values and _tolerance are what mx_reference computes on the host."""
    codes, scales = _packed(_gen(0), 200, 300)
    x = _x(_gen(1), 5, 300)
    w = ref.unpack(codes.cpu().numpy(), scales.cpu().numpy(), 200, 300)
    assert np.array_equal(_values(codes, scales, 200, 300).cpu().numpy(), w)
    for dtype in (torch.float32, torch.bfloat16):
        want = ref.tolerance(w, x.double().cpu().numpy(), dtype)
        np.testing.assert_allclose(_tolerance(_values(codes, scales, 200, 300), x.double(), dtype).cpu().numpy(), want, rtol=1e-9)


def _decode_turns(M, N, K):
    """(CTAs a tile, turns of a cluster) of one matrix and M <= 16 tokens, by the
    rule beside decode_plan in csrc/q4_mx_gemm.cu; (0, 0): the other kernel."""
    Nb, Ku = -(-N // 128), -(-K // 256)
    tiles, stage = -(-M // 8) * Nb, 1.35 if M > 4 else 1.0
    least, best = Nb * Ku / 148 + (30 if M > 8 else 21), (0, 0)
    for split, most in ((1, 148), (2, 74), (4, 33)):
        turns = -(-tiles // most)
        cost = (turns * (-(-Ku // split) + 0.5) + (0 if split == 1 else 5)) * stage
        if cost < least:
            least, best = cost, (split, turns)
    return best


@pytest.mark.parametrize("M,N,K,split", [(1, 28672, 8192, 4), (3, 28500, 8192, 4), (13, 4864, 7040, 4), (13, 9728, 3456, 2),
                                         (1, 128256, 700, 1)])
def test_decode_turns(M, N, K, split):
    """A cluster's sums go through its two slots again and again, and whole tiles
    follow each other in a block: three turns at least, x another each time."""
    took, turns = _decode_turns(M, N, K)
    assert took == split and turns >= 3
    gen = _gen(M + N)
    codes, scales = _packed(gen, N, K)
    w = _values(codes, scales, N, K)
    for i in range(4):
        x = _x(gen, M, K)
        _close(q4.q4_gemm_mx(codes, scales, x, N=N, dtype=(torch.float32, torch.bfloat16)[i % 2]), w, x)


@pytest.mark.parametrize("M,N,K", [(250, 20000, 300), (130, 38000, 1200), (24, 40000, 500), (60, 20100, 1000), (33, 19000, 2200)])
def test_several_tiles_of_a_block(M, N, K):
    """More output tiles than pairs (74) or blocks (148), whole ones and cut
    ones after each other in one run."""
    pair = M > 64
    assert -(-N // (256 if pair else 128)) * -(-M // (120 if pair else 64)) > (2 * 74 if pair else 148)
    gen = _gen(M + N)
    codes, scales = _packed(gen, N, K)
    w = _values(codes, scales, N, K)
    for dtype in (torch.float32, torch.bfloat16):
        x = _x(gen, M, K)
        _close(q4.q4_gemm_mx(codes, scales, x, N=N, dtype=dtype), w, x)


@pytest.mark.parametrize("E,most", [(32, 9), (32, 40), (8, 9), (100, 150)])
@pytest.mark.parametrize("N,K", [(130, 200), (2000, 900)])
def test_experts_with_more_rows_than_a_tile(E, most, N, K):
    """An average share of at most two, where tiles hold 8 rows, and one expert
    with several tiles; rows of no expert behind."""
    gen = _gen(E + most + N)
    rng = np.random.default_rng(E + most)
    T = 2 * E
    counts = np.bincount(rng.integers(1, E, T - most - 5), minlength=E)
    counts[0] = most
    counts = np.roll(counts, E // 3)
    assert q4.q4_gemm_experts_workspace(T, E, N, K) == 0     # tiles of 8, in one launch
    codes, scales = _packed(gen, N, K, E)
    x = _x(gen, T, K)
    offsets = torch.tensor(np.cumsum([0, *counts]), dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((T, N), float("nan"), dtype=dtype, device="cuda")
        q4.q4_gemm_experts(codes, scales, x, offsets, y=y, N=N)
        for e in range(E):
            a, b = int(offsets[e]), int(offsets[e + 1])
            if b > a:
                _close(y[a:b], _values(codes[e], scales[e], N, K), x[a:b])
        assert not y[int(offsets[-1]):].any()


def _guarded(shape, dtype, value):
    """A buffer with 64 guard elements on either side, and its middle."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), value, dtype=dtype, device="cuda")
    return buf, buf[64:64 + n].view(shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(4200, 4200), (4096, 4096), (130, 65544), (3, 2500, 2312), (1025, 100, 8)])
def test_pack_and_dequant_of_large_matrices(shape, dtype):
    """2-byte matrices of 1024 blocks and more, odd numbers of blocks along K and
    stacks among them, have the bits that the same values have as binary32
    (whose kernel the small cases reach), and the reference's in their first
    and last rows; nothing is written outside the outputs."""
    lead, N, K = shape[:-2], *shape[-2:]
    nb, kb = -(-N // 128), -(-K // 128)
    assert int(np.prod(lead)) * nb * kb >= 1024 and K % 8 == 0
    gen = _gen(N + K)
    w = torch.randn(shape, device="cuda", generator=gen) * torch.exp2(torch.randint(-6, 6, (*shape[:-1], 1), device="cuda", generator=gen))
    w = w.to(dtype)
    w[..., ::37, :] = 0
    cbuf, codes = _guarded((*lead, nb, kb, 128, 64), torch.uint8, 0xAB)
    sbuf, scales = _guarded((*lead, nb, kb, 512), torch.uint8, 0xCD)
    q4.q4_pack_mx(w, codes, scales)
    want = q4.q4_pack_mx(w.float())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    for buf, v in ((cbuf, 0xAB), (sbuf, 0xCD)):
        assert (buf[:64] == v).all() and (buf[-64:] == v).all()
    flat, rows = w.reshape(-1, N, K), slice(0, min(N, 128))
    for e, part, block in ((0, rows, 0), (-1, slice(128 * (nb - 1), N), nb - 1)):
        c, s = ref.pack(flat[e, part].double().cpu().numpy())
        assert np.array_equal(codes.view(-1, nb, kb, 128, 64)[e, block].cpu().numpy(), c[0])
        assert np.array_equal(scales.view(-1, nb, kb, 512)[e, block].cpu().numpy(), s[0])
    obuf, out = _guarded(shape, dtype, 7.0)
    q4.q4_dequant_mx(codes, scales, out, N=N, K=K)
    assert torch.equal(out, q4.q4_dequant_mx(codes, scales, N=N, K=K).to(dtype))
    for e, part, block in ((0, rows, 0), (-1, slice(128 * (nb - 1), N), nb - 1)):
        c = codes.view(-1, nb, kb, 128, 64)[e, block][None].cpu().numpy()
        s = scales.view(-1, nb, kb, 512)[e, block][None].cpu().numpy()
        back = ref.unpack(c, s, part.stop - part.start, K)
        assert np.array_equal(out.view(-1, N, K)[e, part].double().cpu().numpy(), torch.from_numpy(back).to(dtype).double().numpy())
    assert (obuf[:64] == 7).all() and (obuf[-64:] == 7).all()
