"""Tokens sorted by expert and back on the GPU: the sort against a serial one,
row movement and its gradients against 64-bit formulas and differences, and
the whole layer as it is used."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_reference as ref
import weight_only_bit_gemv_b200 as q4
from test_gpu_mx import _packed, _x

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    q4.load()


def _ids(rng, M, top, E, dropped=0.1, dtype=np.int32):
    ids = np.minimum(rng.integers(0, E, (M, top)), rng.integers(0, E, (M, top)))
    ids[rng.random((M, top)) < dropped] = -1
    return torch.from_numpy(ids.astype(dtype)).cuda()


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("M,top,E", [(1, 1, 1), (1, 8, 256), (31, 2, 8), (33, 1, 1024), (1000, 3, 60), (1024, 8, 8),
                                     (1025, 8, 1024), (5000, 8, 128), (20001, 1, 2)])
def test_sort(M, top, E, dtype):
    rng = np.random.default_rng(M + E)
    ids = _ids(rng, M, top, E, dtype=dtype)
    offsets, rows, places = q4.q4_sort_experts(ids, E)
    for got, want in zip((offsets, rows, places), ref.sort(ids.cpu().numpy(), E)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)


def test_sort_odd_ids():
    """Ids past either end, all dropped, all alike, and no tokens."""
    big = 1 << 40
    for ids, E in ((torch.tensor([[8, 7], [-5, 0], [1 << 30, 3]], dtype=torch.int32), 8),
                   (torch.tensor([[big, 3], [-big, (1 << 32) + 1]], dtype=torch.int64), 4),
                   (torch.full((700, 2), -1, dtype=torch.int32), 5), (torch.full((9000, 1), 2, dtype=torch.int64), 3)):
        out = q4.q4_sort_experts(ids.cuda(), E)
        for got, want in zip(out, ref.sort(ids.numpy(), E)):
            assert np.array_equal(got.cpu().numpy(), want)
    offsets, rows, places = q4.q4_sort_experts(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    assert not offsets.any() and rows.shape == (0,) and places.shape == (0, 2)


def test_sort_guards_and_stream():
    rng = np.random.default_rng(1)
    M, top, E = 3000, 4, 33
    ids = _ids(rng, M, top, E)
    bufs = [torch.full((n + 64,), 77, dtype=torch.int32, device="cuda") for n in (E + 1, M * top, M * top)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q4.q4_sort_experts(ids, E, bufs[0][32:-32], bufs[1][32:-32], bufs[2][32:-32].view(M, top), stream=side)
    side.synchronize()
    for b, want in zip(bufs, ref.sort(ids.cpu().numpy(), E)):
        assert np.array_equal(b[32:-32].cpu().numpy(), want.reshape(-1))
        assert (b[:32] == 77).all() and (b[-32:] == 77).all()


def _half(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,top,K", [(1, 1, 1), (1, 8, 4096), (7, 2, 33), (50, 3, 130), (20, 9, 2052), (300, 8, 512), (4, 20, 100)])
def test_rows_and_gradients(M, top, K, dtype):
    """dispatch exactly, combine and its gradients within the roundings they make."""
    rng = np.random.default_rng(M * K + top)
    E = 12
    ids = _ids(rng, M, top, E, dropped=0.2)
    _, rows, places = q4.q4_sort_experts(ids, E)
    kept = (places >= 0).cpu().numpy()
    at = np.where(kept, places.cpu().numpy(), -1 - places.cpu().numpy())
    x = torch.from_numpy(rng.standard_normal((M, K))).to(dtype).cuda()
    xs = q4.q4_dispatch(x, places)
    want = x[rows.clamp(min=0).long()] * (rows >= 0)[:, None]
    assert torch.equal(xs, want)

    ys = torch.from_numpy(rng.standard_normal((M * top, K))).to(dtype).cuda()
    wt = torch.from_numpy(rng.random((M, top))).float().cuda()
    y64, w64 = ys.double().cpu().numpy(), wt.double().cpu().numpy() * kept
    terms = y64[at] * w64[..., None]
    for weights, t in ((wt, terms), (None, y64[at] * kept[..., None])):
        out = q4.q4_combine(ys, places, weights)
        # one rounding a product-sum in binary32 for each choice, one to the type
        total = np.abs(t).sum(1)
        bound = total * top * 2.0 ** -24
        bound = bound + _half(dtype) * (np.abs(t.sum(1)) + bound) + 2.0 ** -25 * (dtype == torch.float16)
        assert out.dtype == dtype and np.all(np.abs(out.double().cpu().numpy() - t.sum(1)) <= bound)

    dout = torch.from_numpy(rng.standard_normal((M, K))).to(dtype).cuda()
    dys, dw = q4.q4_combine_grad(dout, ys, places, wt)
    d64 = dout.double().cpu().numpy()
    want = np.zeros((M * top, K))
    want[at.reshape(-1)] = (d64[:, None] * w64[..., None]).reshape(-1, K)
    # the product's rounding in binary32, then the type's
    bound = np.abs(want) * (2.0 ** -24 + _half(dtype) * (1 + 2.0 ** -24)) + 2.0 ** -25 * (dtype == torch.float16)
    assert np.all(np.abs(dys.double().cpu().numpy() - want) <= bound)
    prod = d64[:, None] * y64[at] * kept[..., None]
    # a sum of K products in binary32, in any order
    bound = np.abs(prod).sum(-1) * (K + 1) * 2.0 ** -24
    assert dw.dtype == torch.float32
    assert np.all(np.abs(dw.double().cpu().numpy() - prod.sum(-1)) <= bound)


def test_gradients_against_differences():
    """combine is linear in ys and in weights, dispatch in x: differences of the
    calls' own outputs in binary32 against their gradients."""
    rng = np.random.default_rng(7)
    M, top, K, E = 9, 3, 40, 5
    ids = _ids(rng, M, top, E, dropped=0.2)
    _, _, places = q4.q4_sort_experts(ids, E)

    def normal(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).float().cuda()

    ys, wt, dout, x = normal(M * top, K), normal(M, top), normal(M, K), normal(M, K)
    dys, dw = q4.q4_combine_grad(dout, ys, places, wt)
    for _ in range(4):
        a, b = normal(M * top, K), normal(M, top)
        # f(y + a) - f(y - a) over 2: sums of 2 * M * K * top terms, each a few roundings of 2^-24
        got = (dout.double() * (q4.q4_combine(ys + a, places, wt).double() - q4.q4_combine(ys - a, places, wt).double())).sum() / 2
        want = (dys.double() * a.double()).sum()
        assert abs(got - want) <= 16 * 2.0 ** -24 * (dout.abs().double() * 10 * top).sum()
        got = (dout.double() * (q4.q4_combine(ys, places, wt + b).double() - q4.q4_combine(ys, places, wt - b).double())).sum() / 2
        want = (dw.double() * b.double()).sum()
        assert abs(got - want) <= 16 * 2.0 ** -24 * (dout.abs().double() * 10 * top).sum()
        # <dispatch(x), a> = <x, combine(a)>
        left = (q4.q4_dispatch(x, places).double() * a.double()).sum()
        right = (x.double() * q4.q4_combine(a, places).double()).sum()
        assert abs(left - right) <= 16 * 2.0 ** -24 * (x.abs().double() * 10 * top).sum()


def test_places_outside_are_skipped():
    """Positions past the last row touch nothing."""
    M, top, K = 4, 2, 64
    places = torch.tensor([[0, 8], [1 << 30, 3], [-9, -1 << 31], [-3, 5]], dtype=torch.int32, device="cuda")
    x = torch.randn(M, K, device="cuda")
    buf = torch.full((M * top * K + 128,), 5.0, device="cuda")
    xs = buf[64:-64].view(M * top, K)
    q4.q4_dispatch(x, places, xs)
    assert (buf[:64] == 5).all() and (buf[-64:] == 5).all()
    assert torch.equal(xs[0], x[0]) and torch.equal(xs[3], x[1]) and not xs[2].any() and torch.equal(xs[5], x[3])
    assert (xs[[1, 4, 6, 7]] == 5).all()
    ys = torch.randn(M * top, K, device="cuda")
    out = q4.q4_combine(ys, places)
    assert torch.equal(out[0], ys[0]) and torch.equal(out[1], ys[3]) and not out[2].any() and torch.equal(out[3], ys[5])
    dys = torch.full_like(buf, 5.0)
    _, dw = q4.q4_combine_grad(x, ys, places, torch.ones(M, top, device="cuda"), dys[64:-64].view(M * top, K))
    assert (dys[:64] == 5).all() and (dys[-64:] == 5).all()
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and not dw[2].any() and dw[3, 0] == 0


def _layer(x, ids, wt, gate_up, down, H):
    """Tokens through their experts: sort, gate and up, SiLU, down, back."""
    E = gate_up[0].shape[0]
    offsets, rows, places = q4.q4_sort_experts(ids, E)
    h = q4.q4_gemm_experts(*gate_up, x, offsets, rows, N=2 * H)
    act = (torch.nn.functional.silu(h[:, :H]) * h[:, H:]).to(torch.bfloat16)
    return q4.q4_combine(q4.q4_gemm_experts(*down, act, offsets, N=x.shape[1]), places, wt), act, offsets, rows, places


@pytest.mark.parametrize("M,top,E", [(3, 2, 8), (100, 2, 4)])
def test_whole_layer_in_a_graph(M, top, E):
    """The calls together as a decode step uses them, captured once and
    replayed on other tokens, routes and weights, some of them padding."""
    rng = np.random.default_rng(M)
    K, H = 256, 192
    cg, sg, wg = _packed(rng, 2 * H, K, E)
    cd, sd, wd = _packed(rng, K, H, E)
    x, ids = _x(rng, M, K), _ids(rng, M, top, E)
    wt = torch.from_numpy(rng.random((M, top))).float().cuda()
    _layer(x, ids, wt, (cg, sg), (cd, sd), H)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, act, offsets, rows, places = _layer(x, ids, wt, (cg, sg), (cd, sd), H)
    for _ in range(4):
        x.copy_(_x(rng, M, K))
        ids.copy_(_ids(rng, M, top, E, dropped=0.3))
        wt.copy_(torch.from_numpy(rng.random((M, top))).float())
        g.replay()
        torch.cuda.synchronize()
        o, r, p = ref.sort(ids.cpu().numpy(), E)
        assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(places.cpu().numpy(), p)
        x64, a64 = x.double().cpu().numpy(), act.double().cpu().numpy()
        want, bound = np.zeros((M, K)), np.zeros((M, K))
        for m in range(M):
            for j in range(top):
                if p[m, j] < 0:
                    continue
                e = int(ids[m, j])
                h = x64[m] @ wg[e].T
                gate, up = h[:H], h[H:]
                # the binary32 products' error through SiLU (slope at most 1.1) and the product, then bfloat16's half step
                err = ref.tolerance(wg[e], x64[m:m + 1], torch.float32)[0]
                a = gate / (1 + np.exp(-gate)) * up
                off = 1.1 * err[:H] * (np.abs(up) + err[H:]) + np.abs(gate) * err[H:] + 8 * 2.0 ** -24 * np.abs(a)
                off = off + 2.0 ** -8 * (np.abs(a) + off)
                assert np.all(np.abs(a64[p[m, j]] - a) <= off)
                y = a64[p[m, j]] @ wd[e].T
                want[m] += float(wt[m, j]) * y
                bound[m] += float(wt[m, j]) * (ref.tolerance(wd[e], a64[p[m, j]][None], torch.float32)[0] + 4 * 2.0 ** -24 * np.abs(y))
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound + 1e-30)


def test_backward_in_a_graph():
    """The routing's backward pass, captured and replayed: dys and dweights of
    combine, and dx of dispatch from them, beside autograd's of the same layer."""
    rng = np.random.default_rng(5)
    M, top, E, K = 60, 2, 6, 128
    ids = _ids(rng, M, top, E, dropped=0.2)
    offsets, rows, places = q4.q4_sort_experts(ids, E)
    x = torch.randn(M, K, device="cuda")
    wt = torch.rand(M, top, device="cuda")
    dout = torch.randn(M, K, device="cuda")

    def backward():
        xs = q4.q4_dispatch(x, places)
        ys = xs * xs                                     # the experts, elementwise here
        out = q4.q4_combine(ys, places, wt)
        dys, dw = q4.q4_combine_grad(dout, ys, places, wt)
        return out, q4.q4_combine(2 * xs * dys, places), dw

    backward()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, dx, dw = backward()
    g.replay()
    torch.cuda.synchronize()
    x64 = x.double().requires_grad_()
    w64 = wt.double().requires_grad_()
    kept = (places >= 0).double()
    ref_out = ((x64 ** 2)[:, None] * (w64 * kept)[..., None]).sum(1)
    gx, gw = torch.autograd.grad(ref_out, (x64, w64), dout.double())
    # products of a few binary32 factors, and for dweights a sum of K of them
    assert torch.all((out - ref_out).abs() <= 4 * top * 2.0 ** -24 * ref_out.abs() + 1e-30)
    assert torch.all((dx - gx).abs() <= 8 * top * 2.0 ** -24 * (2 * x64 * dout).abs() * wt.sum(1, keepdim=True) + 1e-30)
    assert torch.all((dw - gw).abs() <= (K + 4) * 2.0 ** -24 * ((x64 ** 2) * dout.abs()).sum(1, keepdim=True))
