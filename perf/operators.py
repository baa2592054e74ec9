"""Cases for the microscaled 4-bit weights and the expert-routed layers built on them.

Five operators, each in a plain form (elementary torch operations) and as the
calls a user makes of the library:

  pack           quantise a weight matrix to 4-bit e2m1 codes with one power-of-two
                 scale for 32 weights along K, and read the values back
  gemm           y = x W^T from the packed matrix, bfloat16 activations
  experts        the same product for tokens grouped by expert, each group with
                 its own matrix of a stack of packed ones
  route          sort the tokens of a batch by expert and gather their rows
  combine        bring the experts' rows back to their tokens with the router's
                 weights, and that step's gradients

Packed matrices are stored in blocks of 128 rows x 128 k: codes
[ceil(N/128)][ceil(K/128)][128][64] bytes (low nibble = even k), scales
[ceil(N/128)][ceil(K/128)][512] bytes, the exponent byte of row r, group g of a
block at (r % 32) * 16 + (r // 32) * 4 + g; W = e2m1(code) * 2^(byte - 127).
"""
import math

import torch

own = False

BLOCK, GROUP = 128, 32
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
DEVICE = "cuda"


def listed():
    return [
        # one small projection of a fine-tuned checkpoint, odd in both directions: packed when an adapter is merged
        {"name": "pack 1001x1056 fp32", "kind": "pack", "N": 1001, "K": 1056, "type": "float32"},
        # the widest projection of a 70B model, packed from its bfloat16 checkpoint at load time
        {"name": "pack 57344x8192 bf16", "kind": "pack", "N": 57344, "K": 8192, "type": "bfloat16"},
        # one token of decode through the attention output projection of a 7B model: the latency case
        {"name": "gemm 1x4096x4096", "kind": "gemm", "M": 1, "N": 4096, "K": 4096, "out": "float32"},
        # a verify batch of drafted tokens through the vocabulary projection
        {"name": "gemm 13x128256x4096", "kind": "gemm", "M": 13, "N": 128256, "K": 4096, "out": "float32"},
        # the last, ragged chunk of a prompt through an 8B model's down projection
        {"name": "gemm 77x4096x14336", "kind": "gemm", "M": 77, "N": 4096, "K": 14336, "out": "float32"},
        # a full prefill chunk through the widest projection of a 70B model
        {"name": "gemm 512x57344x8192", "kind": "gemm", "M": 512, "N": 57344, "K": 8192, "out": "bfloat16"},
        # four sequences decoding one token each through the gate and up projections of eight experts
        {"name": "experts 4 of 8x28672x4096", "kind": "experts", "M": 4, "top": 2, "E": 8, "N": 28672, "K": 4096, "out": "float32"},
        # a prefill chunk through the same experts, loaded as unevenly as a router loads them
        {"name": "experts 2048 of 8x28672x4096", "kind": "experts", "M": 2048, "top": 2, "E": 8, "N": 28672, "K": 4096, "out": "bfloat16"},
        # a decode step's routing, four of its sequences already finished
        {"name": "route 12x2 of 8", "kind": "route", "M": 12, "top": 2, "E": 8, "K": 4096, "padded": 4, "wide": True, "type": "bfloat16"},
        # a training or prefill batch over many small experts
        {"name": "route 16384x8 of 256", "kind": "route", "M": 16384, "top": 8, "E": 256, "K": 2048, "padded": 0, "wide": False, "type": "bfloat16"},
        # a ragged chunk's expert outputs back to their tokens
        {"name": "combine 777x2 of 8", "kind": "combine", "M": 777, "top": 2, "E": 8, "K": 4096, "padded": 9, "grad": False, "type": "bfloat16"},
        # the backward pass of a training batch's combine: gradients of the rows and of the router's weights
        {"name": "combine grad 16384x8 of 256", "kind": "combine", "M": 16384, "top": 8, "E": 256, "K": 2048, "padded": 0, "grad": True, "type": "bfloat16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["pack", "gemm", "gemm", "experts", "route", "combine"])
    width = rng.choice([1, 2, 8, 32, 32, 128])  # what K is a multiple of
    if kind == "pack":
        N, K = _spread(rng, 1, 32000), _spread(rng, 32, 14336)
        return {"kind": kind, "N": N, "K": max(1, K // width) * width, "type": rng.choice(list(TYPES))}
    if kind == "gemm":
        K = _spread(rng, 64, 28672)
        N = _spread(rng, 64, max(64, min(60000, 400_000_000 // K)))
        return {"kind": kind, "M": _spread(rng, 1, 512), "N": N, "K": max(1, K // width) * width, "out": rng.choice(["float32", "bfloat16"])}
    if kind == "experts":
        E = rng.choice([2, 4, 8, 16, 60, 64, 128])
        top = rng.randint(1, min(E, 8))
        K = _spread(rng, 256, 7168)
        N = _spread(rng, 256, max(256, min(14336, 400_000_000 // (K * E))))
        return {"kind": kind, "M": _spread(rng, 1, 8192 // top), "top": top, "E": E, "N": N, "K": max(1, K // width) * width, "out": rng.choice(["float32", "bfloat16"])}
    E = rng.choice([4, 8, 32, 60, 128, 160, 256])
    top = rng.randint(1, min(E, 8))
    K = max(1, _spread(rng, 256, 8192) // width) * width
    M = _spread(rng, 1, max(1, min(20000, 120_000_000 // (K * top))))
    case = {"kind": kind, "M": M, "top": top, "E": E, "K": K, "padded": rng.choice([0, 0, M // 7, M]), "type": rng.choice(list(TYPES))}
    case["wide" if kind == "route" else "grad"] = rng.random() < 0.5
    return case


# ---- making the inputs ------------------------------------------------------


def _up(n, m):
    return -(-n // m) * m


def _two(e):
    """2^e of whole numbers e, exactly: exp2 and pow need not be."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantised(w):
    """(codes 0..15 as uint8, exponent bytes) of w [N, K], K a multiple of GROUP: scale = 2^(floor(log2 max) - 2), nearest code, ties to the even one."""
    groups = w.float().unflatten(-1, (-1, GROUP))
    top = groups.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    e = torch.where(top > 0, e, -127)
    a = groups * _two(-e).float()
    s, a = (a < 0), a.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte()
    return (code + 8 * s.byte()).flatten(-2), (e + 127).squeeze(-1).byte()


def _blocks(code, scale):
    """Codes [N, K] and exponent bytes [N, K / 32] in blocks."""
    N, K = code.shape
    Np, Kp = _up(N, BLOCK), _up(K, BLOCK)
    code = torch.nn.functional.pad(code, (0, Kp - K, 0, Np - N))
    scale = torch.nn.functional.pad(scale, (0, Kp // GROUP - scale.shape[1], 0, Np - N))
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    codes = packed.view(Np // BLOCK, BLOCK, Kp // BLOCK, 64).permute(0, 2, 1, 3).contiguous()
    scales = scale.view(Np // BLOCK, 4, 32, Kp // BLOCK, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes, scales.view(Np // BLOCK, Kp // BLOCK, 512)


def _weights(gen, N, K, spread):
    """A packed matrix drawn from N(0, spread) with some rows far larger than others, as trained projections have them."""
    codes, scales = [], []
    for at in range(0, N, 8192):
        n = min(8192, N - at)
        w = torch.randn(n, _up(K, GROUP), generator=gen, device=DEVICE) * spread
        w *= torch.exp2(torch.randn(n, 1, generator=gen, device=DEVICE))
        w[:, K:] = 0
        c, s = _blocks(*_quantised(w))
        codes.append(c)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def _activations(gen, M, K):
    """bfloat16 rows ~ N(0, 1) with a few channels that stand far out."""
    x = torch.randn(M, K, generator=gen, device=DEVICE)
    x *= 1 + 30 * (torch.rand(K, generator=gen, device=DEVICE) < 0.002)
    return x.bfloat16()


def _ids(gen, case):
    """The router's choices [M, top], distinct in a row, experts not equally loved; -1 for the padded tokens at the end."""
    score = torch.randn(case["M"], case["E"], generator=gen, device=DEVICE) + 0.7 * torch.randn(case["E"], generator=gen, device=DEVICE)
    value, ids = torch.topk(score, case["top"], dim=1)
    if case.get("padded"):
        ids[case["M"] - case["padded"]:] = -1
    return ids, torch.softmax(value, dim=1)


def _sorted(ids, E):
    """offsets [E + 1], rows [T], places [M, top] of the stable order by expert; ids outside 0..E-1 come last, their places as -1 - place."""
    M, top = ids.shape
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E).long()
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(M * top, device=ids.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = (key[:, None] == torch.arange(E, device=ids.device)).sum(0).cumsum(0)
    rows = torch.where(key[order] < E, order // top, -1)
    places = torch.where(key < E, place, -1 - place).view(M, top)
    return offsets.int(), rows.int(), places.int()


def prepare(case, seed):
    gen = torch.Generator(DEVICE)
    gen.manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind == "pack":
        w = torch.randn(case["N"], case["K"], generator=gen, device=DEVICE) * 0.02
        s["w"] = (w * torch.exp2(torch.randn(case["N"], 1, generator=gen, device=DEVICE))).to(TYPES[case["type"]])
    elif kind == "gemm":
        s["codes"], s["scales"] = _weights(gen, case["N"], case["K"], 0.02)
        s["x"] = _activations(gen, case["M"], case["K"])
    elif kind == "experts":
        stack = [_weights(gen, case["N"], case["K"], 0.02) for _ in range(case["E"])]
        s["codes"], s["scales"] = (torch.stack(v) for v in zip(*stack))
        s["x"] = _activations(gen, case["M"], case["K"])
        s["offsets"], s["rows"], _ = _sorted(_ids(gen, case)[0], case["E"])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        ids, weights = _ids(gen, case)
        t = TYPES[case["type"]]
        if kind == "route":
            s["ids"] = ids.long() if case["wide"] else ids.int()
            s["x"] = torch.randn(case["M"], case["K"], generator=gen, device=DEVICE).to(t)
        else:
            s["places"], s["weights"] = _sorted(ids, case["E"])[2], weights
            s["ys"] = torch.randn(case["M"] * case["top"], case["K"], generator=gen, device=DEVICE).to(t)
            if case["grad"]:
                s["dout"] = torch.randn(case["M"], case["K"], generator=gen, device=DEVICE).to(t)
    return s


# ---- the plain forms --------------------------------------------------------


def _values(codes, scales, N, K):
    """W [..., N, K] in 32 bits from its blocks."""
    lead = codes.shape[:-4]
    nb, kb = codes.shape[-4:-2]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    grid = torch.cat([grid, -grid])
    both = torch.arange(256, device=codes.device)
    pairs = torch.stack([grid[both % 16], grid[both // 16]], 1)
    w = pairs[codes.int()].flatten(-2).view(*lead, nb, kb, 4, 32, 4, GROUP)
    scale = _two(scales.view(*lead, nb, kb, 32, 4, 4).transpose(-3, -2).long() - 127).float()
    w = w * scale[..., None]
    return w.view(*lead, nb, kb, BLOCK, BLOCK).transpose(-3, -2).reshape(*lead, nb * BLOCK, kb * BLOCK)[..., :N, :K]


def _plain(s):
    kind = s["kind"]
    if kind == "pack":
        N, K = s["N"], s["K"]
        w = torch.nn.functional.pad(s["w"], (0, _up(K, GROUP) - K))
        return _values(*_blocks(*_quantised(w)), N, K).to(s["w"].dtype)
    if kind == "gemm":
        return (s["x"].float() @ _values(s["codes"], s["scales"], s["N"], s["K"]).T).to(TYPES[s["out"]])
    if kind == "experts":
        E, offsets = s["E"], s["offsets"].long()
        T = s["rows"].numel()
        at = torch.arange(T, device=DEVICE)
        expert = (at[:, None] >= offsets[1:-1]).sum(1)
        inside = at - offsets[expert]
        x = torch.zeros(E, s["most"], s["K"], device=DEVICE)
        x[expert, inside] = s["x"].float()[s["rows"].long()]
        y = torch.bmm(x, _values(s["codes"], s["scales"], s["N"], s["K"]).transpose(1, 2))
        return y[expert, inside].to(TYPES[s["out"]])
    if kind == "route":
        offsets, rows, places = _sorted(s["ids"], s["E"])
        xs = s["x"][rows.clamp(min=0).long()] * (rows >= 0)[:, None]
        return {"offsets": offsets, "rows": rows, "places": places, "xs": xs}
    kept = s["places"] >= 0
    at = torch.where(kept, s["places"], -1 - s["places"]).long()
    ys = s["ys"].float()[at.reshape(-1)].view(*at.shape, -1)
    weights = s["weights"] * kept
    if not s["grad"]:
        return (ys * weights[..., None]).sum(1).to(s["ys"].dtype)
    dout = s["dout"].float()[:, None]
    dys = torch.empty_like(s["ys"])
    dys[at.reshape(-1)] = (dout * weights[..., None]).flatten(0, 1).to(dys.dtype)
    return {"dys": dys, "dweights": (dout * ys).sum(-1) * kept}


def run(state):
    if not own:
        return _plain(state)
    import weight_only_bit_gemv_b200 as q4

    s, kind = state, state["kind"]
    if kind == "pack":
        codes, scales = q4.q4_pack_mx(s["w"])
        return q4.q4_dequant_mx(codes, scales, N=s["N"], K=s["K"], dtype=s["w"].dtype)
    if kind == "gemm":
        return q4.q4_gemm_mx(s["codes"], s["scales"], s["x"], N=s["N"], dtype=TYPES[s["out"]])
    if kind == "experts":
        return q4.q4_gemm_experts(s["codes"], s["scales"], s["x"], s["offsets"], s["rows"], N=s["N"], dtype=TYPES[s["out"]])
    if kind == "route":
        offsets, rows, places = q4.q4_sort_experts(s["ids"], s["E"])
        return {"offsets": offsets, "rows": rows, "places": places, "xs": q4.q4_dispatch(s["x"], places)}
    if not s["grad"]:
        return q4.q4_combine(s["ys"], s["places"], s["weights"])
    dys, dweights = q4.q4_combine_grad(s["dout"], s["ys"], s["places"], s["weights"])
    return {"dys": dys, "dweights": dweights}


def work(case):
    kind, K = case["kind"], case["K"]
    size = lambda t: TYPES[t].itemsize  # noqa: E731
    if kind == "pack":  # the matrix in, codes and scales out, the values they stand for out
        n = case["N"] * K
        return {"bytes": n * 2 * size(case["type"]) + n / 2 + n / GROUP, "flops": 4 * n}
    if kind in ("gemm", "experts"):
        rows, matrices = case["M"] * case.get("top", 1), 1
        if kind == "experts":  # the experts that some token is expected to choose
            matrices = case["E"] * (1 - (1 - case["top"] / case["E"]) ** case["M"])
        n = case["N"] * K
        return {"bytes": matrices * (n / 2 + n / GROUP) + case["M"] * K * 2 + rows * case["N"] * size(case["out"]), "flops": 2 * rows * n}
    row = K * size(case["type"])
    T, kept = case["M"] * case["top"], (case["M"] - case["padded"])
    if kind == "route":  # ids in, offsets, rows and places out; each kept row of x in, all of xs out
        return {"bytes": T * (8 if case["wide"] else 4) + 8 * T + 4 * case["E"] + kept * row + T * row, "flops": T}
    if not case["grad"]:
        return {"bytes": 8 * T + kept * case["top"] * row + case["M"] * row, "flops": 2 * T * K}
    return {"bytes": 12 * T + kept * (case["top"] + 1) * row + T * row, "flops": 3 * T * K}


# ---- the definitions in 64 bits ---------------------------------------------


def _powers():
    """2^-127 .. 2^128 in 64 bits; entry b is what exponent byte b stands for."""
    return torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=torch.float64, device=DEVICE)


def _matrix64(codes, scales, N, K):
    """W [N, K] in 64 bits, code by code from its bits: sign, two bits of exponent, one of mantissa."""
    nb, kb = codes.shape[:2]
    out = torch.empty(nb * BLOCK, kb * BLOCK, dtype=torch.float64, device=codes.device)
    r = torch.arange(BLOCK, device=codes.device)
    g = torch.arange(4, device=codes.device)
    spot = ((r % 32) * 16 + r // 32 * 4)[:, None] + g
    powers = _powers()
    for b in range(nb):
        c = torch.stack([codes[b] & 15, codes[b] >> 4], -1).flatten(-2).short()  # [kb, 128, 128]
        e, m = c >> 1 & 3, (c & 1).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * (1 << (e - 1).clamp(min=0)).double())
        v = torch.where(c >= 8, -v, v)
        f = powers[scales[b][:, spot].long()]  # [kb, 128, 4]
        out[b * BLOCK:(b + 1) * BLOCK] = (v.view(kb, BLOCK, 4, GROUP) * f[..., None]).flatten(-2).transpose(0, 1).reshape(BLOCK, -1)
    return out[:N, :K]


def exact(case, seed):
    s = prepare(case, seed)
    kind, K = case["kind"], case["K"]
    if kind == "pack":
        out = torch.empty(case["N"], K, dtype=torch.float64, device=DEVICE)
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEVICE)
        powers = _powers()
        for at in range(0, case["N"], 2048):
            w = torch.nn.functional.pad(s["w"][at:at + 2048].double(), (0, -K % GROUP)).unflatten(1, (-1, GROUP))
            top = w.abs().amax(2, keepdim=True)
            step = powers[(torch.searchsorted(powers, top, right=True) - 3).clamp(min=0)]
            a = (w.abs() / step).clamp(max=6)
            up = torch.searchsorted(grid, a).clamp(max=7)
            low = (up - 1).clamp(min=0)
            far, near = grid[up] - a, a - grid[low]
            i = torch.where((far < near) | ((far == near) & (up % 2 == 0)), up, low)
            out[at:at + 2048] = (torch.sign(w) * grid[i] * step).flatten(1)[:, :K]
        return out
    if kind == "gemm":
        y = torch.empty(case["M"], case["N"], dtype=torch.float64, device=DEVICE)
        x = s["x"].double()
        for b in range(0, s["codes"].shape[0], 64):
            n = min(64 * BLOCK, case["N"] - b * BLOCK)
            y[:, b * BLOCK:b * BLOCK + n] = x @ _matrix64(s["codes"][b:b + 64], s["scales"][b:b + 64], n, K).T
        return y
    if kind == "experts":
        x, offsets = s["x"].double(), s["offsets"].tolist()
        y = torch.empty(len(s["rows"]), case["N"], dtype=torch.float64, device=DEVICE)
        for e in range(case["E"]):
            if offsets[e + 1] > offsets[e]:
                chosen = s["rows"][offsets[e]:offsets[e + 1]].long()
                y[offsets[e]:offsets[e + 1]] = x[chosen] @ _matrix64(s["codes"][e], s["scales"][e], case["N"], K).T
        return y
    M, top = case["M"], case["top"]
    if kind == "route":
        ids = s["ids"].long().reshape(-1)
        token = torch.arange(M * top, device=DEVICE) // top
        good = (ids >= 0) & (ids < case["E"])
        mine = torch.nonzero(good).flatten()
        mine = mine[torch.sort(ids[mine] * (M * top) + mine).indices]
        xs = torch.zeros(M * top, K, dtype=torch.float64, device=DEVICE)
        xs[:len(mine)] = s["x"].double()[token[mine]]
        return {"offsets": None, "rows": None, "places": None, "xs": xs}
    ys, weights = s["ys"].double(), s["weights"].double()
    out = torch.zeros(M, K, dtype=torch.float64, device=DEVICE)
    dys, dweights = torch.zeros_like(ys), torch.zeros(M, top, dtype=torch.float64, device=DEVICE)
    for j in range(top):
        m = torch.nonzero(s["places"][:, j] >= 0).flatten()
        p = s["places"][m, j].long()
        if case["grad"]:
            d = s["dout"].double()[m]
            dys[p] = d * weights[m, j, None]
            dweights[m, j] = (d * ys[p]).sum(1)
        else:
            out[m] += ys[p] * weights[m, j, None]
    return {"dys": dys, "dweights": dweights} if case["grad"] else out
