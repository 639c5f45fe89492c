"""The measured cases of the library's grouped products and of its 4-bit floating point.

Four operators:

  gemm_grouped      C[r] = sa[r] sb[g] (A[r] B[g]) for the rows r of each group g: the products of a
                    layer of experts, whose rows are sorted by expert; also their input's gradient
  gemm_grouped_dw   dW[g] = sum over the rows of group g of X[r]^T dY[r]: those experts' gradients
  quantize_mx4      blocks of 32 (or 16) values along k to 4-bit floats (E2M1) with one 8-bit scale,
                    and their reading back (dequantize_mx4), which is what the pass returns
  gemm_mx4          C = A B^T of two such operands

`run` computes them in plain torch operations in FP32, or, where `own` is
true, through the library.

4-bit floats: E2M1 has the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Blocks of 32
have a power of two as their scale (E8M0: code - 127 is the exponent), blocks of
16 an E4M3 number and the tensor one FP32 factor.  The scales lie in tiles of
128 rows by 4 blocks: the scale of row r and block b is byte
(r % 32) * 16 + r % 128 // 32 * 4 + b % 4 of tile (r // 128, b // 4).
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through its two experts of a small layer: launch latency is most of it
        {"name": "experts-1", "op": "gemm_grouped", "R": 2, "G": 8, "K": 512, "N": 4096, "dtype": "bf16", "out": "bf16",
         "weight": "nk", "skew": 0.0},
        # a decode step of 32 sequences, two experts each, through the up projections
        {"name": "experts-decode-64", "op": "gemm_grouped", "R": 64, "G": 8, "K": 4096, "N": 14336, "dtype": "bf16",
         "out": "bf16", "weight": "nk", "skew": 0.0},
        # many experts of odd sizes in FP8 with a scale per row and per column, some experts without a row
        {"name": "experts-odd", "op": "gemm_grouped", "R": 1234, "G": 40, "K": 1008, "N": 2003, "dtype": "e4m3",
         "out": "f32", "weight": "nk", "skew": 1.0},
        # the gradient of a training batch's input: the same weights, read along their other dim
        {"name": "experts-train", "op": "gemm_grouped", "R": 8192, "G": 8, "K": 14336, "N": 4096, "dtype": "bf16",
         "out": "bf16", "weight": "kn", "skew": 0.5},
        # gradients of small experts after a short sequence, kept in FP32
        {"name": "dw-small", "op": "gemm_grouped_dw", "R": 130, "G": 16, "K": 512, "N": 1024, "dtype": "f16",
         "out": "f32", "weight": "kn", "skew": 1.0},
        # gradients of a training batch's experts
        {"name": "dw-train", "op": "gemm_grouped_dw", "R": 8192, "G": 8, "K": 4096, "N": 4096, "dtype": "bf16",
         "out": "bf16", "weight": "nk", "skew": 0.5},
        # one token's activations to 4 bits
        {"name": "quantize-1", "op": "quantize_mx4", "R": 1, "K": 4096, "block": 32, "dtype": "bf16", "order": "k"},
        # the activations of a training batch
        {"name": "quantize-8192", "op": "quantize_mx4", "R": 8192, "K": 14336, "block": 16, "dtype": "bf16",
         "order": "k"},
        # a weight along its other dim, as the product of its input's gradient wants it
        {"name": "quantize-turned", "op": "quantize_mx4", "R": 4096, "K": 5000, "block": 32, "dtype": "f16",
         "order": "r"},
        # one token through the decode step's up projection, all in 4 bits
        {"name": "mx4-1", "op": "gemm_mx4", "M": 1, "K": 4096, "N": 14336, "block": 32, "out": "bf16"},
        # a ragged batch, sizes that fill no tile
        {"name": "mx4-odd", "op": "gemm_mx4", "M": 777, "K": 1000, "N": 5003, "block": 16, "out": "f32"},
        # a training batch
        {"name": "mx4-8192", "op": "gemm_mx4", "M": 8192, "K": 4096, "N": 14336, "block": 16, "out": "bf16"},
    ]


MOST = 8192 * 4096 * 14336       # multiply-adds of the largest listed products
MOST_WEIGHTS = 8 * 4096 * 14336  # and their weights


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["gemm_grouped", "gemm_grouped_dw", "quantize_mx4", "gemm_mx4"])
    if op == "quantize_mx4":
        K = _log(rng, 64, 16384)
        return {"op": op, "R": _log(rng, 1, min(16384, 8192 * 14336 // K)), "K": K, "block": rng.choice([16, 32]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "order": rng.choice(["k", "k", "r"])}
    if op == "gemm_mx4":
        K, N = _log(rng, 64, 14336), _log(rng, 64, 14336)
        if rng.random() < 0.7:
            K = max(64, K // 32 * 32)
        return {"op": op, "M": _log(rng, 1, min(8192, MOST // (K * N))), "K": K, "N": N,
                "block": rng.choice([16, 32]), "out": rng.choice(["bf16", "f16", "f32"])}
    # rows of the operands start at multiples of 16 bytes, as framework allocators and layer sizes make them
    dtype = rng.choice(["bf16", "f16", "e4m3"] if op == "gemm_grouped" else ["bf16", "f16"])
    G = _log(rng, 1, 64)
    weight = rng.choice(["nk", "kn"])
    K = max(64, _log(rng, 64, 14336) // 16 * 16)
    N = _log(rng, 64, min(14336, MOST_WEIGHTS // (G * K)))
    if op == "gemm_grouped_dw" or weight == "kn" or rng.random() < 0.5:
        N = max(64, N // 16 * 16)
    return {"op": op, "R": _log(rng, 1, min(8192, MOST // (K * N))), "G": G, "K": K, "N": N, "dtype": dtype,
            "out": rng.choice(["bf16", "f32"]), "weight": weight, "skew": rng.choice([0.0, 0.5, 1.0])}


# ----------------------------------------------------------------- the inputs

def _sizes(case):
    """Rows of each group: R rows that choose among G groups whose popularity falls as 1 / rank ** skew."""
    r = random.Random(case["R"] * 1009 + case["G"])
    popular = [1.0 / (i + 1) ** case["skew"] for i in range(case["G"])]
    sizes = [0] * case["G"]
    for g in r.choices(range(case["G"]), popular, k=case["R"]):
        sizes[g] += 1
    return sizes


def _randn(g, dtype, *shape):
    """Normal values of a type; E4M3 ones at a size that uses its range."""
    if dtype == "e4m3":
        return (torch.randn(*shape, generator=g, device="cuda") * 64).clamp(-448, 448).to(DT[dtype])
    return torch.randn(*shape, generator=g, device="cuda", dtype=DT[dtype])


def _prepare_grouped(case, g, seed):
    R, G, K, N, dtype = case["R"], case["G"], case["K"], case["N"], case["dtype"]
    sizes = _sizes(case)
    random.Random(seed).shuffle(sizes)
    s = {"op": case["op"], "sizes": sizes, "x": _randn(g, dtype, R, K),
         "offsets": torch.tensor([0] + sizes, device="cuda").cumsum(0)}
    if case["op"] == "gemm_grouped_dw":
        s["dy"] = _randn(g, dtype, R, N)
        dw = torch.empty((G, N, K) if case["weight"] == "nk" else (G, K, N), device="cuda", dtype=DT[case["out"]])
        s["dw"] = dw.transpose(1, 2) if case["weight"] == "nk" else dw
        return s
    shape = (N, K) if case["weight"] == "nk" else (K, N)
    w = torch.empty(G, *shape, device="cuda", dtype=DT[dtype])
    for i in range(G):
        w[i] = _randn(g, dtype, *shape) if dtype == "e4m3" else _randn(g, dtype, *shape) * K ** -0.5
    s["w"] = w.transpose(1, 2) if case["weight"] == "nk" else w
    s["sa"] = s["sb"] = None
    if dtype == "e4m3":
        s["sa"] = (torch.rand(R, generator=g, device="cuda") + 0.5) / 64
        s["sb"] = (torch.rand(G, N, generator=g, device="cuda") + 0.5) / (64 * K ** 0.5)
    s["y"] = torch.empty(R, N, device="cuda", dtype=DT[case["out"]])
    return s


def _values(g, R, K):
    """Activations: normal, with a few channels ten times as large."""
    x = torch.randn(R, K, generator=g, device="cuda")
    return x * torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 10.0, 1.0)


def _empty_codes(R, K):
    """Rows of codes that start at multiples of 16 bytes."""
    return torch.zeros(R, (K + 31) // 32 * 16, dtype=torch.uint8, device="cuda")[:, :(K + 1) // 2]


def _tiled(scales):
    """Codes of scales [R, blocks] in the order of their tiles."""
    R, n = scales.shape
    t = torch.zeros((R + 127) // 128 * 128, (n + 3) // 4 * 4, dtype=torch.uint8, device="cuda")
    t[:R, :n] = scales
    return t.view(t.shape[0] // 128, 4, 32, t.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _operand(case, g, R, K, spread):
    """A quantised matrix: its codes, tiled scales and factor."""
    block = case["block"]
    x = _values(g, R, K) * spread
    scale = None if block == 32 else (x.abs().amax() / (6 * 448)).reshape(1)
    e, s = _encode(x, block, scale)
    codes = _empty_codes(R, K)
    codes[:, :K // 2] = e[:, 0:K - 1:2] | (e[:, 1::2] << 4)
    if K % 2:
        codes[:, -1] = e[:, -1]
    return {"codes": codes, "scales": _tiled(s), "scale": scale}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] in ("gemm_grouped", "gemm_grouped_dw"):
        return _prepare_grouped(case, g, seed)
    K, block = case["K"], case["block"]
    s = {"op": case["op"], "K": K, "block": block}
    if case["op"] == "quantize_mx4":
        R, dt = case["R"], DT[case["dtype"]]
        if case["order"] == "k":
            s["x"], s["y"] = _values(g, R, K).to(dt), torch.empty(R, K, device="cuda", dtype=dt)
        else:
            s["x"], s["y"] = _values(g, K, R).to(dt).t(), torch.empty(K, R, device="cuda", dtype=dt).t()
        s["scale"] = None if block == 32 else (s["x"].abs().amax().float() / (6 * 448)).reshape(1)
        s["codes"] = _empty_codes(R, K)
        s["scales"] = torch.empty((R + 127) // 128 * ((-(-K // block) + 3) // 4) * 512, dtype=torch.uint8, device="cuda")
        return s
    s["a"] = _operand(case, g, case["M"], K, 1.0)
    s["b"] = _operand(case, g, case["N"], K, K ** -0.5)
    s["c"] = torch.empty(case["M"], case["N"], device="cuda", dtype=DT[case["out"]])
    return s


# ------------------------------------------------------------------- one pass

def _encode(x, block, scale):
    """Codes of E2M1 (one per byte) and of the scales, rounded to nearest, ties to even.  The largest of a block
    decides its scale: of 32 values, the power of two that brings it to 4 ... 8 (values above 6 become 6); of 16,
    a sixth of it in E4M3, after the factor."""
    R, K = x.shape
    u = x.float() if scale is None else x.float() / scale
    n = -(-K // block)
    u = torch.nn.functional.pad(u, (0, n * block - K)).view(R, n, block)
    top = u.abs().amax(2)
    if block == 32:
        e = (torch.frexp(top)[1] - 3).clamp(min=-127)
        s = (torch.where(top > 0, e, -127) + 127).to(torch.uint8)
    else:
        s = (top / 6).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
    unit = _unit(s, block).unsqueeze(2)
    q = torch.where(unit > 0, u / unit, 0.0)
    m = q.abs()
    e = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
         + 8 * torch.signbit(q).byte())
    return e.view(R, n * block)[:, :K], s


def _unit(s, block):
    """The FP32 values of the scales' codes (E8M0's is a float's exponent; its 0 is half the least normal one)."""
    if block == 16:
        return s.view(torch.float8_e4m3fn).float()
    return torch.where(s > 0, s.int() << 23, 1 << 22).view(torch.float32)


def _decode(codes, tiled, K, block, scale):
    """The FP32 values of a quantised matrix."""
    R, n = codes.shape[0], -(-K // block)
    rows, tiles = (R + 127) // 128, (n + 3) // 4
    s = tiled.view(rows, tiles, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows * 128, tiles * 4)[:R, :n]
    s = _unit(s, block)
    if scale is not None:
        s = s * scale
    e = torch.stack((codes & 15, codes >> 4), 2).view(R, -1)[:, :K].int()
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")[e]
    return v * s.repeat_interleave(block, 1)[:, :K]


def _plain_grouped(s):
    x = s["x"].float()
    y = torch.cat([a @ s["w"][g].float() * (1.0 if s["sb"] is None else s["sb"][g])
                   for g, a in enumerate(x.split(s["sizes"]))])
    return (y if s["sa"] is None else y * s["sa"][:, None]).to(s["y"].dtype)


def _plain_grouped_dw(s):
    parts = zip(s["x"].float().split(s["sizes"]), s["dy"].float().split(s["sizes"]))
    return torch.stack([(a.t() @ b).to(s["dw"].dtype) for a, b in parts])


def _plain_quantize(s):
    e, scales = _encode(s["x"], s["block"], s["scale"])
    e = torch.nn.functional.pad(e, (0, s["K"] % 2))
    codes = e[:, 0::2] | (e[:, 1::2] << 4)
    return _decode(codes, _tiled(scales), s["K"], s["block"], s["scale"]).to(s["y"].dtype)


def _plain_mx4(s):
    a, b = (_decode(o["codes"], o["scales"], s["K"], s["block"], o["scale"]) for o in (s["a"], s["b"]))
    return (a @ b.t()).to(s["c"].dtype)


def run(state):
    s = state
    if own:
        import tcgen05_tmem_gemm_b200 as dg

        if s["op"] == "gemm_grouped":
            return dg.gemm_grouped(s["x"], s["w"], s["y"], s["offsets"], scale_a=s["sa"], scale_b=s["sb"])
        if s["op"] == "gemm_grouped_dw":
            return dg.gemm_grouped_dw(s["x"], s["dy"], s["dw"], s["offsets"])
        if s["op"] == "quantize_mx4":
            dg.quantize_mx4(s["x"], s["codes"], s["scales"], block=s["block"], scale=s["scale"])
            return dg.dequantize_mx4(s["codes"], s["scales"], s["y"], block=s["block"], scale=s["scale"])
        a, b = (dg.mx4(o["codes"], o["scales"], K=s["K"], block=s["block"], scale=o["scale"]) for o in (s["a"], s["b"]))
        return dg.gemm_mx4(a, b, s["c"])
    return {"gemm_grouped": _plain_grouped, "gemm_grouped_dw": _plain_grouped_dw, "quantize_mx4": _plain_quantize,
            "gemm_mx4": _plain_mx4}[s["op"]](s)


def work(case):
    K = case["K"]
    if case["op"] == "quantize_mx4":
        # in, codes and scales out, and the values read back out
        n, R = -(-K // case["block"]), case["R"]
        return {"bytes": R * (2 * K * SIZE[case["dtype"]] + (K + 1) // 2 + n), "flops": 4 * R * K}
    N = case["N"]
    if case["op"] == "gemm_mx4":
        M, n = case["M"], -(-K // case["block"])
        return {"bytes": (M + N) * ((K + 1) // 2 + n) + M * N * SIZE[case["out"]], "flops": 2 * M * K * N}
    R, es, used = case["R"], SIZE[case["dtype"]], sum(c > 0 for c in _sizes(case))
    if case["op"] == "gemm_grouped_dw":
        return {"bytes": R * (K + N) * es + case["G"] * K * N * SIZE[case["out"]], "flops": 2 * R * K * N}
    scales = 4 * (R + used * N) if case["dtype"] == "e4m3" else 0
    return {"bytes": R * K * es + used * K * N * es + R * N * SIZE[case["out"]] + scales, "flops": 2 * R * K * N}


# ---------------------------------------------------- the definitions, in FP64

def _exact_blocks(x, block, scale):
    """The values that a matrix's quantisation stands for.  The value that is quantised is the FP32 quotient of
    the input and the factor; its block's scale is a power of two, or the FP32 quotient by 6 in E4M3."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    u = x.double() if scale is None else (x.double() / scale.double()).float().double()
    out = torch.empty_like(u)
    for k0 in range(0, u.shape[1], block):
        v = u[:, k0:k0 + block]
        top = v.abs().amax(1, keepdim=True)
        if block == 32:
            unit = 2.0 ** (torch.floor(torch.log2(top)) - 2).clamp(min=-127)
        else:
            unit = (top / 6).float().clamp(max=448).to(torch.float8_e4m3fn).double()
        m = torch.where(unit > 0, v.abs() / unit, 0.0)
        # the nearest of the eight magnitudes; between two, the one whose index is even
        at = torch.bucketize(m, table[1:], right=True)
        low, high = table[at], table[(at + 1).clamp(max=7)]
        up = (m - low > high - m) | ((m - low == high - m) & (at % 2 == 1))
        out[:, k0:k0 + block] = torch.where(up, high, low) * unit * torch.sign(v)
    return out if scale is None else out * scale.double()


def _exact_read(o, K, block):
    """The values of a quantised operand, element by element."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    R = o["codes"].shape[0]
    r, k = torch.arange(R, device="cuda")[:, None], torch.arange(K, device="cuda")
    b = k // block
    tile = r // 128 * ((-(-K // block) + 3) // 4) + b // 4
    code = o["scales"][tile * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]
    if block == 32:
        unit = 2.0 ** (code.double() - 127)
    else:
        unit = torch.where(code < 8, code.double() / 512, (1 + (code % 8).double() / 8) * 2.0 ** ((code // 8).double() - 7))
    e = (o["codes"][:, k // 2].int() >> (4 * (k % 2)).int()) % 16
    v = table[e % 8] * torch.where(e > 7, -1.0, 1.0) * unit
    return v if o["scale"] is None else v * o["scale"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize_mx4":
        return _exact_blocks(s["x"], case["block"], s["scale"])
    if case["op"] == "gemm_mx4":
        return torch.einsum("mk,nk->mn", _exact_read(s["a"], case["K"], case["block"]),
                            _exact_read(s["b"], case["K"], case["block"]))
    ends = s["offsets"].tolist()
    x = s["x"].double()
    if case["op"] == "gemm_grouped_dw":
        dw = torch.zeros(case["G"], case["K"], case["N"], dtype=torch.float64, device="cuda")
        for g, (r0, r1) in enumerate(zip(ends, ends[1:])):
            dw[g] = torch.einsum("rk,rn->kn", x[r0:r1], s["dy"][r0:r1].double())
        return dw
    y = torch.empty(case["R"], case["N"], dtype=torch.float64, device="cuda")
    for g, (r0, r1) in enumerate(zip(ends, ends[1:])):
        y[r0:r1] = torch.einsum("rk,kn->rn", x[r0:r1], s["w"][g].double())
        if s["sa"] is not None:
            y[r0:r1] *= s["sa"][r0:r1, None].double() * s["sb"][g].double()
    return y
