"""The measured cases of the library's language-model operators.

Three operators, around the weight of a projection or of the output layer:

  gemv_w4         y = alpha * x W for up to 8 tokens, W held in 4 bits with one
                  scale (and, optionally, one zero point) per group of k
  linear_ce       loss[t] = logsumexp_v(z[t]) - z[t][target[t]], z = alpha * X W,
                  without keeping the logits z
  linear_ce_grad  dX and dW of sum_t dloss[t] * loss[t]

`run` computes them in plain torch operations in FP32, or, where `own` is
true, through the library.  Rows whose target is -100 are padding: their loss
is 0 and they take no part in the gradients.
"""
import math

import torch

own = False

IGNORE = -100
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through a small expert projection: launch latency is most of it
        {"name": "w4-expert-1", "op": "gemv_w4", "R": 1, "K": 512, "N": 4096, "group": 32, "dtype": "bf16",
         "scale": "bf16", "zeros": False, "out": "bf16"},
        # one token through the decode step's up projection
        {"name": "w4-decode-1", "op": "gemv_w4", "R": 1, "K": 4096, "N": 14336, "group": 128, "dtype": "bf16",
         "scale": "bf16", "zeros": True, "out": "bf16"},
        # eight sequences through the down projection
        {"name": "w4-down-8", "op": "gemv_w4", "R": 8, "K": 14336, "N": 4096, "group": 64, "dtype": "f16",
         "scale": "f16", "zeros": True, "out": "f16"},
        # sizes that fill no tile, rows of codes that start at odd multiples of four bytes
        {"name": "w4-odd-3", "op": "gemv_w4", "R": 3, "K": 5000, "N": 5003, "group": 128, "dtype": "f16",
         "scale": "f32", "zeros": False, "out": "f32"},
        # one token's logits over a large vocabulary
        {"name": "w4-head-1", "op": "gemv_w4", "R": 1, "K": 4096, "N": 128000, "group": 128, "dtype": "bf16",
         "scale": "bf16", "zeros": True, "out": "f32"},
        # the score of one token (choosing between candidate answers)
        {"name": "ce-score-1", "op": "linear_ce", "T": 1, "D": 4096, "V": 32000, "dtype": "bf16", "ignored": 0.0},
        # the loss of a training micro-batch
        {"name": "ce-train", "op": "linear_ce", "T": 2048, "D": 4096, "V": 32000, "dtype": "bf16", "ignored": 0.1},
        # a ragged batch with a third of its rows padded, a vocabulary of odd size
        {"name": "ce-odd", "op": "linear_ce", "T": 777, "D": 1000, "V": 50257, "dtype": "f16", "ignored": 0.33},
        # a long sequence over a large vocabulary
        {"name": "ce-long", "op": "linear_ce", "T": 8192, "D": 4096, "V": 128000, "dtype": "bf16", "ignored": 0.0},
        # fine-tuning on one short answer
        {"name": "grad-64", "op": "linear_ce_grad", "T": 64, "D": 4096, "V": 32000, "dtype": "bf16", "ignored": 0.25},
        # the gradient of the ragged batch, with the loss scale of FP16 training
        {"name": "grad-odd", "op": "linear_ce_grad", "T": 777, "D": 1000, "V": 50257, "dtype": "f16", "ignored": 0.33},
        # the gradient of a full training batch
        {"name": "grad-8192", "op": "linear_ce_grad", "T": 8192, "D": 4096, "V": 32000, "dtype": "bf16",
         "ignored": 0.05},
    ]


MOST_W4 = 4096 * 128000          # weights of the largest listed product
MOST_CE = 8192 * 4096 * 32000    # multiply-adds of the largest listed gradient's logits


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv_w4", "linear_ce", "linear_ce_grad"])
    if op == "gemv_w4":
        K = _log(rng, 128, 16384)
        if rng.random() < 0.6:
            K = max(128, K // 64 * 64)
        N = _log(rng, 64, min(128000, MOST_W4 // K))
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "R": rng.randint(1, 8), "K": K, "N": N, "group": rng.choice([32, 64, 128, 256]),
                "dtype": dtype, "scale": rng.choice([dtype, "f32"]), "zeros": rng.random() < 0.5,
                "out": rng.choice([dtype, "f32"])}
    D = _log(rng, 64, 8192)
    if rng.random() < 0.8:
        D = max(64, D // 8 * 8)
    V = _log(rng, 100, 128000)
    T = _log(rng, 1, max(1, min(8192, MOST_CE // (D * V))))
    return {"op": op, "T": T, "D": D, "V": V, "dtype": rng.choice(["bf16", "f16"]),
            "ignored": rng.choice([0.0, 0.05, 0.3])}


# ----------------------------------------------------------------- the inputs

def _prepare_w4(case, g):
    """Weights quantised from normal data to the nearest of 16 steps per group: between the group's extremes
    with zero points, between -7 and 7 times the scale (codes 1 to 15 around 8) without."""
    K, N, G = case["K"], case["N"], case["group"]
    groups = (K + G - 1) // G
    w = torch.randn(N, groups * G, generator=g, device="cuda") * 0.02
    w[:, K:] = 0
    w = w.view(N, groups, G)
    if case["zeros"]:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).to(DT[case["scale"]])
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
    else:
        scale = (w.abs().amax(2) / 7).to(DT[case["scale"]])
        zero = torch.full_like(scale, 8.0, dtype=torch.float32)
    q = (torch.round(w / scale.float().unsqueeze(2)) + zero.unsqueeze(2)).clamp(0, 15)
    q = q.to(torch.uint8).view(N, groups * G)[:, :K + K % 2]
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return {"op": "gemv_w4", "group": G, "K": K,
            "x": torch.randn(case["R"], K, generator=g, device="cuda").to(DT[case["dtype"]]),
            "codes": codes, "scales": scale.contiguous(),
            "zeros": zero.to(torch.uint8).contiguous() if case["zeros"] else None,
            "y": torch.empty(case["R"], N, device="cuda", dtype=DT[case["out"]])}


def _prepare_ce(case, g):
    T, D, V, dt = case["T"], case["D"], case["V"], DT[case["dtype"]]
    x = torch.randn(T, D, generator=g, device="cuda").to(dt)
    weight = (torch.randn(V, D, generator=g, device="cuda") * (2.0 / math.sqrt(D))).to(dt)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    padded = torch.rand(T, generator=g, device="cuda") < case["ignored"]
    target = torch.where(padded, torch.full_like(target, IGNORE), target)
    state = {"op": case["op"], "x": x, "weight": weight, "target": target}
    if case["op"] == "linear_ce":
        state["loss"] = torch.empty(T, device="cuda")
        state["lse"] = torch.empty(T, device="cuda")
        return state
    # the forward pass's logsumexp, which the training program kept
    lse = torch.empty(T, device="cuda")
    for t0 in range(0, T, 1024):
        z = x[t0:t0 + 1024].double() @ weight.double().t()
        lse[t0:t0 + 1024] = torch.logsumexp(z, 1).float()
    scale = 1024.0 if case["dtype"] == "f16" else 1.0
    state["lse"] = lse
    state["dloss"] = torch.full((T,), scale / max(1, int((~padded).sum())), device="cuda")
    state["dx"] = torch.empty_like(x)
    state["dweight"] = torch.empty_like(weight)
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return _prepare_w4(case, g) if case["op"] == "gemv_w4" else _prepare_ce(case, g)


# ------------------------------------------------------------------- one pass

def _plain_w4(s):
    x, codes, K, G = s["x"], s["codes"], s["K"], s["group"]
    q = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1)[:, :K].float()
    scale = s["scales"].float().repeat_interleave(G, 1)[:, :K]
    zero = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(G, 1)[:, :K]
    return (x.float() @ (scale * (q - zero)).t()).to(s["y"].dtype)


def _plain_ce(s):
    z = s["x"].float() @ s["weight"].float().t()
    valid = s["target"] != IGNORE
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    hit = z.gather(1, torch.where(valid, s["target"], 0)[:, None])[:, 0]
    return {"loss": torch.where(valid, lse - hit, 0.0), "lse": lse}


def _plain_ce_grad(s):
    x, w = s["x"].float(), s["weight"].float()
    valid = s["target"] != IGNORE
    p = torch.exp(x @ w.t() - s["lse"][:, None])
    index = torch.where(valid, s["target"], 0)[:, None]
    p.scatter_add_(1, index, torch.full_like(index, -1, dtype=torch.float32))
    p *= torch.where(valid, s["dloss"], 0.0)[:, None]
    return {"dx": (p @ w).to(s["x"].dtype), "dweight": (p.t() @ x).to(s["x"].dtype)}


def run(state):
    s = state
    if own:
        import tcgen05_tmem_gemm_b200 as dg

        if s["op"] == "gemv_w4":
            return dg.gemv_w4(s["x"], s["codes"], s["scales"], s["y"], zeros=s["zeros"], group=s["group"])
        w = s["weight"].t()
        if s["op"] == "linear_ce":
            dg.linear_ce(s["x"], w, s["target"], s["loss"], s["lse"], ignore_index=IGNORE)
            return {"loss": s["loss"], "lse": s["lse"]}
        dg.linear_ce_grad(s["x"], w, s["target"], s["lse"], s["dloss"], dx=s["dx"], dw=s["dweight"].t(),
                          ignore_index=IGNORE)
        return {"dx": s["dx"], "dweight": s["dweight"]}
    return {"gemv_w4": _plain_w4, "linear_ce": _plain_ce, "linear_ce_grad": _plain_ce_grad}[s["op"]](s)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "gemv_w4":
        R, K, N = case["R"], case["K"], case["N"]
        groups = (K + case["group"] - 1) // case["group"]
        weights = N * ((K + 1) // 2) + N * groups * (size[case["scale"]] + (1 if case["zeros"] else 0))
        return {"bytes": weights + R * K * 2 + R * N * size[case["out"]], "flops": 2 * R * K * N}
    T, D, V = case["T"], case["D"], case["V"]
    if case["op"] == "linear_ce":
        return {"bytes": (T * D + V * D) * 2 + T * 16, "flops": 2 * T * D * V}
    # the logits again, and the two products of the gradients
    return {"bytes": 2 * (T * D + V * D) * 2 + T * 16, "flops": 6 * T * D * V}


# ---------------------------------------------------- the definitions, in FP64

def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "gemv_w4":
        K, N = case["K"], case["N"]
        k = torch.arange(K, device="cuda")
        group = k // case["group"]
        y = torch.empty(case["R"], N, dtype=torch.float64, device="cuda")
        for n0 in range(0, N, 16384):
            n1 = min(N, n0 + 16384)
            code = (s["codes"][n0:n1, k // 2].int() >> (4 * (k % 2)).int()) % 16
            zero = s["zeros"][n0:n1, group].int() if case["zeros"] else 8
            y[:, n0:n1] = torch.einsum("rk,nk->rn", x, (code - zero).double() * s["scales"][n0:n1, group].double())
        return y
    w = s["weight"].double()
    T = case["T"]
    if case["op"] == "linear_ce":
        loss, lse = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.empty(T, dtype=torch.float64, device="cuda")
        for t0 in range(0, T, 2048):
            z = torch.einsum("td,vd->tv", x[t0:t0 + 2048], w)
            lse[t0:t0 + 2048] = torch.logsumexp(z, 1)
            y = s["target"][t0:t0 + 2048]
            kept = (y != IGNORE).nonzero()[:, 0]
            loss[t0 + kept] = lse[t0 + kept] - z[kept, y[kept]]
        return {"loss": loss, "lse": lse}
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    kept = (s["target"] != IGNORE).nonzero()[:, 0]
    for t in kept.split(2048):
        p = torch.softmax(torch.einsum("td,vd->tv", x[t], w), 1)
        p[torch.arange(len(t), device="cuda"), s["target"][t]] -= 1
        p *= s["dloss"][t].double()[:, None]
        dx[t] = torch.einsum("tv,vd->td", p, w)
        dw += torch.einsum("tv,td->vd", p, x[t])
    return {"dx": dx, "dweight": dw}
