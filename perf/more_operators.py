"""Measured cases of the 8-bit operators: rows of int8 with one scale each, as the operands of
products (decode and prompt) and as checkpoints of activations that the gradients read.

``run`` computes a case either with elementary torch operations in 32 bits, rounded once at the
end, or, where ``own`` is true, with the package's entry points. A matrix of weights is int8
[N][K], one row and one scale per output channel; activations are int8 [M][K], one row and one
scale per token. M counts rows, K is what a token has before the product and N after it.
"""
import math

import torch

own = False


def listed():
    return [
        # what one short step of eight requests keeps for later: the smallest call, latency counts
        {"name": "checkpoint 8 rows of 4096 fp16", "op": "checkpoint", "M": 8, "K": 4096,
         "type": "fp16"},
        # the gated block's product of one sequence of the prefill configuration, kept in 8 bits
        {"name": "checkpoint 2048 rows of 11008 bf16", "op": "checkpoint", "M": 2048, "K": 11008,
         "type": "bf16"},
        # attention projection of one token
        {"name": "gemv 1 row 4096x4096", "op": "gemv", "M": 1, "K": 4096, "N": 4096},
        # down projection of a 7B layer for a decode batch of eight
        {"name": "gemv 8 rows 11008x4096", "op": "gemv", "M": 8, "K": 11008, "N": 4096},
        # 33 requests decoding at once: an odd row count, the weights' bytes count
        {"name": "gemm 33 rows 4096x11008 fp16", "op": "gemm", "M": 33, "K": 4096, "N": 11008,
         "type": "fp16"},
        # shared expert (hidden 5120) for a ragged batch, results kept in fp32
        {"name": "gemm 777 rows 5120x1536 fp32", "op": "gemm", "M": 777, "K": 5120, "N": 1536,
         "type": "fp32"},
        # the prompt of the prefill configuration
        {"name": "gemm 2048 rows 4096x11008 bf16", "op": "gemm", "M": 2048, "K": 4096, "N": 11008,
         "type": "bf16"},
        # gradient of the down projection for a short ragged batch
        {"name": "backward 150 rows 11008x4096", "op": "backward", "M": 150, "K": 11008,
         "N": 4096},
        # gradient of a 7B feed-forward projection for one sequence
        {"name": "backward 2048 rows 4096x11008", "op": "backward", "M": 2048, "K": 4096,
         "N": 11008},
        # narrow half of an adapter of rank 16 beside the down projection, ragged batch
        {"name": "weight gradient 1999 rows 11008x16", "op": "weight", "M": 1999, "K": 11008,
         "N": 16},
        # weights of a shared expert for a ragged batch
        {"name": "weight gradient 777 rows 5120x1536", "op": "weight", "M": 777, "K": 5120,
         "N": 1536},
        # weights of a 7B feed-forward projection for one sequence
        {"name": "weight gradient 2048 rows 4096x11008", "op": "weight", "M": 2048, "K": 4096,
         "N": 11008},
    ]


TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
MOST = 2048 * 4096 * 11008  # products of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["checkpoint", "gemv", "gemm", "backward", "weight"])
    if op == "checkpoint":
        # any row length, whole or odd
        c = {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 1, 16384)}
        if c["M"] * c["K"] > 2048 * 11008:
            c["M"] = 2048 * 11008 // c["K"]
        c["type"] = rng.choice(["fp32", "fp16", "bf16"])
        return c
    c = {"op": op, "K": 16 * _log(rng, 4, 688), "N": 8 * _log(rng, 1, 1376)}
    if op == "gemv":
        c["M"] = rng.randint(1, 8)
    else:
        c["M"] = min(_log(rng, 1, 4096), MOST // (c["K"] * c["N"]))
    if op == "gemm":
        c["type"] = rng.choice(["fp32", "fp16", "bf16"])
    return c


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(x):
    """Rows of x as int8 and one fp32 scale a row: the scale is the largest magnitude over 127,
    values go to the nearest multiple (ties to the even one). The quotient is taken in 64 bits:
    in 32 a value just beside a half would be taken for one."""
    scale = x.float().abs().amax(dim=1) / 127.0
    q = torch.round(x.double() / scale.double()[:, None]).clamp(-127.0, 127.0)
    q = torch.where(scale[:, None] > 0, q, torch.zeros_like(q))
    return q.to(torch.int8), scale


def _activations(g, M, K):
    """Tokens of differing sizes, with a few channels that are large in every token."""
    size = torch.exp(0.5 * _normal(g, M, 1))
    channel = torch.ones((1, K), device="cuda")
    channel[:, torch.rand((K,), generator=g, device="cuda") < 0.005] = 8.0
    return _normal(g, M, K) * size * channel


def _gradient(g, M, N):
    """Rows of gradients: small, of sizes that differ from token to token."""
    size = torch.exp(_normal(g, M, 1) - 9.0)
    return (_normal(g, M, N) * size).bfloat16()


def prepare(case, seed):
    g = _gen(seed)
    op, M, K = case["op"], case["M"], case["K"]
    s = dict(case)
    if op in ("checkpoint", "gemv"):
        s["x"] = _activations(g, M, K).to(TYPES[case.get("type", "fp32")])
    elif op in ("gemm", "weight"):
        s["X"], s["sx"] = _rows(_activations(g, M, K))
    if op in ("gemv", "gemm", "backward"):
        s["W"], s["sw"] = _rows(_normal(g, case["N"], K) / math.sqrt(K))
    if op in ("backward", "weight"):
        s["dY"] = _gradient(g, M, case["N"])
    return s


# ------------------------------------------------------------------------------ plain form
def _plain(s):
    op = s["op"]
    if op == "checkpoint":
        q, scale = _rows(s["x"])
        return (q.float() * scale[:, None]).to(s["x"].dtype), scale
    if op == "gemv":
        q, scale = _rows(s["x"])
        return (q.float() @ s["W"].float().T) * scale[:, None] * s["sw"]
    if op == "gemm":
        y = (s["X"].float() @ s["W"].float().T) * s["sx"][:, None] * s["sw"]
        return y.to(TYPES[s["type"]])
    if op == "backward":
        return ((s["dY"].float() * s["sw"]) @ s["W"].float()).bfloat16()
    return ((s["dY"].float() * s["sx"][:, None]).T @ s["X"].float()).bfloat16()


def _framework(s):
    import moe_experts_amd as q4
    op = s["op"]
    if op == "checkpoint":
        # kept, and restored where the backward pass needs it
        q, scale = q4.i8_quantize(s["x"])
        return q4.i8_dequantize(q, scale, dtype=s["x"].dtype), scale
    if op == "gemv":
        return q4.i8_gemv(s["x"], s["W"], s["sw"])
    if op == "gemm":
        return q4.i8_gemm(s["X"], s["sx"], s["W"], s["sw"], dtype=TYPES[s["type"]])
    if op == "backward":
        return q4.i8_gemm_backward(s["dY"], s["W"], s["sw"])
    return q4.i8_gemm_backward_weight(s["dY"], s["X"], s["sx"])


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------------------ work
def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "checkpoint":
        size = TYPES[case["type"]].itemsize
        return {"bytes": 2 * size * M * K + 4 * M, "flops": 3.0 * M * K}
    N = case["N"]
    flops = 2.0 * M * K * N
    if op == "gemv":
        return {"bytes": K * N + 4 * N + 4 * M * (K + N), "flops": flops}
    if op == "gemm":
        return {"bytes": K * (M + N) + 4 * (M + N) + TYPES[case["type"]].itemsize * M * N,
                "flops": flops}
    if op == "backward":
        return {"bytes": K * N + 4 * N + 2 * M * (K + N), "flops": flops}
    return {"bytes": M * K + 4 * M + 2 * N * (M + K), "flops": flops}


# ------------------------------------------------------------------------------ in 64 bits
def _nearest64(x):
    """(whole numbers, scale) of the rows of x, in 64 bits; the scale is an fp32 number by
    definition."""
    x = x.to(torch.float64)
    scale = (torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True) / 127).float().double()
    t = x / torch.where(scale == 0, torch.ones_like(scale), scale)
    low = torch.floor(t)
    up = (t - low > 0.5) | ((t - low == 0.5) & (torch.remainder(low, 2) == 1))
    return (low + up).clamp_(-127, 127), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        q, scale = _nearest64(s["x"])
        return q * scale, scale[:, 0]
    if op == "backward":
        return torch.matmul(s["dY"].double(), s["W"].double() * s["sw"].double()[:, None])
    if op == "weight":
        values = s["X"].double() * s["sx"].double()[:, None]
        return torch.matmul(s["dY"].double().t().contiguous(), values)
    weights = s["W"].double() * s["sw"].double()[:, None]
    if op == "gemv":
        q, scale = _nearest64(s["x"])
        values = q * scale
    else:
        values = s["X"].double() * s["sx"].double()[:, None]
    return torch.matmul(values, weights.t())
