"""Measured cases of the dense feed-forward operators over frozen Q4_0 weights: the gated block
(decode, prompt, gradient), the projection with the low-rank adapters of many requests (decode,
prompt), and the gradient of a projection.

``run`` computes a case either with elementary torch operations on the dequantized weights, in
32 bits and rounded once at the end, or, where ``own`` is true, with the package's entry points.
Every size is given as rows M, contraction K and columns N of the Q4_0 matrix [K, N/32 blocks].
"""
import math

import torch

own = False

BLOCK = 32
BLOCK_BYTES = 18


def listed():
    return [
        # the shared expert of one token (hidden 5120, 1536 columns): the smallest call, latency counts
        {"name": "glu 1 row 5120x1536", "op": "glu", "M": 1, "K": 5120, "N": 1536, "act": "silu"},
        # gate and up of a 7B layer for a decode batch of eight
        {"name": "glu 8 rows 4096x11008", "op": "glu", "M": 8, "K": 4096, "N": 11008, "act": "silu"},
        # 33 requests decoding at once, or a short prompt: an odd row count, the weights' bytes count
        {"name": "glu_gemm 33 rows 4096x11008", "op": "glu_gemm", "M": 33, "K": 4096, "N": 11008,
         "act": "gelu", "save": False},
        # the prompt of the prefill configuration, keeping gate and up for the gradient
        {"name": "glu_gemm 2048 rows 4096x11008", "op": "glu_gemm", "M": 2048, "K": 4096,
         "N": 11008, "act": "silu", "save": True},
        # gradient through a shared expert for a ragged batch
        {"name": "glu_backward 777 rows 5120x1536", "op": "glu_backward", "M": 777, "K": 5120,
         "N": 1536, "act": "gelu"},
        # gradient through the 7B feed-forward for one sequence of 2048 tokens
        {"name": "glu_backward 2048 rows 4096x11008", "op": "glu_backward", "M": 2048, "K": 4096,
         "N": 11008, "act": "silu"},
        # attention projection of one request with its own adapter
        {"name": "gemv_lora 1 row 4096x4096 r16", "op": "gemv_lora", "M": 1, "K": 4096, "N": 4096,
         "R": 16, "L": 8, "none": 0.0, "run": 1},
        # down projection of eight requests with eight adapters of rank 64
        {"name": "gemv_lora 8 rows 11008x4096 r64", "op": "gemv_lora", "M": 8, "K": 11008,
         "N": 4096, "R": 64, "L": 16, "none": 0.1, "run": 1},
        # 48 requests decoding at once, nearly every one with another adapter, some with none
        {"name": "gemm_lora 48 rows 4096x4096 r16", "op": "gemm_lora", "M": 48, "K": 4096,
         "N": 4096, "R": 16, "L": 40, "none": 0.1, "run": 1},
        # the prompts of about seven requests in one batch through the down projection
        {"name": "gemm_lora 2000 rows 11008x4096 r32", "op": "gemm_lora", "M": 2000, "K": 11008,
         "N": 4096, "R": 32, "L": 7, "none": 0.1, "run": 300},
        # gradient of the down projection for a short ragged batch
        {"name": "gemm_backward 150 rows 11008x4096", "op": "gemm_backward", "M": 150, "K": 11008,
         "N": 4096},
        # gradient of an attention projection for one sequence
        {"name": "gemm_backward 2048 rows 4096x4096", "op": "gemm_backward", "M": 2048, "K": 4096,
         "N": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu", "glu_gemm", "glu_backward", "gemv_lora", "gemm_lora", "gemm_backward"])
    if op in ("glu", "gemv_lora"):
        # decode: any K, N a multiple of the block
        c = {"op": op, "M": rng.randint(1, 8), "K": _log(rng, 200, 11008),
             "N": BLOCK * _log(rng, 8, 344)}
        if op == "gemv_lora":
            c["K"] = max(8, c["K"] // 8 * 8)
    else:
        c = {"op": op, "M": _log(rng, 1, 2048), "K": 64 * _log(rng, 4, 172),
             "N": 64 * _log(rng, 4, 172)}
        while 2.0 * c["M"] * c["K"] * c["N"] > 2.0 * 2048 * 4096 * 11008:
            c["M"] = c["M"] // 2 + 1
    if op.startswith("glu"):
        c["act"] = rng.choice(["silu", "gelu"])
    if op == "glu_gemm":
        c["save"] = rng.random() < 0.5
    if op.endswith("lora"):
        c["R"] = 8 * rng.choice([1, 2, 3, 4, 8])
        c["L"] = _log(rng, 1, 48)
        c["none"] = rng.choice([0.0, 0.1, 0.5])
        c["run"] = 1 if c["M"] <= 64 else _log(rng, 1, 600)
    return c


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, K, N):
    """A normal matrix of deviation 1/sqrt(K), rounded to Q4_0: each block of 32 columns by its
    largest value, which becomes -8. uint8 [K, N/32, 18]."""
    w = _normal(g, K, N // BLOCK, BLOCK) / math.sqrt(K)
    at = w.abs().argmax(dim=-1, keepdim=True)
    d = (w.gather(-1, at) / -8.0).half()
    q = (w / d.float()).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
    out = torch.empty((K, N // BLOCK, BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    out[..., :2] = d.view(torch.uint8)
    out[..., 2:] = q[..., 0::2] | (q[..., 1::2] << 4)
    return out


def _gradient(g, M, N):
    """Rows of gradients: small, of sizes that differ from token to token."""
    size = torch.exp(_normal(g, M, 1) - 9.0)
    return (_normal(g, M, N) * size).bfloat16()


def _adapters(g, case, s):
    M, K, N, R, L = (case[k] for k in "MKNRL")
    a = _normal(g, L, R, K) / math.sqrt(K)
    b = _normal(g, L, N, R) * 0.05
    # every third adapter has half the rank: the rest of its rows and columns are zero
    a[2::3, R // 2:] = 0
    s["A"], s["Bl"] = a.half(), b.half()
    s["scale"] = torch.rand((L,), generator=g, device="cuda") * 1.5 + 0.5
    # requests are consecutive rows of about `run` rows each; some carry no adapter
    n = M // case["run"] + 1
    ids = torch.randint(0, L, (n,), generator=g, device="cuda", dtype=torch.int32)
    bare = torch.rand((n,), generator=g, device="cuda") < case["none"]
    ids = torch.where(bare, torch.full_like(ids, -1), ids)
    cuts = torch.sort(torch.randint(0, M + 1, (n - 1,), generator=g, device="cuda")).values
    rows = torch.arange(M, device="cuda")
    of = rows if case["run"] == 1 else torch.bucketize(rows, cuts, right=True)
    s["ids"] = ids[of].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    s = dict(case)
    if op.startswith("glu"):
        s["Wg"], s["Wu"] = _weights(g, K, N), _weights(g, K, N)
    else:
        s["B"] = _weights(g, K, N)
    if op in ("glu", "gemv_lora"):
        s["x"] = _normal(g, M, K)
    elif op in ("glu_gemm", "gemm_lora"):
        s["x"] = _normal(g, M, K).half()
    elif op == "glu_backward":
        s["dH"] = _gradient(g, M, N)
        s["G"], s["U"] = _normal(g, M, N).half(), _normal(g, M, N).half()
    else:
        s["dY"] = _gradient(g, M, N)
    if op.endswith("lora"):
        _adapters(g, case, s)
    return s


# ------------------------------------------------------------------------------ plain form
def _dequantized(B):
    """Q4_0 bytes [K, N/32, 18] -> fp32 [K, N]: (q - 8) * d, the low nibble first."""
    K = B.shape[0]
    d = B[..., :2].contiguous().view(torch.float16).float()
    qs = B[..., 2:]
    q = torch.stack((qs & 15, qs >> 4), dim=-1).float().reshape(K, -1, BLOCK)
    return ((q - 8.0) * d).reshape(K, -1)


_C = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.tanh(_C * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    t = torch.tanh(_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)


def _adapter_part(x, A, Bl, ids, scale):
    """scale[id] * (x . A[id]^T) . Bl[id]^T of each row, as one product over all adapters in which
    every row keeps only its own."""
    L, R, K = A.shape
    mine = (ids[:, None] == torch.arange(L, device=ids.device)).float() * scale
    t = (x @ A.float().reshape(L * R, K).T).reshape(-1, L, R) * mine[:, :, None]
    return t.reshape(-1, L * R) @ Bl.float().permute(0, 2, 1).reshape(L * R, -1)


def _plain(s):
    op = s["op"]
    if op == "glu":
        return _act(s["x"] @ _dequantized(s["Wg"]), s["act"]) * (s["x"] @ _dequantized(s["Wu"]))
    if op == "glu_gemm":
        x = s["x"].float()
        g, u = x @ _dequantized(s["Wg"]), x @ _dequantized(s["Wu"])
        h = (_act(g, s["act"]) * u).half()
        return (h, g.half(), u.half()) if s["save"] else h
    if op == "glu_backward":
        dh, g, u = s["dH"].float(), s["G"].float(), s["U"].float()
        dg, du = dh * u * _act_slope(g, s["act"]), dh * _act(g, s["act"])
        return (dg @ _dequantized(s["Wg"]).T + du @ _dequantized(s["Wu"]).T).bfloat16()
    if op == "gemm_backward":
        return (s["dY"].float() @ _dequantized(s["B"]).T).bfloat16()
    x = s["x"].float()
    y = x @ _dequantized(s["B"]) + _adapter_part(x, s["A"], s["Bl"], s["ids"], s["scale"])
    return y if op == "gemv_lora" else y.half()


def _framework(s):
    import moe_experts_amd as q4
    op = s["op"]
    if op == "glu":
        return q4.q4_0_glu(s["x"], s["Wg"], s["Wu"], s["N"], act=s["act"])
    if op == "glu_gemm":
        return q4.q4_0_glu_gemm(s["x"], s["Wg"], s["Wu"], s["N"], act=s["act"], save=s["save"])
    if op == "glu_backward":
        return q4.q4_0_glu_backward(s["dH"], s["G"], s["U"], s["Wg"], s["Wu"], s["K"],
                                    act=s["act"])
    if op == "gemm_backward":
        return q4.q4_0_gemm_backward(s["dY"], s["B"], s["K"])
    call = q4.q4_0_gemv_lora if op == "gemv_lora" else q4.q4_0_gemm_lora
    return call(s["x"], s["B"], s["N"], s["A"], s["Bl"], s["ids"], s["scale"])


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------------------ work
def work(case):
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    matrix = K * (N // BLOCK) * BLOCK_BYTES
    flops = 2.0 * M * K * N
    if op == "glu":
        return {"bytes": 2 * matrix + 4 * M * (K + N), "flops": 2 * flops}
    if op == "glu_gemm":
        return {"bytes": 2 * matrix + 2 * M * K + 2 * M * N * (3 if case["save"] else 1),
                "flops": 2 * flops}
    if op == "glu_backward":
        return {"bytes": 2 * matrix + 2 * M * (3 * N + K), "flops": 2 * flops}
    if op == "gemm_backward":
        return {"bytes": matrix + 2 * M * (N + K), "flops": flops}
    # adapters in use: at most one a request
    used = min(case["L"], M // case["run"] + 1)
    size = 4 if op == "gemv_lora" else 2
    return {"bytes": matrix + size * M * (K + N) + 2 * used * case["R"] * (K + N) + 4 * M,
            "flops": flops + 2.0 * M * case["R"] * (K + N)}


# ------------------------------------------------------------------------------ in 64 bits
def _values64(B):
    """The weights of Q4_0 bytes in 64 bits: nibble i of a block is column i."""
    K, nb = B.shape[:2]
    raw = B.to(torch.int64)
    d = (raw[..., 0] | (raw[..., 1] << 8)).to(torch.int16).view(torch.float16).double()
    w = torch.empty((K, nb, BLOCK), dtype=torch.float64, device=B.device)
    w[..., 0::2] = (raw[..., 2:] % 16 - 8).double()
    w[..., 1::2] = (raw[..., 2:] // 16 - 8).double()
    return w.mul_(d[..., None]).reshape(K, nb * BLOCK)


def _act64(z, act):
    """Activation and slope: z * sigmoid(p(z)), with p(z) = z or, since (1 + tanh a) / 2 =
    sigmoid(2a), the cubic of the tanh form of GELU."""
    c = 2.0 * math.sqrt(2.0 / math.pi)
    p = z if act == "silu" else c * (z + 0.044715 * z ** 3)
    dp = torch.ones_like(z) if act == "silu" else c * (1.0 + 0.134145 * z ** 2)
    sig = torch.sigmoid(p)
    return z * sig, sig + z * sig * torch.sigmoid(-p) * dp


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("glu", "glu_gemm"):
        x = s["x"].double()
        g, u = torch.matmul(x, _values64(s["Wg"])), torch.matmul(x, _values64(s["Wu"]))
        h = _act64(g, case["act"])[0] * u
        return (h, g, u) if case.get("save") else h
    if op == "glu_backward":
        dh, g, u = (s[k].double() for k in ("dH", "G", "U"))
        a, slope = _act64(g, case["act"])
        dx = torch.matmul(dh * slope * u, _values64(s["Wg"]).t())
        return dx.add_(torch.matmul(dh * a, _values64(s["Wu"]).t()))
    if op == "gemm_backward":
        return torch.matmul(s["dY"].double(), _values64(s["B"]).t())
    x = s["x"].double()
    y = torch.matmul(x, _values64(s["B"]))
    for i in range(case["L"]):
        rows = (s["ids"] == i).nonzero()[:, 0]
        if rows.numel():
            t = torch.matmul(x[rows], s["A"][i].double().t())
            y[rows] += s["scale"][i].double() * torch.matmul(t, s["Bl"][i].double().t())
    return y
