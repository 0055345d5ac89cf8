"""The 8-bit and block-boundary operators of the library as calls to be measured.

listed() names real calls over the operators' range and draw() gives more of them; prepare() makes
the inputs, run() is one call (the library's kernels where `own` is true, elementary torch
operations where it is not), work() the bytes and operations the call cannot do without, and
exact() its outputs in 64 bits.

Operators ("op" of a case):
  quant  x [rows][K] -> int8 rows of T(x) with a scale per row, returned as the values they stand
         for, and the scales
  gemm   int8 rows x int8 rows, scaled per token and per output channel, optional bias
  norm   norm after a block, gate, residual add, norm before the next block
  step   a block boundary as it is served: norm with int8 rows out, then the 8-bit product
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5


def listed():
    return [
        # activations of four decoding requests ahead of an 8-bit layer: launch latency
        dict(name="quant_decode_4x8192", op="quant", rows=4, K=8192, x="bf16", block=256),
        # a prompt's activations ahead of the down projection: one pass over HBM
        dict(name="quant_prefill_2048x28672", op="quant", rows=2048, K=28672, x="bf16", block=256),
        # offline: a weight matrix's rows (output channels), no whitening, fp32 masters
        dict(name="quant_weight_8192x8192", op="quant", rows=8192, K=8192, x="f32", block=0),
        # single-token decode through a 7B-sized projection: the smallest product, latency
        dict(name="gemm_b1_4096x4096", op="gemm", rows=1, K=4096, N=4096, y="bf16", bias=False),
        # sixteen requests through a 70B-sized down projection: the weights stream from HBM
        dict(name="gemm_b16_28672x8192", op="gemm", rows=16, K=28672, N=8192, y="f32", bias=False),
        # a ragged batch on a layer whose sizes divide nothing, with a bias
        dict(name="gemm_b77_4100x1003", op="gemm", rows=77, K=4100, N=1003, y="f16", bias=True),
        # a prompt through a 70B-sized gate/up projection: tensor-core bound
        dict(name="gemm_b2048_8192x28672", op="gemm", rows=2048, K=8192, N=28672, y="bf16",
             bias=False),
        # single-token decode between attention and the MLP: latency of one row
        dict(name="norm_b1_8192", op="norm", rows=1, K=8192, h="f32", r="bf16", y="bf16",
             kind="rms", gate_tokens=0),
        # a prompt at the same place, with a gate per channel: one pass over HBM
        dict(name="norm_b2048_8192", op="norm", rows=2048, K=8192, h="f32", r="bf16", y="bf16",
             kind="rms", gate_tokens=2048),
        # layer norms with a gate row per 64 tokens on an odd width, fp32 residual stream
        dict(name="norm_b333_4097_layer", op="norm", rows=333, K=4097, h="f16", r="f32", y="f32",
             kind="layer", gate_tokens=64),
        # one decoded token across a block boundary into an 8-bit gate/up projection
        dict(name="step_b1_8192x28672", op="step", rows=1, K=8192, N=28672, h="f32", r="bf16",
             y="bf16", block=256),
        # a prompt across a block boundary into an 8-bit square projection
        dict(name="step_b1024_8192x8192", op="step", rows=1024, K=8192, N=8192, h="f32",
             r="bf16", y="bf16", block=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "gemm", "gemm", "norm", "step"))
    rows = _log_int(rng, 1, 4096)
    if op == "quant":
        # values that T mixes in fp32 lie next to rounding borders of the codes: 16-bit inputs
        block = rng.choice((0, 0, 64, 256, 256, 1024))
        K = _log_int(rng, 128, 28672)
        K = max(block, K // block * block) if block else K
        rows = min(rows, 2048 * 28672 // K)
        x = rng.choice(("bf16", "f16")) if block else rng.choice(("bf16", "f16", "f32"))
        return dict(op=op, rows=rows, K=K, x=x, block=block)
    if op == "norm":
        K = _log_int(rng, 128, 16384)
        K = K if rng.random() < 0.4 else max(8, K // 8 * 8)
        rows = min(rows, 2048 * 8192 // K)
        return dict(op=op, rows=rows, K=K, h=rng.choice(("f32", "bf16", "f16")),
                    r=rng.choice(("f32", "bf16", "f16")), y=rng.choice(("f32", "bf16", "f16")),
                    kind=rng.choice(("rms", "rms", "layer")),
                    gate_tokens=rng.choice((0, 1, 64, rows)))
    N = _log_int(rng, 128, 28672)
    if op == "step":
        K = 256 * _log_int(rng, 1, 40)
        rows = max(1, min(rows, 2 * 10 ** 11 // (K * N)))
        return dict(op=op, rows=rows, K=K, N=N, h=rng.choice(("f32", "bf16")), r="bf16",
                    y="bf16", block=256)
    K = _log_int(rng, 128, 28672)
    K = K if rng.random() < 0.3 else max(16, K // 16 * 16)
    rows = max(1, min(rows, 4 * 10 ** 11 // (K * N)))
    return dict(op=op, rows=rows, K=K, N=N, y=rng.choice(("f32", "bf16", "f16")),
                bias=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs


def _hadamard(block, dtype, dev):
    i = torch.arange(block, device=dev)
    bits = i[:, None] & i[None, :]
    for s in (8, 4, 2, 1):
        bits = bits ^ (bits >> s)
    return (1 - 2 * (bits & 1)).to(dtype)


def _activations(gen, rows, K, dtype, dev):
    """N(0, 1) rows; every second one has 1 % of its inputs times 20."""
    x = torch.randn(rows, K, generator=gen, device=dev)
    big = torch.rand(rows, K, generator=gen, device=dev) < 0.01
    big[1::2] = False
    return torch.where(big, 20 * x, x).to(dtype)


def _int8_rows(gen, rows, K, spread, dev):
    """Int8 codes of Gaussian rows and a scale per row; rows padded to 16 bytes with zeros."""
    v = torch.randn(rows, K, generator=gen, device=dev)
    a = v.abs().amax(1, keepdim=True)
    q = torch.zeros(rows, (K + 15) // 16 * 16, dtype=torch.int8, device=dev)
    q[:, :K] = torch.round(v * (127 / a)).to(torch.int8)
    return q, (a[:, 0] / 127 * spread).contiguous()


def _vector(gen, K, dtype, dev):
    return (1 + 0.1 * torch.randn(K, generator=gen, device=dev)).to(dtype)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, rows, K = case["op"], case["rows"], case["K"]
    s = dict(case=case)
    block = case.get("block", 0)
    if block:
        s["sign"] = torch.randint(0, 2, (K,), generator=gen, device=dev).to(torch.int8) * 2 - 1
        s["H"] = _hadamard(block, torch.float32, dev)
    if op == "quant":
        s["x"] = _activations(gen, rows, K, _DTYPES[case["x"]], dev)
    if op in ("gemm", "step"):
        s["wq"], s["ws"] = _int8_rows(gen, case["N"], K, 1 / math.sqrt(K), dev)
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    if op == "gemm":
        s["xq"], s["xs"] = _int8_rows(gen, rows, K, 1.0, dev)
        s["bias"] = torch.randn(case["N"], generator=gen, device=dev) if case["bias"] else None
    if op in ("norm", "step"):
        rdt = _DTYPES[case["r"]]
        s["h"] = _activations(gen, rows, K, _DTYPES[case["h"]], dev)
        s["r"] = (4 * torch.randn(rows, K, generator=gen, device=dev)).to(rdt)
        s["kind"] = case.get("kind", "rms")
        s["post_w"], s["pre_w"] = _vector(gen, K, rdt, dev), _vector(gen, K, rdt, dev)
        layer = s["kind"] == "layer"
        s["post_b"] = (_vector(gen, K, rdt, dev) - 1) if layer else None
        s["pre_b"] = (_vector(gen, K, rdt, dev) - 1) if layer else None
        gt = case.get("gate_tokens", 0)
        s["gate"] = None
        if gt:
            s["gate"] = (0.5 + 0.2 * torch.randn((rows + gt - 1) // gt, K, generator=gen,
                                                 device=dev)).to(rdt)
        s["gate_tokens"] = gt
        # residual and branch multipliers of a depth-scaled stack
        s["residual_scale"], s["branch_scale"] = 0.9, 0.22
    return s


# ------------------------------------------------------------------ plain forms


def _whiten_plain(s, v):
    block = s["case"].get("block", 0)
    if not block:
        return v
    t = (v * s["sign"]).reshape(-1, block) @ s["H"]
    return (t / math.sqrt(block)).reshape(v.shape)


def _quant_plain(v):
    """(codes as fp32 values, scales) of fp32 rows."""
    a = v.abs().amax(1, keepdim=True)
    # values next to a rounding border: the quotient in 64 bits
    q = torch.round(127 * v.double() / a.double())
    q = torch.where((a > 0) & torch.isfinite(a), q, torch.zeros_like(q)).float()
    scale = torch.where(torch.isfinite(a), a / 127, torch.full_like(a, math.nan))
    return q, scale


def _product_plain(q, scale, s):
    case = s["case"]
    y = (q @ s["wq"][:, :case["K"]].float().t()) * scale * s["ws"]
    if s.get("bias") is not None:
        y = y + s["bias"]
    return y.to(_DTYPES[case["y"]])


def _norm_plain(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    u = v * torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS) * w.float()
    return u if b is None else u + b.float()


def _boundary_plain(s):
    u = _norm_plain(s["h"].float(), s["kind"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        t = torch.arange(u.shape[0], device=u.device) // s["gate_tokens"]
        u = u * s["gate"].float()[t]
    r = s["residual_scale"] * s["r"].float() + s["branch_scale"] * u
    return r, _norm_plain(r, s["kind"], s["pre_w"], s["pre_b"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quant":
        q, scale = _quant_plain(_whiten_plain(s, s["x"].float()))
        return (q * scale).to(s["x"].dtype), scale[:, 0]
    if case["op"] == "gemm":
        return _product_plain(s["xq"][:, :case["K"]].float(), s["xs"][:, None], s)
    r, n = _boundary_plain(s)
    if case["op"] == "norm":
        return r.to(s["r"].dtype), n.to(_DTYPES[case["y"]])
    q, scale = _quant_plain(_whiten_plain(s, n))
    return r.to(s["r"].dtype), _product_plain(q, scale, s)


# ------------------------------------------------------------------ the library's calls


def _run_own(s):
    import fractional_bit_weight_b200 as lq
    case = s["case"]
    block = case.get("block", 0)
    if case["op"] == "quant":
        _, scale, values = lq.quant_i8(s["x"], sign=s.get("sign"), block=block, values=True)
        return values, scale
    if case["op"] == "gemm":
        return lq.gemm_i8(s["xq"], s["xs"], s["wq"], s["ws"], K=case["K"], bias=s["bias"],
                          dtype=_DTYPES[case["y"]], workspace=s["workspace"])
    if "post" not in s:     # the norms' descriptors are made once, as a layer would
        s["post"] = lq.Norm(s["kind"], s["post_w"], s["post_b"], _EPS)
        s["pre"] = lq.Norm(s["kind"], s["pre_w"], s["pre_b"], _EPS)
    if case["op"] == "norm":
        r, n = lq.norm_residual(s["h"], s["r"], post=s["post"], pre=s["pre"], gate=s["gate"],
                                gate_tokens=s["gate_tokens"], branch_scale=s["branch_scale"],
                                residual_scale=s["residual_scale"], dtype=_DTYPES[case["y"]])
        return r, n
    r, q, scale = lq.norm_residual_i8(s["h"], s["r"], post=s["post"], pre=s["pre"],
                                      branch_scale=s["branch_scale"],
                                      residual_scale=s["residual_scale"], sign=s["sign"],
                                      block=block)
    return r, lq.gemm_i8(q, scale, s["wq"], s["ws"], K=case["K"], dtype=_DTYPES[case["y"]],
                         workspace=s["workspace"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, rows, K = case["op"], case["rows"], case["K"]
    block = case.get("block", 0)
    whiten = rows * K * (math.log2(block) + 2) if block else 0
    if op == "quant":
        xb = _BYTES[case["x"]]
        return dict(bytes=rows * K * (2 * xb + 1) + 4 * rows + (K if block else 0),
                    flops=4 * rows * K + whiten)
    nbytes = flops = 0
    if op in ("norm", "step"):
        hb, rb = _BYTES[case["h"]], _BYTES[case["r"]]
        gt = case.get("gate_tokens", 0)
        vectors = 4 if case.get("kind") == "layer" else 2
        nbytes += rows * K * (hb + 2 * rb) + vectors * K * rb
        nbytes += -(-rows // gt) * K * rb if gt else 0
        flops += 12 * rows * K
    if op == "norm":
        nbytes += rows * K * _BYTES[case["y"]]
    else:
        N = case["N"]
        nbytes += N * K + 4 * N + rows * N * _BYTES[case["y"]]
        nbytes += (4 * N if case.get("bias") else 0)
        nbytes += rows * K + 4 * rows if op == "gemm" else K
        flops += 2 * rows * N * K + whiten
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------------------ 64 bits


def _exact_whiten(s, v):
    """T by butterflies."""
    block = s["case"].get("block", 0)
    if not block:
        return v
    v = v * s["sign"].double()
    shape, h = v.shape, 1
    while h < block:
        p = v.reshape(-1, 2, h)
        v = torch.stack((p[:, 0] + p[:, 1], p[:, 0] - p[:, 1]), 1)
        h *= 2
    return v.reshape(shape) * block ** -0.5


def _exact_codes(v):
    top = torch.max(v.abs(), 1, keepdim=True).values
    step = top / 127
    code = torch.round(v * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    return code, step


def _exact_norm(v, kind, w, b):
    n = v.shape[1]
    if kind == "layer":
        v = v - (v.sum(1) / n)[:, None]
    u = v / torch.sqrt(torch.linalg.vecdot(v, v) / n + _EPS)[:, None]
    u = u * w.double()
    return u + b.double() if b is not None else u


def _exact_product(code, step, s):
    K = s["case"]["K"]
    acc = torch.mm(code, s["wq"].double()[:, :K].t())
    y = torch.outer(step, s["ws"].double()) * acc
    return y + s["bias"].double() if s.get("bias") is not None else y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        code, step = _exact_codes(_exact_whiten(s, s["x"].double()))
        return code * step, step[:, 0]
    if op == "gemm":
        return _exact_product(s["xq"].double()[:, :case["K"]], s["xs"].double(), s)
    branch = _exact_norm(s["h"].double(), s["kind"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        branch = branch * s["gate"].double().repeat_interleave(s["gate_tokens"],
                                                               0)[:case["rows"]]
    r = branch * s["branch_scale"] + s["r"].double() * s["residual_scale"]
    n = _exact_norm(r, s["kind"], s["pre_w"], s["pre_b"])
    if op == "norm":
        return r, n
    code, step = _exact_codes(_exact_whiten(s, n))
    return r, _exact_product(code, step[:, 0], s)
