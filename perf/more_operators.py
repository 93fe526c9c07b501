"""What the operators between a model's projections are measured on.

Four groups of operators that a model with binarized projections needs around
them:

- the root-mean-square norm before a projection: the residual's addition, the
  norm, and its result in 16 bits and / or in 8 or 4 bits with block scales,
  forward and backward;
- microscaled quantisation (OCP MX: blocks of 32 values share a power of two;
  values in E4M3 or E2M1) of weights and activations, and back;
- the linear layer on such operands, for the projections that cannot do with
  signs, and its input gradient;
- the global norm of many gradients and clipping by it, the last step before
  the optimiser's.

Every case is a dict; ``op`` names the operator. ``run`` computes it either in
its plain form (elementary torch operations, rounded once) or, with ``own``
set, through the library's entry points. ``exact`` is the definition in 64
bits. What is held in 8 or 4 bits is returned as the values it stands for.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32
# format: mantissa bits, smallest normal exponent, largest exponent, largest value, bytes a value
_FORMAT = {"e4m3": (3, -6, 8, 448.0, 1.0), "e2m1": (1, 0, 2, 6.0, 0.5)}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 16 requests: residual, norm, straight to the 4-bit operand of the next projection
        {"name": "norm_decode", "op": "norm", "T": 16, "N": 4096, "dtype": "bf16", "residual": True, "out": False,
         "format": "e2m1"},
        # a long prompt: the 16-bit result for a binarized projection and its adapters, 8 bits for the one beside it
        {"name": "norm_prompt", "op": "norm", "T": 8192, "N": 4096, "dtype": "bf16", "residual": True, "out": True,
         "format": "e4m3"},
        # a training step's backward, the residual stream's gradient added in
        {"name": "norm_bwd", "op": "norm_bwd", "T": 4096, "N": 4096, "dtype": "bf16", "residual": True},
        # the same at odd sizes and in full precision
        {"name": "norm_bwd_odd", "op": "norm_bwd", "T": 777, "N": 4093, "dtype": "f32", "residual": False},
        # a projection's weights, laid out once when a model is loaded
        {"name": "quantize_weight", "op": "quantize", "R": 11008, "K": 4096, "dtype": "bf16", "format": "e2m1"},
        # activations whose width is no whole number of blocks
        {"name": "quantize_odd", "op": "quantize", "R": 1500, "K": 4100, "dtype": "f16", "format": "e4m3"},
        # one request generating one token, the wide MLP projection: the weights' bytes and latency
        {"name": "linear_token", "op": "linear", "M": 1, "N": 11008, "K": 4096, "dtype": "bf16", "out": "bf16",
         "format": "e2m1"},
        # a prompt or a training step through the MLP's second projection
        {"name": "linear_prompt", "op": "linear", "M": 8192, "N": 4096, "K": 11008, "dtype": "bf16", "out": "bf16",
         "format": "e2m1"},
        # a training step's input gradient on the square projection
        {"name": "linear_bwd", "op": "linear_bwd", "M": 4096, "N": 4096, "K": 4096, "format": "e4m3"},
        # the same at ragged sizes
        {"name": "linear_bwd_odd", "op": "linear_bwd", "M": 777, "N": 4093, "K": 4100, "format": "e2m1"},
        # two adapters beside one projection
        {"name": "clip_few", "op": "clip", "count": 4, "size": 65536, "ragged": False, "dtype": "f32", "clip": True},
        # adapters beside every projection of a deep model
        {"name": "clip_many", "op": "clip", "count": 448, "size": 88064, "ragged": True, "dtype": "f32", "clip": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo=128, hi=11008):
    """A layer's width: mostly whole 64s, now and then odd."""
    w = _log_int(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "quantize", "linear", "linear", "linear", "linear_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    fmt = rng.choice(["e4m3", "e2m1"])
    if op == "norm":
        N = _width(rng)
        fmt = rng.choice([fmt, fmt, "none"])
        return {"op": op, "T": _log_int(rng, 1, min(8192, 8192 * 4096 // N)), "N": N, "dtype": dtype,
                "residual": rng.random() < 0.7, "out": fmt == "none" or rng.random() < 0.5, "format": fmt}
    if op == "norm_bwd":
        N = _width(rng)
        return {"op": op, "T": _log_int(rng, 1, min(8192, 8192 * 4096 // N)), "N": N, "dtype": dtype,
                "residual": rng.random() < 0.5}
    if op == "quantize":
        return {"op": op, "R": _log_int(rng, 1, 11008), "K": _width(rng), "dtype": dtype, "format": fmt}
    if op == "linear":
        M = _log_int(rng, 1, 64) if rng.random() < 0.5 else _log_int(rng, 16, 8192)
        N, K = _width(rng), _width(rng)
        M = min(M, 8192 * 4096 * 11008 // (N * K))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "out": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "format": fmt}
    if op == "linear_bwd":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _width(rng, hi=8192), "K": _width(rng, hi=8192), "format": fmt}
    count = _log_int(rng, 1, 448)
    return {"op": op, "count": count, "size": _log_int(rng, 64, min(1 << 22, 448 * 88064 // count)),
            "ragged": rng.random() < 0.5, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
            "clip": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
EPS = 1e-6


def _normal(gen, dt, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dt)


def _activations(gen, dt, T, N):
    """A residual stream: a few channels far larger than the others, tokens of different size."""
    x = torch.randn(T, N, generator=gen, device=DEV)
    x *= torch.where(torch.rand(N, generator=gen, device=DEV) < 0.01, 20.0, 1.0)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=gen, device=DEV))
    return x.to(dt)


def _sizes(case):
    """Elements of every gradient; the ragged ones are odd and start anywhere in the buffer that holds them all."""
    r = random.Random(case["count"])
    return [max(1, int(case["size"] * r.uniform(0.1, 1.9))) if case["ragged"] else case["size"]
            for _ in range(case["count"])]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if own:
        import xnor_popcount_gemm_gb300 as bt
        st["bt"] = bt
        st["code"] = {"e4m3": bt.BT_CODE_E4M3, "e2m1": bt.BT_CODE_E2M1}.get(case.get("format"))
    if op in ("norm", "norm_bwd"):
        T, N, dt = case["T"], case["N"], _DT[case["dtype"]]
        st["x"] = _activations(gen, dt, T, N)
        st["w"] = (1.0 + 0.2 * torch.randn(N, generator=gen, device=DEV)).to(dt)
        st["r"] = _normal(gen, dt, T, N, std=0.5) if op == "norm" and case["residual"] else None
        if op == "norm_bwd":
            st["g"] = _normal(gen, dt, T, N, std=0.01)
            st["gsum"] = _normal(gen, dt, T, N, std=0.01) if case["residual"] else None
    elif op == "quantize":
        st["x"] = _activations(gen, _DT[case["dtype"]], case["R"], case["K"])
    elif op in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        w = _normal(gen, torch.bfloat16, N, K, std=0.02)
        if op == "linear":
            st["x"] = _activations(gen, _DT[case["dtype"]], M, K)
        else:
            st["g"] = _normal(gen, torch.bfloat16, M, N, std=0.01)
        if own:                                   # laid out once, when the model is loaded
            st["wq"] = st["bt"].bt_mx_quantize(w, st["code"])
            if op == "linear_bwd":
                st["wt"] = st["bt"].bt_mx_transpose(st["wq"])
        else:
            st["wd"] = _quantized(w.float(), case["format"])
        st["w"] = w
    else:
        sizes = _sizes(case)
        flat = torch.randn(sum(sizes), generator=gen, device=DEV)
        scale = torch.exp(torch.randn(len(sizes), generator=gen, device=DEV))
        flat *= torch.repeat_interleave(scale, torch.tensor(sizes, device=DEV))
        st["flat"] = (flat * 1e-3).to(_DT[case["dtype"]])
        st["grads"] = list(st["flat"].split(sizes))
        st["max_norm"] = (0.1 if case["clip"] else 1e3) * 1e-3 * math.sqrt(sum(sizes))
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _quantized(x, fmt):
    """The values that x [R, K] has in blocks of 32 along K: a power of two each, from the largest magnitude's
    exponent, and values rounded to the format, ties to even, beyond its largest to that. Products and quotients by
    powers of two are exact in 32 bits."""
    mant, emin, emax, vmax, _ = _FORMAT[fmt]
    R, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(R, -1, BLOCK)
    amax = v.abs().amax(dim=2, keepdim=True)
    e = (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(v, -e)
    step = torch.frexp(v)[1] - 1
    step = step.clamp(min=emin) - mant
    v = torch.ldexp(torch.ldexp(v, -step).round(), step).clamp(-vmax, vmax)
    return torch.ldexp(v, e).view(R, -1)[:, :K].contiguous()


def _plain_norm(st, case):
    dt = _DT[case["dtype"]]
    h = st["x"] if st["r"] is None else (st["x"].float() + st["r"].float()).to(dt)
    # values next to a border of the 8- or 4-bit format decide in 64 bits
    v = h.float() if case["format"] == "none" else h.double()
    y = (v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * st["w"].to(v.dtype)).float().to(dt)
    return {"sum": h if st["r"] is not None else None, "out": y if case["out"] else None,
            "values": None if case["format"] == "none" else _quantized(y.float(), case["format"]).to(torch.bfloat16)}


def _plain_norm_bwd(st, case):
    h, g, w = st["x"].float(), st["g"].float(), st["w"].float()
    rms = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    n = h * rms
    gn = g * w
    gx = rms * (gn - n * (gn * n).mean(dim=1, keepdim=True))
    if st["gsum"] is not None:
        gx = gx + st["gsum"].float()
    return {"grad_x": gx.to(_DT[case["dtype"]]), "grad_weight": (g * n).sum(dim=0)}


def _plain_clip(st):
    sums = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]])
    norm = sums.sum().sqrt().float()
    factor = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [g.copy_(g.float() * factor) for g in st["grads"]]
    return {"norm": norm, "grads": st["flat"]}


def run(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        if not own:
            return _plain_norm(st, case)
        bt = st["bt"]
        out, total, q = bt.bt_rms_norm(st["x"], st["w"], EPS, residual=st["r"], want_out=case["out"], code=st["code"])
        return {"sum": total, "out": out, "values": None if q is None else bt.bt_mx_dequantize(q, torch.bfloat16)}
    if op == "norm_bwd":
        if not own:
            return _plain_norm_bwd(st, case)
        gx, gw = st["bt"].bt_rms_norm_backward(st["g"], st["x"], st["w"], EPS, grad_sum=st["gsum"])
        return {"grad_x": gx, "grad_weight": gw}
    if op == "quantize":
        if not own:
            return {"values": _quantized(st["x"], case["format"]).to(torch.bfloat16)}
        q = st["bt"].bt_mx_quantize(st["x"], st["code"])
        return {"values": st["bt"].bt_mx_dequantize(q, torch.bfloat16)}
    if op == "linear":
        if not own:
            return (_quantized(st["x"], case["format"]) @ st["wd"].t()).to(_DT[case["out"]])
        return st["bt"].bt_mx_linear(st["x"], st["wq"], out_dtype=_DT[case["out"]])
    if op == "linear_bwd":
        if not own:
            return (st["g"].float() @ st["wd"]).to(torch.bfloat16)
        return st["bt"].bt_mx_linear_backward(st["g"], st["wt"])
    if not own:
        return _plain_clip(st)
    norm = st["bt"].bt_clip_grads(st["grads"], st["max_norm"])
    return {"norm": norm, "grads": st["flat"]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, e = case["T"] * case["N"], _SIZE[case["dtype"]]
        if op == "norm":
            b = n * e * (1 + 2 * case["residual"] + case["out"]) + case["N"] * e
            b += 2 * n if case["format"] != "none" else 0
            return {"bytes": b, "flops": 8 * n}
        return {"bytes": n * e * (3 + case["residual"]) + case["N"] * (e + 4), "flops": 12 * n}
    if op == "quantize":
        n = case["R"] * case["K"]
        return {"bytes": n * (_SIZE[case["dtype"]] + 2), "flops": 4 * n}
    if op == "clip":
        n = sum(_sizes(case))
        return {"bytes": n * _SIZE[case["dtype"]] * (2 if case["clip"] else 1), "flops": 3 * n}
    M, N, K = case["M"], case["N"], case["K"]
    held = N * K * (_FORMAT[case["format"]][4] + 1 / BLOCK)
    if op == "linear":
        return {"bytes": M * K * _SIZE[case["dtype"]] + held + M * N * _SIZE[case["out"]], "flops": 2.0 * M * N * K}
    return {"bytes": 2 * (M * N + M * K) + held, "flops": 2.0 * M * N * K}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_quantized(x, fmt):
    """Nearest of the format's own values, by a table of them; ties to the one with the even code."""
    mant, emin, emax, vmax, _ = _FORMAT[fmt]
    values = [0.0]
    code = 0
    while values[-1] < vmax:
        code += 1
        e, m = code >> mant, code & ((1 << mant) - 1)
        values.append(math.ldexp(m, emin - mant) if e == 0 else math.ldexp((1 << mant) + m, emin + e - 1 - mant))
    table = torch.tensor(values, dtype=torch.float64, device=x.device)
    R, K = x.shape
    out = torch.empty(R, K, dtype=torch.float64, device=x.device)
    for lo in range(0, R, 2048):                  # the double intermediates of large weights in pieces
        v = x[lo:lo + 2048].double()
        v = torch.cat([v, v.new_zeros(v.shape[0], -K % BLOCK)], dim=1).reshape(v.shape[0], -1, BLOCK)
        top = v.abs().max(dim=2, keepdim=True).values
        # the exponent of the largest, exactly: log2 may round up to the next whole number
        e = torch.log2(top.clamp(min=1e-300)).floor()
        e = e - (torch.exp2(e) > top).double() + (torch.exp2(e + 1) <= top).double()
        scale = torch.exp2((e - emax).clamp(-127, 127))
        a = (v / scale).abs()
        mid = (table[1:] + table[:-1]) / 2
        i = torch.bucketize(a, mid)
        tie = (i < len(mid)) & (a == mid[i.clamp(max=len(mid) - 1)]) & (i % 2 == 1)
        q = table[i + tie.long()] * torch.sign(v) * scale
        out[lo:lo + 2048] = q.reshape(v.shape[0], -1)[:, :K]
    return out


def exact(case, seed):
    op = case["op"]
    if op == "linear" and case["M"] * case["N"] * case["K"] > 1 << 40:
        return None
    st = prepare(case, seed)
    if op == "norm":
        dt = _DT[case["dtype"]]
        h = st["x"].double()
        if st["r"] is not None:
            h = (h + st["r"].double()).float().to(dt).double()      # the sum is kept in its type
        y = h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["N"] + EPS) * st["w"].double()
        return {"sum": h if st["r"] is not None else None, "out": y if case["out"] else None,
                "values": None if case["format"] == "none" else _exact_quantized(y.float().to(dt), case["format"])}
    if op == "norm_bwd":
        h, g, w = st["x"].double(), st["g"].double(), st["w"].double()
        inv = 1.0 / torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["N"] + EPS)
        dot = (g * w * h).sum(dim=1, keepdim=True)
        gx = g * w * inv - h * inv ** 3 * dot / case["N"]
        if st["gsum"] is not None:
            gx = gx + st["gsum"].double()
        return {"grad_x": gx, "grad_weight": (g * h * inv).sum(dim=0)}
    if op == "quantize":
        return {"values": _exact_quantized(st["x"], case["format"])}
    if op == "linear":
        return _exact_quantized(st["x"], case["format"]) @ _exact_quantized(st["w"], case["format"]).t()
    if op == "linear_bwd":
        return st["g"].double() @ _exact_quantized(st["w"], case["format"])
    flat = st["flat"].double()
    norm = (flat * flat).sum().sqrt()
    return {"norm": norm, "grads": flat * min(1.0, st["max_norm"] / (float(norm) + 1e-6))}
