"""Measured cases of the operators beside the block-scaled GEMMs: low-rank
adapters of many requests, and activation checkpoints held in 8 bits.

``run`` makes one pass through an operator: with ``own`` false in its plain
form (elementary torch operations in binary32, rounded once at the end), with
``own`` true through the library's entry points.

Operators (``case["op"]``):

* ``adapters``            out = y + s[id] (x A[id]^T) B[id]^T per token, u = x A[id]^T
* ``adapters_backward``   dx, dA and dB of the same, x in bfloat16 or as an MXFP8 checkpoint
* ``gated_act``           h = act(gate) * up as a GEMM operand, gate and up kept in 8 bits
* ``gated_act_backward``  d_gate, d_up (and h again) from those 8 bits
* ``linear_backward_checkpoint``  dX and dW of a linear layer whose input was kept in 8 bits
"""

import math

import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# --------------------------------------------------------------------------- #
# Cases                                                                       #
# --------------------------------------------------------------------------- #

def _adapters(name, T, K, N, R, L, y, order):
    return {"name": name, "op": "adapters", "T": T, "K": K, "N": N, "R": R, "L": L, "y": y, "order": order}


def _adapters_backward(name, T, K, N, R, L, x, grad, order):
    return {"name": name, "op": "adapters_backward", "T": T, "K": K, "N": N, "R": R, "L": L, "x": x, "grad": grad,
            "order": order}


def _gated(name, M, I, act, h, code, scale):
    return {"name": name, "op": "gated_act", "M": M, "I": I, "act": act, "h": h, "code": code, "scale": scale}


def _gated_backward(name, M, I, act, code, scale, h):
    return {"name": name, "op": "gated_act_backward", "M": M, "I": I, "act": act, "code": code, "scale": scale, "h": h}


def _linear(name, M, N, K, code, scale, fp8):
    return {"name": name, "op": "linear_backward_checkpoint", "M": M, "N": N, "K": K, "code": code, "scale": scale,
            "fp8": fp8}


def listed():
    return [
        # one request's next token: latency counts
        _adapters("adapters one token", 1, 4096, 4096, 16, 8, "bf16", "mixed"),
        # a decode step of 64 requests, nearly every one with an adapter of its own
        _adapters("adapters 64 requests", 64, 4096, 4096, 16, 64, "bf16", "mixed"),
        # a ragged batch of short prompts, a rank that is no power of two, binary32 sums
        _adapters("adapters 777 tokens r24", 777, 2048, 8192, 24, 5, "f32", "runs"),
        # a full prefill batch of eight long prompts
        _adapters("adapters 8192 tokens r64", 8192, 8192, 8192, 64, 8, "bf16", "runs"),
        # a small fine-tuning step, tokens of three adapters interleaved
        _adapters_backward("adapters backward 1333", 1333, 2048, 2048, 8, 3, "bf16", "f32", "mixed"),
        # a full fine-tuning step whose input was kept as the forward GEMM's MXFP8 operand
        _adapters_backward("adapters backward 8192", 8192, 8192, 8192, 16, 4, "e4m3", "f32", "runs"),
        # serving: a few tokens, nothing kept for a backward pass
        _gated("gated 3 tokens", 3, 8192, "silu", "e4m3", "none", "none"),
        # training: a full batch, gate and up kept as INT8 per 1 x 128
        _gated("gated 8192 int8", 8192, 8192, "silu", "e4m3", "int8", "f32"),
        # a ragged micro-batch, gate and up kept as MXFP8
        _gated_backward("gated backward 1001 mxfp8", 1001, 2048, "gelu", "e4m3", "ue8m0", True),
        # the full batch's backward pass
        _gated_backward("gated backward 8192 int8", 8192, 8192, "silu", "int8", "f32", True),
        # a small layer
        _linear("linear backward 1024", 1024, 2048, 2048, "int8", "f32", "e4m3"),
        # the MXFP8 backward workload of bench.py, X kept as the forward GEMM's operand
        _linear("linear backward 16384", 16384, 8192, 8192, "e4m3", "ue8m0", "e5m2"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_backward", "gated_act", "gated_act_backward",
                     "linear_backward_checkpoint"])
    kept = rng.choice([("int8", "f32"), ("e4m3", "f32"), ("e4m3", "ue8m0"), ("e5m2", "ue8m0")])
    if op in ("adapters", "adapters_backward"):
        step = rng.choice([1, 8, 8, 128])  # odd widths, the vector path's, the usual ones
        c = {"op": op, "T": _log(rng, 1 if op == "adapters" else 16, 8192), "K": _mult(rng, 512, 8192, step),
             "N": _mult(rng, 512, 8192, step), "R": rng.choice([4, 8, 8, 12, 16, 16, 24, 32, 64]),
             "L": _log(rng, 1, 64 if op == "adapters" else 8)}
        c["order"] = "mixed" if c["T"] < 256 else rng.choice(["runs", "runs", "mixed"])
        if op == "adapters":
            c["y"] = rng.choice(["bf16", "bf16", "f32"])
        else:
            c["x"] = rng.choice(["bf16", "e4m3"])
            c["grad"] = rng.choice(["f32", "bf16"])
            if c["x"] == "e4m3":
                c["K"] = max(32, c["K"] // 32 * 32)
        return c
    if op == "linear_backward_checkpoint":
        code, scale = kept
        return {"op": op, "M": _mult(rng, 256, 16384, 32), "N": _mult(rng, 512, 8192, 32),
                "K": _mult(rng, 512, 8192, 128 if scale == "f32" else 32), "code": code, "scale": scale,
                "fp8": rng.choice(["e5m2", "e4m3"])}
    c = {"op": op, "M": _log(rng, 1 if op == "gated_act" else 16, 8192),
         "I": _mult(rng, 512, 8192, 128 if kept[1] == "f32" else 32), "act": rng.choice(["silu", "silu", "gelu"]),
         "code": kept[0], "scale": kept[1]}
    if op == "gated_act":
        c["h"] = rng.choice(["e4m3", "e4m3", "e5m2", "bf16"])
        if c["M"] < 64:
            c["code"] = c["scale"] = "none"
    else:
        c["h"] = rng.choice([True, False])
    return c


# --------------------------------------------------------------------------- #
# Inputs                                                                      #
# --------------------------------------------------------------------------- #

def _randn(shape, seed, stream, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + stream)
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _ids(T, L, order, seed):
    """Each token's adapter: -1 for about one request in ten; 'runs' are
    consecutive tokens of one request, 'mixed' has no order."""
    g = torch.Generator()
    g.manual_seed(seed * 1_000_003 + 77)
    if order == "runs":
        starts = torch.sort(torch.randint(0, T, (2 * L - 1,), generator=g)).values
        run = torch.bucketize(torch.arange(T), starts, right=True)
        adapter = torch.randint(0, L, (2 * L,), generator=g)
        adapter[torch.rand(2 * L, generator=g) < 0.1] = -1
        ids = adapter[run]
    else:
        ids = torch.randint(0, L, (T,), generator=g) if T != L else torch.randperm(L, generator=g)
        ids[torch.rand(T, generator=g) < 0.1] = -1
    if T == 1:
        ids[0] = seed % L
    return ids.to(torch.int32).to(DEV)


def _block_quantize(x, block, code, scale):
    """Absmax quantization of each row in blocks: codes (float8 or int8) and
    one scale per block, binary32 or the exponent byte of a power of two."""
    rows, cols = x.shape
    xb = x.float().view(rows, cols // block, block)
    amax = xb.abs().amax(-1)
    r = amax / QMAX[code]
    if scale == "ue8m0":
        m, e = torch.frexp(r)
        e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
        e = torch.where(amax == 0, torch.zeros_like(e), e)
        s = torch.ldexp(torch.ones_like(r), e)
        stored = (e + 127).to(torch.uint8)
    else:
        s = torch.where(amax == 0, torch.ones_like(r), r) if code == "int8" else r.clamp_min(1e-10)
        stored = s
    q = (xb / s[..., None]).clamp(-QMAX[code], QMAX[code]).view(rows, cols)
    return (torch.round(q).to(torch.int8) if code == "int8" else q.to(FP8[code])), stored


def _block_values(codes, scales):
    """The values that _block_quantize's codes and scales stand for."""
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.to(torch.int32) - 127) \
        if scales.dtype == torch.uint8 else scales
    rows, cols = codes.shape
    return (codes.float().view(rows, s.shape[1], -1) * s[..., None]).view(rows, cols)


def _block(scale):
    return 128 if scale == "f32" else 32


def prepare(case, seed):
    c, op = case, case["op"]
    s = {"case": dict(c)}
    if op in ("adapters", "adapters_backward"):
        T, K, N, R, L = c["T"], c["K"], c["N"], c["R"], c["L"]
        s["x"] = _randn((T, K), seed, 1)
        s["a"] = _randn((L, R, K), seed, 2, K ** -0.5)
        s["b"] = _randn((L, N, R), seed, 3, R ** -0.5)
        s["ids"] = _ids(T, L, c["order"], seed)
        s["scaling"] = 0.25 + 0.25 * (torch.arange(L, device=DEV) % 8).float()
        if op == "adapters":
            dt = torch.float32 if c["y"] == "f32" else torch.bfloat16
            s["y"] = _randn((T, N), seed, 4, 1.0, dt)  # the shared projection's product
            s["out"], s["u"] = torch.empty_like(s["y"]), torch.empty((T, R), device=DEV)
        else:
            s["dy"] = _randn((T, N), seed, 5)
            s["dx_base"] = _randn((T, K), seed, 6)  # the shared projection's own dX
            s["u"] = _low_rank(s["x"].float(), s["a"].float(), s["ids"])
            if c["x"] != "bf16":
                codes, scales = _block_quantize(s.pop("x"), 32, c["x"], "ue8m0")
                s["x"], s["x_scales"] = codes.view(torch.uint8), scales
    elif op in ("gated_act", "gated_act_backward"):
        M, I = c["M"], c["I"]
        gu = _randn((M, 2 * I), seed, 1, 1.5)
        if op == "gated_act":
            s["gate_up"] = gu
        else:
            codes, s["scales"] = _block_quantize(gu, _block(c["scale"]), c["code"], c["scale"])
            s["codes"] = codes if c["code"] == "int8" else codes.view(torch.uint8)
            s["dh"] = _randn((M, I), seed, 2)
    else:
        M, N, K = c["M"], c["N"], c["K"]
        s["dY"], s["W"] = _randn((M, N), seed, 1), _randn((N, K), seed, 2, 0.02)
        codes, s["x_scales"] = _block_quantize(_randn((M, K), seed, 3), _block(c["scale"]), c["code"], c["scale"])
        s["x_codes"] = codes if c["code"] == "int8" else codes.view(torch.uint8)
    return s


# --------------------------------------------------------------------------- #
# Plain forms                                                                 #
# --------------------------------------------------------------------------- #

def _select(ids, L):
    """[T, L, 1]: 1 at each token's adapter, no 1 for a token without one."""
    return (ids[:, None] == torch.arange(L, device=ids.device, dtype=ids.dtype)).float()[..., None]


def _gathers(T, L):
    """Whether gathering each token's adapter is less work than multiplying
    every token with every adapter and selecting."""
    return 50 * T < L * (T + 30)


def _low_rank(x, a, ids):
    T, (L, R, K) = x.shape[0], a.shape
    if _gathers(T, L):
        u = torch.bmm(a[ids.clamp_min(0).long()], x[..., None])[..., 0]
        return torch.where(ids[:, None] >= 0, u, torch.zeros_like(u))
    return ((x @ a.view(L * R, K).t()).view(T, L, R) * _select(ids, L)).sum(1)


def _plain_adapters(s):
    x, a, b, ids = s["x"].float(), s["a"].float(), s["b"].float(), s["ids"]
    T, (L, N, R) = x.shape[0], b.shape
    u = _low_rank(x, a, ids)
    at = ids.clamp_min(0).long()
    us = u * s["scaling"][at][:, None]
    if _gathers(T, L):
        d = torch.bmm(b[at], us[..., None])[..., 0]
    else:
        d = (us[:, None, :] * _select(ids, L)).view(T, L * R) @ b.transpose(1, 2).reshape(L * R, N)
    return {"out": (s["y"].float() + d).to(s["y"].dtype), "u": u}


def _plain_adapters_backward(s):
    c = s["case"]
    x = s["x"].float() if c["x"] == "bf16" else _block_values(s["x"].view(FP8[c["x"]]), s["x_scales"])
    a, b, dy, u, ids = s["a"].float(), s["b"].float(), s["dy"].float(), s["u"], s["ids"]
    T, (L, N, R), K = x.shape[0], b.shape, x.shape[1]
    scaled = _select(ids, L) * s["scaling"][:, None]
    du = ((dy @ b.transpose(1, 2).reshape(L * R, N).t()).view(T, L, R) * scaled).view(T, L * R)
    us = (u[:, None, :] * scaled).view(T, L * R)
    grad = torch.float32 if c["grad"] == "f32" else torch.bfloat16
    return {"dx": (s["dx_base"].float() + du @ a.view(L * R, K)).to(torch.bfloat16),
            "da": (du.t() @ x).view(L, R, K).to(grad),
            "db": (us.t() @ dy).view(L, R, N).transpose(1, 2).contiguous().to(grad)}


def _act(g, act):
    return g / (1 + torch.exp(-g)) if act == "silu" else 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _act_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _as_scale(scales):
    return scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales


def _plain_gated(s):
    c, gu = s["case"], s["gate_up"]
    I = c["I"]
    h = _act(gu[:, :I].float(), c["act"]) * gu[:, I:].float()
    r = {}
    if c["h"] == "bf16":
        r["h"] = h.to(torch.bfloat16)
    else:
        r["h"], hs = _block_quantize(h, 32, c["h"], "ue8m0")
        r["h_scales"] = _as_scale(hs)
    if c["code"] != "none":
        r["codes"], ks = _block_quantize(gu, _block(c["scale"]), c["code"], c["scale"])
        r["scales"] = _as_scale(ks)
    return r


def _plain_gated_backward(s):
    c, I = s["case"], s["case"]["I"]
    codes = s["codes"] if c["code"] == "int8" else s["codes"].view(FP8[c["code"]])
    gu, dh = _block_values(codes, s["scales"]), s["dh"].float()
    g, up = gu[:, :I], gu[:, I:]
    f = _act(g, c["act"])
    r = {"d_gate_up": torch.cat([dh * up * _act_slope(g, c["act"]), dh * f], 1).to(torch.bfloat16)}
    if c["h"]:
        r["h"] = (f * up).to(torch.bfloat16)
    return r


def _requantized(x, fp8):
    """[rows, cols] quantized down its columns in blocks of 32 rows (MXFP8), as values."""
    codes, scales = _block_quantize(x.t().contiguous(), 32, fp8, "ue8m0")
    return _block_values(codes, scales).t()


def _plain_linear(s):
    c = s["case"]
    codes = s["x_codes"] if c["code"] == "int8" else s["x_codes"].view(FP8[c["code"]])
    x, dy, w = _block_values(codes, s["x_scales"]), s["dY"].float(), s["W"].float()
    dy_n = _block_values(*_block_quantize(dy, 32, c["fp8"], "ue8m0"))
    return {"dX": (dy_n @ _requantized(w, c["fp8"])).to(torch.bfloat16),
            "dW": (_requantized(dy, c["fp8"]).t() @ _requantized(x, c["fp8"])).to(torch.bfloat16)}


PLAIN = {"adapters": _plain_adapters, "adapters_backward": _plain_adapters_backward, "gated_act": _plain_gated,
         "gated_act_backward": _plain_gated_backward, "linear_backward_checkpoint": _plain_linear}


# --------------------------------------------------------------------------- #
# The library's calls                                                         #
# --------------------------------------------------------------------------- #

def _own(s):
    import block_scaled_precision_gemm_gb300 as bsmm
    c, op = s["case"], s["case"]["op"]
    if op == "adapters":
        out, u = bsmm.adapters(s["x"], s["a"], s["b"], s["ids"], y=s["y"], scaling=s["scaling"], out=s["out"],
                               u=s["u"])
        return {"out": out, "u": u}
    if op == "adapters_backward":
        dx, da, db = bsmm.adapters_backward(s["dy"], s["x"], s["a"], s["b"], s["ids"], s["u"],
                                            scaling=s["scaling"], dx_base=s["dx_base"], x_scales=s.get("x_scales"),
                                            grad_dtype=torch.float32 if c["grad"] == "f32" else torch.bfloat16)
        return {"dx": dx, "da": da, "db": db}
    if op == "gated_act":
        keep = None if c["code"] == "none" else c["code"]
        h, hs, codes, scales = bsmm.gated_act(s["gate_up"], act=c["act"], h_type=c["h"], code=keep,
                                              scale=c["scale"] if keep else "f32")
        r = {"h": h if c["h"] == "bf16" else h.view(FP8[c["h"]])}
        if c["h"] != "bf16":
            r["h_scales"] = _as_scale(hs)
        if keep:
            r["codes"] = codes if keep == "int8" else codes.view(FP8[keep])
            r["scales"] = _as_scale(scales)
        return r
    if op == "gated_act_backward":
        d, h = bsmm.gated_act_backward(s["dh"], s["codes"], s["scales"], act=c["act"], code=c["code"],
                                       scale=c["scale"], return_h=c["h"])
        return {"d_gate_up": d, "h": h} if c["h"] else {"d_gate_up": d}
    dX, dW = bsmm.linear_backward_checkpoint(s["dY"], s["W"], s["x_codes"], s["x_scales"], x_code=c["code"],
                                             x_scale=c["scale"], fp8=c["fp8"])
    return {"dX": dX, "dW": dW}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------- #
# What a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def work(case):
    c, op = case, case["op"]
    if op in ("adapters", "adapters_backward"):
        T, K, N, R, L = c["T"], c["K"], c["N"], c["R"], c["L"]
        if op == "adapters":
            y = 4 if c["y"] == "f32" else 2
            return {"bytes": T * K * 2 + min(L, T) * R * (K + N) * 2 + 2 * T * N * y + T * R * 4 + T * 4,
                    "flops": 2 * T * R * (K + N)}
        x = 2 if c["x"] == "bf16" else 1 + 1 / 32
        g = 4 if c["grad"] == "f32" else 2
        return {"bytes": T * N * 2 + T * K * (x + 4) + L * R * (K + N) * (2 + g) + T * R * 4 + T * 4,
                "flops": 4 * T * R * (K + N)}
    if op in ("gated_act", "gated_act_backward"):
        n = c["M"] * c["I"]
        kept = 0 if c["code"] == "none" else 2 * (1 + (4 / 128 if c["scale"] == "f32" else 1 / 32))
        if op == "gated_act":
            return {"bytes": n * (4 + kept + (2 if c["h"] == "bf16" else 1 + 1 / 32)), "flops": 10 * n}
        return {"bytes": n * (2 + kept + 4 + (2 if c["h"] else 0)), "flops": 15 * n}
    M, N, K = c["M"], c["N"], c["K"]
    kept = 1 + (4 / 128 if c["scale"] == "f32" else 1 / 32)
    return {"bytes": M * N * 2 + N * K * 2 + M * K * kept + M * K * 2 + N * K * 2, "flops": 4 * M * N * K}


# --------------------------------------------------------------------------- #
# From the definitions, in 64 bits                                            #
# --------------------------------------------------------------------------- #

def _mx64(x, block, code, power_of_two):
    """Code values and scales of x's rows in blocks, binary64, rounding to nearest even by the grid's spacing."""
    rows, cols = x.shape
    xb = x.reshape(rows, cols // block, block)
    amax = xb.abs().amax(-1)
    ratio = amax / QMAX[code]
    if power_of_two:
        e = torch.ceil(torch.log2(torch.where(amax == 0, torch.ones_like(ratio), ratio))).clamp(-127, 127)
        s = torch.exp2(e)
    else:
        s = torch.where(amax == 0, torch.ones_like(ratio), ratio) if code == "int8" else ratio.clamp_min(1e-10)
    q = xb / s[..., None]
    if code == "int8":
        q = torch.round(q)
    else:
        bits, low = (3, -6) if code == "e4m3" else (2, -14)
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** low))) - bits)
        q = torch.round(q / step) * step
    return q.clamp(-QMAX[code], QMAX[code]).reshape(rows, cols), s


def _values64(codes, scales, code):
    """What a checkpoint's codes stand for: binary32(code * scale), by definition."""
    v = codes.double() if code == "int8" else codes.view(FP8[code]).double()
    s = torch.exp2(scales.double() - 127) if scales.dtype == torch.uint8 else scales.double()
    return (v.reshape(v.shape[0], s.shape[1], -1) * s[..., None]).reshape(v.shape).float().double()


def _down64(x, fp8):
    q, s = _mx64(x.t().contiguous(), 32, fp8, True)
    return (q.reshape(q.shape[0], s.shape[1], -1) * s[..., None]).reshape(q.shape).t()


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "adapters":
        x, ids = s["x"].double(), s["ids"].long()
        u = torch.zeros((c["T"], c["R"]), dtype=torch.float64, device=DEV)
        y = s["y"].double()
        for k in range(c["L"]):
            at = torch.nonzero(ids == k)[:, 0]
            u[at] = x[at] @ s["a"][k].double().t()
            y[at] += float(s["scaling"][k]) * (u[at] @ s["b"][k].double().t())
        return {"out": y, "u": u}
    if op == "adapters_backward":
        x = s["x"].double() if c["x"] == "bf16" else _values64(s["x"], s["x_scales"], c["x"])
        dy, u, ids, dx = s["dy"].double(), s["u"].double(), s["ids"].long(), s["dx_base"].double()
        da = torch.zeros(s["a"].shape, dtype=torch.float64, device=DEV)
        db = torch.zeros(s["b"].shape, dtype=torch.float64, device=DEV)
        for k in range(c["L"]):
            at = torch.nonzero(ids == k)[:, 0]
            du = float(s["scaling"][k]) * (dy[at] @ s["b"][k].double())
            dx[at] += du @ s["a"][k].double()
            da[k] = du.t() @ x[at]
            db[k] = float(s["scaling"][k]) * (dy[at].t() @ u[at])
        return {"dx": dx, "da": da, "db": db}
    if op in ("gated_act", "gated_act_backward"):
        I = c["I"]
        gu = s["gate_up"].double() if op == "gated_act" else _values64(s["codes"], s["scales"], c["code"])
        g, up = gu[:, :I], gu[:, I:]
        cdf = torch.sigmoid(g) if c["act"] == "silu" else torch.special.ndtr(g)
        h = g * cdf * up
        if op == "gated_act":
            r = {}
            if c["h"] == "bf16":
                r["h"] = h
            else:
                r["h"], r["h_scales"] = _mx64(h, 32, c["h"], True)
            if c["code"] != "none":
                q, sc = _mx64(gu, _block(c["scale"]), c["code"], c["scale"] == "ue8m0")
                r["codes"], r["scales"] = None if c["code"] == "int8" else q, sc
            return r
        density = cdf * (1 - cdf) if c["act"] == "silu" else torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        dh = s["dh"].double()
        r = {"d_gate_up": torch.cat([dh * up * (cdf + g * density), dh * g * cdf], 1)}
        if c["h"]:
            r["h"] = h
        return r
    x, dy, w = _values64(s["x_codes"], s["x_scales"], c["code"]), s["dY"].double(), s["W"].double()
    q, sc = _mx64(dy, 32, c["fp8"], True)
    dy_n = (q.reshape(q.shape[0], sc.shape[1], -1) * sc[..., None]).reshape(q.shape)
    return {"dX": dy_n @ _down64(w, c["fp8"]), "dW": _down64(dy, c["fp8"]).t() @ _down64(x, c["fp8"])}
