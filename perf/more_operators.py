"""Measured cases of a mixture-of-experts layer in MXFP8, served and trained:
the router, the products grouped by expert with their gradients, the weighted
sum of the experts' results, and the AdamW step over all weights at once.

``run`` makes one pass through an operator: with ``own`` false in its plain
form (elementary torch operations in binary32, rounded once at the end), with
``own`` true through the library's entry points.

Operators (``case["op"]``):

* ``route``             the k largest logits of each token, their softmax, and the tokens' layout by expert
* ``route_backward``    the logits' gradient from the weights'
* ``gemm``              y[s] = W[expert of s] x[rows[s]], MXFP8 codes, ragged numbers of rows an expert
* ``backward``          dX and dW of the same from bfloat16, quantized on the way
* ``combine``           out[t] = sum over j of weights[t, j] y[slots[t, j]]
* ``combine_backward``  dy and the weights' gradient
* ``adamw``             one step over many tensors, states in 32 or in 8 bits
"""

import math

import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- #
# Cases                                                                       #
# --------------------------------------------------------------------------- #

def _route(name, op, T, E, k, renormalize, logits):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "renormalize": renormalize, "logits": logits}


def _gemm(name, T, k, E, N, K, gather, skew, x, w):
    return {"name": name, "op": "gemm", "T": T, "k": k, "E": E, "N": N, "K": K, "gather": gather, "skew": skew, "x": x,
            "w": w}


def _backward(name, T, k, E, N, K, gather, skew, fp8):
    return {"name": name, "op": "backward", "T": T, "k": k, "E": E, "N": N, "K": K, "gather": gather, "skew": skew,
            "fp8": fp8}


def _combine(name, op, T, k, N, out):
    return {"name": name, "op": op, "T": T, "k": k, "N": N, "out": out}


def _adamw(name, tensors, size, odd, params, grads, states, copy):
    return {"name": name, "op": "adamw", "tensors": tensors, "size": size, "odd": odd, "params": params, "grads": grads,
            "states": states, "copy": copy}


def listed():
    return [
        # a decode step of 16 requests: latency counts
        _route("route 16 tokens", "route", 16, 64, 4, True, "f32"),
        # a training batch over many experts; bfloat16 logits tie often
        _route("route 65536 tokens", "route", 65536, 256, 8, False, "bf16"),
        # that batch's backward pass
        _route("route backward 65536", "route_backward", 65536, 256, 8, False, "bf16"),
        # a decode step of 8 requests over 16 experts: the weights' bytes
        _gemm("experts 8 tokens", 8, 2, 16, 4096, 4096, True, False, "e4m3", "e4m3"),
        # a ragged prefill of a small layer, some experts far busier than others, the tokens gathered by row
        _gemm("experts 1501 tokens", 1501, 2, 8, 2048, 4096, True, True, "e4m3", "e4m3"),
        # a full training batch, rows already in the experts' order (the second projection)
        _gemm("experts 65536 rows", 16384, 4, 32, 4096, 4096, False, False, "e4m3", "e4m3"),
        # the gradients of a small ragged step
        _backward("experts backward 1001", 1001, 2, 8, 2048, 1024, True, True, "e5m2"),
        # the gradients of a full batch, tokens gathered by row (the first projection)
        _backward("experts backward 32768", 16384, 2, 16, 4096, 4096, True, False, "e5m2"),
        # a decode step's sum of results
        _combine("combine 16 tokens", "combine", 16, 4, 4096, "bf16"),
        # a full batch's backward pass
        _combine("combine backward 16384", "combine_backward", 16384, 4, 4096, "bf16"),
        # a model's small tensors (norms, biases, odd shapes), plain states
        _adamw("adamw 100 small tensors", 100, 20000, True, "f32", "f32", "f32", False),
        # an expert layer's weights: states in 8 bits, the GEMMs' bfloat16 copy written in the same pass
        _adamw("adamw 8 bits", 4, 67108864, False, "f32", "bf16", "e4m3", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["route", "route_backward", "gemm", "gemm", "gemm", "backward", "backward", "combine",
                     "combine_backward", "adamw", "adamw"])
    if op in ("route", "route_backward"):
        E = rng.choice([rng.randint(2, 8), 16, 64, rng.randint(9, 256), 128, 256])
        return {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(E, 8)),
                "renormalize": rng.choice([True, False]), "logits": rng.choice(["f32", "bf16"])}
    if op in ("combine", "combine_backward"):
        return {"op": op, "T": _log(rng, 1, 16384), "k": rng.choice([1, 2, 2, 4, 6, 8]),
                "N": _mult(rng, 512, 8192, rng.choice([1, 8, 128])), "out": rng.choice(["bf16", "f32"])} \
            if rng.random() < 0.5 else \
            {"op": op, "T": _log(rng, 1, 16384), "k": rng.choice([1, 2, 4]), "N": rng.choice([1024, 2048, 4096]), "out": "bf16"}
    if op in ("gemm", "backward"):
        step = rng.choice([32, 128, 128])
        E = rng.choice([4, 8, 16, rng.randint(1, 32), 32])
        c = {"op": op, "T": _log(rng, 1 if op == "gemm" else 16, 16384), "k": rng.randint(1, min(E, 4)), "E": E,
             "N": _mult(rng, 512, 4096, step), "K": _mult(rng, 512, 4096, step), "gather": rng.choice([True, False]),
             "skew": rng.choice([True, False])}
        if op == "gemm":
            c["x"], c["w"] = rng.choice([("e4m3", "e4m3"), ("e4m3", "e4m3"), ("e5m2", "e4m3")])
        else:
            c["T"] = min(c["T"], 32768 // c["k"])
            c["fp8"] = rng.choice(["e5m2", "e4m3"])
        return c
    states = rng.choice(["f32", "e4m3"])
    tensors = _log(rng, 1, 200)
    return {"op": op, "tensors": tensors, "size": _log(rng, 1000, min(67108864, 200000000 // tensors)),
            "odd": rng.choice([True, False]), "params": rng.choice(["f32", "f32", "bf16"]),
            "grads": rng.choice(["f32", "bf16"]), "states": states, "copy": rng.choice([True, False])}


# --------------------------------------------------------------------------- #
# Inputs                                                                      #
# --------------------------------------------------------------------------- #

def _randn(shape, seed, stream, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + stream)
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _block_quantize(x, block, code, scale):
    """Absmax quantization of each row in blocks: float8 codes and one scale
    per block, binary32 or the exponent byte of a power of two."""
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
        s = torch.where(amax == 0, torch.ones_like(r), r.clamp_min(2.0 ** -126))
        stored = s
    q = (xb / s[..., None]).clamp(-QMAX[code], QMAX[code]).view(rows, cols)
    return q.to(FP8[code]), stored


def _block_values(codes, scales):
    """The values that _block_quantize's codes and scales stand for."""
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.to(torch.int32) - 127) \
        if scales.dtype == torch.uint8 else scales
    rows, cols = codes.shape
    return (codes.float().view(rows, s.shape[1], -1) * s[..., None]).view(rows, cols)


def _atoms(scales):
    """Row-major scale bytes [E, N, K / 32] in the tensor cores' layout: per
    128 rows x 4 blocks 512 bytes, row tiles in pairs, neutral padding."""
    E, N, B = scales.shape
    rt, ks = (N + 255) // 256 * 2, (B + 3) // 4
    full = torch.full((E, rt * 128, ks * 4), 127, dtype=torch.uint8, device=scales.device)
    full[:, :N, :B] = scales
    return full.view(E, rt, 4, 32, ks, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def _layout(T, k, E, skew, seed):
    """Each token's k experts, and the rows in the experts' order."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + 77)
    score = torch.rand((T, E), generator=g, device=DEV)
    if skew:  # some experts are preferred
        score = score + 0.3 * torch.rand((1, E), generator=g, device=DEV)
    ids = score.topk(k, dim=1).indices
    order = torch.argsort(ids.flatten(), stable=True)
    counts = torch.bincount(ids.flatten(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    slots = torch.empty(T * k, dtype=torch.int32, device=DEV)
    slots[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    return offsets, (order // k).to(torch.int32), slots.view(T, k), int(counts.max())


def _sizes(c):
    n, size = c["tensors"], c["size"]
    return [max(1, size + (i * 7919) % 257 - 128) if c["odd"] else max(128, size // 128 * 128) for i in range(n)]


def prepare(case, seed):
    c, op = case, case["op"]
    s = {"case": dict(c)}
    if op in ("route", "route_backward"):
        s["logits"] = _randn((c["T"], c["E"]), seed, 1, 1.5, DTYPE[c["logits"]])
        if op == "route_backward":
            s["weights"], s["ids"] = _choose(s["logits"], c["k"], c["renormalize"])
            s["d_weights"] = _randn((c["T"], c["k"]), seed, 2, 1.0, torch.float32)
    elif op in ("gemm", "backward"):
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        s["offsets"], rows, _, s["most"] = _layout(T, k, E, c["skew"], seed)
        s["rows"] = rows if c["gather"] else None
        x = _randn((T if c["gather"] else T * k, K), seed, 1)
        if op == "gemm":
            s["x"], s["x_scales"] = _block_quantize(x, 32, c["x"], "ue8m0")
            w, ws = _block_quantize(_randn((E * N, K), seed, 2, K ** -0.5), 32, c["w"], "ue8m0")
            s["w"], s["w_scales"] = w.view(E, N, K), ws.view(E, N, K // 32)
            s["w_atoms"] = _atoms(s["w_scales"])  # laid out once, with the weights
        else:
            s["X"], s["W"] = x, _randn((E, N, K), seed, 2, K ** -0.5)
            s["dY"] = _randn((T * k, N), seed, 3)
    elif op in ("combine", "combine_backward"):
        T, k, N = c["T"], c["k"], c["N"]
        _, _, s["slots"], _ = _layout(T, k, max(k, 16), False, seed)
        s["y"] = _randn((T * k, N), seed, 1)
        s["weights"] = torch.softmax(_randn((T, k), seed, 2, 1.0, torch.float32), 1)
        if op == "combine_backward":
            s["d_out"] = _randn((T, N), seed, 3, 1.0, DTYPE[c["out"]])
    else:
        # the tensors lie in one buffer a kind, each from a multiple of 128 on, as a program keeps them that
        # gathers or saves them at once; the gaps hold zeros
        sizes = _sizes(c)
        padded = [(n + 127) // 128 * 128 for n in sizes]
        flat, real = sum(padded), torch.zeros(sum(padded), dtype=torch.bool, device=DEV)
        for t, n in zip(real.split(padded), sizes):
            t[:n] = True
        s["flat"] = {"params": _randn((flat,), seed, 1, 0.02, DTYPE[c["params"]]) * real,
                     "grads": _randn((flat,), seed, 2, 1e-3, DTYPE[c["grads"]]) * real}
        m = _randn((flat,), seed, 3, 3e-4, torch.float32) * real
        v = (_randn((flat,), seed, 4, 1e-3, torch.float32).square() + 1e-8) * real
        if c["states"] == "f32":
            s["flat"] |= {"m": m, "v": v}
        else:
            s["flat"]["m"], s["flat"]["m_scales"] = _state(m)
            s["flat"]["v"], s["flat"]["v_scales"] = _root_state(v)
        if c["copy"]:
            s["flat"]["copies"] = s["flat"]["params"].to(torch.bfloat16)
        for name, t in s["flat"].items():
            blocks = name.endswith("scales")
            parts = t.split([n // 128 for n in padded] if blocks else padded)
            s[name] = list(parts) if blocks else [x[:n] for x, n in zip(parts, sizes)]
    return s


# --------------------------------------------------------------------------- #
# Plain forms                                                                 #
# --------------------------------------------------------------------------- #

def _choose(logits, k, renormalize):
    """Weights and experts of each token: its k largest logits, ties to the lowest index."""
    l = logits.float()
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].to(torch.int32)
    e = torch.exp(top - top[:, :1])
    total = e.sum(1, keepdim=True) if renormalize else torch.exp(l - top[:, :1]).sum(1, keepdim=True)
    return e / total, ids


def _plain_route(s):
    c = s["case"]
    k, E = c["k"], c["E"]
    weights, ids = _choose(s["logits"], k, c["renormalize"])
    keys, order = torch.sort(ids.flatten(), stable=True)
    offsets = torch.searchsorted(keys, torch.arange(E + 1, dtype=torch.int32, device=DEV)).to(torch.int32)
    slots = torch.empty_like(keys)
    slots[order] = torch.arange(keys.numel(), dtype=torch.int32, device=DEV)
    return {"weights": weights, "ids": ids, "offsets": offsets, "rows": (order // k).to(torch.int32),
            "slots": slots.view(-1, k)}


def _plain_route_backward(s):
    c, l = s["case"], s["logits"].float()
    w, dw, ids = s["weights"], s["d_weights"], s["ids"].long()
    mean = (w * dw).sum(1, keepdim=True)
    if c["renormalize"]:
        d = torch.zeros_like(l).scatter_(1, ids, w * (dw - mean))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        d = (-mean * (e / e.sum(1, keepdim=True))).scatter_add_(1, ids, w * dw)
    return {"d_logits": d.to(s["logits"].dtype)}


def _padded(s, most):
    """Index of each expert's i-th row [E, most] (any row past its last), and whether it is one."""
    first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = first[:, None] + torch.arange(most, device=DEV)
    real = at < last[:, None]
    return torch.where(real, at, torch.zeros_like(at)), real


def _unpadded(s, y, S):
    """Rows [S, N] of y [E, most, N]."""
    at = torch.arange(S, device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return y[e, at - s["offsets"].long()[e]]


def _by_row(x, rows):
    return x if rows is None else x[rows.long()]


def _plain_gemm(s):
    c = s["case"]
    E, N, K = c["E"], c["N"], c["K"]
    x = _by_row(_block_values(s["x"], s["x_scales"]), s["rows"])
    w = _block_values(s["w"].view(E * N, K), s["w_scales"].view(E * N, K // 32)).view(E, N, K)
    at, _ = _padded(s, s["most"])
    return {"y": _unpadded(s, torch.bmm(x[at], w.transpose(1, 2)), x.shape[0]).to(torch.bfloat16)}


def _along_rows(x, fp8):
    """[E, rows, cols] quantized down each expert's rows in blocks of 32, as values [E, cols, rows]."""
    E, rows, cols = x.shape
    codes, scales = _block_quantize(x.transpose(1, 2).reshape(E * cols, rows), 32, fp8, "ue8m0")
    return _block_values(codes, scales).view(E, cols, rows)


def _plain_backward(s):
    c, fp8 = s["case"], s["case"]["fp8"]
    dy, x, w = s["dY"].float(), _by_row(s["X"], s["rows"]).float(), s["W"].float()
    at, real = _padded(s, (s["most"] + 31) // 32 * 32)
    dx = torch.bmm(_block_values(*_block_quantize(dy, 32, fp8, "ue8m0"))[at], _along_rows(w, fp8).transpose(1, 2))
    dyt, xt = (_along_rows(t[at] * real[..., None], fp8) for t in (dy, x))
    return {"dX": _unpadded(s, dx, dy.shape[0]).to(torch.bfloat16),
            "dW": torch.bmm(dyt, xt.transpose(1, 2)).to(torch.bfloat16)}


def _plain_combine(s):
    y = s["y"].float()[s["slots"].long()]
    return {"out": (y * s["weights"][..., None]).sum(1).to(DTYPE[s["case"]["out"]])}


def _plain_combine_backward(s):
    at, d = s["slots"].long(), s["d_out"].float()
    dy = torch.empty_like(s["y"])
    dy[at.flatten()] = (s["weights"][..., None] * d[:, None]).to(torch.bfloat16).view(-1, dy.shape[1])
    return {"dy": dy, "d_weights": (s["y"].float()[at] * d[:, None]).sum(-1)}


STEP, LR, BETA1, BETA2, EPS, DECAY = 100, 1e-3, 0.9, 0.95, 1e-8, 0.1


def _state(m):
    """A state in E4M3 per 128 numbers."""
    codes, scales = _block_quantize(m.view(1, -1), 128, "e4m3", "f32")
    return codes.view(-1), scales.view(-1)


def _root_state(v):
    """The root of the second moment, which never falls to zero by rounding."""
    root = torch.sqrt(v)
    codes, scales = _state(root)
    lost = (root > 0) & (codes.float() == 0)
    return torch.where(lost, torch.ones_like(codes, dtype=torch.uint8), codes.view(torch.uint8)).view(codes.dtype), scales


def _state_values(codes, scales):
    return (codes.float().view(-1, 128) * scales[:, None]).view(-1)


def _plain_adamw(s):
    c, f = s["case"], s["flat"]
    p, g, kept = f["params"].float(), f["grads"].float(), c["states"] != "f32"
    m = _state_values(f["m"], f["m_scales"]) if kept else f["m"]
    v = _state_values(f["v"], f["v_scales"]).square() if kept else f["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + ((1 - BETA2) * g) * g
    move = m / (torch.sqrt(v) / math.sqrt(1 - BETA2 ** STEP) + EPS)
    p = p * (1 - LR * DECAY) - (LR / (1 - BETA1 ** STEP)) * move
    f["params"].copy_(p)
    if c["copy"]:
        f["copies"].copy_(p)
    if kept:
        for name, (codes, scales) in (("m", _state(m)), ("v", _root_state(v))):
            f[name].copy_(codes)
            f[name + "_scales"].copy_(scales)
    else:
        f["m"].copy_(m)
        f["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """The updated tensors and states, each kind's buffer as a whole."""
    return {n: t for n, t in s["flat"].items() if n != "grads"}


PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "gemm": _plain_gemm, "backward": _plain_backward,
         "combine": _plain_combine, "combine_backward": _plain_combine_backward, "adamw": _plain_adamw}


# --------------------------------------------------------------------------- #
# The library's calls                                                         #
# --------------------------------------------------------------------------- #

def _own(s):
    import block_scaled_precision_gemm_gb300 as bsmm
    c, op = s["case"], s["case"]["op"]
    if op == "route":
        weights, ids, offsets, rows, slots = bsmm.route(s["logits"], c["k"], renormalize=c["renormalize"])
        return {"weights": weights, "ids": ids, "offsets": offsets, "rows": rows, "slots": slots}
    if op == "route_backward":
        return {"d_logits": bsmm.route_backward(s["d_weights"], s["logits"], s["ids"], s["weights"],
                                                renormalize=c["renormalize"])}
    if op == "gemm":
        return {"y": bsmm.expert_gemm(s["x"], s["x_scales"], s["w"], s["w_atoms"], s["offsets"], rows=s["rows"],
                                      x_type=c["x"], w_type=c["w"])}
    if op == "backward":
        dX, dW = bsmm.expert_backward(s["dY"], s["W"], s["X"], s["offsets"], rows=s["rows"], fp8=c["fp8"])
        return {"dX": dX, "dW": dW}
    if op == "combine":
        return {"out": bsmm.expert_combine(s["y"], s["slots"], s["weights"], out_dtype=DTYPE[c["out"]])}
    if op == "combine_backward":
        dy, d_weights = bsmm.expert_combine_backward(s["d_out"], s["y"], s["slots"], s["weights"])
        return {"dy": dy, "d_weights": d_weights}
    bsmm.adamw(s["params"], s["grads"], s["m"], s["v"], STEP, lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
               m_scales=s.get("m_scales"), v_scales=s.get("v_scales"), copies=s.get("copies"))
    return _adamw_outputs(s)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------- #
# What a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def work(case):
    c, op = case, case["op"]
    if op in ("route", "route_backward"):
        n, size = c["T"] * c["E"], 4 if c["logits"] == "f32" else 2
        if op == "route":
            return {"bytes": n * size + c["T"] * c["k"] * 16 + (c["E"] + 1) * 4, "flops": 4 * n}
        return {"bytes": n * size * (1 if c["renormalize"] else 2) + c["T"] * c["k"] * 12, "flops": 4 * n}
    if op in ("gemm", "backward"):
        T, k, N, K = c["T"], c["k"], c["N"], c["K"]
        S, X = T * k, T if c["gather"] else T * k
        weights = min(c["E"], S) * N * K
        if op == "gemm":
            return {"bytes": (weights + X * K) * (1 + 1 / 32) + S * N * 2 + (S * 4 if c["gather"] else 0), "flops": 2 * S * N * K}
        return {"bytes": S * (N + K) * 2 + X * K * 2 + weights * 2 + c["E"] * N * K * 2 + (S * 4 if c["gather"] else 0),
                "flops": 4 * S * N * K}
    if op in ("combine", "combine_backward"):
        T, k, N = c["T"], c["k"], c["N"]
        out = 4 if c["out"] == "f32" else 2
        if op == "combine":
            return {"bytes": T * k * (N * 2 + 8) + T * N * out, "flops": 2 * T * k * N}
        return {"bytes": T * k * (N * 4 + 12) + T * N * out, "flops": 3 * T * k * N}
    n = sum(_sizes(c))
    p, g = (4 if c["params"] == "f32" else 2), (4 if c["grads"] == "f32" else 2)
    state = 8 if c["states"] == "f32" else 2 * (1 + 4 / 128)
    return {"bytes": n * (2 * p + g + 2 * state + (2 if c["copy"] else 0)), "flops": 15 * n}


# --------------------------------------------------------------------------- #
# From the definitions, in 64 bits                                            #
# --------------------------------------------------------------------------- #

def _grid64(q, code):
    """q rounded to the code's grid, to nearest even by the grid's spacing."""
    bits, low = (3, -6) if code == "e4m3" else (2, -14)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** low))) - bits)
    return (torch.round(q / step) * step).clamp(-QMAX[code], QMAX[code])


def _mx64(x, code):
    """Values of x's rows quantized in blocks of 32 (the last may be shorter) with power-of-two scales."""
    rows, cols = x.shape
    xb = torch.cat([x, x.new_zeros(rows, -cols % 32)], 1).reshape(rows, -1, 32)
    ratio = xb.abs().amax(-1, keepdim=True) / QMAX[code]
    scale = torch.exp2(torch.ceil(torch.log2(torch.where(ratio == 0, torch.ones_like(ratio), ratio))).clamp(-127, 127))
    return (_grid64(xb / scale, code) * scale).reshape(rows, -1)[:, :cols]


def _kept64(codes, scales):
    s = torch.exp2(scales.double() - 127)
    return (codes.double().reshape(s.shape[0], s.shape[1], 32) * s[..., None]).reshape(s.shape[0], -1)


def _flat_blocks64(x):
    """E4M3 codes and scales of a flat array per 128 numbers."""
    xb = x.reshape(-1, 128)
    top = xb.abs().amax(1)
    scale = torch.where(top == 0, torch.ones_like(top), top / 448)
    return _grid64(xb / scale[:, None], "e4m3").reshape(-1), scale


def exact(case, seed):
    c, op = case, case["op"]
    if op in ("gemm", "backward") and c["T"] * c["k"] * c["N"] * c["K"] > 3e12:
        return None
    s = prepare(case, seed)
    if op in ("route", "route_backward"):
        l, k = s["logits"].double(), c["k"]
        p = torch.softmax(l, 1)
        if op == "route":
            ids = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
            w = p.gather(1, ids)
            r = _layout_of(ids, c["E"])
            return {"weights": w / w.sum(1, keepdim=True) if c["renormalize"] else w, "ids": ids.to(torch.int32), **r}
        w, dw, ids = s["weights"].double(), s["d_weights"].double(), s["ids"].long()
        chosen = torch.zeros_like(l).scatter_(1, ids, w)
        d = torch.zeros_like(l).scatter_(1, ids, w * dw)
        mean = (w * dw).sum(1, keepdim=True)
        return {"d_logits": d - (chosen if c["renormalize"] else p) * mean}
    if op in ("gemm", "backward"):
        bounds = s["offsets"].tolist()
        rows = s["rows"].long() if c["gather"] else torch.arange(c["T"] * c["k"], device=DEV)
        spans = [(e, slice(bounds[e], bounds[e + 1])) for e in range(c["E"]) if bounds[e + 1] > bounds[e]]
        if op == "gemm":
            y = torch.empty((c["T"] * c["k"], c["N"]), dtype=torch.float64, device=DEV)
            x = _kept64(s["x"], s["x_scales"])
            for e, at in spans:
                y[at] = x[rows[at]] @ _kept64(s["w"][e], s["w_scales"][e]).t()
            return {"y": y}
        dx = torch.empty((c["T"] * c["k"], c["K"]), dtype=torch.float64, device=DEV)
        dw = torch.zeros(s["W"].shape, dtype=torch.float64, device=DEV)
        for e, at in spans:
            dy, x = s["dY"][at].double(), s["X"][rows[at]].double()
            dx[at] = _mx64(dy, c["fp8"]) @ _mx64(s["W"][e].double().t().contiguous(), c["fp8"]).t()
            dw[e] = _mx64(dy.t().contiguous(), c["fp8"]) @ _mx64(x.t().contiguous(), c["fp8"]).t()
        return {"dX": dx, "dW": dw}
    if op in ("combine", "combine_backward"):
        y, at, w = s["y"].double(), s["slots"].long(), s["weights"].double()
        if op == "combine":
            return {"out": torch.einsum("tk,tkn->tn", w, y[at])}
        d = s["d_out"].double()
        dy = torch.zeros_like(y)
        dy.index_put_((at,), w[..., None] * d[:, None])
        return {"dy": dy, "d_weights": torch.einsum("tn,tkn->tk", d, y[at])}
    p, g, m, v = (s["flat"][n].double() for n in ("params", "grads", "m", "v"))
    kept = c["states"] == "e4m3"
    if kept:
        block = torch.arange(p.numel(), device=DEV) // 128
        m, v = m * s["flat"]["m_scales"].double()[block], (v * s["flat"]["v_scales"].double()[block]) ** 2
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    hat_m, hat_v = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    r = {"params": p - LR * (hat_m / (hat_v.sqrt() + EPS) + DECAY * p)}
    if c["copy"]:
        r["copies"] = r["params"]
    if not kept:
        return {**r, "m": m, "v": v}
    r["m"], r["m_scales"] = _flat_blocks64(m)
    codes, r["v_scales"] = _flat_blocks64(v.sqrt())
    r["v"] = torch.where((v > 0) & (codes == 0), torch.full_like(codes, 2.0 ** -9), codes)
    return r


def _layout_of(ids, E):
    """Offsets, rows and slots of the (token, choice) pairs by expert, from counts alone."""
    flat = ids.flatten()
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.argsort(flat * flat.numel() + torch.arange(flat.numel(), device=DEV))
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=DEV)
    return {"offsets": offsets.to(torch.int32), "rows": (order // ids.shape[1]).to(torch.int32),
            "slots": slots.view(ids.shape).to(torch.int32)}
