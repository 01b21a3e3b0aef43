"""The sharded optimizer step and the 4-bit product: what is measured of them, and in which sizes.

Five operators: the global gradient norm with its clip factor, AdamW over many shards with states in 32 or
8 bits, microscaled 4-bit quantisation, and the product of 4-bit operands (a linear layer's forward pass on
stored weights, and a training step with both gradients).
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128                     # elements that share a scale in an 8-bit state
E4M3_MAX = 448.0
LR, B1, B2, EPS, WD = 3e-4, 0.9, 0.95, 1e-8, 0.1
GOLDEN, MUL1, MUL2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the shards of the uneven workload, 10,000,019 fp32 gradients over 8 ranks: no shard but the first starts on 16 bytes
        {"name": "norm_ragged_shards", "op": "norm", "shards": 8, "len": 1_250_003, "g": "f32"},
        # the eight full 25,000,000-element buckets of the headline layer, 8 shards each
        {"name": "norm_layer", "op": "norm", "shards": 64, "len": 3_125_000, "g": "bf16"},
        # norm weights and biases: many small tensors, where the launch counts
        {"name": "adamw_small_tensors", "op": "adamw", "shards": 16, "len": 4_099, "p": "f32", "g": "f32", "copy": False},
        # the layer's shards with fp32 masters, bf16 gradients, and the bf16 copy that is gathered next
        {"name": "adamw_layer", "op": "adamw", "shards": 64, "len": 3_125_000, "p": "f32", "g": "bf16", "copy": True},
        # the uneven workload's shards in plain bf16 training with 8-bit states
        {"name": "adamw8_ragged_shards", "op": "adamw8", "shards": 8, "len": 1_250_003, "p": "bf16", "g": "bf16", "copy": False, "stochastic": False},
        # the layer's shards with 8-bit states, stochastically rounded
        {"name": "adamw8_layer", "op": "adamw8", "shards": 64, "len": 3_125_000, "p": "f32", "g": "bf16", "copy": True, "stochastic": True},
        # a ragged batch of fp32 activations, for the forward product only
        {"name": "quantize_ragged", "op": "quantize", "rows": 1000, "cols": 2049, "x": "f32", "both": False},
        # the layer's gate matrix after its update: for the forward product, and transposed for the backward one
        {"name": "quantize_gate", "op": "quantize", "rows": 14336, "cols": 4096, "x": "bf16", "both": True},
        # one token through the gate matrix
        {"name": "linear_token", "op": "linear", "m": 1, "n": 14336, "k": 4096, "y": "bf16"},
        # a small batch through a small odd-sized layer
        {"name": "linear_ragged", "op": "linear", "m": 201, "n": 1000, "k": 2000, "y": "f32"},
        # a long prompt through the gate matrix
        {"name": "linear_prompt", "op": "linear", "m": 8192, "n": 14336, "k": 4096, "y": "bf16"},
        # a training step of the attention output layer: output, input gradient, weight gradient
        {"name": "linear_train", "op": "train", "m": 4096, "n": 4096, "k": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "adamw", "adamw8", "quantize", "linear", "train"])
    if op in ("norm", "adamw", "adamw8"):
        shards = _log(rng, 1, 64)
        case = {"op": op, "shards": shards, "len": _log(rng, 1_000, min(20_000_000, 150_000_000 // shards)), "g": rng.choice(["f32", "bf16"])}
        if op != "norm":
            case["p"] = rng.choice(["f32", "bf16"])
            case["copy"] = case["p"] == "f32" and rng.random() < 0.5
        if op == "adamw8":
            case["stochastic"] = rng.random() < 0.5
        return case
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 14336), "cols": _log(rng, 32, 4096), "x": rng.choice(["f32", "bf16"]), "both": rng.random() < 0.5}
    case = {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 16, 8192), "k": _log(rng, 32, 4096)}
    if op == "linear":
        case["y"] = rng.choice(["f32", "bf16"])
    else:
        case["m"] = _log(rng, 32, 4096)
        case["n"] = min(case["n"], 4096)
    return case


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _blocks(x):
    """[T, L] as [T, ceil(L / 128), 128], the last block filled up with zeros."""
    t, n = x.shape
    return torch.nn.functional.pad(x, (0, -n % BLOCK)).view(t, -1, BLOCK)


def _optimizer_state(case, gen):
    shape = (case["shards"], case["len"])
    s = {"g": _normal(gen, shape, 1e-3, DTYPES[case["g"]])}
    s["p"] = _normal(gen, shape, 0.02, DTYPES[case["p"]])
    s["copy"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    m = _normal(gen, shape, 3e-4)
    v = (_normal(gen, shape, 1e-3) * (0.2 + torch.rand(shape, generator=gen, device=DEV))).square()
    if case["op"] == "adamw":
        s["m"], s["v"] = m, v
    else:
        r = v.sqrt()
        mb, rb = _blocks(m), _blocks(r)
        s["scales"] = torch.stack([mb.abs().amax(2), rb.amax(2)], 2) / E4M3_MAX
        for name, b, at in (("m", mb, 0), ("v", rb, 1)):
            q = (b / s["scales"][:, :, at:at + 1]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s[name] = q.view(torch.uint8).view(shape[0], -1)[:, :shape[1]].contiguous().view(torch.float8_e4m3fn)
        del mb, rb
    s["clip"] = torch.full((), 0.75, device=DEV)
    s["t"] = 1 + int(torch.randint(0, 1000, (), generator=gen, device=DEV))
    s["seed"] = 1 + int(torch.randint(0, 1 << 40, (), generator=gen, device=DEV))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        s["g"] = _normal(gen, (case["shards"], case["len"]), 1e-3, DTYPES[case["g"]])
        s["max_norm"] = 1.0
        s["step"] = torch.zeros((), dtype=torch.int32, device=DEV)
        s["skipped"] = torch.zeros((), dtype=torch.int32, device=DEV)
        if own:
            import gradient_sync_amd as dps
            s["plan"] = dps.GradNorm(list(s["g"]))
    elif op in ("adamw", "adamw8"):
        s |= _optimizer_state(case, gen)
        if own:
            import gradient_sync_amd as dps
            rows = {k: None if s.get(k) is None else list(s[k]) for k in ("p", "g", "m", "v", "copy", "scales")}
            s["ctrl"] = dps.StepCtrl(scale=0.75, step=s["t"])
            s["plan"] = dps.AdamW(rows["p"], rows["g"], rows["m"], rows["v"], copies=rows["copy"], scales=rows["scales"],
                                  lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD,
                                  seed=s["seed"] if case.get("stochastic") else None)
    elif op == "quantize":
        s["x"] = _normal(gen, (case["rows"], case["cols"]), 0.5, DTYPES[case["x"]])
        s["x"] *= torch.exp2(torch.randint(-6, 7, (case["rows"], 1), generator=gen, device=DEV).float()).to(s["x"].dtype)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = _normal(gen, (m, k), 1.0, torch.bfloat16)
        w = _normal(gen, (n, k), 0.02, torch.bfloat16)
        if op == "train":
            s["w"] = w
            s["dy"] = _normal(gen, (m, n), 1.0, torch.bfloat16)
        elif own:
            import gradient_sync_amd as dps
            s["weight"] = dps.dp_mxfp4_quantize(w)
        else:
            s["codes"], s["exps"] = _quantize(w.float())
    return s


# ------------------------------------------------------------------ plain forms

def _signed(x):
    return x - (1 << 64) if x >= 1 << 63 else x


def _mix(x):
    """SplitMix64's output function, on Python integers."""
    mask = (1 << 64) - 1
    x = ((x ^ (x >> 30)) * MUL1) & mask
    x = ((x ^ (x >> 27)) * MUL2) & mask
    return x ^ (x >> 31)


def _mix_tensor(x):
    """The same on int64 tensors: products wrap, and a logical shift is an arithmetic one with the sign's copies cleared."""
    x = (x ^ ((x >> 30) & ((1 << 34) - 1))) * _signed(MUL1)
    x = (x ^ ((x >> 27) & ((1 << 37) - 1))) * _signed(MUL2)
    return x ^ ((x >> 31) & ((1 << 33) - 1))


def _random(s, shape):
    """16 random bits for m and 16 for sqrt(v) of each element, as fractions: a counter hashed with (seed, step, shard)."""
    t, n = shape
    mask = (1 << 64) - 1
    key = _mix((s["seed"] + s["t"] * GOLDEN) & mask)
    shard = torch.arange(1, t + 1, device=DEV)
    pair = torch.arange(1, (n + 1) // 2 + 1, device=DEV)
    z = _mix_tensor(_mix_tensor(_signed(key) + shard * _signed(GOLDEN)).unsqueeze(1) + pair * _signed(GOLDEN))
    bits = [((z >> at) & 0xFFFF).float() / 65536 for at in (0, 32, 16, 48)]
    return [torch.stack(bits[at:at + 2], 2).view(t, -1)[:, :n] for at in (0, 2)]


def _to_e4m3(y, u):
    """y in [-448, 448] to 8 bits: nearest, or up with the probability of the remainder where `u` is given."""
    if u is not None:
        a = y.abs()
        e = (torch.frexp(a)[1] - 1).clamp(min=-6) - 3
        up = ((127 - e) << 23).view(torch.float32)
        down = ((127 + e) << 23).view(torch.float32)
        y = torch.copysign(torch.floor(a * up + u).mul_(down).clamp_(max=E4M3_MAX), y)
    return y.to(torch.float8_e4m3fn)


def _adamw(s):
    case, t = s["case"], s["t"]
    eight = case["op"] == "adamw8"
    g = s["g"].float() * s["clip"]
    if eight:
        n = case["len"]
        spread = lambda at: s["scales"][:, :, at].repeat_interleave(BLOCK, 1)[:, :n]
        m, v = s["m"].float() * spread(0), (s["v"].float() * spread(1)).square()
    else:
        m, v = s["m"], s["v"]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * g) * (1 - B2)
    r = v.sqrt()
    del g
    p = s["p"].float() * (1 - LR * WD) - m / (r * (1 / math.sqrt(1 - B2 ** t)) + EPS) * (LR / (1 - B1 ** t))
    s["p"].copy_(p)
    out = {"p": s["p"]}
    if s["copy"] is not None:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    del p
    if eight:
        del v
        u = _random(s, m.shape) if case["stochastic"] else (None, None)
        amax = [_blocks(x).abs().amax(2, keepdim=True) for x in (m, r)]
        inv = [torch.where(a >= 2.0 ** -100, E4M3_MAX / a, 0.0).expand(-1, -1, BLOCK).reshape(m.shape[0], -1)[:, :n] for a in amax]
        s["scales"].copy_(torch.where(torch.cat(amax, 2) >= 2.0 ** -100, torch.cat(amax, 2) / E4M3_MAX, 0.0))
        s["m"].copy_(_to_e4m3((m * inv[0]).clamp_(-E4M3_MAX, E4M3_MAX), u[0]))
        y = r * inv[1]
        q = _to_e4m3(y.clamp(max=E4M3_MAX), u[1])
        s["v"].copy_(torch.where((y > 0) & (q.float() == 0), 2.0 ** -9, q.float()))
        out["scales"] = s["scales"]
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    out["m"], out["v"] = s["m"], s["v"]
    return out


def _quantize(x):
    """Codes 0..15 [rows, 32 * blocks] and exponents [rows, blocks] of fp32 rows, 32 columns a block."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 32)).view(x.shape[0], -1, 32)
    a = x.abs()
    top = a.amax(2, keepdim=True)
    e = torch.where(top > 0, (torch.frexp(top)[1] - 3).clamp(min=-127), -127)
    a = a * ((127 - e) << 23).view(torch.float32)
    c = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)) + 8 * torch.signbit(x)
    return c.to(torch.uint8).view(x.shape[0], -1), e.squeeze(2).to(torch.int16)


def _values(codes, exps):
    """What codes and exponents stand for, in fp32."""
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    scale = torch.exp2(exps.double()).float()
    return (e2m1[codes.int()].view(codes.shape[0], -1, 32) * scale.unsqueeze(2)).view(codes.shape)


def _rounded(x):
    return _values(*_quantize(x.float()))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        norm = s["g"].double().square().sum().sqrt()
        fine = torch.isfinite(norm)
        s["step"] += fine
        s["skipped"] += ~fine
        scale = torch.where(fine, torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0), 0.0)
        return {"norm": norm.float(), "scale": scale.float(), "step": s["step"], "skipped": s["skipped"]}
    if op in ("adamw", "adamw8"):
        return _adamw(s)
    if op == "quantize":
        out = {"rows": _rounded(s["x"])[:, :case["cols"]].bfloat16()}
        if case["both"]:
            out["cols"] = _rounded(s["x"].t().contiguous())[:, :case["rows"]].bfloat16()
        return out
    if op == "linear":
        return _rounded(s["x"]).matmul(_values(s["codes"], s["exps"]).t()).to(DTYPES[case["y"]])
    x, w, dy = s["x"], s["w"], s["dy"]
    return {"y": _rounded(x).matmul(_rounded(w).t()).bfloat16(),
            "dx": _rounded(dy).matmul(_rounded(w.t().contiguous()).t()).bfloat16(),
            "dw": _rounded(dy.t().contiguous()).matmul(_rounded(x.t().contiguous()).t())}


def _own(s):
    import gradient_sync_amd as dps
    case = s["case"]
    op = case["op"]
    if op == "norm":
        ctrl = s["plan"].run(max_norm=s["max_norm"])
        return {"norm": ctrl.norm, "scale": ctrl.scale, "step": ctrl.step, "skipped": ctrl.skipped}
    if op in ("adamw", "adamw8"):
        s["plan"].step(ctrl=s["ctrl"])
        out = {k: s[k] for k in ("p", "m", "v")}
        if s["copy"] is not None:
            out["copy"] = s["copy"]
        if op == "adamw8":
            out["scales"] = s["scales"]
        return out
    if op == "quantize":
        q = dps.dp_mxfp4_quantize(s["x"], transposed="also" if case["both"] else "no")
        if not case["both"]:
            return {"rows": dps.dp_mxfp4_dequantize(q)}
        return {"rows": dps.dp_mxfp4_dequantize(q[0]), "cols": dps.dp_mxfp4_dequantize(q[1])}
    if op == "linear":
        return dps.dp_mxfp4_linear(s["x"], s["weight"], dtype=DTYPES[case["y"]])
    x, xt = dps.dp_mxfp4_quantize(s["x"], transposed="also")
    w, wt = dps.dp_mxfp4_quantize(s["w"], transposed="also")
    dy, dyt = dps.dp_mxfp4_quantize(s["dy"], transposed="also")
    return {"y": dps.dp_gemm_mxfp4(x, w), "dx": dps.dp_gemm_mxfp4(dy, wt),
            "dw": dps.dp_gemm_mxfp4(dyt, xt, dtype=torch.float32)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op in ("norm", "adamw", "adamw8"):
        n = case["shards"] * case["len"]
        if op == "norm":
            return {"bytes": n * size[case["g"]] + 16, "flops": 2 * n}
        states = 16 if op == "adamw" else 4 + 16 / BLOCK
        return {"bytes": n * (2 * size[case["p"]] + size[case["g"]] + states + (2 if case["copy"] else 0)), "flops": 14 * n}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x"]] + (4 if case["both"] else 2)), "flops": n * (6 if case["both"] else 3)}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear":
        return {"bytes": 2 * m * k + n * k * 17 / 32 + m * n * size[case["y"]], "flops": 2 * m * n * k}
    return {"bytes": 2 * (m * k + n * k + m * n) + 2 * m * n + 2 * m * k + 4 * n * k, "flops": 6 * m * n * k}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _power_of_two(e):
    """2^e, whose bits are its exponent's."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_fp4(x):
    """Each row's blocks of 32 to the nearest multiple that e2m1 has of 2^(floor(log2 max) - 2), in 64 bits: the grid's step is 2^-1 below 2, 1 below 4, and 2 above."""
    rows, cols = x.shape
    b = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=DEV)
    b[:, :cols] = x.double()
    b = b.view(rows, -1, 32)
    _, e = torch.frexp(b.abs().max(2, keepdim=True).values)
    unit = _power_of_two((e - 3).clamp(min=-127))
    y = b / unit
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    y = (y / step).round() * step            # round() takes ties to even
    return (y.clamp(-6, 6) * unit).view(rows, -1)


def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    s = prepare(case, seed)
    globals()["own"] = was
    op = case["op"]
    if op == "norm":
        norm = torch.linalg.vector_norm(s["g"].double())
        return {"norm": norm, "scale": torch.clamp(s["max_norm"] / norm, max=1.0), "step": None, "skipped": None}
    if op in ("adamw", "adamw8"):
        t = s["t"]
        if op == "adamw":
            m0, v0 = s["m"].double(), s["v"].double()
        else:
            block = torch.arange(case["len"], device=DEV) // BLOCK
            m0 = s["m"].double() * s["scales"][:, :, 0].double()[:, block]
            v0 = (s["v"].double() * s["scales"][:, :, 1].double()[:, block]) ** 2
        g = s["g"].double() * 0.75
        m = B1 * m0 + (1 - B1) * g
        v = B2 * v0 + (1 - B2) * g ** 2
        del m0, v0, g
        p = (1 - LR * WD) * s["p"].double()
        p -= LR * (m / (1 - B1 ** t)) / (torch.sqrt(v / (1 - B2 ** t)) + EPS)
        out = {"p": p, "copy": p} if case["copy"] else {"p": p}
        if op == "adamw":
            return out | {"m": m, "v": v}
        r = v.sqrt()
        scales = torch.stack([_blocks(x).abs().amax(2) / E4M3_MAX for x in (m, r)], 2)
        # a rounding at random has no one value in 64 bits
        if case["stochastic"]:
            return out | {"scales": scales, "m": None, "v": None}
        return out | {"scales": scales, "m": m / scales[:, :, 0][:, block], "v": r / scales[:, :, 1][:, block]}
    if op == "quantize":
        out = {"rows": _nearest_fp4(s["x"])[:, :case["cols"]]}
        if case["both"]:
            out["cols"] = _nearest_fp4(s["x"].t())[:, :case["rows"]]
        return out
    x = _nearest_fp4(s["x"])
    if op == "linear":
        e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        c = s["codes"].long()
        w = e2m1[c % 8] * (1 - 2 * (c // 8)) * _power_of_two(s["exps"]).repeat_interleave(32, 1)
        return x @ w.T
    return {"y": x @ _nearest_fp4(s["w"]).T,
            "dx": _nearest_fp4(s["dy"]) @ _nearest_fp4(s["w"].t()).T,
            "dw": _nearest_fp4(s["dy"].t()) @ _nearest_fp4(s["x"].t()).T}
