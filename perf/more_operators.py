"""What is measured of the 4-bit parameter and layer-norm operators.

Operators around the step: they read the parameters that it writes, and leave
the gradients that it takes.

  quantize  a matrix to 4-bit floating point (E2M1) in blocks along its rows,
            and along its columns for products that sum over the rows.  "nv":
            16 elements to an E4M3 scale, one power of two per matrix; "mx": 32
            elements to an E8M0 scale.  A scale is the least of its type that
            takes the block's largest magnitude to at most 6; elements go to
            the nearest value, ties to even, or are rounded up with the
            probability of their distance (random bits of Philox4x32-10).
  product   C = A B^T of two quantised matrices, or C += A B^T
  linear    a layer's forward pass and both gradients in 4-bit products
  norm      layer norm; norm_back its gradients, the gain's and the bias's
            summed over the rows

With `own` the calls go to the library; without it the same results come from
elementary torch operations in fp32.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
BLOCK = {"nv": 16, "mx": 32}


def listed():
    return [
        # the smallest call: the smallest weight of a tiny network
        {"name": "quantize_tiny", "op": "quantize", "rows": 32, "cols": 64, "in": "bf16", "format": "nv",
         "sides": "row", "seed": 0},
        # an output gradient before the products that take it, stochastic, odd sizes, both orientations
        {"name": "quantize_gradient", "op": "quantize", "rows": 4099, "cols": 1531, "in": "bf16", "format": "nv",
         "sides": "both", "seed": 77},
        # the masters of the largest weight of an 8B Llama-3-shaped layer, both orientations
        {"name": "quantize_master", "op": "quantize", "rows": 14336, "cols": 4096, "in": "f32", "format": "mx",
         "sides": "both", "seed": 0},
        # a few tokens through the same weight: the weight's bytes bound it
        {"name": "product_few", "op": "product", "m": 8, "n": 14336, "k": 4096, "format": "nv", "out": "bf16",
         "add": False},
        # attention input projection of a GPT-2-small-shaped model: short sums
        {"name": "product_gpt2", "op": "product", "m": 4096, "n": 2304, "k": 768, "format": "mx", "out": "bf16",
         "add": False},
        # a weight gradient added to its fp32 accumulator, odd sizes, long sums
        {"name": "product_gradient", "op": "product", "m": 1111, "n": 777, "k": 5003, "format": "mx",
         "out": "f32", "add": True},
        # tokens of a microbatch through a weight of an 8B Llama-3-shaped layer
        {"name": "product_llama8b", "op": "product", "m": 8192, "n": 14336, "k": 4096, "format": "nv",
         "out": "bf16", "add": False},
        # forward pass and both gradients of a 1B Llama-shaped layer's weight
        {"name": "linear_llama1b", "op": "linear", "rows": 4096, "m": 8192, "k": 2048, "format": "nv", "seed": 5},
        # the smallest norm
        {"name": "norm_tiny", "op": "norm", "rows": 32, "cols": 64, "in": "f32", "bias": True},
        # norm before a layer of an 8B Llama-3-shaped model
        {"name": "norm_llama8b", "op": "norm", "rows": 16384, "cols": 4096, "in": "bf16", "bias": False},
        # gradients of a GPT-2-small-shaped norm: few columns, many rows to sum over
        {"name": "norm_back_gpt2", "op": "norm_back", "rows": 8192, "cols": 768, "in": "bf16", "bias": True},
        # gradients of the norm before a layer of an 8B Llama-3-shaped model
        {"name": "norm_back_llama8b", "op": "norm_back", "rows": 16384, "cols": 4096, "in": "bf16", "bias": True},
    ]


def _dim(rng, hi):
    n = int(round(math.exp(rng.uniform(0.0, math.log(hi)))))
    if n > 64 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(1, n)


def draw(rng):
    op = rng.choice(["quantize", "quantize", "product", "product", "linear", "norm", "norm_back"])
    while True:
        if op == "quantize":
            case = {"op": op, "rows": _dim(rng, 32768), "cols": _dim(rng, 16384), "in": rng.choice(["bf16", "f32"]),
                    "format": rng.choice(["nv", "mx"]), "sides": rng.choice(["row", "col", "both"]),
                    "seed": rng.choice([0, rng.randint(1, 2 ** 62)])}
            fits = case["rows"] * case["cols"] <= 50e6
        elif op == "product":
            case = {"op": op, "m": _dim(rng, 16384), "n": _dim(rng, 16384), "k": _dim(rng, 16384),
                    "format": rng.choice(["nv", "mx"]), "out": rng.choice(["bf16", "f32"])}
            case["add"] = case["out"] == "f32" and rng.random() < 0.5
            fits = 2.0 * case["m"] * case["n"] * case["k"] <= 9e11 and case["m"] * case["n"] <= 1e8
        elif op == "linear":
            case = {"op": op, "rows": _dim(rng, 8192), "m": _dim(rng, 8192), "k": _dim(rng, 8192),
                    "format": rng.choice(["nv", "mx"]), "seed": rng.randint(1, 2 ** 62)}
            fits = 6.0 * case["rows"] * case["m"] * case["k"] <= 4e11
        else:
            # (over two columns the gradient is what rounding leaves of a difference)
            case = {"op": op, "rows": _dim(rng, 65536), "cols": 7 + _dim(rng, 16377), "in": rng.choice(["bf16", "f32"]),
                    "bias": rng.random() < 0.7}
            fits = case["rows"] * case["cols"] <= 60e6
        if fits:
            return case


def _packed(case):
    """Bytes of a quantised element: four bits and its share of a scale."""
    return 0.5 + 1.0 / BLOCK[case["format"]]


def work(case):
    if case["op"] == "quantize":
        n = float(case["rows"] * case["cols"])
        sides = 2 if case["sides"] == "both" else 1
        # read; each orientation written, and the values it stands for
        return {"bytes": n * ((2 if case["in"] == "bf16" else 4) + sides * (_packed(case) + 2)), "flops": 4 * n * sides}
    if case["op"] == "product":
        m, n, k = float(case["m"]), float(case["n"]), float(case["k"])
        out = (2 if case["out"] == "bf16" else 4) * (2 if case["add"] else 1)
        return {"bytes": (m + n) * k * _packed(case) + m * n * out, "flops": 2 * m * n * k}
    if case["op"] == "linear":
        t, m, k = float(case["rows"]), float(case["m"]), float(case["k"])
        # x, dy and both forms of the weight read; y, dx and dw written
        return {"bytes": t * (m + k) * 4 + m * k * (2 * _packed(case) + 2), "flops": 6 * t * m * k}
    n, e = float(case["rows"] * case["cols"]), 2 if case["in"] == "bf16" else 4
    return {"bytes": n * e * (2 if case["op"] == "norm" else 3), "flops": n * (8 if case["op"] == "norm" else 16)}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _philox(seed, side, rows, cols):
    """16 random bits of each element of a rows x cols matrix: those of element
    (r, c) are half-word c mod 8 of the four words for the counter
    (r ceil(cols / 8) + c // 8, side)."""
    per = (cols + 7) // 8
    at = torch.arange(rows * per, device="cuda", dtype=torch.int64)
    mask = 0xFFFFFFFF
    x, key = [at & mask, at >> 32, torch.full_like(at, side), torch.zeros_like(at)], [seed & mask, seed >> 32]
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57       # (products mod 2^64: their bits are right)
        x = [(b >> 32 & mask) ^ x[1] ^ key[0], b & mask, (a >> 32 & mask) ^ x[3] ^ key[1], a & mask]
        key = [(key[0] + 0x9E3779B9) & mask, (key[1] + 0xBB67AE85) & mask]
    u = torch.stack([h for w in x for h in (w & 0xFFFF, w >> 16)], -1)
    return u.view(rows, per * 8)[:, :cols]


def _exponent(x):
    """floor(log2(x)) of positive x, exactly."""
    return torch.frexp(x)[1] - 1


def _power(e):
    """2^e in fp32, e from -127 on."""
    return torch.where(e >= -126, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantized(x, fmt, seed=0, side=0):
    """The values that the quantised form of x stands for, in fp32."""
    x = x.float()
    rows, cols = x.shape
    b = BLOCK[fmt]
    finite = x.isfinite()
    v = torch.where(finite, x, 0.0).abs()
    pad = (-cols) % b
    v = torch.nn.functional.pad(v, (0, pad)).view(rows, -1, b)
    top = v.amax(2, keepdim=True)
    unit = 1.0
    if fmt == "nv":
        most = v.amax()
        e = _exponent(most)
        unit = _power((e - 11 + (most > _power(e) * 1.3125)).clamp_min(-126))
        v, top = v / unit, top / unit
        q = top.double() / 6
        step = _power(_exponent(q).clamp_min(-6) - 3)
        s = (torch.ceil(q / step) * step).float()
    else:
        e = _exponent(top)
        e = (e - 2 + (top > _power(e) * 1.5)).clamp_min(-127)
        s = _power(torch.where(top > 0, e, -127))
    y = v / torch.where(s > 0, s, 1.0)
    gap = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    if seed:
        u = torch.nn.functional.pad(_philox(seed, side, rows, cols), (0, pad)).view(v.shape).float()
        low = torch.floor(y / gap) * gap
        y = torch.where(v - low * s > (2 * u + 1) * 2.0 ** -17 * gap * s, low + gap, low)
    else:
        y = torch.round(y / gap) * gap
    y = (y * s * unit).view(rows, -1)[:, :cols]
    bad = torch.nn.functional.pad(~finite, (0, pad)).view(rows, -1, b).any(2, keepdim=True)
    y = torch.where(bad.expand(-1, -1, b).reshape(rows, -1)[:, :cols], float("nan"), y)
    return torch.where(x < 0, -y, y)


def _values(state, x, seed, sides):
    fmt = state["case"]["format"]
    got = {}
    if sides != "col":
        got["row"] = _quantized(x, fmt, seed, 0)
    if sides != "row":
        got["col"] = _quantized(x.t(), fmt, seed, 1)
    return got


def _norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    return d, mean, rstd


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype = torch.float32 if case.get("in") == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def spread(rows, cols):
        # rows and columns of unlike size, as activations and gradients have
        return normal(rows, cols) * torch.exp(0.7 * normal(rows, 1)) * torch.exp(0.5 * normal(1, cols))

    s = {"case": dict(case)}
    if own:
        import zero_optimizer_step_gb300 as dpg
        s["dpg"] = dpg
        fmt = {"nv": dpg.DPG_NVFP4, "mx": dpg.DPG_MXFP4}.get(case.get("format"))
    if case["op"] == "quantize":
        rows, cols, sides = case["rows"], case["cols"], case["sides"]
        s["x"] = (1e-3 * spread(rows, cols)).to(dtype)
        s["seed"] = torch.tensor([case["seed"]], device="cuda") if case["seed"] else None
        s["out"] = {}
        if sides != "col":
            s["out"]["row"] = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
        if sides != "row":
            s["out"]["col"] = torch.empty(cols, rows, device="cuda", dtype=torch.bfloat16)
        if own:
            s["q"] = {k: dpg.Fp4(*t.shape, fmt) for k, t in s["out"].items()}
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a, b = spread(m, k).to(dtype), (0.02 * normal(n, k)).to(dtype)
        out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["c"] = normal(m, n).to(out) if case["add"] else torch.empty(m, n, device="cuda", dtype=out)
        if own:
            s["a"], s["b"] = dpg.Fp4(m, k, fmt), dpg.Fp4(n, k, fmt)
            dpg.dpg_fp4_quantize(a, s["a"])
            dpg.dpg_fp4_quantize(b, s["b"])
        else:
            s["a"], s["b"] = _quantized(a, case["format"]), _quantized(b, case["format"])
    elif case["op"] == "linear":
        t, m, k = case["rows"], case["m"], case["k"]
        s["x"], s["dy"] = spread(t, k).to(dtype), (1e-3 * spread(t, m)).to(dtype)
        w = 0.02 * normal(m, k)                      # masters
        s["seed"] = torch.tensor([case["seed"]], device="cuda")
        s["y"] = torch.empty(t, m, device="cuda", dtype=torch.bfloat16)
        s["dx"] = torch.empty(t, k, device="cuda", dtype=torch.bfloat16)
        s["dw"] = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
        if own:
            s["w"] = {"row": dpg.Fp4(m, k, fmt), "col": dpg.Fp4(k, m, fmt)}
            dpg.dpg_fp4_quantize(w, s["w"]["row"], s["w"]["col"])
            s["xq"] = {"row": dpg.Fp4(t, k, fmt), "col": dpg.Fp4(k, t, fmt)}
            s["gq"] = {"row": dpg.Fp4(t, m, fmt), "col": dpg.Fp4(m, t, fmt)}
        else:
            s["w"] = _values(s, w, 0, "both")
    else:
        rows, cols = case["rows"], case["cols"]
        s["x"] = (normal(rows, cols) * (1 + torch.rand(rows, 1, device="cuda", generator=gen)) + normal(rows, 1)).to(dtype)
        s["gain"] = (1 + 0.1 * normal(cols)).to(dtype)
        s["bias"] = (0.1 * normal(cols)).to(dtype) if case["bias"] else None
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        s["y"] = torch.empty_like(s["x"])
        if case["op"] == "norm_back":
            _, mean, rstd = _norm(s)                 # what the forward pass kept
            s["mean"], s["rstd"] = mean[:, 0].contiguous(), rstd[:, 0].contiguous()
            s["dy"] = (1e-3 * normal(rows, cols)).to(dtype)
            s["dx"] = s.pop("y")
            s["dgain"] = torch.empty_like(s["gain"])
            s["dbias"] = torch.empty_like(s["bias"]) if case["bias"] else None
            if own:
                s["workspace"] = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), device="cuda", dtype=torch.uint8)
    return s


def _run_own(s):
    dpg, case = s["dpg"], s["case"]
    if case["op"] == "quantize":
        q = s["q"]
        dpg.dpg_fp4_quantize(s["x"], q.get("row"), q.get("col"), seed=s["seed"])
        for k, t in s["out"].items():
            dpg.dpg_fp4_dequantize(q[k], t)
        return s["out"]
    if case["op"] == "product":
        dpg.dpg_fp4_product(s["a"], s["b"], s["c"], accumulate=case["add"])
        return {"c": s["c"]}
    if case["op"] == "linear":
        x, g, w = s["xq"], s["gq"], s["w"]
        dpg.dpg_fp4_quantize(s["x"], x["row"], x["col"])
        dpg.dpg_fp4_product(x["row"], w["row"], s["y"])
        dpg.dpg_fp4_quantize(s["dy"], g["row"], g["col"], seed=s["seed"])
        dpg.dpg_fp4_product(g["row"], w["col"], s["dx"])
        dpg.dpg_fp4_product(g["col"], x["col"], s["dw"])
        return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    if case["op"] == "norm":
        dpg.dpg_layer_norm(s["x"], s["gain"], s["bias"], EPS, s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    dpg.dpg_layer_norm_backward(s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], s["dx"], s["dgain"], s["dbias"],
                                s["workspace"])
    return {"dx": s["dx"], "dgain": s["dgain"], "dbias": s["dbias"]}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "quantize":
        got = _values(s, s["x"], case["seed"], case["sides"])
        return {k: s["out"][k].copy_(t) for k, t in got.items()}
    if case["op"] == "product":
        c = s["a"] @ s["b"].t()
        return {"c": s["c"].copy_(s["c"] + c if case["add"] else c)}
    if case["op"] == "linear":
        x, w = _values(s, s["x"], 0, "both"), s["w"]
        g = _values(s, s["dy"], case["seed"], "both")
        return {"y": s["y"].copy_(x["row"] @ w["row"].t()), "dx": s["dx"].copy_(g["row"] @ w["col"].t()),
                "dw": s["dw"].copy_(g["col"] @ x["col"].t())}
    if case["op"] == "norm":
        d, mean, rstd = _norm(s)
        y = d * rstd * s["gain"].float()
        s["y"].copy_(y + s["bias"].float() if case["bias"] else y)
        s["mean"].copy_(mean[:, 0])
        s["rstd"].copy_(rstd[:, 0])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    n = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gain"].float()
    s["dx"].copy_(rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)))
    s["dgain"].copy_((dy * n).sum(0))
    if case["bias"]:
        s["dbias"].copy_(dy.sum(0))
    return {"dx": s["dx"], "dgain": s["dgain"], "dbias": s["dbias"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _random_bits(seed, side, rows, cols):
    """Philox4x32-10 (Salmon et al. 2011) on the host, in 64-bit unsigned integers."""
    per = -(-cols // 8)
    n = np.arange(rows * per, dtype=np.uint64)
    low, bits = np.uint64(0xFFFFFFFF), np.uint64(32)
    c0, c1 = n & low, n >> bits
    c2, c3 = np.full_like(n, side), np.zeros_like(n)
    k0, k1 = seed % 2 ** 32, seed // 2 ** 32
    for _ in range(10):
        p, q = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = (q >> bits) ^ c1 ^ np.uint64(k0), q & low, (p >> bits) ^ c3 ^ np.uint64(k1), p & low
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    words = np.stack([c0, c1, c2, c3], 1).astype(np.uint32)
    halves = np.stack([words & 0xFFFF, words >> 16], 2).reshape(rows, per * 8)[:, :cols]
    return torch.from_numpy(halves.astype(np.float64)).cuda()


def _exact_values(x, fmt, seed=0, side=0):
    """Every value of every scale type is listed and searched."""
    x = x.double()
    rows, cols = x.shape
    b = BLOCK[fmt]
    blocks = -(-cols // b)
    a = torch.zeros(rows, blocks * b, dtype=torch.float64, device="cuda")
    a[:, :cols] = x.abs()
    a = a.view(rows, blocks, b)
    top = a.max(2).values
    unit = 1.0
    if fmt == "nv":
        unit = 2.0 ** max(-126, math.ceil(math.log2(float(a.max()) / 2688)))
        if float(a.max()) > 2688 * unit:       # (the logarithm is rounded)
            unit *= 2
        elif unit > 2.0 ** -126 and float(a.max()) <= 1344 * unit:
            unit /= 2
        scales = [k * 2.0 ** -9 for k in range(8)] + [(8 + k) * 2.0 ** (e - 3) for e in range(-6, 9) for k in range(8)][:-1]
    else:
        scales = [2.0 ** e for e in range(-127, 128)]
    scales = torch.tensor(scales, dtype=torch.float64, device="cuda")
    s = scales[torch.searchsorted(6 * scales, (top / unit).contiguous())][..., None] * unit
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 8], dtype=torch.float64, device="cuda")
    y = a / torch.where(s > 0, s, 1.0)
    at = (torch.searchsorted(levels, y.contiguous(), right=True) - 1).clamp_max(7)
    low, high = levels[at], levels[at + 1]
    if seed:
        u = torch.zeros(rows, blocks * b, dtype=torch.float64, device="cuda")
        u[:, :cols] = _random_bits(seed, side, rows, cols)
        up = a - low * s > (high - low) * s * (u.view(a.shape) + 0.5) / 65536
    else:
        middle = (low + high) / 2
        up = (y > middle) | ((y == middle) & (at % 2 == 1))
    y = (torch.where(up, high, low) * s).view(rows, -1)[:, :cols]
    return torch.copysign(y, x)


def exact(case, seed):
    if case["op"] == "quantize":
        s = prepare(case, seed)
        got = {}
        if case["sides"] != "col":
            got["row"] = _exact_values(s["x"], case["format"], case["seed"], 0)
        if case["sides"] != "row":
            got["col"] = _exact_values(s["x"].t(), case["format"], case["seed"], 1)
        return got
    # the operands are the same values in 64 bits: the plain form's are exact
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "product":
        c = s["a"].double() @ s["b"].double().t()
        return {"c": c + s["c"] if case["add"] else c}
    if case["op"] == "linear":
        fmt, w = case["format"], {k: t.double() for k, t in s["w"].items()}
        g = _exact_values(s["dy"], fmt, case["seed"], 0), _exact_values(s["dy"].t(), fmt, case["seed"], 1)
        return {"y": _exact_values(s["x"], fmt) @ w["row"].t(), "dx": g[0] @ w["col"].t(),
                "dw": g[1] @ _exact_values(s["x"].t(), fmt).t()}
    x, gain = s["x"].double(), s["gain"].double()
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS) ** -0.5
        y = (x - mean) * rstd * gain
        return {"y": y + s["bias"].double() if case["bias"] else y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    n = (x - s["mean"].double()[:, None]) * rstd
    c = x.shape[1]
    g = dy * gain
    dx = rstd * (g - g.sum(1, keepdim=True) / c - n * ((g * n).sum(1, keepdim=True) / c))
    return {"dx": dx, "dgain": torch.einsum("rc,rc->c", dy, n), "dbias": dy.sum(0) if case["bias"] else None}
