"""What is measured of the matrix-orthogonalising optimizer (Muon) operators.

Three operators over the flat buffers of a bucket plan:

  momentum   the R replica gradients summed in rank order, scaled by 1/G (G the
             global valid-token count), folded into the momentum, and the
             (Nesterov) update written out
  ortho      the update of every matrix orthogonalised by Newton-Schulz steps
             X <- aX + (bA + cA^2)X, A = XX^T, from X = U / max(|U|_F, eps)
  apply      decoupled weight decay and the orthogonalised update applied to
             the fp32 master weights, and the bf16 parameter views written

A case names its matrices as "ROWSxCOLSxCOUNT" groups; a group is one stacked
parameter (the same weight of COUNT layers, or a fused projection's parts).
With `own` the calls go to the library; without it the same results come from
elementary torch operations in fp32.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
MOMENTUM = 0.95
LR = 0.02
WEIGHT_DECAY = 0.1


def listed():
    return [
        # the step's smallest call: three small weights, four replicas
        {"name": "momentum_tiny", "op": "momentum", "mats": "64x32x1,32x10x1", "R": 4,
         "grads": "bf16", "out": "bf16", "nesterov": True},
        # attention weights of a GPT-2-small-shaped model, eight replicas
        {"name": "momentum_gpt2_attn", "op": "momentum", "mats": "768x2304x12,768x768x12", "R": 8,
         "grads": "bf16", "out": "bf16", "nesterov": True},
        # two layers of a 1B Llama-shaped model, eight replicas, fp32 update
        {"name": "momentum_llama1b", "op": "momentum", "mats": "2048x2048x8,8192x2048x4,2048x8192x2",
         "R": 8, "grads": "bf16", "out": "f32", "nesterov": True},
        # fp32 accumulation buffers of four replicas, plain momentum
        {"name": "momentum_acc_f32", "op": "momentum", "mats": "4096x4096x2,1024x4096x2", "R": 4,
         "grads": "f32", "out": "bf16", "nesterov": False},
        # latency: two matrices far below a tile
        {"name": "ortho_tiny", "op": "ortho", "mats": "64x32x1,32x10x1", "in": "bf16"},
        # odd sizes, a single row, tall and wide
        {"name": "ortho_ragged", "op": "ortho", "mats": "1000x333x1,517x1031x2,1x777x1,641x129x1",
         "in": "f32"},
        # attention weights of a few GPT-2-small-shaped layers
        {"name": "ortho_gpt2_attn", "op": "ortho", "mats": "768x2304x4,768x768x4", "in": "bf16"},
        # one layer of a 1B Llama-shaped model
        {"name": "ortho_llama1b", "op": "ortho", "mats": "2048x2048x4,8192x2048x2,2048x8192x1",
         "in": "bf16"},
        # one layer of an 8B Llama-3-shaped model
        {"name": "ortho_llama8b", "op": "ortho",
         "mats": "4096x4096x2,1024x4096x2,14336x4096x2,4096x14336x1", "in": "bf16"},
        # a small model's weights, every replica's own view written
        {"name": "apply_gpt2_attn", "op": "apply", "mats": "768x2304x12,768x768x12", "views": 4,
         "rule": "rms"},
        # two layers of a 1B Llama-shaped model, one shared view
        {"name": "apply_llama1b", "op": "apply", "mats": "2048x2048x8,8192x2048x4,2048x8192x2",
         "views": 1, "rule": "spectral"},
    ]


def _dim(rng, hi):
    n = int(round(math.exp(rng.uniform(0.0, math.log(hi)))))
    if n > 64 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(1, n)


def draw(rng):
    op = rng.choice(["momentum", "ortho", "ortho", "apply"])
    hi = 6000 if op == "ortho" else 8192
    budget = 3e12 if op == "ortho" else 60e6   # of flops, or of elements
    groups, spent = [], 0.0
    for _ in range(rng.randint(1, 5)):
        r, c, k = _dim(rng, hi), _dim(rng, hi), rng.choice([1, 1, 2, 3])
        cost = _ortho_flops(r, c) * k if op == "ortho" else float(r * c * k)
        if not groups or spent + cost <= budget:
            groups.append((r, c, k))
            spent += cost
    case = {"op": op, "mats": ",".join("%dx%dx%d" % g for g in groups)}
    if op == "momentum":
        case.update(R=rng.choice([1, 2, 3, 4, 5, 8]), grads=rng.choice(["bf16", "bf16", "f32"]),
                    out=rng.choice(["bf16", "f32"]), nesterov=rng.random() < 0.7)
    elif op == "ortho":
        case["in"] = rng.choice(["bf16", "f32"])
    else:
        case.update(views=rng.choice([1, 1, 2, 8]), rule=rng.choice(["rms", "spectral"]))
    return case


def _groups(case):
    return [tuple(int(x) for x in g.split("x")) for g in case["mats"].split(",")]


def _layout(groups, R):
    """Offsets of the stacked parameters in one bucket: last parameter first,
    slices on multiples of 8, the bucket padded to a multiple of 8 R."""
    offset, fill = [0] * len(groups), 0
    for k in reversed(range(len(groups))):
        r, c, n = groups[k]
        offset[k] = (fill + 7) // 8 * 8
        fill = offset[k] + r * c * n
    return offset, (fill + 8 * R - 1) // (8 * R) * (8 * R)


def _ortho_flops(r, c):
    m, n = float(min(r, c)), float(max(r, c))
    return STEPS * (3.0 * m * m * n + m * m * m)


def work(case):
    groups = _groups(case)
    n = float(sum(r * c * k for r, c, k in groups))
    if case["op"] == "momentum":
        g, u = (2 if case["grads"] == "bf16" else 4), (2 if case["out"] == "bf16" else 4)
        return {"bytes": n * (g * case["R"] + 8 + u), "flops": n * (case["R"] + 6)}
    if case["op"] == "apply":
        return {"bytes": n * (2 + 8 + 2 * case["views"]), "flops": n * 4}
    # A and A^2 are symmetric: half of their products
    return {"bytes": n * ((2 if case["in"] == "bf16" else 4) + 2),
            "flops": sum(_ortho_flops(r, c) * k for r, c, k in groups)}


def _flat(groups, offset, total, make):
    """A flat fp32 buffer: make(rows, cols, count) in every slice, zero elsewhere."""
    t = torch.zeros(total, device="cuda")
    for (r, c, k), o in zip(groups, offset):
        t[o:o + r * c * k] = make(r, c, k).reshape(-1)
    return t


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    groups, R = _groups(case), int(case.get("R", 1))
    offset, total = _layout(groups, R)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def gradient(r, c, k):
        # noise and a few strong directions, as a layer's gradient has
        low = normal(k, r, 4) @ normal(k, 4, c)
        return 1e-3 * (normal(k, r, c) + 0.5 * low)

    state = {"case": dict(case), "groups": groups, "offset": offset, "total": total}
    if case["op"] == "momentum":
        dtype = torch.bfloat16 if case["grads"] == "bf16" else torch.float32
        state["tokens"] = torch.randint(3000, 4097, (R,), generator=torch.Generator().manual_seed(int(seed))).tolist()
        state["grads"] = [_flat(groups, offset, total, lambda r, c, k: 1e-3 * normal(k, r, c)).to(dtype)
                          for _ in range(R)]
        scale = 1.0 / sum(state["tokens"])
        state["momentum"] = _flat(groups, offset, total, lambda r, c, k: (1e-3 * scale) * normal(k, r, c))
        state["update"] = torch.zeros(total, device="cuda",
                                      dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    elif case["op"] == "ortho":
        u = _flat(groups, offset, total, gradient)
        state["update"] = u.to(torch.bfloat16) if case["in"] == "bf16" else u
        state["out"] = torch.zeros(total, device="cuda", dtype=torch.bfloat16)
    else:
        state["ortho"] = _flat(groups, offset, total,
                               lambda r, c, k: normal(k, r, c) / math.sqrt(max(r, c))).to(torch.bfloat16)
        state["master"] = _flat(groups, offset, total, lambda r, c, k: 0.02 * normal(k, r, c))
        state["views"] = [torch.zeros(total, device="cuda", dtype=torch.bfloat16)
                          for _ in range(case["views"])]
    if own:
        # the handles that a training loop makes once and keeps
        import zero_optimizer_step_gb300 as dpg
        plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in groups], 1 << 50, R)
        assert plan.total_padded == total and plan.param_offset.tolist() == offset
        state["dpg"], state["plan"] = dpg, plan
        state["hp"] = dpg.MuonHParams(
            lr=LR, momentum=MOMENTUM, weight_decay=WEIGHT_DECAY, eps=EPS,
            nesterov=bool(case.get("nesterov", True)), coeffs=[COEFFS] * STEPS,
            scale_rule=dpg.DPG_SCALE_RMS if case.get("rule") == "rms" else dpg.DPG_SCALE_SPECTRAL)
        state["matrices"] = dpg.dpg_plan_matrices(plan, [g[0] for g in groups], [g[1] for g in groups])
    return state


def _run_own(s):
    dpg, case = s["dpg"], s["case"]
    if case["op"] == "momentum":
        dpg.dpg_muon_momentum(s["plan"], s["grads"], s["tokens"], s["hp"], s["momentum"], s["update"])
        return {"momentum": s["momentum"], "update": s["update"]}
    if case["op"] == "ortho":
        dpg.dpg_orthogonalize(s["matrices"], s["update"], s["hp"], s["out"])
        return {"out": s["out"]}
    dpg.dpg_muon_apply(s["matrices"], s["ortho"], s["hp"], s["master"], s["views"])
    return {"master": s["master"], "views": s["views"]}


def _newton_schulz(u):
    """[count, rows, cols] in fp32; the Gram matrix is taken on the shorter side."""
    x = u.float()
    x = x / x.square().sum((1, 2), keepdim=True).sqrt().clamp_min(EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    a, b, c = COEFFS
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


def _scale(case, r, c):
    return 0.2 * math.sqrt(max(r, c)) if case["rule"] == "rms" else math.sqrt(max(1.0, r / c))


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "momentum":
        g = sum(x.float() for x in s["grads"]) * (1.0 / sum(s["tokens"]))
        m = s["momentum"].mul_(MOMENTUM).add_(g, alpha=1.0 - MOMENTUM)
        u = g * (1.0 - MOMENTUM) + m * MOMENTUM if case["nesterov"] else m
        s["update"].copy_(u)
        return {"momentum": m, "update": s["update"]}
    for (r, c, k), o in zip(s["groups"], s["offset"]):
        piece = slice(o, o + r * c * k)
        if case["op"] == "ortho":
            s["out"][piece] = _newton_schulz(s["update"][piece].view(k, r, c)).reshape(-1)
        else:
            w = s["master"][piece]
            w.mul_(1.0 - LR * WEIGHT_DECAY).sub_(s["ortho"][piece].float() * (LR * _scale(case, r, c)))
    if case["op"] == "ortho":
        return {"out": s["out"]}
    for v in s["views"]:
        v.copy_(s["master"])
    return {"master": s["master"], "views": s["views"]}


def exact(case, seed):
    if case["op"] == "ortho" and sum(min(r, c) ** 3 * k for r, c, k in _groups(case)) > 1e11:
        return None
    s = prepare(case, seed)
    if case["op"] == "momentum":
        total = torch.zeros(s["total"], dtype=torch.float64, device="cuda")
        for x in s["grads"]:
            total += x
        total /= sum(s["tokens"])
        m = MOMENTUM * s["momentum"].double() + (1.0 - MOMENTUM) * total
        return {"momentum": m, "update": (1.0 - MOMENTUM) * total + MOMENTUM * m if case["nesterov"] else m}
    if case["op"] == "apply":
        w = s["master"].double()
        for (r, c, k), o in zip(s["groups"], s["offset"]):
            e = o + r * c * k
            w[o:e] -= LR * WEIGHT_DECAY * w[o:e] + LR * _scale(case, r, c) * s["ortho"][o:e].double()
        return {"master": w, "views": [w] * case["views"]}
    out = torch.zeros(s["total"], dtype=torch.float64, device="cuda")
    for (r, c, k), o in zip(s["groups"], s["offset"]):
        for i in range(k):
            at = slice(o + i * r * c, o + (i + 1) * r * c)
            u = s["update"][at].double().view(r, c)
            u = u / max(float(u.norm()), EPS)
            u = u if r <= c else u.T
            # every step multiplies each singular direction by a + b l + c l^2,
            # l the square of its singular value
            l, v = torch.linalg.eigh(u @ u.T)
            f = torch.ones_like(l)
            for _ in range(STEPS):
                h = COEFFS[0] + COEFFS[1] * l + COEFFS[2] * l * l
                f, l = f * h, l * h * h
            y = (v * f) @ (v.T @ u)
            out[at] = (y if r <= c else y.T).reshape(-1)
    return {"out": out}
