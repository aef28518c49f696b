"""Cases of the list operators around an optimizer step: the global gradient norm, clipping by it,
and AdamW over a list of tensors.

Every list lies in flat buckets, one per type, its tensors packed one behind the other without
padding, as a flat-parameter shard or a gradient bucket holds them: after an odd-sized tensor the
next one starts at any element.  ``run`` returns the buckets.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP_EPS = 1e-6
ADAM = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
LAYER = "4096x4096*4,4096x11008*2,11008x4096"


def listed():
    return [
        # Two norm vectors of one layer: a call whose cost is its latency.
        {"name": "norm 2 vectors bf16", "op": "norm", "kind": "l2", "shapes": "4096*2", "grads": "bf16",
         "offset": 0, "size": 3.0},
        # The gradients of one 4096-hidden decoder layer.
        {"name": "norm layer bf16", "op": "norm", "kind": "l2", "shapes": LAYER, "grads": "bf16", "offset": 0,
         "size": 3.0},
        # 512 small matrices with fp32 gradients (accumulated over micro-batches).
        {"name": "norm 512 small f32", "op": "norm", "kind": "l2",
         "shapes": "256x256*128,512x2048*128,768x768*128,1024x1024*128", "grads": "f32", "offset": 0, "size": 3.0},
        # Odd sizes, single values and both types in one list, behind an odd offset: the largest magnitude.
        {"name": "norm ragged inf", "op": "norm", "kind": "inf", "shapes": "1x1,37x129*5,1000003,3*7,511x257*9",
         "grads": "mixed", "offset": 3, "size": 3.0},
        # The 65 norm vectors of a 32-layer decoder, fp32.
        {"name": "clip 65 vectors f32", "op": "clip", "kind": "l2", "shapes": "4096*65", "grads": "f32", "offset": 0,
         "size": 5.0, "max_norm": 1.0},
        # One decoder layer early in training, when the norm is over the limit.
        {"name": "clip layer bf16", "op": "clip", "kind": "l2", "shapes": LAYER, "grads": "bf16", "offset": 0,
         "size": 14.0, "max_norm": 1.0},
        # Many small matrices behind an odd offset.
        {"name": "clip 512 small bf16", "op": "clip", "kind": "l2",
         "shapes": "256x256*128,512x2048*128,768x768*128,1024x1024*128", "grads": "bf16", "offset": 1, "size": 4.0,
         "max_norm": 1.0},
        # One owner's 28 matrices of a 32-layer decoder in a settled run: the norm is below the limit.
        {"name": "clip 28 settled f32", "op": "clip", "kind": "l2",
         "shapes": "4096x4096*16,4096x11008*8,11008x4096*4", "grads": "f32", "offset": 0, "size": 0.3,
         "max_norm": 1.0},
        # The norm vectors again, updated: fp32 throughout, no decay.
        {"name": "adamw 65 vectors f32", "op": "adamw", "shapes": "4096*65", "params": "f32", "grads": "f32",
         "offset": 0, "size": 0.5, "max_norm": 0.0, "step": 1000},
        # Embedding and output head: bf16 parameters with fp32 masters, clipped by a norm in hand.
        {"name": "adamw embeddings master", "op": "adamw", "shapes": "32000x4096*2", "params": "master",
         "grads": "bf16", "offset": 0, "size": 5.0, "max_norm": 1.0, "step": 7},
        # bf16 parameters without masters, gradients accumulated in fp32.
        {"name": "adamw 16 matrices bf16", "op": "adamw", "shapes": "1024x4096*16", "params": "bf16", "grads": "f32",
         "offset": 0, "size": 5.0, "max_norm": 1.0, "step": 1},
        # Odd sizes: matrices in bf16 with masters, vectors in fp32 without decay, behind an odd offset.
        {"name": "adamw ragged mixed", "op": "adamw", "shapes": "1031x517*6,4097*13,1,77x3*4,50257x129",
         "params": "mixed", "grads": "mixed", "offset": 5, "size": 2.0, "max_norm": 1.0, "step": 250},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "clip", "adamw"])
    room = spread(1, 200_000_000 if op != "adamw" else 100_000_000)
    kinds = rng.randint(1, 8)
    shapes = []
    for _ in range(kinds):
        share = max(1, room // kinds)
        many = spread(1, min(64, share))
        each = max(1, share // many)
        if rng.random() < 0.4:
            shapes.append("%d*%d" % (each, many))
        else:
            rows = spread(1, each)
            shapes.append("%dx%d*%d" % (rows, max(1, each // rows), many))
    case = {"op": op, "shapes": ",".join(shapes), "offset": rng.choice([0, 0, 1, 2, 3, 4, 8, 13]),
            "grads": rng.choice(["bf16", "f32", "mixed"])}
    if op == "adamw":
        case["params"] = rng.choice(["f32", "bf16", "master", "mixed"])
        if case["params"] == "mixed" or case["grads"] == "mixed":
            case["params"] = case["grads"] = "mixed"
        case |= {"size": rng.uniform(0.2, 8.0), "max_norm": rng.choice([0.0, 1.0]), "step": spread(1, 100_000)}
    else:
        case |= {"kind": rng.choice(["l2", "l2", "inf"]), "size": rng.uniform(2.0, 8.0)}
        if op == "clip":
            case["max_norm"] = 1.0
            if case["kind"] == "inf":
                case["max_norm"] = 1e-4
    return case


# --- lists and buckets ---------------------------------------------------------------------------

def tensors(case):
    """(numel, is a matrix) of each tensor of the list."""
    out = []
    for part in case["shapes"].split(","):
        dims, _, many = part.partition("*")
        dims = [int(d) for d in dims.split("x")]
        out += [(math.prod(dims), len(dims) > 1)] * int(many or 1)
    return out


def groups(case):
    """The list as buckets: (params kind, grads type, decay, numels).  A mixed list holds its
    matrices in bf16 (with masters, decayed) and its vectors in fp32 (not decayed)."""
    ts = tensors(case)
    if "mixed" in (case["grads"], case.get("params")):
        both = [("master", "bf16", 1.0, [n for n, matrix in ts if matrix]),
                ("f32", "f32", 0.0, [n for n, matrix in ts if not matrix])]
        return [g for g in both if g[3]]
    return [(case.get("params"), case["grads"], 1.0, [n for n, _ in ts])]


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    gs = groups(case)
    total = sum(sum(g[3]) for g in gs)
    std = case["size"] / math.sqrt(total)

    def bucket(n, dtype):
        return torch.empty(n + case["offset"], device=DEVICE, dtype=dtype)[case["offset"]:]

    def normal(n, scale):
        return torch.randn(n, device=DEVICE, generator=gen).mul_(scale)

    state = {"case": case, "buckets": []}
    for params, grads, decay, numels in gs:
        n = sum(numels)
        b = {"numels": numels, "decay": decay, "g": bucket(n, TYPES[grads])}
        # Layers differ in the size of their gradients.
        sizes = (torch.rand(len(numels), device=DEVICE, generator=gen) + 0.5).tolist()
        values = normal(n, std)
        for part, s in zip(values.split(numels), sizes):
            part.mul_(s)
        b["g"].copy_(values)
        if case["op"] == "adamw":
            values = normal(n, 0.02)
            b["p"] = bucket(n, torch.float32 if params == "f32" else torch.bfloat16)
            b["p"].copy_(values)
            if params == "master":
                b["w"] = bucket(n, torch.float32)
                b["w"].copy_(values)
            b["m"] = bucket(n, torch.float32)
            b["m"].copy_(normal(n, 0.3 * std))
            b["v"] = bucket(n, torch.float32)
            b["v"].copy_(torch.rand(n, device=DEVICE, generator=gen).add_(0.5).mul_(std * std))
        state["buckets"].append(b)
    if case["op"] == "adamw":
        # The global norm, as the reduction over all ranks left it.
        state["norm"] = torch.full((), case["size"] * 1.01, device=DEVICE)
    if own:
        import newton_schulz_02_amd as nm

        def views(name):
            return [t for b in state["buckets"] for t in (b[name].split(b["numels"]) if name in b else
                                                          [None] * len(b["numels"]))]

        if case["op"] == "adamw":
            decays = [b["decay"] for b in state["buckets"] for _ in b["numels"]]
            state["plan"] = nm.AdamWStep(views("p"), views("g"), views("m"), views("v"), masters=views("w"),
                                         decays=decays, **ADAM)
        else:
            state["plan"] = nm.GradClip(views("g"))
    return state


# --- one pass ------------------------------------------------------------------------------------

def plain_norm(buckets, kind):
    if kind == "inf":
        return torch.stack([b["g"].float().abs().max() for b in buckets]).max()
    sums = [b["g"].float().square().sum(dtype=torch.float64) for b in buckets]
    return torch.stack(sums).sum().sqrt().float()


def plain_scale(norm, max_norm):
    return (max_norm / (norm + CLIP_EPS)).clamp(max=1.0)


def plain_adamw(b, step, scale):
    g = b["g"].float()
    if scale is not None:
        g = g * scale
    w = b["w"] if "w" in b else b["p"].float()
    b["m"].mul_(ADAM["beta1"]).add_(g, alpha=1.0 - ADAM["beta1"])
    b["v"].mul_(ADAM["beta2"]).add_(g * g, alpha=1.0 - ADAM["beta2"])
    down = (b["v"] / (1.0 - ADAM["beta2"] ** step)).sqrt_().add_(ADAM["eps"])
    update = (b["m"] / (1.0 - ADAM["beta1"] ** step)).div_(down)
    update.add_(w, alpha=ADAM["weight_decay"] * b["decay"])
    w = w.sub_(update, alpha=ADAM["lr"])
    if w is not b["p"]:
        b["p"].copy_(w)


def run(state):
    case, buckets = state["case"], state["buckets"]
    if case["op"] == "norm":
        norm = state["plan"].norm(kind=case["kind"]) if own else plain_norm(buckets, case["kind"])
        return {"norm": norm}
    if case["op"] == "clip":
        if own:
            norm = state["plan"].clip_norm(case["max_norm"], kind=case["kind"])
        else:
            norm = plain_norm(buckets, case["kind"])
            scale = plain_scale(norm, case["max_norm"])
            for b in buckets:
                b["g"].copy_(b["g"].float() * scale)
        return {"norm": norm, "grads": [b["g"] for b in buckets]}
    limit = case["max_norm"]
    if own:
        state["plan"](case["step"], clip=(state["norm"], limit) if limit else None)
    else:
        scale = plain_scale(state["norm"], limit) if limit else None
        for b in buckets:
            plain_adamw(b, case["step"], scale)
    return {name: [b[name] for b in buckets if name in b] for name in ("p", "m", "v", "w")}


def work(case):
    gs = groups(case)
    width = {"bf16": 2, "f32": 4}
    grad_bytes = sum(sum(n) * width[g] for _, g, _, n in gs)
    total = sum(sum(n) for _, _, _, n in gs)
    if case["op"] == "norm":
        return {"bytes": grad_bytes + 4, "flops": 2 * total}
    if case["op"] == "clip":
        # Clipped gradients are written once; the norm has to be known before, but what was read for it
        # counts once.
        clips = case["kind"] == "inf" or case["size"] > case["max_norm"]
        return {"bytes": grad_bytes * (2 if clips else 1) + 4, "flops": (3 if clips else 2) * total}
    param = {"bf16": 4, "f32": 8, "master": 10}  # read and written; a master's bf16 copy is only written
    return {"bytes": sum(sum(n) * (16 + param[p] + width[g]) for p, g, _, n in gs), "flops": 16 * total}


# --- the definition in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    f64 = torch.float64

    def join(parts):
        return torch.cat([p.reshape(-1) for p in parts])

    lists = [[(t, b) for t in b["g"].split(b["numels"])] for b in state["buckets"]]
    if case["op"] in ("norm", "clip"):
        if case["kind"] == "inf":
            norm = max(float(torch.linalg.vector_norm(t.to(f64), ord=math.inf)) for ts in lists for t, _ in ts)
        else:
            norm = math.sqrt(math.fsum(float(torch.dot(x, x)) for ts in lists for t, _ in ts for x in [t.to(f64)]))
        out = {"norm": torch.tensor(norm, dtype=f64)}
        if case["op"] == "clip":
            c = case["max_norm"] / (norm + CLIP_EPS)
            out["grads"] = [join([t.to(f64) * min(1.0, c) for t, _ in ts]) for ts in lists]
        return out
    c = 1.0
    if case["max_norm"]:
        c = min(1.0, case["max_norm"] / (float(state["norm"]) + CLIP_EPS))
    b1, b2, t = ADAM["beta1"], ADAM["beta2"], case["step"]
    out = {"p": [], "m": [], "v": [], "w": []}
    for b in state["buckets"]:
        g = b["g"].to(f64) * c
        first = b["m"].to(f64) * b1 + g * (1 - b1)
        second = b["v"].to(f64) * b2 + g.pow(2) * (1 - b2)
        del g
        at = b.get("w", b["p"]).to(f64)
        move = first / (1 - b1 ** t) / (torch.sqrt(second / (1 - b2 ** t)) + ADAM["eps"])
        at = at * (1 - ADAM["lr"] * ADAM["weight_decay"] * b["decay"]) - ADAM["lr"] * move
        out["p"].append(at)
        out["m"].append(first)
        out["v"].append(second)
        if "w" in b:
            out["w"].append(at)
    return out
