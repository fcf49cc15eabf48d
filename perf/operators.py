"""The operators of a training step around the SSIM loss, as cases to measure.

Three paths, each in a plain form (elementary torch operations in fp32 or fp64) and, with ``own`` set, through
``ssim_loss_amd``'s entry points:

  clip   the global norm of many gradients, and the gradients scaled to at most ``max_norm``
  adamw  one AdamW update of many parameters, its gradients clipped by their global norm
  norm   the joint between two blocks of an image network: the norm after a block, its gate, the scaled residual
         sum and the norm before the next block; ``train`` adds the gradient of all of it

``exact`` computes the same from the definitions in 64 bits, by another way than the plain forms.
"""
import math

import torch

own = False

EPS_NORM = 1e-6    # under the roots of the norms
MAX_NORM = 1.0     # the clipping threshold
LR, BETA1, BETA2, EPS_ADAM, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
FIRST_STEP = 10    # updates done before the measured one


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a small splatting scene's gradients: six tensors, the whole step is a few microseconds
        {"name": "clip-scene-2k", "path": "clip", "layout": "scene", "size": 2000, "depth": 0, "half": ""},
        # an image network's gradients in bf16 with fp32 norm weights, packed end to end in buckets
        {"name": "clip-layers-520", "path": "clip", "layout": "layers", "size": 520, "depth": 16, "half": "bfloat16"},
        # a full splatting scene: three million points, 708 MB of gradients
        {"name": "clip-scene-3m", "path": "clip", "layout": "scene", "size": 3000000, "depth": 0, "half": ""},
        # the update of a small scene
        {"name": "adamw-scene-2k", "path": "adamw", "layout": "scene", "size": 2000, "depth": 0, "half": ""},
        # an image network in bf16 with fp32 master weights
        {"name": "adamw-layers-520", "path": "adamw", "layout": "layers", "size": 520, "depth": 16, "half": "bfloat16"},
        # the update of a scene of a million points
        {"name": "adamw-scene-1m", "path": "adamw", "layout": "scene", "size": 1000000, "depth": 0, "half": ""},
        # one token of a network that generates its image token by token
        {"name": "norm-token", "path": "norm", "train": False, "batch": 1, "tokens": 1, "width": 4096,
         "half": "bfloat16", "wide_residual": False, "gate": "token", "act": "none"},
        # inference on a batch of images of 32 x 32 patches and one more token, an odd width, one gate per image
        {"name": "norm-image-1153", "path": "norm", "train": False, "batch": 4, "tokens": 1025, "width": 1153,
         "half": "float16", "wide_residual": False, "gate": "sample", "act": "sigmoid"},
        # a large batch, bf16 blocks on an fp32 residual stream, a gate for each token
        {"name": "norm-batch-2048", "path": "norm", "train": False, "batch": 8, "tokens": 4096, "width": 2048,
         "half": "bfloat16", "wide_residual": True, "gate": "token", "act": "none"},
        # training a small image network in fp32: 16 x 16 patches and one more token
        {"name": "norm-train-384", "path": "norm", "train": True, "batch": 1, "tokens": 257, "width": 384,
         "half": "", "wide_residual": False, "gate": "sample", "act": "none"},
        # training in fp16 at an odd width, a sigmoid gate for each token
        {"name": "norm-train-1001", "path": "norm", "train": True, "batch": 6, "tokens": 577, "width": 1001,
         "half": "float16", "wide_residual": False, "gate": "token", "act": "sigmoid"},
        # training a large network in bf16, one gate per image
        {"name": "norm-train-4096", "path": "norm", "train": True, "batch": 4, "tokens": 4096, "width": 4096,
         "half": "bfloat16", "wide_residual": False, "gate": "sample", "act": "none"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    path = rng.choice(["clip", "adamw", "norm", "norm"])
    if path != "norm":
        half = rng.choice(["", "bfloat16", "float16"])
        if rng.random() < 0.5:
            return {"path": path, "layout": "scene", "size": _spread(rng, 1, 1000000), "depth": 0, "half": half}
        size = _spread(rng, 17, 900)
        depth = rng.randint(1, max(1, min(40, 50000000 // (12 * size * size))))
        return {"path": path, "layout": "layers", "size": size, "depth": depth, "half": half}
    train = rng.random() < 0.5
    half = rng.choice(["", "bfloat16", "bfloat16", "float16"])
    width = _spread(rng, 48, 8192)
    if rng.random() < 0.6:
        width = max(64, width // 64 * 64)
    tokens = _spread(rng, 1, 4096)
    batch = _spread(rng, 1, max(1, min(16, 30000000 // (tokens * width))))
    return {"path": path, "train": train, "batch": batch, "tokens": tokens, "width": width + (width == 3072),
            "half": half, "wide_residual": bool(half) and rng.random() < 0.4, "gate": rng.choice(["token", "sample", ""]),
            "act": rng.choice(["none", "sigmoid"])}


# ------------------------------------------------------------------------------------------------ inputs
def _shapes(case):
    """The parameters' shapes, and for each whether a half-precision run keeps it in the half type."""
    n, found = case["size"], []
    if case["layout"] == "scene":  # positions, scales, rotations, opacities, colours
        return [((n, 3), True), ((n, 3), True), ((n, 4), True), ((n, 1), True), ((n, 1, 3), True), ((n, 15, 3), True)]
    for _ in range(case["depth"]):
        found += [((3 * n, n), True), ((n, n), True), ((4 * n, n), True), ((n, 4 * n), True),
                  ((3 * n,), True), ((n,), True), ((4 * n,), True), ((n,), True), ((n,), False), ((n,), False)]
    return found


def _views(flat, shapes, places):
    return [flat[at:at + math.prod(shape)].view(shape) for shape, at in zip(shapes, places)]


def _lists(case, half):
    """{dtype: (shapes, places in the flat tensor, its length)}: scenes' tensors start at 512 bytes, as tensors of
    their own do; networks' are packed end to end, as buckets hold them."""
    found = {}
    for shape, low in _shapes(case):
        shapes, places, end = found.setdefault(half if half and low else torch.float32, ([], [], [0]))
        at = -(-end[0] // 256) * 256 if case["layout"] == "scene" else end[0]
        shapes.append(shape)
        places.append(at)
        end[0] = at + math.prod(shape)
    return {t: (shapes, places, end[0]) for t, (shapes, places, end) in found.items()}


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(seed)
    half = getattr(torch, case["half"]) if case["half"] else None

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=rng, device=dev) * std + mean).to(dtype)

    if case["path"] == "norm":
        b, t, d = case["batch"], case["tokens"], case["width"]
        low = half or torch.float32
        wide = torch.float32 if case["wide_residual"] else low
        s = {"path": "norm", "train": case["train"], "act": case["act"], "x": normal(b, t, d, std=2.0, dtype=wide),
             "branch": normal(b, t, d, std=0.7, mean=0.1, dtype=low), "scale": normal(d, std=0.02, mean=0.2),
             "post_weight": normal(d, std=0.1, mean=1.0), "pre_weight": normal(d, std=0.1, mean=1.0), "gate": None}
        if case["gate"]:
            s["gate"] = normal(b, t if case["gate"] == "token" else 1, d, dtype=low)
        if case["train"]:
            s["d_residual"] = normal(b, t, d, std=1e-2, dtype=wide)
            s["d_normed"] = normal(b, t, d, std=1e-2, dtype=low)
            s["leaves"] = [s[k] for k in ("x", "branch", "scale", "post_weight", "pre_weight")]
            s["leaves"] += [s["gate"]] if s["gate"] is not None else []
            s["leaves"] = [x.requires_grad_(True) for x in s["leaves"]]
        return s

    s = {"path": case["path"], "flat": {}, "grads": [], "params": [], "exp_avgs": [], "exp_avg_sqs": [], "masters": [],
         "out": [], "step": FIRST_STEP}
    for dtype, (shapes, places, total) in _lists(case, half).items():
        name = str(dtype).replace("torch.", "")
        std = 10.0 ** (2.0 * torch.rand((), generator=rng, device=dev) - 3.0)  # some networks' gradients are small
        flat = {"grads": normal(total, std=std, dtype=dtype)}
        if case["path"] == "clip":
            flat["out"] = torch.zeros_like(flat["grads"])
        else:
            master = normal(total, std=0.05)
            flat["params"] = master.to(dtype) if dtype != torch.float32 else master
            flat["exp_avgs"] = normal(total, std=1e-3)
            flat["exp_avg_sqs"] = torch.rand(total, generator=rng, device=dev) * 1e-5
            if half:
                flat["masters"] = master if dtype != torch.float32 else master.clone()
        for key, whole in flat.items():
            s["flat"][key + "." + name] = whole
            s[key] += _views(whole, shapes, places)
    if case["path"] == "adamw" and own:
        import ssim_loss_amd as S

        # the handle of a training program: it keeps the moments, the master weights and the count of updates
        s["optimizer"] = S.AdamW(s["params"], lr=LR, betas=(BETA1, BETA2), eps=EPS_ADAM, weight_decay=DECAY,
                                 max_norm=MAX_NORM, exp_avgs=s["exp_avgs"], exp_avg_sqs=s["exp_avg_sqs"],
                                 masters=s["masters"] or None, step=FIRST_STEP)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"clip": _clip, "adamw": _adamw, "norm": _norm}[s["path"]](s)


def _run_own(s):
    import ssim_loss_amd as S

    if s["path"] == "clip":
        norm = S.clip_grads_(s["grads"], MAX_NORM, out=s["out"])
        return {"norm": norm, **{k: v for k, v in s["flat"].items() if k.startswith("out")}}
    if s["path"] == "adamw":
        norm = s["optimizer"].step(s["grads"])
        return {"norm": norm, **{k: v for k, v in s["flat"].items() if not k.startswith("grads")}}
    args = (s["x"], s["branch"])
    kw = dict(gate=s["gate"], scale=s["scale"], post_weight=s["post_weight"], pre_weight=s["pre_weight"], eps=EPS_NORM,
              gate_act=s["act"])
    if not s["train"]:
        return S.block_norm(*args, **kw)
    residual, normed = S.block_norm(*args, **kw)
    grads = torch.autograd.grad((residual, normed), s["leaves"], (s["d_residual"], s["d_normed"]))
    return (residual.detach(), normed.detach(), *grads)


def _coefficient(grads):
    norm = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    return norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()


def _clip(s):
    norm, c = _coefficient(s["grads"])
    [o.copy_(g.float() * c) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm.float(), **{k: v for k, v in s["flat"].items() if k.startswith("out")}}


def _adamw_one(p, w, g, m, v, c, t):
    g = g.float() * c
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * g * (1 - BETA2))
    step = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS_ADAM)
    w.copy_(w * (1 - LR * DECAY) - LR * step)
    return w if w is p else p.copy_(w)


def _adamw(s):
    norm, c = _coefficient(s["grads"])
    s["step"] += 1
    [_adamw_one(p, w, g, m, v, c, s["step"])
     for p, w, g, m, v in zip(s["params"], s["masters"] or s["params"], s["grads"], s["exp_avgs"], s["exp_avg_sqs"])]
    return {"norm": norm.float(), **{k: v for k, v in s["flat"].items() if not k.startswith("grads")}}


def _norm(s):
    with torch.no_grad():
        x, b = s["x"].float(), s["branch"].float()
        inv_b = (b.square().mean(-1, keepdim=True) + EPS_NORM).rsqrt()
        bh = b * inv_b
        c = s["scale"] * s["post_weight"]
        g = None if s["gate"] is None else s["gate"].float()
        a = 1.0 if g is None else torch.sigmoid(g) if s["act"] == "sigmoid" else g
        r = x + a * c * bh
        inv_r = (r.square().mean(-1, keepdim=True) + EPS_NORM).rsqrt()
        rh = r * inv_r
        out = (r.to(s["x"].dtype), (rh * s["pre_weight"]).to(s["branch"].dtype))
        if not s["train"]:
            return out
        dh = s["d_normed"].float()
        wd = dh * s["pre_weight"]
        e = s["d_residual"].float() + inv_r * (wd - rh * (wd * rh).mean(-1, keepdim=True))
        t = e * a * c
        db = inv_b * (t - bh * (t * bh).mean(-1, keepdim=True))
        rows = (0, 1)
        total = (e * a * bh).double().sum(rows)
        grads = [e.to(s["x"].dtype), db.to(s["branch"].dtype), (total * s["post_weight"]).float(),
                 (total * s["scale"]).float(), (dh * rh).double().sum(rows).float()]
        if g is not None:
            dg = e * c * bh
            dg = dg * a * (1 - a) if s["act"] == "sigmoid" else dg
            dg = dg.double().sum(1, keepdim=True) if g.shape[1] != x.shape[1] else dg
            grads.append(dg.to(s["gate"].dtype))
        return (*out, *grads)


# ------------------------------------------------------------------------------------------------ what it has to move
def work(case):
    half = 2 if case["half"] else 4
    if case["path"] == "norm":
        rows, d = case["batch"] * case["tokens"], case["width"]
        n = rows * d
        wide = 4 if case["wide_residual"] else half
        gate = {"token": n, "sample": case["batch"] * d, "": 0}[case["gate"]] * half
        there = (2 * wide + 2 * half) * n + gate + 3 * 4 * d  # x, residual, branch, normed; the gate; three weights
        if not case["train"]:
            return {"bytes": there, "flops": 12 * n}
        # two gradients come in; those of x, the branch, the gate and the weights go out
        return {"bytes": there + 2 * (wide + half) * n + gate + 3 * 4 * d, "flops": 40 * n}
    low = sum(math.prod(shape) for shape, is_low in _shapes(case) if is_low and case["half"])
    rest = sum(math.prod(shape) for shape, is_low in _shapes(case)) - low
    n = low + rest
    if case["path"] == "clip":
        return {"bytes": 2 * (2 * low + 4 * rest) + 4, "flops": 3 * n}
    # gradient in, moments and weights in and out; in a half run the weights are the masters and the parameters go out
    state = 16 * n + (2 * low + 4 * rest)
    weights = 8 * n + (2 * low + 4 * rest if case["half"] else 0)
    return {"bytes": state + weights + 4, "flops": 20 * n}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["path"] == "norm":
        return _exact_norm(s)
    whole = {k: v.double() for k, v in s["flat"].items()}
    kinds = [k.split(".", 1)[1] for k in whole if k.startswith("grads")]
    # (the places between tensors hold gradients that belong to no tensor: they are left out)
    inside = {}
    half = getattr(torch, case["half"]) if case["half"] else None
    for dtype, (shapes, places, total) in _lists(case, half).items():
        marks = torch.zeros(total, dtype=torch.bool, device="cuda")
        for shape, at in zip(shapes, places):
            marks[at:at + math.prod(shape)] = True
        inside[str(dtype).replace("torch.", "")] = marks
    grads = {k: torch.where(inside[k], whole["grads." + k], 0.0) for k in kinds}
    norm = math.sqrt(sum(float(torch.dot(g, g)) for g in grads.values()))
    c = min(1.0, MAX_NORM / (norm + 1e-6))
    found = {"norm": norm}
    for k in kinds:
        if case["path"] == "clip":
            found["out." + k] = grads[k] * c
            continue
        m = torch.lerp(whole["exp_avgs." + k], grads[k] * c, 1 - BETA1)
        v = torch.lerp(whole["exp_avg_sqs." + k], (grads[k] * c) ** 2, 1 - BETA2)
        w = whole["masters." + k] if s["masters"] else whole["params." + k]
        t = FIRST_STEP + 1
        m_hat, v_hat = m / -math.expm1(t * math.log(BETA1)), v / -math.expm1(t * math.log(BETA2))
        w_new = w - LR * (DECAY * w + m_hat / (torch.sqrt(v_hat) + EPS_ADAM))
        now = {"exp_avgs": m, "exp_avg_sqs": v, "params": w_new}
        if s["masters"]:
            now["masters"] = w_new
        for name, value in now.items():
            found[name + "." + k] = torch.where(inside[k], value, whole[name + "." + k])
    return found


def _exact_norm(s):
    names = [n for n in ("x", "branch", "scale", "post_weight", "pre_weight", "gate") if s[n] is not None]
    leaf = {n: s[n].detach().double().requires_grad_(s["train"]) for n in names}

    def rms(v):
        return v / torch.sqrt(torch.sum(v * v, -1, keepdim=True) / v.shape[-1] + EPS_NORM)

    update = rms(leaf["branch"]) * leaf["post_weight"] * leaf["scale"]
    if "gate" in leaf:
        update = update * (1 / (1 + torch.exp(-leaf["gate"])) if s["act"] == "sigmoid" else leaf["gate"])
    residual = leaf["x"] + update
    normed = rms(residual) * leaf["pre_weight"]
    if not s["train"]:
        return residual, normed
    grads = torch.autograd.grad((residual, normed), [leaf[n] for n in names],
                                (s["d_residual"].double(), s["d_normed"].double()))
    return (residual.detach(), normed.detach(), *grads)
