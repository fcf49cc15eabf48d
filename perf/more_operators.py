"""The operators inside a block of an image network, as cases to measure.

Three paths, each in a plain form (elementary torch operations in fp32, angles in fp64) and, with ``own`` set,
through ``ssim_loss_amd``'s entry points:

  rotary     queries and keys turned by their positions along several axes (time, height, width)
  attention  softmax attention with shared key heads, ragged lengths and causal order
  gated      both projections of a gated feed-forward block, the activation and the product

``train`` adds the gradients.  ``exact`` computes the same from the definitions in 64 bits, by another way than the
plain forms.
"""
import math

import torch

own = False

BASE = 10000.0  # of the rotary frequencies
GRAD = 1e-2     # standard deviation of the gradients that come in


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a network that generates its image token by token: three axes, the angles of a far frame
        {"name": "rotary-token", "path": "rotary", "train": False, "batch": 1, "tokens": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "axes": "32,48,48", "pairs": "adjacent", "half": "bfloat16", "spot": "far"},
        # inference on images of 32 x 32 patches and one more token: height and width, part of the head unturned
        {"name": "rotary-image-72", "path": "rotary", "train": False, "batch": 4, "tokens": 1025, "heads": 16,
         "kv_heads": 16, "dim": 72, "axes": "32,32", "pairs": "halves", "half": "float16", "spot": "grid"},
        # training on video of 16 frames of 32 x 32 patches, two clips at once
        {"name": "rotary-train-16384", "path": "rotary", "train": True, "batch": 2, "tokens": 16384, "heads": 16,
         "kv_heads": 16, "dim": 128, "axes": "32,48,48", "pairs": "halves", "half": "bfloat16", "spot": "grid"},
        # one more token against the keys of 8 images of different lengths, four query heads to a key head
        {"name": "attention-token", "path": "attention", "train": False, "batch": 8, "queries": 1, "keys": 8193,
         "heads": 32, "kv_heads": 8, "dim": 128, "half": "bfloat16", "causal": True, "lengths": True},
        # inference on images of 32 x 32 patches and one more token
        {"name": "attention-image-72", "path": "attention", "train": False, "batch": 4, "queries": 1025, "keys": 1025,
         "heads": 16, "kv_heads": 16, "dim": 72, "half": "float16", "causal": False, "lengths": False},
        # inference on a clip of 16 frames of 32 x 32 patches
        {"name": "attention-video-16384", "path": "attention", "train": False, "batch": 1, "queries": 16384,
         "keys": 16384, "heads": 16, "kv_heads": 16, "dim": 128, "half": "bfloat16", "causal": False, "lengths": False},
        # training a small image network in fp32: 16 x 16 patches and one more token
        {"name": "attention-train-257", "path": "attention", "train": True, "batch": 2, "queries": 257, "keys": 257,
         "heads": 6, "kv_heads": 6, "dim": 64, "half": "", "causal": False, "lengths": False},
        # training token by token order on images padded to one length, two query heads to a key head
        {"name": "attention-train-4096", "path": "attention", "train": True, "batch": 4, "queries": 4096, "keys": 4096,
         "heads": 16, "kv_heads": 8, "dim": 128, "half": "bfloat16", "causal": True, "lengths": True},
        # one token of a network that generates its image token by token
        {"name": "gated-token", "path": "gated", "train": False, "rows": 1, "width": 4096, "hidden": 10944,
         "half": "bfloat16", "act": "silu", "bias": False},
        # inference on images of 32 x 32 patches and one more token, odd widths
        {"name": "gated-image-1153", "path": "gated", "train": False, "rows": 4100, "width": 1153, "hidden": 2997,
         "half": "float16", "act": "gelu", "bias": True},
        # training a small image network in fp32
        {"name": "gated-train-384", "path": "gated", "train": True, "rows": 514, "width": 384, "hidden": 1024,
         "half": "", "act": "silu", "bias": True},
        # training a large network in bf16
        {"name": "gated-train-4096", "path": "gated", "train": True, "rows": 16384, "width": 4096, "hidden": 10944,
         "half": "bfloat16", "act": "silu", "bias": False},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _axes_of(rng, dim):
    """Even sizes that fill the head or leave a part of it."""
    count = rng.randint(1, 3)
    each = max(2, dim // count // 2 * 2)
    sizes = [each] * count
    if rng.random() < 0.5:
        sizes[0] = max(2, sizes[0] - 2 * rng.randint(0, each // 2 - 1))
    return ",".join(str(s) for s in sizes)


def draw(rng):
    path = rng.choice(["rotary", "attention", "attention", "gated"])
    half = rng.choice(["", "bfloat16", "bfloat16", "float16"])
    train = rng.random() < 0.5
    case = {"path": path, "train": train, "half": half}
    if path == "gated":
        width, hidden = _spread(rng, 24, 4096), _spread(rng, 24, 8192)
        if rng.random() < 0.6:
            width, hidden = max(8, width // 8 * 8), max(8, hidden // 8 * 8)
        most = (1 << 36 if half else 1 << 33) // (width * hidden)
        rows = _spread(rng, 1, max(1, min(16384, most)))
        return {**case, "rows": rows, "width": width, "hidden": hidden, "act": rng.choice(["silu", "gelu", "sigmoid"]),
                "bias": rng.random() < 0.5}
    dim = 8 * rng.randint(2, 16)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4])
    batch = rng.randint(1, 5)
    if path == "rotary":
        tokens = _spread(rng, 1, max(2, min(16384, 50000000 // (batch * heads * dim))))
        return {**case, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "axes": _axes_of(rng, dim), "pairs": rng.choice(["adjacent", "halves"]),
                "spot": rng.choice(["grid", "grid", "far"])}
    keys = _spread(rng, 1, 6000)
    queries = keys if rng.random() < 0.5 else 1 if rng.random() < 0.4 else _spread(rng, 1, keys)
    most = 4e9 if half else 5e8  # pairs of a query and a key over all heads
    batch = max(1, min(batch, int(most / (heads * queries * keys))))
    return {**case, "batch": batch, "queries": queries, "keys": keys, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": rng.random() < 0.5, "lengths": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------------ inputs
def _grid(batch, tokens, axes):
    """Patches in reading order of a clip that is about twice as many frames as it takes."""
    side = max(1, int(round(math.sqrt(tokens / 2 if axes > 2 else tokens))))
    t = torch.arange(tokens, device="cuda")
    found = {1: [t], 2: [t // side, t % side]}.get(axes, [t // (side * side), t // side % side, t % side])
    return torch.stack(found, 1).float().expand(batch, tokens, axes).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(seed)
    low = getattr(torch, case["half"]) if case["half"] else torch.float32

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=rng, device=dev) * std + mean).to(low)

    s = {k: case[k] for k in ("path", "train")}
    if case["path"] == "gated":
        rows, width, hidden = case["rows"], case["width"], case["hidden"]
        s.update(act=case["act"], x=normal(rows, width), w_gate=normal(hidden, width, std=width ** -0.5),
                 w_up=normal(hidden, width, std=width ** -0.5), b_gate=None, b_up=None)
        if case["bias"]:
            s.update(b_gate=normal(hidden, std=0.1), b_up=normal(hidden, std=0.1))
        names = [k for k in ("x", "w_gate", "w_up", "b_gate", "b_up") if s[k] is not None]
        if case["train"]:
            s["d_out"] = normal(rows, hidden, std=GRAD)
    elif case["path"] == "rotary":
        b, t, h, kv, d = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "dim"))
        axes = [int(a) for a in case["axes"].split(",")]
        # queries, keys and values of one projection, of which the turned parts are views
        whole = normal(b, t, h + 2 * kv, d)
        s.update(axes=axes, pairs=case["pairs"], q=whole[:, :, :h], k=whole[:, :, h:h + kv])
        s["positions"] = _grid(b, t, len(axes))
        if case["spot"] == "far":  # late in a long stream of frames, between pixels
            s["positions"] = s["positions"] + 1e5 * torch.rand(b, 1, len(axes), generator=rng, device=dev)
        names = ["q", "k"]
        if case["train"]:
            s["d_q"], s["d_k"] = normal(b, t, h, d, std=GRAD), normal(b, t, kv, d, std=GRAD)
            s["q"], s["k"] = s["q"].detach(), s["k"].detach()
    else:
        b, n, m, h, kv, d = (case[k] for k in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
        s.update(causal=case["causal"], q=normal(b, n, h, d, std=1.3), k=normal(b, m, kv, d, mean=0.1),
                 v=normal(b, m, kv, d, mean=0.2), lengths=None)
        if case["lengths"]:  # half of the padded length to all of it
            part = torch.rand(b, generator=rng, device=dev)
            s["lengths"] = (m - (part * (m // 2)).floor()).to(torch.int32)
        # as many queries as keys: they are of the same tokens, and end where these do
        s["query_lengths"] = s["lengths"] if n == m else None
        names = ["q", "k", "v"]
        if case["train"]:
            s["d_out"] = normal(b, n, h, d, std=GRAD)
    if case["train"]:
        s["leaves"] = [s[k].requires_grad_(True) for k in names]
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        return {"rotary": _rotary, "attention": _attention, "gated": _gated}[s["path"]](s)


def _run_own(s):
    import ssim_loss_amd as S

    if s["path"] == "rotary":
        outs = S.rotary(s["q"], s["k"], s["positions"], s["axes"], base=BASE, pairs=s["pairs"])
        given = (s["d_q"], s["d_k"]) if s["train"] else None
    elif s["path"] == "attention":
        # (causal: the last query sees the last key)
        outs = (S.attention(s["q"], s["k"], s["v"], causal=s["causal"], query_lengths=s["query_lengths"],
                            key_lengths=s["lengths"]),)
        given = (s["d_out"],) if s["train"] else None
    else:
        outs = (S.gated_linear(s["x"], s["w_gate"], s["w_up"], b_gate=s["b_gate"], b_up=s["b_up"], act=s["act"]),)
        given = (s["d_out"],) if s["train"] else None
    if given is None:
        return outs
    grads = torch.autograd.grad(outs, s["leaves"], given)
    return (*(o.detach() for o in outs), *grads)


def _turn(x, cos, sin, places, sign):
    first, second = places
    x = x.float()
    y = x.clone()
    y[..., first] = x[..., first] * cos - sign * x[..., second] * sin
    y[..., second] = x[..., second] * cos + sign * x[..., first] * sin
    return y


def _places(axes, pairs):
    """The two elements of each pair, axis after axis."""
    first, second, at = [], [], 0
    for size in axes:
        for i in range(size // 2):
            first.append(at + (2 * i if pairs == "adjacent" else i))
            second.append(at + (2 * i + 1 if pairs == "adjacent" else i + size // 2))
        at += size
    return torch.tensor(first, device="cuda"), torch.tensor(second, device="cuda")


def _rotary(s):
    angles = []
    for a, size in enumerate(s["axes"]):
        i = torch.arange(size // 2, device="cuda", dtype=torch.float64)
        angles.append(s["positions"][..., a:a + 1].double() * torch.exp(i * (-2.0 / size * math.log(BASE))))
    angle = torch.cat(angles, -1).unsqueeze(2)
    cos, sin = angle.cos().float(), angle.sin().float()
    places = _places(s["axes"], s["pairs"])
    low = s["q"].dtype
    out = [_turn(s[k], cos, sin, places, 1.0).to(low) for k in ("q", "k")]
    if s["train"]:
        out += [_turn(s[k], cos, sin, places, -1.0).to(low) for k in ("d_q", "d_k")]
    return tuple(out)


def _mask(s, b, n, m):
    """[n, m], true where query i of sequence b sees key j; None: everywhere."""
    if not s["causal"] and s["lengths"] is None:
        return None
    length = m if s["lengths"] is None else s["lengths"][b].long()
    last = n if s["query_lengths"] is None else s["query_lengths"][b].long()
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")
    seen = (j < length) & (i < last)
    return seen & (j <= i + (length - last)) if s["causal"] else seen


def _attention(s):
    """One sequence and key head at a time: the probabilities of all together would not fit."""
    q, k, v = s["q"], s["k"], s["v"]
    (batch, n, heads, d), m, kv = q.shape, k.shape[1], k.shape[2]
    group, scale, low = heads // kv, d ** -0.5, q.dtype
    out = torch.empty(q.shape, dtype=low, device="cuda")
    grads = [torch.empty(x.shape, dtype=low, device="cuda") for x in (q, k, v)] if s["train"] else []
    for b in range(batch):
        seen = _mask(s, b, n, m)
        for c in range(kv):
            some = slice(c * group, (c + 1) * group)
            qc = q[b, :, some].float().transpose(0, 1).contiguous()  # [group, n, d]
            kc, vc = k[b, :, c].float(), v[b, :, c].float()
            p = torch.matmul(qc, kc.t().contiguous()) * scale
            if seen is not None:
                p = torch.where(seen, p, -math.inf)
            top = p.amax(-1, keepdim=True)
            p = torch.exp(p - torch.where(top == -math.inf, 0.0, top))
            p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
            o = torch.matmul(p, vc)
            out[b, :, some] = o.transpose(0, 1).to(low)
            if not s["train"]:
                continue
            do = s["d_out"][b, :, some].float().transpose(0, 1).contiguous()
            ds = p * (torch.matmul(do, vc.t().contiguous()) - (do * o).sum(-1, keepdim=True))
            grads[0][b, :, some] = (torch.matmul(ds, kc) * scale).transpose(0, 1).to(low)
            flat = lambda x: x.reshape(group * n, -1)
            grads[1][b, :, c] = (torch.matmul(flat(ds).t().contiguous(), flat(qc)) * scale).to(low)
            grads[2][b, :, c] = torch.matmul(flat(p).t().contiguous(), flat(do)).to(low)
    return (out, *grads)


def _act(g, act):
    """act(g) and its derivative."""
    if act == "gelu":
        phi = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    a = 1 / (1 + torch.exp(-g))
    b = 1 / (1 + torch.exp(g))
    return (a, a * b) if act == "sigmoid" else (g * a, a * (1 + g * b))


def _gated(s):
    x, wg, wu, low = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["x"].dtype
    g, u = torch.matmul(x, wg.t().contiguous()), torch.matmul(x, wu.t().contiguous())
    if s["b_gate"] is not None:
        g, u = g + s["b_gate"].float(), u + s["b_up"].float()
    a, slope = _act(g, s["act"])
    out = ((a * u).to(low),)
    if not s["train"]:
        return out
    dh = s["d_out"].float()
    dg, du = dh * u * slope, dh * a
    grads = [torch.matmul(dg, wg) + torch.matmul(du, wu), torch.matmul(dg.t().contiguous(), x),
             torch.matmul(du.t().contiguous(), x)]
    if s["b_gate"] is not None:
        grads += [dg.sum(0), du.sum(0)]
    return (*out, *(t.to(low) for t in grads))


# ------------------------------------------------------------------------------------------------ what it has to do
def work(case):
    half = 2 if case["half"] else 4
    train = case["train"]
    if case["path"] == "gated":
        rows, width, hidden = case["rows"], case["width"], case["hidden"]
        weights = 2 * hidden * (width + (1 if case["bias"] else 0))
        there = rows * width + weights + rows * hidden
        # backward: the gradient of h comes in, those of x and of the weights go out
        return {"bytes": half * (2 * there if train else there),
                "flops": (12 if train else 4) * rows * width * hidden}
    heads, kv, d, b = case["heads"], case["kv_heads"], case["dim"], case["batch"]
    if case["path"] == "rotary":
        n = b * case["tokens"]
        moved = 2 * n * (heads + kv) * d * half
        places = 4 * n * len(case["axes"].split(","))
        return {"bytes": (2 if train else 1) * moved + places, "flops": (2 if train else 1) * 3 * n * (heads + kv) * d}
    n, m = case["queries"], case["keys"]
    seen = m * 0.75 if case["lengths"] else m  # the mean length
    real = seen if n == m else min(n, seen)  # rows that see a key
    pairs = real * seen - (real * (real - 1) / 2 if case["causal"] else 0)
    per = b * heads * pairs * d
    moved = b * (2 * n * heads + 2 * seen * kv) * d * half
    # backward: two products of the scores and the gradients of p, three of the gradients of q, k and v
    return {"bytes": moved * (2 if train else 1), "flops": (14 if train else 4) * per}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "attention": _exact_attention, "gated": _exact_gated}[case["path"]](s)


def _exact_rotary(s):
    def turned(x, way):
        x = x.detach().double()
        parts, at = [], 0
        for a, size in enumerate(s["axes"]):
            part = x[..., at:at + size]
            rate = torch.pow(torch.tensor(BASE, dtype=torch.float64, device="cuda"),
                             -2.0 * torch.arange(size // 2, device="cuda").double() / size)
            spin = torch.polar(torch.ones_like(rate), way * s["positions"][..., a, None].double() * rate).unsqueeze(2)
            if s["pairs"] == "adjacent":
                z = torch.view_as_complex(part.reshape(*part.shape[:-1], size // 2, 2).contiguous()) * spin
                parts.append(torch.view_as_real(z).flatten(-2))
            else:
                z = torch.complex(part[..., :size // 2], part[..., size // 2:]) * spin
                parts.append(torch.cat([z.real, z.imag], -1))
            at += size
        return torch.cat([*parts, x[..., at:]], -1)

    out = [turned(s["q"], 1.0), turned(s["k"], 1.0)]
    return tuple(out + ([turned(s["d_q"], -1.0), turned(s["d_k"], -1.0)] if s["train"] else []))


def _exact_attention(s):
    """By torch's own gradients of the definition, one query head at a time."""
    q, k, v = (s[x].detach().double() for x in ("q", "k", "v"))
    (batch, n, heads, d), m = q.shape, k.shape[1]
    group = heads // k.shape[2]
    out = torch.zeros_like(q)
    grads = [torch.zeros_like(x) for x in (q, k, v)] if s["train"] else []
    for b in range(batch):
        length = m if s["lengths"] is None else int(s["lengths"][b])
        last = n if s["query_lengths"] is None else int(s["query_lengths"][b])
        rows = slice(max(0, last - length) if s["causal"] else 0, last)  # the others see nothing
        count = rows.stop - rows.start
        if count == 0 or length == 0:
            continue
        for h in range(heads):
            c = h // group
            leaf = [x.clone().requires_grad_(s["train"]) for x in (q[b, rows, h], k[b, :length, c], v[b, :length, c])]
            score = leaf[0] @ leaf[1].t() / math.sqrt(d)
            if s["causal"]:
                score = score + torch.full_like(score, -math.inf).triu(length - count + 1)
            o = torch.softmax(score, -1) @ leaf[2]
            out[b, rows, h] = o.detach()
            if s["train"]:
                found = torch.autograd.grad(o, leaf, s["d_out"][b, rows, h].double())
                grads[0][b, rows, h] = found[0]
                grads[1][b, :length, c] += found[1]
                grads[2][b, :length, c] += found[2]
    return (out, *grads)


def _exact_gated(s):
    names = [n for n in ("x", "w_gate", "w_up", "b_gate", "b_up") if s[n] is not None]
    leaf = {n: s[n].detach().double().requires_grad_(s["train"]) for n in names}
    g, u = leaf["x"] @ leaf["w_gate"].t(), leaf["x"] @ leaf["w_up"].t()
    if "b_gate" in leaf:
        g, u = g + leaf["b_gate"], u + leaf["b_up"]
    act = {"silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid,
           "gelu": lambda t: t * torch.special.ndtr(t)}[s["act"]]
    h = act(g) * u
    if not s["train"]:
        return (h,)
    grads = torch.autograd.grad(h, [leaf[n] for n in names], s["d_out"].double())
    return (h.detach(), *grads)
