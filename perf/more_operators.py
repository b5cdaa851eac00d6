"""Cases of the operators that complete a training step, with their plain forms.

Three operators: layer norm of rows (the encoder's frames or the label embedding's rows, ragged
lengths) and its gradients, the global norm of many gradients and their clipping, and the AdamW
update of many tensors (of the weights that the orthogonalised update leaves to another method),
which takes the clipping's scale and writes the bf16 copies that the loss reads.

``own = False`` runs elementary torch operations in 32 bits (long sums in 64); ``own = True`` runs
the package's entry points on the same inputs.  ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

EPS_NORM, EPS_CLIP, EPS_ADAM = 1e-5, 1e-6, 1e-8
BETA1, BETA2, DECAY, LR = 0.9, 0.999, 0.01, 1e-3
MAX_NORM = 1.0

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}

# Largest listed work in elements of frames: drawn cases stay below.
MAX_ELEMENTS = 1024 * 1000 * 512


def listed():
    """Sizes are those of the package's synthetic workloads unless the comment says otherwise."""
    return [
        # a streaming encoder or one decoding step: one row of each of 8 streams
        dict(name="ln step 8x1x512", op="ln_fwd", B=8, T=1, C=512, dtype="bf16", out="bf16",
             labels=False, ragged=False),
        # the label rows of a 40 s batch of 1024 samples
        dict(name="ln labels 1024x101x512", op="ln_fwd", B=1024, T=101, C=512, dtype="bf16",
             out="bf16", labels=True, ragged=True),
        # the frames of the 40 s batch, lengths 0.3 to 1 of 1000
        dict(name="ln 1024x1000x512", op="ln_fwd", B=1024, T=1000, C=512, dtype="bf16",
             out="bf16", labels=False, ragged=True),
        # odd sizes (333 frames of 360 channels), fp32, with the gradients
        dict(name="ln grad 7x333x360", op="ln_bwd", B=7, T=333, C=360, dtype="f32", out="f32",
             labels=False, ragged=True),
        # the frames of the large-vocabulary workload: an fp32 residual stream, bf16 rows for the loss
        dict(name="ln grad 16x400x1024 mixed", op="ln_bwd", B=16, T=400, C=1024, dtype="f32",
             out="bf16", labels=False, ragged=True),
        # the 40 s batch's frames with the gradients
        dict(name="ln grad 1024x1000x512", op="ln_bwd", B=1024, T=1000, C=512, dtype="bf16",
             out="bf16", labels=False, ragged=True),
        # gradients of the smallest workload's eight parameters
        dict(name="clip tiny", op="clip", L=0, H=64, F=256, V=32, grad="f32"),
        # gradients of the 40 s workload's eight parameters (4.7 million)
        dict(name="clip 40s", op="clip", L=0, H=512, F=2048, V=4096, grad="f32"),
        # the large vocabulary under an encoder of 24 blocks of 1024 (336 million, 296 tensors),
        # gradients in bf16
        dict(name="clip 24x1024 bf16", op="clip", L=24, H=1024, F=4096, V=16384, grad="bf16"),
        # a whole step (norm of the gradients, then the update with its scale) of the same three kinds
        dict(name="adamw tiny", op="adamw", L=0, H=64, F=256, V=32, grad="f32"),
        # the 20 s workload under an encoder of 16 blocks of 640 (80 million)
        dict(name="adamw 16x640 bf16", op="adamw", L=16, H=640, F=2560, V=1024, grad="bf16"),
        dict(name="adamw 24x1024", op="adamw", L=24, H=1024, F=4096, V=16384, grad="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ln_bwd", "clip", "adamw"])
    if op.startswith("ln"):
        C = rng.choice([_log(rng, 16, 4096), 8 * _log(rng, 2, 512), 8 * _log(rng, 2, 512)])
        T = _log(rng, 1, 4000)
        B = _log(rng, 1, max(1, min(1024, MAX_ELEMENTS // (2 * T * C))))
        return dict(op=op, B=B, T=T, C=C, dtype=rng.choice(["f32", "bf16"]),
                    out=rng.choice(["f32", "bf16"]), labels=rng.random() < 0.4,
                    ragged=rng.random() < 0.7)
    H = rng.choice([_log(rng, 32, 1024), 8 * _log(rng, 4, 128)])
    return dict(op=op, L=rng.choice([0, rng.randint(1, 24)]), H=H, F=H * rng.choice([1, 2, 4]),
                V=_log(rng, 32, 16384), grad=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(n, lo, hi, g):
    """Lengths of [lo, hi], the first of them hi."""
    t = torch.randint(lo, hi + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    t[0] = hi
    return t


def _shapes(c):
    """W^A, W^L, b^Z, W^O, b^O, the label table, a norm, then the encoder's blocks."""
    L, H, F, V = c["L"], c["H"], c["F"], c["V"]
    block = [(H,), (H,), (H, H), (H, H), (H, H), (H, H), (H,), (H,), (F, H), (F,), (H, F), (H,)]
    return [(H, H), (H, H), (H,), (V, H), (V,), (V, H), (H,), (H,)] + block * L


def _places(shapes):
    """Where each tensor lies in one buffer, at multiples of 16 elements, and the buffer's length."""
    at, end = [], 0
    for shape in shapes:
        at.append(end)
        end += -(-math.prod(shape) // 16) * 16
    return at, end


def _views(flat, shapes, at):
    return [flat[a:a + math.prod(s)].view(s) for s, a in zip(shapes, at)]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = dict(case=c)
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    if c["op"].startswith("ln"):
        B, T, C = c["B"], c["T"], c["C"]
        x = r(B, T, C)
        x.mul_(r(C).exp_()).add_(r(C))  # channels of unlike scales and offsets
        s["x"] = x.to(DT[c["dtype"]])
        del x
        s["gamma"] = 1 + 0.2 * r(C)
        s["beta"] = 0.2 * r(C)
        # frame lengths name the frames that exist, label lengths the last label row
        top = T - 1 if c["labels"] else T
        s["len"] = _lengths(B, math.ceil(0.3 * top) if c["ragged"] else top, top, g)
        if c["op"] == "ln_bwd":
            s["dy"] = (r(B, T, C) * 0.02).to(DT[c["out"]])
        return s
    shapes = _shapes(c)
    at, n = _places(shapes)
    live = torch.zeros(n, device="cuda")  # 1 in the tensors, 0 in the gaps between them
    scale = torch.zeros(n, device="cuda")
    std = torch.rand(len(shapes), device="cuda", generator=g).mul_(4).sub_(4).exp_()
    for v, w, k in zip(_views(live, shapes, at), _views(scale, shapes, at), std):
        v.fill_(1)
        w.copy_(k.expand(v.shape))  # tensors whose gradients differ by up to e^4
    s["shapes"], s["at"] = shapes, at
    # a norm of several times the largest one, as early in training
    size = 5 * MAX_NORM / math.sqrt(n)
    s["g"] = (r(n) * scale * size).to(DT[c["grad"]])
    if c["op"] == "adamw":
        s["p"] = r(n) * live * 0.03
        s["m"] = 0.3 * r(n) * scale * size
        s["v"] = (0.1 + torch.rand(n, device="cuda", generator=g)) * (scale * size) ** 2
        s["steps"] = 1000 + seed % 1000  # updates taken before this one
        # biases, norms and tables are not decayed
        s["decay"] = [DECAY if len(k) > 1 and i != 5 else 0.0 for i, k in enumerate(shapes)]
        live.zero_()
        for v, d in zip(_views(live, shapes, at), s["decay"]):
            v.fill_(d)
        s["decay_flat"] = live
    return s


# ---------------------------------------------------------------- the package's entry points

def _plan(s):
    """The plan and the output buffers, as a program keeps them between calls."""
    if "plan" not in s:
        import asr_tiled_tanh_gb300 as rn
        c = s["case"]
        if c["op"].startswith("ln"):
            s["plan"] = rn.LayerNorm(c["B"], c["T"], c["C"], dtype=c["dtype"], out_dtype=c["out"],
                                     eps=EPS_NORM, label_rows=c["labels"])
            shape = (c["B"], c["T"], c["C"])
            s["y"] = torch.empty(shape, dtype=DT[c["out"]], device="cuda")
            if c["op"] == "ln_bwd":
                s["dx"] = torch.empty(shape, dtype=DT[c["dtype"]], device="cuda")
            return s["plan"]
        shapes, at = s["shapes"], s["at"]
        s["plan"] = rn.GradClip(shapes, max_norm=MAX_NORM, dtype=c["grad"], eps=EPS_CLIP)
        s["g list"] = _views(s["g"], shapes, at)
        if c["op"] == "clip":
            s["clipped"] = torch.zeros_like(s["g"])
            s["out list"] = _views(s["clipped"], shapes, at)
        else:
            s["adamw"] = rn.AdamW(shapes, grad_dtype=c["grad"], betas=(BETA1, BETA2), eps=EPS_ADAM,
                                  weight_decay=s["decay"], m=_views(s["m"], shapes, at),
                                  v=_views(s["v"], shapes, at), steps=s["steps"])
            s["low"] = torch.zeros_like(s["p"], dtype=torch.bfloat16)
            s["p list"] = _views(s["p"], shapes, at)
            s["low list"] = _views(s["low"], shapes, at)
    return s["plan"]


def _run_own(s):
    op = s["case"]["op"]
    plan = _plan(s)
    if op == "ln_fwd":
        return plan.fwd(s["x"], s["gamma"], s["beta"], s["len"], y=s["y"])
    if op == "ln_bwd":  # a training step: the forward, then the backward on its statistics
        y = plan.fwd(s["x"], s["gamma"], s["beta"], s["len"], y=s["y"])
        dx, dgamma, dbeta = plan.bwd(s["x"], s["dy"], s["gamma"], s["len"], dx=s["dx"])
        return [y, dx, dgamma, dbeta]
    if op == "clip":
        norm = plan.clip(s["g list"], into=s["out list"])
        return [s["clipped"], norm]
    norm = plan.norm(s["g list"])
    s["adamw"].step(s["p list"], s["g list"], LR, clip=norm, low=s["low list"])
    return [s["p"], s["m"], s["v"], s["low"], norm]


# ---------------------------------------------------------------- the plain forms

def _plain_ln(s):
    c = s["case"]
    x = s["x"].float()
    t = torch.arange(c["T"], device="cuda")
    m = (t < s["len"][:, None] + int(c["labels"])).float()[..., None]
    mean = x.sum(2, keepdim=True) / c["C"]
    xc = (x - mean) * m
    del x
    rstd = ((xc * xc).sum(2, keepdim=True) / c["C"] + EPS_NORM).rsqrt()
    xh = xc * rstd
    y = ((xh * s["gamma"] + s["beta"]) * m).to(DT[c["out"]])
    if c["op"] == "ln_fwd":
        return y
    g = s["dy"].float() * m
    dgamma = (g * xh).sum((0, 1), dtype=torch.float64).float()
    dbeta = g.sum((0, 1), dtype=torch.float64).float()
    g = g * s["gamma"]
    m1 = g.sum(2, keepdim=True) / c["C"]
    m2 = (g * xh).sum(2, keepdim=True) / c["C"]
    dx = ((g - m1 - xh * m2) * rstd * m).to(DT[c["dtype"]])
    return [y, dx, dgamma, dbeta]


def _plain_norm(g):
    """(norm, scale) of a buffer of gradients."""
    norm = (g * g).sum(dtype=torch.float64).sqrt().float()
    return torch.stack([norm, (MAX_NORM / (norm + EPS_CLIP)).clamp(max=1)])


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"].startswith("ln"):
        return _plain_ln(s)
    g = s["g"].float()
    norm = _plain_norm(g)
    if c["op"] == "clip":
        return [(g * norm[1]).to(DT[c["grad"]]), norm]
    g = g * norm[1]
    s["steps"] += 1
    p, m, v = s["p"], s["m"], s["v"]
    m.copy_(BETA1 * m + (1 - BETA1) * g)
    v.copy_(BETA2 * v + (1 - BETA2) * (g * g))
    p.copy_(p - LR * s["decay_flat"] * p - LR / (1 - BETA1 ** s["steps"]) * m
            / ((v / (1 - BETA2 ** s["steps"])).sqrt() + EPS_ADAM))
    return [p, m, v, p.bfloat16(), norm]


# ---------------------------------------------------------------- work and exact values

def work(case):
    c = case
    if c["op"].startswith("ln"):
        n = c["B"] * c["T"] * c["C"]
        live = n * (0.65 if c["ragged"] else 1.0)  # of ragged rows about 0.65 exist
        x, y = SIZE[c["dtype"]], SIZE[c["out"]]
        if c["op"] == "ln_fwd":
            return dict(bytes=live * x + n * y, flops=8 * live)
        # forward: x in, y out; backward, another call: x and dy in, dx out
        return dict(bytes=live * (2 * x + y) + n * (x + y), flops=22 * live)
    n = sum(math.prod(k) for k in _shapes(c))
    g = SIZE[c["grad"]]
    if c["op"] == "clip":
        return dict(bytes=2 * n * g, flops=3 * n)
    return dict(bytes=n * (g + 3 * 4 + 3 * 4 + 2), flops=18 * n)


def _exact_ln(c, s):
    """Row by row of one sample at a time, by the derivative of the normalised row."""
    B, T, C = c["B"], c["T"], c["C"]
    gamma, beta = s["gamma"].double(), s["beta"].double()
    y = torch.zeros(B, T, C, dtype=torch.float64, device="cuda")
    dx, dgamma, dbeta = torch.zeros_like(y), torch.zeros_like(gamma), torch.zeros_like(beta)
    for b, n in enumerate(s["len"].tolist()):
        n += int(c["labels"])
        x = s["x"][b, :n].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        std = torch.sqrt(var + EPS_NORM)
        z = (x - mean) / std
        y[b, :n] = torch.addcmul(beta, z, gamma)
        if c["op"] == "ln_fwd":
            continue
        d = s["dy"][b, :n].double()
        dgamma += torch.einsum("tc,tc->c", d, z)
        dbeta += d.sum(0)
        d = d * gamma
        d = d - d.mean(1, keepdim=True)
        dx[b, :n] = (d - z * torch.einsum("tc,tc->t", d, z)[:, None] / C) / std
    return y if c["op"] == "ln_fwd" else [y, dx, dgamma, dbeta]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("ln"):
        return _exact_ln(c, s)
    grads = [g.double() for g in _views(s["g"], s["shapes"], s["at"])]
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g) for g in grads]))
    scale = min(1.0, MAX_NORM / (float(norm) + EPS_CLIP))
    both = torch.tensor([float(norm), scale], dtype=torch.float64, device="cuda")
    if c["op"] == "clip":
        out = torch.zeros(s["g"].shape, dtype=torch.float64, device="cuda")
        for o, g in zip(_views(out, s["shapes"], s["at"]), grads):
            torch.mul(g, scale, out=o)
        return [out, both]
    t = s["steps"] + 1
    P, M, V = (s[k].double() for k in ("p", "m", "v"))
    every = (_views(f, s["shapes"], s["at"]) for f in (P, M, V))
    for p, m, v, g, decay in zip(*every, grads, s["decay"]):
        g = g * scale
        m.lerp_(g, 1 - BETA1)
        v.lerp_(g.square(), 1 - BETA2)
        mh = m / -math.expm1(t * math.log(BETA1))
        vh = v / -math.expm1(t * math.log(BETA2))
        p.mul_(1 - LR * decay).sub_(mh / (vh.sqrt() + EPS_ADAM), alpha=LR)
    return [P, M, V, P, both]
