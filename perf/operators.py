"""Cases of the operators around the transducer loss, with their plain forms.

Three operators make a training step out of the loss: the prediction network's label
embedding and its gradient (the rows hL the joint network reads, and what dhL does to the
table), the group norm with an activation of the encoder's frames and its gradient (the rows
hA, channels last, ragged lengths), and the orthogonalised update of the weight matrices by
Newton-Schulz products (what a Muon step does with dW^A, dW^L and dW^O).

``own = False`` runs elementary torch operations in 32 bits; ``own = True`` runs the package's
entry points on the same inputs.  ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

# The quintic of the Newton-Schulz iteration as the Muon optimiser states it.
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}

# Largest listed work, in elements and in multiply-adds: drawn cases stay below.
MAX_FRAMES = 1024 * 1000 * 512
MAX_MACS = 1024 * 1024 * 16384


def listed():
    """Sizes are those of the package's synthetic workloads unless the comment says otherwise."""
    return [
        # one decoding step of 8 hypotheses: the last label of each, one row each
        dict(name="embed step 8x1", op="embed_fwd", B=8, U1=1, V=1024, D=512, dtype="bf16",
             out="bf16", sos=False, ids="uniform", ragged=False),
        # the label rows of a 40 s batch of 1024 samples
        dict(name="embed 1024x101", op="embed_fwd", B=1024, U1=101, V=4096, D=512, dtype="bf16",
             out="bf16", sos=True, ids="uniform", ragged=True),
        # a large vocabulary with Zipf labels: few tokens, long repeats, a table of 67 MB to write
        dict(name="embed grad 16x81 Zipf", op="embed_bwd", B=16, U1=81, V=16384, D=1024,
             dtype="f32", out="f32", sos=True, ids="zipf", ragged=True),
        # the 40 s batch's gradient in the bf16 hand-off of the encoder gradients
        dict(name="embed grad 1024x101", op="embed_bwd", B=1024, U1=101, V=4096, D=512,
             dtype="bf16", out="f32", sos=True, ids="uniform", ragged=True),
        # a streaming encoder: one frame of each of 8 streams
        dict(name="norm frame 8x1x512", op="norm_fwd", B=8, T=1, C=512, G=32, dtype="bf16",
             act="silu", ragged=False),
        # odd sizes (15 channels a group, 333 frames), fp32, with the gradients
        dict(name="norm grad 7x333x360", op="norm_bwd", B=7, T=333, C=360, G=24, dtype="f32",
             act="silu", ragged=True),
        # the frames of the 40 s batch, lengths 0.3 to 1 of 1000
        dict(name="norm 1024x1000x512", op="norm_fwd", B=1024, T=1000, C=512, G=32,
             dtype="bf16", act="silu", ragged=True),
        dict(name="norm grad 1024x1000x512", op="norm_bwd", B=1024, T=1000, C=512, G=32,
             dtype="bf16", act="silu", ragged=True),
        # W^A of the smallest workload, whose parameters and gradients are fp32 throughout
        dict(name="orth 64x64", op="orth", N=1, R=64, K=64, dtype="f32", out="f32", steps=5),
        # W^A and W^L of the 20 s workload, both in one call
        dict(name="orth 2x640x640", op="orth", N=2, R=640, K=640, dtype="f32", out="bf16",
             steps=5),
        # W^O of the 40 s workload, kept in fp32
        dict(name="orth 4096x512 f32", op="orth", N=1, R=4096, K=512, dtype="f32", out="f32",
             steps=5),
        # W^O of the large vocabulary
        dict(name="orth 16384x1024", op="orth", N=1, R=16384, K=1024, dtype="f32", out="bf16",
             steps=5),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "orth"])
    if op.startswith("embed"):
        sos = rng.random() < 0.7
        return dict(op=op, B=_log(rng, 1, 1024), U1=_log(rng, 1, 101), V=_log(rng, 16, 16384),
                    D=rng.choice([_log(rng, 16, 1024), 8 * _log(rng, 2, 128)]),
                    dtype=rng.choice(["f32", "bf16"]),
                    out="f32" if op == "embed_bwd" else rng.choice(["f32", "bf16"]), sos=sos,
                    ids=rng.choice(["uniform", "zipf"]), ragged=rng.random() < 0.7)
    if op.startswith("norm"):
        G = rng.choice([1, 2, 4, 8, 16, 24, 32])
        C = G * rng.choice([_log(rng, 1, 1024 // G), 16])
        T = _log(rng, 1, 4000)
        B = _log(rng, 1, max(1, min(1024, MAX_FRAMES // (2 * T * C))))
        return dict(op=op, B=B, T=T, C=C, G=G, dtype=rng.choice(["f32", "bf16"]),
                    act=rng.choice(["none", "silu", "silu", "relu"]), ragged=rng.random() < 0.7)
    while True:
        R, K = _log(rng, 16, 16384), _log(rng, 16, 2048)
        N = rng.choice([1, 1, 1, 2, 4])
        if N * R * K * min(R, K) <= MAX_MACS:
            return dict(op=op, N=N, R=R, K=K, dtype=rng.choice(["f32", "bf16"]),
                        out=rng.choice(["f32", "bf16"]), steps=5)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(n, lo, hi, g):
    """Lengths of [lo, hi], the first of them hi."""
    t = torch.randint(lo, hi + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    t[0] = hi
    return t


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = dict(case=c)
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    if c["op"].startswith("embed"):
        B, U1, V, D = c["B"], c["U1"], c["V"], c["D"]
        first = 1 if c["sos"] else 0  # labels never name the blank, index 0
        u = torch.rand(B, U1, device="cuda", generator=g)
        if c["ids"] == "zipf":  # probability of label k about 1 / k
            ids = torch.exp(u * math.log(V)).long().clamp_(first, V - 1)
        else:
            ids = first + (u * (V - first)).long().clamp_(0, V - 1 - first)
        s["ids"] = ids.to(torch.int32)
        lo = math.ceil(0.3 * (U1 - 1)) if c["ragged"] else U1 - 1
        s["U_len"] = _lengths(B, lo, U1 - 1, g)
        s["scale"] = math.sqrt(D)  # rows of variance 1 / D, scaled to variance 1
        if c["op"] == "embed_fwd":
            s["table"] = (r(V, D) / math.sqrt(D)).to(DT[c["dtype"]])
        else:
            s["dout"] = (r(B, U1, D) * 0.02).to(DT[c["dtype"]])
        return s
    if c["op"].startswith("norm"):
        B, T, C = c["B"], c["T"], c["C"]
        x = r(B, T, C)
        x.mul_(r(C).exp_()).add_(r(C))  # channels of unlike scales and offsets
        s["x"] = x.to(DT[c["dtype"]])
        del x
        s["gamma"] = 1 + 0.2 * r(C)
        s["beta"] = 0.2 * r(C)
        s["T_len"] = _lengths(B, math.ceil(0.3 * T) if c["ragged"] else T, T, g)
        if c["op"] == "norm_bwd":
            s["dy"] = (r(B, T, C) * 0.02).to(DT[c["dtype"]])
        return s
    # a weight gradient: a few strong directions, a tail, and noise
    N, R, K = c["N"], c["R"], c["K"]
    k = max(1, min(R, K) // 8)
    d = torch.arange(1, k + 1, device="cuda", dtype=torch.float32) ** -0.5
    s["G"] = (1e-3 * (torch.matmul(r(N, R, k) * d, r(N, k, K)) + 0.1 * r(N, R, K))).to(
        DT[c["dtype"]])
    return s


# ---------------------------------------------------------------- the package's entry points

def _plan(s):
    """The plan and the output buffers, as a program keeps them between calls."""
    if "plan" not in s:
        import asr_tiled_tanh_gb300 as rn
        c = s["case"]
        e = lambda shape, dt: torch.empty(shape, dtype=DT[dt], device="cuda")  # noqa: E731
        if c["op"].startswith("embed"):
            fwd = c["op"] == "embed_fwd"
            s["plan"] = rn.LabelEmbedding(c["B"], c["U1"], c["V"], c["D"], dtype=c["dtype"],
                                          out_dtype=c["out"] if fwd else c["dtype"],
                                          scale=s["scale"], sos=c["sos"])
            s["out"] = e((c["B"], c["U1"], c["D"]), c["out"]) if fwd else e((c["V"], c["D"]), "f32")
        elif c["op"].startswith("norm"):
            s["plan"] = rn.FrameNorm(c["B"], c["T"], c["C"], c["G"], act=c["act"],
                                     dtype=c["dtype"], eps=1e-5)
            s["y"] = e((c["B"], c["T"], c["C"]), c["dtype"])
            if c["op"] == "norm_bwd":
                s["dx"] = e((c["B"], c["T"], c["C"]), c["dtype"])
        else:
            s["plan"] = rn.Orthogonalizer(c["R"], c["K"], batch=c["N"], dtype=c["dtype"],
                                          out_dtype=c["out"], steps=c["steps"])
            s["out"] = e((c["N"], c["R"], c["K"]), c["out"])
    return s["plan"]


def _run_own(s):
    op = s["case"]["op"]
    plan = _plan(s)
    if op == "embed_fwd":
        return plan.fwd(s["table"], s["ids"], s["U_len"], out=s["out"])
    if op == "embed_bwd":
        return plan.bwd(s["dout"], s["ids"], s["U_len"], dtable=s["out"])
    if op == "norm_fwd":
        return plan.fwd(s["x"], s["gamma"], s["beta"], s["T_len"], y=s["y"])
    if op == "norm_bwd":  # a training step: the forward, then the backward on its statistics
        y = plan.fwd(s["x"], s["gamma"], s["beta"], s["T_len"], y=s["y"])
        dx, dgamma, dbeta = plan.bwd(s["x"], s["dy"], s["gamma"], s["beta"], s["T_len"],
                                     dx=s["dx"])
        return [y, dx, dgamma, dbeta]
    return plan.run(s["G"], out=s["out"])


# ---------------------------------------------------------------- the plain forms

def _embed_mask(s, dtype):
    """ids with the blank in front where it is prepended, and the rows that exist."""
    c, ids = s["case"], s["ids"].long()
    u = torch.arange(c["U1"], device="cuda")
    if c["sos"]:
        ids = torch.where(u == 0, 0, ids)
    return ids, (u <= s["U_len"][:, None]).to(dtype)[..., None]


def _norm_parts(s):
    """x in 32 bits split into groups, the frames that exist, and the group statistics."""
    c = s["case"]
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    x = s["x"].float().view(B, T, G, C // G)
    here = torch.arange(T, device="cuda") < s["T_len"][:, None]
    m = here.float()[:, :, None, None]
    n = (s["T_len"].float() * (C // G)).clamp(min=1)[:, None, None, None]
    mean = (x * m).sum((1, 3), keepdim=True) / n
    xc = (x - mean) * m
    rstd = ((xc * xc).sum((1, 3), keepdim=True) / n + 1e-5).rsqrt()
    return xc * rstd, rstd, m, n


def _plain_norm(s):
    c = s["case"]
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    xh, rstd, m, n = _norm_parts(s)
    gamma, beta = s["gamma"].view(1, 1, G, -1), s["beta"].view(1, 1, G, -1)
    u = xh * gamma + beta
    if c["act"] == "silu":
        sig = 1 / (1 + torch.exp(-u))
        y = u * sig
    elif c["act"] == "relu":
        y = u.clamp(min=0)
    else:
        y = u
    y = (y * m).to(s["x"].dtype).view(B, T, C)
    if c["op"] == "norm_fwd":
        return y
    g = s["dy"].float().view(B, T, G, -1) * m
    if c["act"] == "silu":
        g = g * (sig * (1 + u * (1 - sig)))
    elif c["act"] == "relu":
        g = g * (u > 0)
    del u
    dgamma, dbeta = (g * xh).sum((0, 1)).view(C), g.sum((0, 1)).view(C)
    g = g * gamma
    m1 = g.sum((1, 3), keepdim=True) / n
    m2 = (g * xh).sum((1, 3), keepdim=True) / n
    dx = ((g - m1 - xh * m2) * rstd * m).to(s["x"].dtype).view(B, T, C)
    return [y, dx, dgamma, dbeta]


def _plain_orth(s):
    c = s["case"]
    X = s["G"].float()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    wide = c["R"] <= c["K"]
    X = X if wide else X.transpose(1, 2)
    for _ in range(c["steps"]):
        A = torch.matmul(X, X.transpose(1, 2))
        X = NS_A * X + torch.matmul(NS_B * A + NS_C * torch.matmul(A, A), X)
    X = X if wide else X.transpose(1, 2)
    return X.to(DT[c["out"]]).contiguous()


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "embed_fwd":
        ids, m = _embed_mask(s, torch.float32)
        return (s["table"][ids].float() * s["scale"] * m).to(DT[c["out"]])
    if c["op"] == "embed_bwd":
        ids, m = _embed_mask(s, torch.float32)
        rows = (s["dout"].float() * m * s["scale"]).view(-1, c["D"])
        return torch.zeros(c["V"], c["D"], device="cuda").index_add_(0, ids.view(-1), rows)
    if c["op"].startswith("norm"):
        return _plain_norm(s)
    return _plain_orth(s)


# ---------------------------------------------------------------- work and exact values

def work(case):
    c = case
    if c["op"].startswith("embed"):
        rows = c["B"] * c["U1"]
        # of ragged label rows about 0.65 exist; a lookup reads each table row that is named once
        live = rows * (0.65 if c["ragged"] else 1.0)
        if c["op"] == "embed_fwd":
            return dict(bytes=min(c["V"], live) * c["D"] * SIZE[c["dtype"]]
                        + rows * c["D"] * SIZE[c["out"]] + 4 * rows, flops=live * c["D"])
        return dict(bytes=live * c["D"] * SIZE[c["dtype"]] + c["V"] * c["D"] * 4 + 4 * rows,
                    flops=live * c["D"])
    if c["op"].startswith("norm"):
        full = c["B"] * c["T"] * c["C"] * SIZE[c["dtype"]]
        live = full * (0.65 if c["ragged"] else 1.0)
        if c["op"] == "norm_fwd":
            return dict(bytes=live + full, flops=8 * live / SIZE[c["dtype"]])
        # forward: x in, y out; backward, another call: x and dy in, dx out
        return dict(bytes=3 * live + 2 * full, flops=24 * live / SIZE[c["dtype"]])
    R, K = c["R"], c["K"]
    m, n = min(R, K), max(R, K)
    # X X^T and A A are symmetric (half of each), B X is not
    return dict(bytes=c["N"] * R * K * (SIZE[c["dtype"]] + SIZE[c["out"]]),
                flops=c["N"] * c["steps"] * (m * m * n + m ** 3 + 2 * m * m * n))


def _exact_norm(c, s):
    """By the derivatives of the definition, one sample group of frames at a time."""
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    gamma, beta = s["gamma"].double(), s["beta"].double()
    out = dict(y=torch.zeros(B, T, C, dtype=torch.float64, device="cuda"))
    bwd = c["op"] == "norm_bwd"
    if bwd:
        out["dx"] = torch.zeros_like(out["y"])
        dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(beta)
    lengths = s["T_len"].tolist()
    for b in range(B):
        t = lengths[b]
        x = s["x"][b, :t].double()
        xg = x.view(t, G, C // G)
        var, mean = torch.var_mean(xg, (0, 2), correction=0, keepdim=True)
        std = (var + 1e-5).sqrt()
        z = ((xg - mean) / std).view(t, C)
        u = z * gamma + beta
        f = (u * torch.sigmoid(u) if c["act"] == "silu" else
             torch.relu(u) if c["act"] == "relu" else u)
        out["y"][b, :t] = f
        if not bwd:
            continue
        d = (torch.sigmoid(u) + f * (1 - torch.sigmoid(u)) if c["act"] == "silu" else
             (u > 0).double() if c["act"] == "relu" else torch.ones_like(u))
        d = d * s["dy"][b, :t].double()
        dgamma += (d * z).sum(0)
        dbeta += d.sum(0)
        dz = (d * gamma).view(t, G, C // G)
        zg = z.view(t, G, C // G)
        dzm = dz - dz.mean((0, 2), keepdim=True)
        out["dx"][b, :t] = ((dzm - zg * (zg * dz).mean((0, 2), keepdim=True)) / std).view(t, C)
    return [out["y"], out["dx"], dgamma, dbeta] if bwd else out["y"]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("embed"):
        ids = s["ids"].clone()
        if c["sos"]:
            ids[:, 0] = 0
        u = torch.arange(c["U1"], device="cuda")
        gone = u[None, :] > s["U_len"][:, None]
        if c["op"] == "embed_fwd":
            rows = s["table"].double().index_select(0, ids.view(-1).long()) * s["scale"]
            return rows.view(c["B"], c["U1"], c["D"]).masked_fill_(gone[..., None], 0.0)
        # the table's gradient as a product with the one-hot rows, a range of labels at a time
        rows = s["dout"].double().masked_fill(gone[..., None], 0.0).view(-1, c["D"])
        out = torch.empty(c["V"], c["D"], dtype=torch.float64, device="cuda")
        for v in range(0, c["V"], 2048):
            w = torch.arange(v, min(c["V"], v + 2048), device="cuda")
            out[v:v + 2048] = (w[:, None] == ids.view(1, -1)).double() @ rows * s["scale"]
        return out
    if c["op"].startswith("norm"):
        return _exact_norm(c, s)
    out = []
    for G in s["G"].double():
        # Q(S) = a I + S (b I + c S) on the smaller side's S, applied from that side
        X = G / (torch.linalg.matrix_norm(G) + 1e-7)
        tall = c["R"] > c["K"]
        I = torch.eye(min(c["R"], c["K"]), dtype=torch.float64, device="cuda")
        for _ in range(c["steps"]):
            S = X.T @ X if tall else X @ X.T
            Q = NS_A * I + S @ (NS_B * I + NS_C * S)
            X = X @ Q if tall else Q @ X
        out.append(X)
    return torch.stack(out)
