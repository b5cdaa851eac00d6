"""One training step of a small transducer with the library's operators.

    frames [B,T,C] --FrameNorm--> hA --+
                                       +--> joint network, output layer, loss (Rnnt) and gradients
    labels [B,U+1] --LabelEmbedding, LayerNorm--> hL --+

    dhA --FrameNorm.bwd--> d frames, d gamma, d beta
    dhL --LayerNorm.bwd, LabelEmbedding.bwd--> d scale, d shift, d table
    all gradients --GradClip--> their norm and the scale that limits it
    dW^A, dW^L --Orthogonalizer--> weight updates (momentum, then Newton-Schulz products)
    the others --AdamW--> weights and their bf16 copies

The hidden matrices take the orthogonalised update, the output layer, the label table, biases
and norms AdamW; a step whose gradients are not finite changes none of them.  The encoder that
would make the frames and take their gradient is left out: the frames are a fixed synthetic batch
whose features carry the labels, so the loss falls as the step repeats.
Run:  python examples/training_step.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import asr_tiled_tanh_gb300 as rn  # noqa: E402


class Transducer:
    """fp32 master weights, bf16 activations; plans and buffers are made once."""

    def __init__(self, B, T, U1, C, H, V, groups=32, lr=0.02, momentum=0.9, max_norm=5.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std: std * torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        one, zero = (lambda n: torch.ones(n, device="cuda")), (lambda n: torch.zeros(n, device="cuda"))
        self.lr, self.mu = lr, momentum
        self.matrices = {"WA": r(H, C, std=C ** -0.5), "WL": r(H, H, std=H ** -0.5)}
        self.others = {"WO": r(V, H, std=H ** -0.5), "table": r(V, H, std=H ** -0.5),
                       "bZ": zero(H), "bO": zero(V), "gamma": one(C), "beta": zero(C),
                       "scale": one(H), "shift": zero(H)}
        self.velocity = {k: torch.zeros_like(v) for k, v in self.matrices.items()}
        # what the loss reads: AdamW keeps the copies of its own weights
        self.low = {k: v.bfloat16() for k, v in {**self.matrices, **self.others}.items()
                    if k in ("WA", "WL", "WO", "bZ", "bO")}
        self.norm = rn.FrameNorm(B, T, C, groups, act="silu", dtype="bf16")
        self.embed = rn.LabelEmbedding(B, U1, V, H, dtype="f32", out_dtype="bf16",
                                       scale=math.sqrt(H))
        self.rows = rn.LayerNorm(B, U1, H, dtype="bf16", label_rows=True)
        self.rnnt = rn.Rnnt(B, T, U1, C, H, H, V, dtype="bf16")
        self.orth = {k: rn.Orthogonalizer(*w.shape, out_dtype="f32")
                     for k, w in self.matrices.items()}
        weights = [*self.matrices.values(), *self.others.values()]
        self.clip = rn.GradClip([w.shape for w in weights], max_norm=max_norm)
        self.adamw = rn.AdamW([w.shape for w in self.others.values()],
                              weight_decay=[0.01 if k == "WO" else 0.0 for k in self.others])

    def step(self, frames, labels, T_len, U_len):
        """One update; returns (loss per sample, d frames)."""
        m, v = self.matrices, self.others
        hA = self.norm.fwd(frames, v["gamma"], v["beta"], T_len)
        e = self.embed.fwd(v["table"], labels, U_len)
        hL = self.rows.fwd(e, v["scale"], v["shift"], U_len)
        params = rn.make_params(*(self.low[k] for k in ("WA", "WL", "bZ", "WO", "bO")))
        args = (hA, hL, params, labels, T_len, U_len)
        count = frames.shape[0]
        loss = self.rnnt.fwd(*args)
        d = self.rnnt.bwd_ex(*args, grad_loss=torch.full_like(loss, 1 / count), enc_dtype="bf16")
        dframes, dgamma, dbeta = self.norm.bwd(frames, d["dhA"], v["gamma"], v["beta"], T_len)
        de, dscale, dshift = self.rows.bwd(e, d["dhL"], v["scale"], U_len)
        grads = {"WA": d["dWA"], "WL": d["dWL"], "WO": d["dWO"],
                 "table": self.embed.bwd(de, labels, U_len), "bZ": d["dbZ"], "bO": d["dbO"],
                 "gamma": dgamma, "beta": dbeta, "scale": dscale, "shift": dshift}
        clip = self.clip.norm([grads[k] for k in (*m, *v)])
        # (AdamW leaves an update out whose norm is not finite; so do these: a product with 0
        # would keep a NaN)
        ok = torch.isfinite(clip[0])
        for k, w in m.items():  # an update of singular values near 1, whatever the gradient's
            old = self.velocity[k]
            vel = torch.where(ok, self.mu * old + grads[k] * clip[1], old)
            rate = self.lr * math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
            w.copy_(torch.where(ok, w - rate * self.orth[k].run(vel), w))
            old.copy_(vel)
            self.low[k].copy_(w)
        self.adamw.step(list(v.values()), [grads[k] for k in v], 0.5 * self.lr, clip=clip,
                        low=[self.low.get(k) for k in v])
        return loss, dframes * count

    def status(self):
        """0 when no call found a problem on the device."""
        ops = [self.norm, self.embed, self.rows, *self.orth.values()]
        return max([self.rnnt.status()[0], *(o.status()[0] for o in ops)])


def batch(B, T, U1, C, V, seed=0):
    """Frames whose features name the label that is spoken in them, and the labels."""
    g = torch.Generator().manual_seed(seed)
    labels = torch.randint(1, V, (B, U1), generator=g, dtype=torch.int32)
    labels[:, 0] = 0
    T_len = torch.randint(T // 2, T + 1, (B,), generator=g, dtype=torch.int32)
    U_len = torch.randint((U1 - 1) // 2, U1, (B,), generator=g, dtype=torch.int32)
    T_len[0], U_len[0] = T, U1 - 1
    code = torch.randn(V, C, generator=g)
    t = torch.arange(T)[None]
    spoken = (t * U_len[:, None] // T_len[:, None]).clamp(max=U1 - 2) + 1
    frames = code[labels.long().gather(1, spoken.long())] + 0.5 * torch.randn(B, T, C, generator=g)
    return [x.cuda() for x in (frames.bfloat16(), labels, T_len, U_len)]


def main(steps=30, B=8, T=60, U1=9, C=256, H=256, V=128):
    rn.load(build_if_missing=True)
    model = Transducer(B, T, U1, C, H, V)
    data = batch(B, T, U1, C, V)
    losses = []
    for i in range(steps):
        loss, _ = model.step(*data)
        losses.append(loss.mean().item())
        if i % 5 == 0 or i + 1 == steps:
            print(f"step {i:3d}  loss per sample {losses[-1]:.3f}")
    if model.status() != 0:
        raise RuntimeError("a kernel reported a problem")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
