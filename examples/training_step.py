"""One training step of a small transducer with the library's operators.

    frames [B,T,C] --FrameNorm--> hA --+
                                       +--> joint network, output layer, loss (Rnnt) and gradients
    labels [B,U+1] --LabelEmbedding--> hL --+

    dhA --FrameNorm.bwd--> d frames, d gamma, d beta     dhL --LabelEmbedding.bwd--> d table
    dW^A, dW^L, dW^O --Orthogonalizer--> weight updates (momentum, then Newton-Schulz products)

Every matrix takes the orthogonalised update here, the output layer's as well (Muon as published
leaves that one to another method).  The encoder that would make the frames and take their
gradient is left out: the frames are a fixed synthetic batch whose features carry the labels, so
the loss falls as the step repeats.
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

    def __init__(self, B, T, U1, C, H, V, groups=32, lr=0.02, momentum=0.9, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std: std * torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.lr, self.mu = lr, momentum
        self.matrices = {"WA": r(H, C, std=C ** -0.5), "WL": r(H, H, std=H ** -0.5),
                         "WO": r(V, H, std=H ** -0.5)}
        self.vectors = {"bZ": torch.zeros(H, device="cuda"), "bO": torch.zeros(V, device="cuda"),
                        "gamma": torch.ones(C, device="cuda"), "beta": torch.zeros(C, device="cuda"),
                        "table": r(V, H, std=H ** -0.5)}
        self.velocity = {k: torch.zeros_like(v) for k, v in {**self.matrices, **self.vectors}.items()}
        self.norm = rn.FrameNorm(B, T, C, groups, act="silu", dtype="bf16")
        self.embed = rn.LabelEmbedding(B, U1, V, H, dtype="f32", out_dtype="bf16",
                                       scale=math.sqrt(H))
        self.rnnt = rn.Rnnt(B, T, U1, C, H, H, V, dtype="bf16")
        self.orth = {k: rn.Orthogonalizer(*w.shape, out_dtype="f32")
                     for k, w in self.matrices.items()}

    def step(self, frames, labels, T_len, U_len):
        """One update; returns (loss per sample, d frames)."""
        m, v = self.matrices, self.vectors
        hA = self.norm.fwd(frames, v["gamma"], v["beta"], T_len)
        hL = self.embed.fwd(v["table"], labels, U_len)
        low = {k: p.bfloat16() for k, p in {**m, "bZ": v["bZ"], "bO": v["bO"]}.items()}
        params = rn.make_params(low["WA"], low["WL"], low["bZ"], low["WO"], low["bO"])
        args = (hA, hL, params, labels, T_len, U_len)
        loss = self.rnnt.fwd(*args)
        d = self.rnnt.bwd_ex(*args, enc_dtype="bf16")
        dframes, dgamma, dbeta = self.norm.bwd(frames, d["dhA"], v["gamma"], v["beta"], T_len)
        dtable = self.embed.bwd(d["dhL"], labels, U_len)
        grads = {"WA": d["dWA"], "WL": d["dWL"], "WO": d["dWO"], "bZ": d["dbZ"], "bO": d["dbO"],
                 "gamma": dgamma, "beta": dbeta, "table": dtable}
        count = float(frames.shape[0])
        for k, grad in grads.items():
            vel = self.velocity[k].mul_(self.mu).add_(grad, alpha=1 / count)
            if k in m:  # an update of singular values near 1, whatever the gradient's
                scale = self.lr * math.sqrt(max(1.0, m[k].shape[0] / m[k].shape[1]))
                m[k].sub_(self.orth[k].run(vel), alpha=scale)
            else:
                v[k].sub_(vel, alpha=0.1 * self.lr)
        return loss, dframes

    def status(self):
        """0 when no call found a problem on the device."""
        ops = [self.norm, self.embed, *self.orth.values()]
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
