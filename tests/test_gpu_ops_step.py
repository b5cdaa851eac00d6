"""Label embedding, layer norm, clipping and AdamW together, against 64 bits (GPU).

The loss is linear in the normalised rows, so autograd on the CPU gives the gradients.  They are
at most k u (1 + r) of their terms off (u = 2^-24, k = 64, r a row's mean over its deviation), a
few 1e-5 of a gradient's root mean square s; with second moments of s^2 and more an update moves by
at most a tenth of that over s, so 1e-4 of the learning rate holds it with room, beside the
weight's own half step.
"""
import numpy as np
import pytest
import torch

import asr_tiled_tanh_gb300 as rn
from tests.test_gpu_ops_streams import _stream_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rn.load(build_if_missing=True)


def _model(seed=0, B=12, U1=14, V=50, D=72):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ids = torch.randint(1, V, (B, U1), generator=g, dtype=torch.int32)
    U_len = torch.randint(0, U1, (B,), generator=g, dtype=torch.int32)
    U_len[0], U_len[1] = U1 - 1, 0
    return n(V, D) / D ** 0.5, 1 + 0.2 * n(D), 0.2 * n(D), ids, U_len, n(B, U1, D)


def _gradients64(table, scale, shift, ids, U_len, w):
    p = [t.detach().double().clone().requires_grad_() for t in (table, scale, shift)]
    D = table.shape[1]
    ids = ids.long().clone()
    ids[:, 0] = 0
    live = (torch.arange(ids.shape[1])[None] <= U_len[:, None])[..., None]
    e = p[0][ids] * D ** 0.5
    xc = e - e.mean(2, keepdim=True)
    y = xc / ((xc * xc).mean(2, keepdim=True) + 1e-5).sqrt() * p[1] + p[2]
    ((y * w.double()) * live).sum().backward()
    return [t.grad for t in p]


def _step(weights, grads64, m, v, t, lr, decays, max_norm):
    norm = float(np.sqrt(sum(float((g ** 2).sum()) for g in grads64)))
    s = min(1.0, max_norm / (norm + 1e-6))
    out = []
    for p, g, a, b, d in zip(weights, grads64, m, v, decays):
        a, b = 0.9 * a + 0.1 * s * g, 0.999 * b + 0.001 * (s * g) ** 2
        out.append((p - lr * (d * p + a / (1 - 0.9 ** t)
                              / ((b / (1 - 0.999 ** t)).sqrt() + 1e-8)), a, b))
    return [list(x) for x in zip(*out)]


@pytest.mark.parametrize("graph", [False, True])
def test_embedding_norm_clip_and_update(graph):
    table, scale, shift, ids, U_len, w = _model()
    B, U1, D, V = *ids.shape, table.shape[1], table.shape[0]
    lr, decays, t0, max_norm = 2.0 ** -7, [0.0, 0.25, 0.0], 500, 3.0
    g0 = _gradients64(table, scale, shift, ids, U_len, w)
    s = [float((g ** 2).mean().sqrt()) for g in g0]
    ref = [x.double() for x in (table, scale, shift)]
    rm, rv = [0.1 * g for g in g0], [2 * k * k + 0 * g for k, g in zip(s, g0)]

    dev = [x.cuda() for x in (table, scale, shift)]
    m, v = ([x.float().cuda() for x in y] for y in (rm, rv))
    shapes = [x.shape for x in dev]
    embed = rn.LabelEmbedding(B, U1, V, D, dtype="f32", out_dtype="f32", scale=D ** 0.5)
    rows = rn.LayerNorm(B, U1, D, dtype="f32", label_rows=True)
    clip = rn.GradClip(shapes, max_norm=max_norm)
    adamw = rn.AdamW(shapes, weight_decay=decays, m=m, v=v, steps=t0)
    low = [None, torch.zeros(D, dtype=torch.bfloat16, device="cuda"), None]
    idg, ulg, dy = ids.cuda(), U_len.cuda(), w.cuda()

    def step():
        e = embed.fwd(dev[0], idg, ulg)
        y = rows.fwd(e, dev[1], dev[2], ulg)
        de, dscale, dshift = rows.bwd(e, dy, dev[1], ulg)
        grads = [embed.bwd(de, idg, ulg), dscale, dshift]
        adamw.step(dev, grads, lr, clip=clip.norm(grads), low=low)
        return y

    if graph:
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            step()
    for k in range(3):
        G.replay() if graph else step()
        grads = _gradients64(*ref, ids, U_len, w)
        ref, rm, rv = _step(ref, grads, rm, rv, t0 + k + 1, lr, decays, max_norm)
        torch.cuda.synchronize()
        for a, b in zip(dev, ref):
            err = (a.cpu().double() - b).abs()
            assert torch.all(err <= (k + 1) * (1e-4 * lr + 2.0 ** -23 * b.abs())), float(err.max())
        assert torch.equal(low[1], dev[1].bfloat16())
    assert adamw.steps.tolist() == [t0 + 3, 0]
    assert embed.status() == rows.status() == (0, 0)


@pytest.mark.parametrize("how", ["stream", "handle", "current"])
def test_results_belong_to_the_calls_stream(how):
    x, dy = torch.randn(4, 9, 64, device="cuda"), torch.randn(4, 9, 64, device="cuda")
    g = [torch.randn(300, 7, device="cuda"), torch.randn(5, device="cuda")]
    n, c = rn.LayerNorm(4, 9, 64, dtype="f32"), rn.GradClip([(300, 7), (5,)])

    def run(**k):
        return [n.fwd(x, **k), *n.bwd(x, dy, **k), c.norm(g, **k)]

    ref = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    if how == "current":
        with torch.cuda.stream(s):
            got = run()
    else:
        got = run(stream=s if how == "stream" else s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert [_stream_of(t) for t in got] == [s.cuda_stream] * len(got)


def test_the_helper_and_python_say_the_same():
    # (what is refused, and the same results where csrc/lists.cpp was not built)
    x = torch.randn(3, 5, 40, device="cuda")
    g = [torch.randn(30, device="cuda"), torch.randn(4, 4, device="cuda").bfloat16()]
    n = rn.LayerNorm(3, 5, 40, dtype="f32")
    c = rn.GradClip([(30,), (4, 4)], dtype=["f32", "bf16"])
    assert n._fast is not None and c._take_list is not None
    out = []
    for fast in (True, False):
        if not fast:
            n._fast = c._fast = c._take_list = None
        out.append([n.fwd(x), *n.bwd(x, x), c.norm(g)])
        for bad in (x.bfloat16(), x[:2], x.cpu(), x.transpose(0, 1), x[:, :, ::2], x.expand(3, 5, 40)
                    .transpose(1, 2), torch.zeros(5, 3, 40, device="cuda"), None):
            with pytest.raises((ValueError, AttributeError)):
                n.fwd(bad)
        for bad in ([g[0]], g[::-1], [g[0], g[1].float()], [g[0], g[1].t()[:2]], [g[0][::2], g[1]],
                    [g[0].cpu(), g[1]], [g[0].double(), g[1]], [g[0].view(5, 6), g[1]]):
            with pytest.raises(ValueError):
                c.norm(bad)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_plans_of_several_host_threads():
    # each thread with plans, tensors and a stream of its own
    import threading
    wrong = []

    def work(seed, stream):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *k: torch.randn(*k, device="cuda", generator=gen)  # noqa: E731
        with torch.cuda.stream(stream):
            C = (512, 333, 64, 1280)[seed % 4]
            x, dy, scale = r(9, 50, C), r(9, 50, C), r(C)
            shapes = [(1000 * (i + 1) + seed,) for i in range(4 + 12 * seed)]
            grads, p = [r(*k) for k in shapes], [r(*k) for k in shapes]
            q = [t.clone() for t in p]
            n, c = rn.LayerNorm(9, 50, C, dtype="f32"), rn.GradClip(shapes)
            a, b = rn.AdamW(shapes), rn.AdamW(shapes)
            ref = None
            for _ in range(25):
                out = [n.fwd(x, scale, scale), *n.bwd(x, dy, scale), c.norm(grads)]
                a.step(p, grads, 1e-3, clip=out[-1])
                stream.synchronize()
                ref = ref or [t.clone() for t in out]
                if not all(torch.equal(u, w) for u, w in zip(out, ref)):
                    wrong.append(("results", seed))
            for _ in range(25):
                b.step(q, grads, 1e-3, clip=ref[-1])
            stream.synchronize()
            if not all(torch.equal(u, w) for u, w in zip(p, q)) or a.steps.tolist() != [25, 0]:
                wrong.append(("update", seed))

    threads = [threading.Thread(target=work, args=(k, torch.cuda.Stream())) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
