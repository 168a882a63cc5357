"""The operators as a training step uses them: gated front kept in 8 bits,
down projection, head loss, and the way back from the checkpoints to an SGD
step on both adapters - against the same step in 64 bits on the kept values."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import dev_f32, host, rel_err, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,F,r,V,name", [(40, 136, 192, 8, 500, "bf16"), (300, 264, 320, 16, 1003, "bf16"),
                                            (300, 264, 320, 16, 1003, "f16"), (12, 72, 64, 8, 130, "f16")])
def test_training_step(M, K, F, r, V, name):
    import torch
    say(f"training step M={M} K={K} F={F} V={V} {name}")
    T = {"bf16": torch.bfloat16, "f16": torch.float16}[name]
    rng = np.random.default_rng(M + V)
    dev = lambda *s, std=1.0: (torch.from_numpy(rng.standard_normal(s).astype(np.float32)) * std).to(T).cuda()
    Kd = 64 * (-(-K // 64))            # the down projection's output, a multiple of 64
    c, lr = 0.5, 0.1
    states, Ws = [], []
    for shape in ((K, F), (K, F), (F, Kd)):
        st, _ = qn.nf4_quantize(dev_f32(rng.standard_normal(shape) / np.sqrt(shape[0])))
        states.append(st)
        Ws.append(host(qn.nf4_dequantize(st, name)).reshape(shape).astype(np.float64))
    X, A, B = dev(M, K), dev(K, 2 * r, std=1 / np.sqrt(K)), dev(r, 2 * F, std=0.2)
    Ad, Bd, head = dev(F, r, std=1 / np.sqrt(F)), dev(r, Kd, std=0.2), dev(V, Kd, std=1 / np.sqrt(Kd))
    t = torch.from_numpy(rng.integers(0, V, M)).cuda()
    t[::5] = -100
    n = int((t != -100).sum())
    w = torch.full((M,), (64.0 if name == "f16" else 1.0) / n, device="cuda")

    H, Z, gu = qn.qlora_gated_fwd(X, states[:2], A, B, c, K, F, save="8")
    x8, h8 = qn.act8_encode(X), qn.act8_encode(H)
    Y, Zd = qn.qlora_linear_fwd(H, states[2], Ad, Bd, c, F, Kd)
    loss, lse, dY = qn.qlora_head_loss(Y, head, t, weights=w)
    dH, dAd, dBd = qn.qlora_linear_bwd(dY, h8, Zd, states[2], Ad, Bd, c, F, Kd)
    dX, dA, dB = qn.qlora_gated_bwd(dH, x8, Z, gu, states[:2], A, B, c, K, F)

    f64 = lambda v: host(v).astype(np.float64)
    # each operator on what it was given: no error is carried from one to the next
    H0, Z0, _, _ = oo.gated_forward(f64(X), Ws[0], Ws[1], f64(A), f64(B), c, "silu")
    loss0, lse0, dY0 = oo.head_loss(f64(Y), f64(head), host(t), f64(w))
    hk = f64(qn.act8_decode(h8))
    dZd = c * f64(dY) @ f64(Bd).T
    kept = f64(qn.act8_decode(gu))
    back = oo.gated_backward(f64(dH), f64(qn.act8_decode(x8)), f64(Z), kept[:, :F], kept[:, F:], Ws[0], Ws[1], f64(A),
                             f64(B), c, "silu")
    # every 16-bit rounding is below 2^-8 (bf16) of its value; at most three follow each other
    tol = 3 * {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[name] + 1e-5
    for what, g, ref in (("H", H, H0), ("Z", Z, Z0), ("loss", loss, loss0), ("lse", lse, lse0), ("dY", dY, dY0),
                         ("dH", dH, f64(dY) @ Ws[2].T + dZd @ f64(Ad).T), ("dAd", dAd, hk.T @ dZd),
                         ("dBd", dBd, c * f64(Zd).T @ f64(dY)), ("dX", dX, back[0]), ("dA", dA, back[1]),
                         ("dB", dB, back[2])):
        err = rel_err(host(g), ref)
        say(f"  {what} {err:.2e}")
        assert err <= tol, what
    # the step moves both adapters against their gradients
    for a, b, da, db in ((A, B, dA, dB), (Ad, Bd, dAd, dBd)):
        a0, b0 = a.clone(), b.clone()
        if a is A:      # the pair's adapters side by side: one call over the whole matrices
            qn.qlora_sgd_step(a, b[:, :F].contiguous(), da, db[:, :F].contiguous(), lr)
            want = (a0.float() - lr * da).to(T)
            np.testing.assert_array_equal(host(a), host(want))
            continue
        qn.qlora_sgd_step(a, b, da, db, lr)
        np.testing.assert_array_equal(host(a), host((a0.float() - lr * da).to(T)))
        np.testing.assert_array_equal(host(b), host((b0.float() - lr * db).to(T)))


def test_wrappers_refuse_shapes_and_types():
    import torch
    say("refusals")
    b, K, F, r = torch.bfloat16, 64, 128, 8
    z = lambda *s, t=b: torch.zeros(*s, dtype=t, device="cuda")
    states = [qn.nf4_quantize(z(K * F, t=torch.float32) + 1)[0] for _ in range(2)]
    X, A, B, dH, Z = z(4, K), z(K, 2 * r), z(r, 2 * F), z(4, F), z(4, 2 * r)
    ok = dict(c=1.0, K=K, F=F)
    qn.qlora_gated_fwd(X, states, A, B, **ok)
    for args, kw in (((X[:, :32], states, A, B), {}), ((X, states, A[:32], B), {}), ((X, states, A, B[:, :F]), {}),
                     ((X, states, A, B), {"H": z(4, K)}), ((X, states, A, B), {"Z": z(4, r)}),
                     ((X, states, A, B), {"saved": z(4, F)}), ((X, states, A, B), {"saved": z(4, 2 * F, t=torch.float16)}),
                     ((X, states, A, B.half()), {}), ((X, states, A, B), {"H": z(F, 4).T}),
                     ((X, states, A, B), {"H": torch.zeros(4, F, dtype=b)})):
        with pytest.raises(ValueError):
            qn.qlora_gated_fwd(*args, **ok, **kw)
    kept = qn.act8_encode(X)
    for args, kw in (((dH[:3], X, Z, None), {}), ((dH, kept, Z, None), {}), ((dH, X, Z[:, :r], None), {}),
                     ((dH, X, Z, None), {"grad_dtype": torch.float16}), ((dH, X, Z, None), {"dA": z(K, 2 * r)}),
                     ((dH, X, Z, None), {"dX": z(K, 4)})):
        with pytest.raises(ValueError):
            qn.qlora_gated_bwd(*args, states, A, B, **ok, **kw)
    with pytest.raises(RuntimeError):                       # a workspace that is too small
        qn.qlora_gated_fwd(X, states, A, B, **ok, workspace=z(256, t=torch.uint8))
    W, t = z(30, K), z(4, t=torch.int64)
    qn.qlora_head_loss(X, W, t)
    for args, kw in (((X, W[:, :32], t), {}), ((X, W, t[:3]), {}), ((X, W, t.int()), {}), ((X, W.half(), t), {}),
                     ((X, W, t), {"weights": z(4)}), ((X, W, t), {"loss": z(3, t=torch.float32)}),
                     ((X, W, t), {"dX": z(4, K, t=torch.float32)}), ((X, W, t.cpu()), {})):
        with pytest.raises(ValueError):
            qn.qlora_head_loss(*args, **kw)
    torch.cuda.synchronize()


def test_split_products_captured_and_on_two_streams():
    """Products whose reductions are split, in two graphs that share no
    workspace and on two streams at once: the bits of the eager calls."""
    import torch
    say("split products, captured")
    b = torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(9)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(b)
    M, K, F, r = 300, 1544, 16704, 8
    states = [qn.nf4_quantize(torch.randn(K * F, generator=gen, device="cuda") * 0.05)[0] for _ in range(2)]
    X, A, B, dH = n(M, K), n(K, 2 * r, std=0.1), n(r, 2 * F, std=0.1), n(M, F)
    Y, W = n(40, 2056), n(700, 2056, std=0.02)
    t = torch.arange(40, device="cuda") * 17
    wide = n(30, K)

    def block():
        H, Z, kept = qn.qlora_gated_fwd(X, states, A, B, 0.5, K, F, save="8")
        return [H, Z, kept.codes, kept.absmax, *qn.qlora_gated_bwd(dH, X, Z, kept, states, A, B, 0.5, K, F)]

    def loss():
        few = qn.qlora_gated_fwd(wide, states, A, B, 0.5, K, F)
        return [*qn.qlora_head_loss(Y, W, t), *few[:2]]

    want = [[host(v).copy() for v in f()] for f in (block, loss)]
    graphs = []
    side = torch.cuda.Stream()
    for f in (block, loss):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for _ in range(3):
        for v in graphs[0][1] + graphs[1][1]:
            v.zero_()
        block()                                     # eager work between the replays
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
            again = loss()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            for o, v in zip(out, w):
                np.testing.assert_array_equal(host(o), v)
        for o, v in zip(again, want[1]):
            np.testing.assert_array_equal(host(o), v)
