"""The operators at the ends of their documented ranges: the shortest reductions,
the most rows, the widest outputs.  Large outputs are checked on sampled rows or
columns, against 64 bits."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import host, say
from tests.test_gpu_gated import F32, HALF, TINY, Case, _check_backward, _close, _torch_type
from tests.test_gpu_gated_edges import _check_kept
from tests.test_gpu_head import _compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,F,r", [(1, 8, 64, 8), (17, 8, 128, 8), (40, 16, 64, 128), (257, 8, 64, 8), (300, 24, 320, 16),
                                     (2100, 8, 3776, 8)])
def test_gated_of_the_shortest_reductions(M, K, F, r, name):
    say(f"gated, K={K} M={M} F={F} r={r} {name}")
    k = Case(M, K, F, r, name)
    H, Z, gu = k.forward("silu", "16")
    _check_kept(k, "silu", H, Z, gu)
    pair = host(gu).astype(np.float64)
    got = k.backward("silu", k.X, Z, gu)
    _check_backward(k, "silu", k.x, Z, pair[:, :F], pair[:, F:], got, None)
    x8 = qn.act8_encode(k.X)
    for g, w in zip(k.backward("silu", x8, Z, gu), k.backward("silu", qn.act8_decode(x8), Z, gu)):
        np.testing.assert_array_equal(host(g), host(w))


def _sampled_gated(M, K, F, r, name, rows, cols):
    """Forward and backward with random device inputs; H, the kept pair, Z and dX of
    `rows` x `cols` in 64 bits (dA and dB on sampled rows and columns)."""
    import torch
    T, d, c = _torch_type(name), HALF[name], 0.5
    gen = torch.Generator("cuda").manual_seed(M + F)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(T)
    states = [qn.nf4_quantize(torch.randn(K * F, generator=gen, device="cuda") / K ** 0.5)[0] for _ in range(2)]
    X, A, B, dH = n(M, K), n(K, 2 * r, std=K ** -0.5), n(r, 2 * F, std=0.3), n(M, F)
    H, Z, gu = qn.qlora_gated_fwd(X, states, A, B, c, K, F, save="16")
    W = [qn.nf4_dequantize(s, {"bf16": "bf16", "f16": "f16"}[name]).view(K, F) for s in states]
    f64 = lambda t: host(t).astype(np.float64)
    both = np.concatenate((cols, F + cols))
    x, a, b = f64(X[rows]), f64(A), f64(B[:, torch.from_numpy(both).cuda()])
    w = [f64(v[:, torch.from_numpy(cols).cuda()]) for v in W]
    m = len(cols)
    H0, Z0, G0, U0 = oo.gated_forward(x, w[0], w[1], a, b, c, "silu")
    steps = (K + 2 * r + 4) * F32
    zabs = np.abs(x) @ np.abs(a)
    at = torch.from_numpy(cols).cuda()
    _close(Z[rows], Z0, d * np.abs(Z0) + steps * zabs + TINY[name] + 1e-30, "Z")
    e = [d * d * c * (np.abs(Z0[:, i * r:(i + 1) * r]) @ np.abs(b[:, i * m:(i + 1) * m])) + TINY[name] * np.abs(b[:, i * m:(i + 1) * m]).sum(0)
         + steps * (np.abs(x) @ np.abs(w[i]) + c * (zabs[:, i * r:(i + 1) * r] @ np.abs(b[:, i * m:(i + 1) * m]))) for i in (0, 1)]
    for what, got, want, err in (("G", gu[rows][:, at], G0, e[0]), ("U", gu[rows][:, F + at], U0, e[1])):
        _close(got, want, err + d * (np.abs(want) + err) + TINY[name] + 1e-30, what)
    f = oo.act("silu", G0)[0]
    _close(H[rows][:, at], H0, 1.13 * e[0] * (np.abs(U0) + e[1]) + np.abs(f) * e[1] + (d + 1e-5) * (np.abs(H0) + e[0] * e[1])
           + 1e-6 * np.abs(U0) + TINY[name] + 1e-30, "H")
    # the backward of the sampled rows: all columns
    dX, dA, dB = qn.qlora_gated_bwd(dH, X, Z, gu, states, A, B, c, K, F)
    pair = f64(gu[rows])
    got = oo.gated_backward(f64(dH[rows]), x, f64(Z[rows]), pair[:, :F], pair[:, F:], f64(W[0]), f64(W[1]), a, f64(B), c, "silu")
    f, df = oo.act("silu", pair[:, :F])
    dh = f64(dH[rows])
    dY = np.abs(np.hstack((dh * pair[:, F:] * df, dh * f)))
    eY = d * dY + 2e-5 * np.abs(np.hstack((dh * pair[:, F:], dh * pair[:, :F]))) + TINY[name]
    # column sums of the weights' magnitudes, in two steps so that wide F fits: sums over the packed axis
    Wabs = np.abs(np.hstack((f64(W[0]), f64(W[1]))))
    nsum = (2 * F + 2 * r + 8) * F32
    babs = np.abs(f64(B))
    bound = eY @ Wabs.T + nsum * (dY @ Wabs.T)
    for i in (0, 1):
        s = slice(i * F, (i + 1) * F)
        zi = c * (dY[:, s] @ babs[:, s].T)
        ez = c * (eY[:, s] @ babs[:, s].T) * 1.01 + (d + nsum) * zi + TINY[name]
        bound += 1.01 * (ez + nsum * zi) @ np.abs(a[:, i * r:(i + 1) * r]).T
    _close(dX[rows], got[0], bound + d * (np.abs(got[0]) + bound) + TINY[name] + 1e-30, "dX")
    assert bool(torch.isfinite(dA).all()) and bool(torch.isfinite(dB).all()) and bool(torch.isfinite(dX).all())


@pytest.mark.parametrize("M,K,F,r,name", [((1 << 20) - 3, 8, 64, 8, "bf16"), (200003, 40, 320, 16, "f16"),
                                          (255, 8, 1 << 18, 8, "bf16"), (16, 64, 1 << 19, 8, "f16"), (300, 8, 1 << 18, 8, "bf16")])
def test_gated_of_many_rows_and_of_wide_outputs(M, K, F, r, name):
    say(f"gated, M={M} K={K} F={F} {name}")
    rng = np.random.default_rng(2)
    rows = np.unique(np.concatenate(([0, M - 1], rng.integers(0, M, 10 if F > 1000 else 60))))
    cols = np.unique(np.concatenate(([0, F - 1, F // 2], rng.integers(0, F, 60))))
    _sampled_gated(M, K, F, r, name, rows, cols)


def _head(M, K, V, name, rows, need_dx=True, std=None):
    import torch
    T = _torch_type(name)
    gen = torch.Generator("cuda").manual_seed(V)
    W = (torch.randn(V, K, generator=gen, device="cuda") * (K ** -0.5 if std is None else std)).to(T)
    X = torch.randn(M, K, generator=gen, device="cuda").to(T)
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[::7] = -100
    w = torch.rand(M, generator=gen, device="cuda")
    got = qn.qlora_head_loss(X, W, t, weights=w, need_dx=need_dx)
    at = torch.from_numpy(rows).cuda()
    _compare(X[at], W, t[at], w[at], [None if g is None else g[at] for g in got], name)
    assert all(bool(torch.isfinite(g).all()) for g in got if g is not None)


@pytest.mark.parametrize("M,K,V,name", [(1 << 20, 8, 300, "bf16"), ((1 << 20) - 5, 16, 700, "f16")])
def test_head_of_the_most_rows(M, K, V, name):
    say(f"head, M={M} V={V} {name}")
    rows = np.unique(np.concatenate(([0, M - 1], np.random.default_rng(1).integers(0, M, 300))))
    for need_dx in (True, False):
        _head(M, K, V, name, rows, need_dx)


@pytest.mark.parametrize("M,K,V,name", [(1, 8, 1 << 22, "bf16"), (5, 16, 3000017, "f16")])
def test_head_of_wide_vocabularies(M, K, V, name):
    say(f"head, V={V} M={M} {name}")
    _head(M, K, V, name, np.arange(M))


def test_head_of_the_longest_rows():
    """K = 2^20: a piece of the vocabulary is 512 of its rows."""
    import torch
    say("head, K = 2^20")
    M, K, V = 3, 1 << 20, 700
    gen = torch.Generator("cuda").manual_seed(5)
    W = (torch.randn(V, K, generator=gen, device="cuda") / K ** 0.5).bfloat16()
    X = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    t = torch.tensor([0, V - 1, 511], device="cuda")
    loss, lse, dX = qn.qlora_head_loss(X, W, t)
    s = torch.cat([X.double() @ W[i:i + 100].double().T.contiguous() for i in range(0, V, 100)], 1)
    want = torch.logsumexp(s, 1)
    p = torch.exp(s - want[:, None])
    ref = sum(p[:, i:i + 100] @ W[i:i + 100].double() for i in range(0, V, 100)) - W[t].double()
    mag = sum(p[:, i:i + 100] @ W[i:i + 100].double().abs() for i in range(0, V, 100)) + W[t].double().abs()
    # an fp32 sum of 2^20 terms with random signs: far below 2^-24 times 2^10 of its largest partial sum
    np.testing.assert_allclose(host(lse), want.cpu().numpy(), atol=1e-3)
    np.testing.assert_allclose(host(loss), (want - s.gather(1, t[:, None])[:, 0]).cpu().numpy(), atol=1e-3)
    bound = 2.0 ** -8 * 1.1 * ref.abs() + (2.0 ** -8 + 2e-3) * mag
    assert bool(((dX.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("rows,cols,name", [((1 << 25) + 3, 8, "bf16"), (3, 1 << 26, "f16"), (300007, 1016, "bf16")])
def test_checkpoints_of_large_matrices(rows, cols, name):
    import torch
    say(f"act8, {rows} x {cols} {name}")
    gen = torch.Generator("cuda").manual_seed(rows)
    X = torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float32).to(_torch_type(name))
    kept = qn.act8_encode(X)
    back = qn.act8_decode(kept)
    for at in (slice(0, 2), slice(rows // 2, rows // 2 + 1), slice(rows - 1, rows)):
        x = host(X[at])[:, -200000:] if cols > 200000 else host(X[at])
        part = kept.codes[at][:, -200000:] if cols > 200000 else kept.codes[at]
        am = kept.absmax[at][:, -3125:] if cols > 200000 else kept.absmax[at]
        codes, absmax = oo.act8_encode(x)
        np.testing.assert_array_equal(host(part), codes)
        np.testing.assert_array_equal(host(am), absmax)
        b = host(back[at])[:, -200000:] if cols > 200000 else host(back[at])
        np.testing.assert_array_equal(b, oo.act8_decode(codes, absmax, name))
    # every element within half a step of its block, and its rounding
    step = kept.absmax.float() / 254
    worst = 0.0
    for i in range(0, rows, max(1, (1 << 25) // cols)):
        j = min(rows, i + max(1, (1 << 25) // cols))
        s = step[i:j].repeat_interleave(64, 1)[:, :cols]
        err = (back[i:j].float() - X[i:j].float()).abs() - s * 1.0001 - HALF[name] * back[i:j].float().abs()
        worst = max(worst, float(err.max()))
    assert worst <= 2.0 ** -24
