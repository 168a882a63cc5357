"""The gated front where its roundings, ranges and paths meet: gates past the
16-bit type's range, adapters that carry the whole output, factors c of either
sign and above 1, the kept pair on every path."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import dev_f32, host, say
from tests.test_gpu_gated import ACT, F32, HALF, TINY, Case, _check_backward, _close, _dev

pytestmark = pytest.mark.gpu


def _set_weights(k, *weights):
    """Other weights for the case: what they are stored as is what counts."""
    k.states, k.W = [], []
    for w in weights:
        state, status = qn.nf4_quantize(dev_f32(w))
        assert qn.nf4_status_read(status) == 0
        k.states.append(state)
        k.W.append(host(qn.nf4_dequantize(state, k.name)).reshape(k.K, k.F).astype(np.float64))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [4, 40, 300])
def test_gates_below_fp16_have_no_gradient(M, act):
    """G below -65504 is kept as -inf: act and act' are 0 there, not inf * 0."""
    say(f"gated, gates below fp16 M={M} {act}")
    k = Case(M, 64, 192, 8, "f16")
    rng = np.random.default_rng(M)
    _set_weights(k, -np.abs(rng.standard_normal((64, 192))) * 0.19, rng.standard_normal((64, 192)) * 1e-4)
    k.A.zero_()
    k.a[:] = 0
    # every third row small, the others with gates around -65504
    scale = np.where(np.arange(M) % 3 == 0, 0.02, 8400.0)[:, None]
    k.X = _dev(np.abs(rng.standard_normal((M, 64))) * scale, "f16")
    k.x = host(k.X).astype(np.float64)
    H, Z, gu = k.forward(act, "16")
    pair = host(gu).astype(np.float64)
    far = np.isneginf(pair[:, :k.F])
    assert 0.1 < far.mean() < 0.9 and np.isfinite(pair[:, k.F:]).all() and np.isfinite(host(H)).all()
    assert not host(H)[far].any()
    G = np.where(far, -7e4, pair[:, :k.F])
    got = k.backward(act, k.X, Z, gu)
    _check_backward(k, act, k.x, Z, G, pair[:, k.F:], got, None)
    for g, w in zip(k.backward(act, k.X, Z, None), got):
        np.testing.assert_array_equal(host(g), host(w))
    # a NaN gate stays one
    gu[1, 5] = float("nan")
    assert np.isnan(host(k.backward(act, k.X, Z, gu)[0])[1]).all()


def _check_kept(k, act, H, Z, gu):
    """H and the kept pair against 64 bits.  Z's own rounding is no part of the
    bounds: it enters the products as two 16-bit parts, off by d of d of it (fp16:
    by half its smallest step, times the power of two up to 2 |c| that B carries)."""
    d, n, c = HALF[k.name], k.K + 2 * k.r + 4, abs(k.c)
    H0, Z0, G0, U0 = oo.gated_forward(k.x, k.W[0], k.W[1], k.a, k.b, k.c, act)
    zabs = np.abs(k.x) @ np.abs(k.a)
    _close(Z, Z0, d * np.abs(Z0) + n * F32 * zabs + TINY[k.name] + 1e-30, "Z")
    e = []
    for i in range(2):
        b, z = np.abs(k.b[:, i * k.F:(i + 1) * k.F]), zabs[:, i * k.r:(i + 1) * k.r]
        z0 = np.abs(Z0[:, i * k.r:(i + 1) * k.r])
        e.append(d * d * c * (z0 @ b) + n * F32 * (np.abs(k.x) @ np.abs(k.W[i]) + c * (z @ b))
                 + max(1.0, 2 * c) * TINY[k.name] * b.sum(0)[None])
    pair = host(gu)
    for what, got, want, err in (("G", pair[:, :k.F], G0, e[0]), ("U", pair[:, k.F:], U0, e[1])):
        bound = err + d * (np.abs(want) + err) + TINY[k.name] + 1e-30
        worst = np.max(np.abs(got - want) / bound)
        say(f"  {what}: worst error / bound {worst:.3f}")
        assert worst <= 1.0, what
    f = oo.act(act, G0)[0]
    # |act'| <= 1.13; past an argument of 80 the sigmoid is 0 or 1 to below 1e-30
    bound = 1.13 * e[0] * (np.abs(U0) + e[1]) + np.abs(f) * e[1] + (d + ACT) * (np.abs(H0) + e[0] * e[1]) \
        + 1e-6 * np.abs(U0) + TINY[k.name] + 1e-30
    # from 65520 on the nearest fp16 value is an infinity: where H0 lies past it by
    # more than the bound that is the answer, within the bound of it either will do
    h, end = host(H).astype(np.float64), {"bf16": np.inf, "f16": 65520.0}[k.name]
    over = np.isinf(h) & (np.abs(H0) + bound >= end) & (np.sign(h) == np.sign(H0))
    assert np.isinf(h)[np.abs(H0) - bound > end].all()
    h = np.where(over, H0, h)
    assert np.isfinite(h).all()
    worst = np.max(np.abs(h - H0) / bound)
    say(f"  H: worst error / bound {worst:.3f}, {int(over.sum())} past the type's range")
    assert worst <= 1.0


# few rows on every tile count, many rows with and without a split reduction, the
# last round of tiles alone split
KEPT = [(1, 264, 192, 8, 0.5), (3, 72, 128, 8, 2.0), (16, 520, 320, 40, -3.0), (29, 136, 192, 128, -0.37),
        (40, 264, 448, 16, 2.0), (100, 1032, 320, 24, -3.0), (256, 72, 128, 8, 1.5), (257, 136, 192, 8, -3.0),
        (300, 520, 704, 40, 2.0), (300, 2056, 192, 128, -0.37), (2100, 72, 3712, 8, 1.0), (700, 1544, 11072, 8, -1.25)]


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,F,r,c", KEPT)
def test_kept_pair_where_the_adapter_carries_it(M, K, F, r, c, name):
    say(f"gated, kept pair M={M} K={K} F={F} r={r} c={c} {name}")
    act = "gelu" if (M + r) % 3 == 0 else "silu"
    k = Case(M, K, F, r, name, c=c)
    rng = np.random.default_rng(M + F)
    _set_weights(k, *(rng.standard_normal((K, F)) * 1e-3 / np.sqrt(K) for _ in range(2)))
    k.B = _dev(rng.standard_normal((r, 2 * F)), name)
    k.b = host(k.B).astype(np.float64)
    H, Z, gu = k.forward(act, "16")
    _check_kept(k, act, H, Z, gu)
    H8, Z8, gu8 = k.forward(act, "8")
    same = qn.act8_encode(gu)
    for g, w in ((H8, H), (Z8, Z), (gu8.codes, same.codes), (gu8.absmax, same.absmax)):
        np.testing.assert_array_equal(host(g), host(w))


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,F,r,c", KEPT)
def test_kept_pair_of_ordinary_weights(M, K, F, r, c, name):
    say(f"gated, kept pair, weights M={M} K={K} F={F} r={r} c={c} {name}")
    act = "silu" if (M + r) % 3 == 0 else "gelu"
    k = Case(M, K, F, r, name, c=c)
    H, Z, gu = k.forward(act, "16")
    _check_kept(k, act, H, Z, gu)


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,F,r,c", [(3, 72, 128, 8, 2.0), (40, 264, 192, 16, -3.0), (300, 520, 704, 40, 0.5),
                                       (520, 264, 320, 128, -0.25)])
def test_adapter_gradients_of_exact_output_gradients(M, K, F, r, c, name):
    """Gates of 0 and 64 and U of +-1 or 2 make dG and dU exact, so dA and dB show
    the adapter products' own error: dZ goes into dA as two 16-bit parts."""
    import torch
    say(f"gated, adapter gradients M={M} K={K} F={F} r={r} c={c} {name}")
    k = Case(M, K, F, r, name, c=c)
    rng = np.random.default_rng(K)
    pair = np.hstack((rng.choice([0.0, 64.0], (M, F)), rng.choice([-1.0, 1.0, 2.0], (M, F))))
    z = _dev(rng.standard_normal((M, 2 * r)), name)
    dX0, dA0, dB0 = oo.gated_backward(k.dh, k.x, host(z), pair[:, :F], pair[:, F:], k.W[0], k.W[1], k.a, k.b, c, "silu")
    f, df = oo.act("silu", pair[:, :F])
    dY = (np.abs(k.dh * pair[:, F:] * np.round(2 * df) / 2), np.abs(k.dh * np.round(f)))
    d, n = HALF[name], F + 8
    for x in (k.X, qn.act8_encode(k.X)):
        xv = k.x
        if isinstance(x, qn.Act8):
            xv = host(qn.act8_decode(x)).astype(np.float64)
            dA0 = oo.gated_backward(k.dh, xv, host(z), pair[:, :F], pair[:, F:], k.W[0], k.W[1], k.a, k.b, c, "silu")[1]
        _, dA, dB = k.backward("silu", x, z, _dev(pair, name))
        eA, eB = [], []
        for i in range(2):
            zabs = abs(c) * (dY[i] @ np.abs(k.b[:, i * F:(i + 1) * F]).T)
            dz = np.abs(c * (((k.dh * pair[:, F:] * df) if i == 0 else (k.dh * f)) @ k.b[:, i * F:(i + 1) * F].T))
            eA.append(np.abs(xv).T @ (d * d * dz + n * F32 * zabs + TINY[name]) + (2 * M + 8) * F32 * (np.abs(xv).T @ (zabs + TINY[name])))
            eB.append(abs(c) * (M + 8) * F32 * (np.abs(host(z)[:, i * r:(i + 1) * r]).T @ dY[i]))
        _close(dA, dA0, np.hstack(eA) + F32 * np.abs(dA0) + 1e-30, "dA")
        _close(dB, dB0, np.hstack(eB) + F32 * np.abs(dB0) + 1e-30, "dB")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,name,scale", [(4, "f16", 50.0), (64, "f16", 50.0), (300, "f16", 50.0), (300, "bf16", 50.0),
                                          (300, "bf16", 3e4), (64, "bf16", 3e4)])
def test_far_gates_element_by_element(M, name, scale, act):
    say(f"gated, far gates M={M} {name} {scale} {act}")
    k = Case(M, 64, 192, 8, name)
    k.X = _dev(k.x * scale, name)
    k.x = host(k.X).astype(np.float64)
    H, Z, gu = k.forward(act, "16")
    _check_kept(k, act, H, Z, gu)
    for g in k.backward(act, k.X, Z, gu):
        assert np.isfinite(host(g)).all()


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_nan_gate_of_many_rows(name):
    say(f"gated, NaN row of 300 {name}")
    k = Case(300, 64, 192, 8, name)
    k.X[277, 3] = float("nan")
    for save in ("16", "8", "none"):
        H, Z, gu = k.forward("gelu", save)
        bad = np.isnan(host(H)).all(axis=1)
        assert bad[277] and bad.sum() == 1 and np.isfinite(np.delete(host(H), 277, axis=0)).all()
        dX = host(k.backward("gelu", k.X, Z, gu)[0])
        assert np.isnan(dX[277]).all() and np.isfinite(np.delete(dX, 277, axis=0)).all()
