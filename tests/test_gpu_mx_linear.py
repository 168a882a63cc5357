"""The layer on an MXFP4 weight against its 64-bit reference.  Bounds are elementwise
and counted from the roundings: half a step (d) for every value held in 16 bits on the
way, 2^-24 per added term for fp32 sums."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import host, say
from tests.test_gpu_mxfp4 import HALF, _dev, _state, _torch_type

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -24
TINY = {"bf16": 0.0, "f16": 2.0 ** -25}


class Case:
    def __init__(self, M, K, N, r, name, c=0.5, seed=None):
        rng = np.random.default_rng(M * 31 + K + N if seed is None else seed)
        self.M, self.K, self.N, self.r, self.c, self.name = M, K, N, r, c, name
        codes, scales = oo.mxfp4_quantize(rng.standard_normal((N, K)) / np.sqrt(K))
        self.W, self.w = _state(codes, scales, K), oo.mxfp4_values(codes, scales, K)
        self.X, self.A, self.B, self.G = (_dev(rng.standard_normal(s) * std, name) for s, std in (
            ((M, K), 1.0), ((K, r), 1.0 / np.sqrt(K)), ((r, N), 0.3), ((M, N), 1.0)))
        self.x, self.a, self.b, self.g = (host(t).astype(np.float64) for t in (self.X, self.A, self.B, self.G))

    def forward(self, **kw):
        return qn.qlora_mx_linear_fwd(self.X, self.W, self.A, self.B, self.c, **kw)

    def backward(self, Z, X=None, **kw):
        return qn.qlora_mx_linear_bwd(self.G, self.X if X is None else X, Z, self.W, self.A, self.B, self.c, **kw)


def close(got, want, bound, what):
    got = host(got).astype(np.float64)
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - want) / bound)
    say(f"  {what}: worst error / bound {worst:.3f}")
    assert worst <= 1.0, what


def check_forward(t, Y, Z):
    d, tiny, c = HALF[t.name], TINY[t.name], abs(t.c)
    y, z = oo.mx_linear_forward(t.x, t.w, t.a, t.b, t.c)
    ax, aa, ab = np.abs(t.x), np.abs(t.a), np.abs(t.b)
    dz = t.K * F32 * (ax @ aa)                                  # before its rounding
    close(Z, z, d * np.abs(z) + 1.01 * dz + tiny, "Z")
    q = np.abs(oo.mxfp4_values(*oo.mxfp4_quantize(t.x), t.K)) @ np.abs(t.w).T
    zb = np.abs(z) @ ab
    adapter = c * (2.02 * d * zb + 1.02 * (dz @ ab) + 2 * tiny * (ab.sum(0) + np.abs(z).sum(1)[:, None]))
    close(Y, y, d * np.abs(y) + 1.01 * (adapter + (t.K + t.r) * F32 * (q + c * zb)) + tiny, "Y")


def check_backward(t, Z, dX, dA, dB, grad16, x=None):
    d, tiny, c = HALF[t.name], TINY[t.name], abs(t.c)
    z = host(Z).astype(np.float64)
    x = t.x if x is None else x
    gx, ga, gb = oo.mx_linear_backward(t.g, x, z, t.w, t.a, t.b, t.c)
    dz = c * np.abs(t.g @ t.b.T)
    near = d * dz + 1.01 * c * t.N * F32 * (np.abs(t.g) @ np.abs(t.b).T) + tiny   # dZ in 16 bits
    close(dA, ga, (d * np.abs(ga) + tiny) * grad16 + 1.01 * (np.abs(x).T @ near) + t.M * F32 * (np.abs(x).T @ dz) + 1e-30, "dA")
    close(dB, gb, (d * np.abs(gb) + tiny) * grad16 + (t.M + 2) * F32 * c * (np.abs(z).T @ np.abs(t.g)) + 1e-30, "dB")
    if dX is not None:
        w = np.abs(t.w)
        sub = TINY[t.name] * np.abs(t.g).sum(1)[:, None]       # weights below fp16's normal range
        close(dX, gx, d * np.abs(gx) + sub + 1.01 * (near @ np.abs(t.a).T) +
              (t.N + t.r) * F32 * (np.abs(t.g) @ w + dz @ np.abs(t.a).T) + tiny, "dX")


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,r", [(1, 8, 8, 8), (1, 520, 264, 8), (2, 4096, 512, 64), (5, 1032, 1000, 24),
                                     (16, 2056, 520, 256), (17, 64, 72, 8), (33, 776, 328, 40), (100, 1544, 1000, 136),
                                     (255, 512, 264, 16), (256, 1024, 256, 64), (777, 2056, 1336, 24)])
def test_layer(M, K, N, r, name):
    say(f"mx layer M={M} K={K} N={N} r={r} {name}")
    t = Case(M, K, N, r, name)
    Y, Z = t.forward()
    check_forward(t, Y, Z)
    Y2, none = t.forward(return_z=False)
    assert none is None and host(Y2).tobytes() == host(Y).tobytes()
    dX, dA, dB = t.backward(Z)
    check_backward(t, Z, dX, dA, dB, False)
    none, dA16, dB16 = t.backward(Z, need_dx=False, grad_dtype=_torch_type(name))
    assert none is None
    check_backward(t, Z, None, dA16, dB16, True)


@pytest.mark.parametrize("c", [0.0, -2.0, 0.3])
def test_scales_of_the_adapter(c):
    say(f"mx layer c={c}")
    t = Case(40, 520, 136, 16, "bf16", c=c)
    Y, Z = t.forward()
    check_forward(t, Y, Z)
    check_backward(t, Z, *t.backward(Z), False)


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_backward_from_an_8_bit_checkpoint(name):
    say(f"mx backward from 8 bits {name}")
    t = Case(130, 520, 264, 24, name)
    _, Z = t.forward()
    kept = qn.act8_encode(t.X)
    dense = qn.act8_decode(kept)
    got, want = t.backward(Z, X=kept), t.backward(Z, X=dense)
    for a, b in zip(got, want):
        assert host(a).tobytes() == host(b).tobytes()
    check_backward(t, Z, *got, False, x=host(dense).astype(np.float64))


def test_weight_quantised_from_a_checkpoint_matrix():
    """A K x N fp32 weight through mxfp4_quantize, then the layer on it."""
    import torch
    say("mx layer from a K x N weight")
    t = Case(64, 1032, 520, 16, "bf16")
    rng = np.random.default_rng(9)
    w = (rng.standard_normal((1032, 520)) / 32).astype(np.float32)
    t.W = qn.mxfp4_quantize(torch.from_numpy(w).cuda(), transpose=True)
    t.w = oo.mxfp4_values(*oo.mxfp4_quantize(w.T), 1032)
    Y, Z = t.forward()
    check_forward(t, Y, Z)
    check_backward(t, Z, *t.backward(Z), False)


def test_rows_that_are_not_finite_stay_their_own():
    """A NaN in one row of X reaches that row's outputs and no other's."""
    import torch
    say("mx layer with a NaN row")
    for M in (3, 40, 300):
        t = Case(M, 520, 264, 16, "bf16")
        clean, _ = t.forward()
        t.X[1, 100] = float("nan")
        Y, _ = t.forward()
        assert torch.isnan(Y[1]).all()
        rest = torch.arange(M, device="cuda") != 1
        assert torch.equal(Y[rest], clean[rest])


@pytest.mark.parametrize("name,c", [("bf16", 1.0 / 3), ("f16", 1.0 / 3), ("f16", 3e4), ("f16", 1e-7), ("f16", -7e-5), ("bf16", 1e-39)])
@pytest.mark.parametrize("K,N,r", [(264, 2056, 16), (4104, 2056, 96)])
def test_the_adapter_is_scaled_alike_on_every_path(K, N, r, name, c):
    """A row's adapter term does not depend on the rows beside it: c multiplies the fp32 sum
    Z B, and neither c B nor c Z is rounded to 16 bits (c B here passes fp16's largest
    number, or its normal numbers).  W is zero and Z B whole numbers, so Y = RNE(fl32(c) Z B)
    with one rounding to fp32 before it."""
    import torch
    say(f"mx adapter scaled by {c} {name} K={K} r={r}")
    rng = np.random.default_rng(K + r)
    M = 1100
    x = np.zeros((M, K), dtype=np.float32)
    x[:, 7] = rng.integers(-2, 3, size=M)
    x[:, 40] = rng.integers(-900, 900, size=M) // 4 * 4 * (rng.random(M) < 0.5)
    a = np.zeros((K, r), dtype=np.float32)
    a[7, 0] = a[40, 1] = a[7, r - 1] = 1.0
    b = rng.integers(-3, 4, size=(r, N)).astype(np.float32)
    X, A, B = (_dev(v, name) for v in (x, a, b))
    W = qn.mxfp4_quantize(torch.zeros(N, K, device="cuda"))
    x = host(X).astype(np.float64)
    with np.errstate(over="ignore", under="ignore"):
        want = oo.round16((np.float32(c) * (x @ a @ b).astype(np.float32)).astype(np.float32), name)
    for rows in (3, 16, 40, 100, M):      # in the product, waves with chunks of their own, panels, tiles
        Y, Z = qn.qlora_mx_linear_fwd(X[:rows].contiguous(), W, A, B, c)
        np.testing.assert_array_equal(host(Z), x[:rows] @ a)
        np.testing.assert_array_equal(host(Y), want[:rows], err_msg=f"{rows} rows")


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("r", [8, 32, 40, 64, 72, 128, 136, 200, 256])
@pytest.mark.parametrize("M,K,N", [(1100, 264, 2056), (257, 2056, 8264)])
def test_every_rank_by_tiles_in_whole_numbers(M, K, N, r, name):
    """The adapter's products in parts of 64, the last one of 32 or less: with whole numbers
    and c = 1/2 every sum is exact."""
    import torch
    from tests.test_gpu_mxfp4 import _whole
    say(f"mx tiles M={M} K={K} N={N} r={r} {name}")
    rng = np.random.default_rng(M + r)
    codes, scales = _whole(rng, N, K, 0, 0)
    W, w = _state(codes, scales, K), oo.mxfp4_values(codes, scales, K)
    x = rng.integers(-2, 3, size=(M, K)).astype(np.float32)
    x[:, ::32] = 2.0          # every block's scale is 1/2, and -2 .. 2 are kept as they are
    a = np.zeros((K, r), dtype=np.float32)
    a[rng.integers(0, K, size=r), np.arange(r)] = rng.choice([-1.0, 1.0], size=r)
    b = rng.integers(-3, 4, size=(r, N)).astype(np.float32)
    Y, Z = qn.qlora_mx_linear_fwd(_dev(x, name), W, _dev(a, name), _dev(b, name), 0.5)
    z = x.astype(np.float64) @ a
    np.testing.assert_array_equal(host(Z), z)
    np.testing.assert_array_equal(host(Y), oo.round16(x @ w.T + 0.5 * (z @ b), name))
