"""Host-side refusals of the MXFP4 calls, and their reference against values worked
out by hand.  No GPU work is issued."""
import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo

C = ctypes.c_float(1.0)


def _mx(rows=64, cols=64, codes=0x1000, scales=0x2000):
    return ctypes.byref(qn._Mx(rows, cols, codes, scales))


BAD_STATES = [None, _mx(codes=None), _mx(scales=None), _mx(codes=0x1008), _mx(scales=0x2004), _mx(rows=0), _mx(cols=0),
              _mx(cols=12), _mx(rows=1 << 26), _mx(rows=1 << 40, cols=1 << 30)]


def _refused(call, ok, changes):
    for change in changes:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert call(*args) == qn.NF4_EINVAL, change


def test_sizes():
    for rows, cols in [(1, 8), (1, 32), (17, 40), (16, 512), (33, 520), (22016, 8192)]:
        blocks = -(-cols // 32)
        assert qn.mxfp4_sizes(rows, cols) == (rows * blocks * 16, -(-rows // 16) * -(-blocks // 16) * 256)
    for rows, cols in [(0, 8), (1, 0), (1, 4), (1, 12), (1 << 26, 8), (8, 1 << 26), (1 << 40, 1 << 40), (-1, 8)]:
        with pytest.raises(qn.NF4Error):
            qn.mxfp4_sizes(rows, cols)


def test_quantize_refusals():
    L = qn.lib()
    for transposed in (0, 1):
        ok = [1, transposed, 0x100, 64, _mx(), None]
        bad = [{0: 3}, {0: -1}, {2: None}, {2: 0x108}, {3: 56}, {3: 68}, {3: 1 << 26}, {3: 1 << 62}] + [{4: s} for s in BAD_STATES]
        _refused(L.mxfp4_quantize, ok, bad)
        for change in bad:      # (type, transposed, in, X, ld)
            args = list(ok)
            for i, v in change.items():
                args[i] = v
            args[2], args[3], args[4] = args[4], args[2], args[3]
            assert L.mxfp4_dequantize(*args) == qn.NF4_EINVAL, change
    _refused(L.mxfp4_quantize, [1, 1, 0x100, 72, _mx(rows=65), None], [{}])      # rows % 8 across


def test_matmul_refusals():
    L = qn.lib()
    n = ctypes.c_int64()
    for shape in [(0, 64, 64), (4, 60, 64), (4, 0, 64), (4, 64, 12), (4, 64, 0), ((1 << 20) + 1, 64, 8),
                  (1 << 20, 512, 8), (4, (1 << 24) + 8, 8), (8, 64, 1 << 26)]:
        assert L.mxfp4_matmul_workspace_bytes(*shape, ctypes.byref(n)) == qn.NF4_EINVAL, shape
    assert L.mxfp4_matmul_workspace_bytes(4, 64, 64, ctypes.byref(n)) == qn.NF4_OK
    ok = [1, _mx(rows=5), _mx(), 0x100, 0x10000, 1 << 30, None]
    _refused(L.mxfp4_matmul, ok, [{0: 3}, {1: _mx(cols=32)}, {2: _mx(cols=32)}, {2: _mx(rows=60)}, {3: None}, {3: 0x108},
                                  {4: None}, {4: 0x10080}, {5: -1}] + [{1: s} for s in BAD_STATES] + [{2: s} for s in BAD_STATES])


def test_layer_refusals():
    L = qn.lib()
    f, b = ctypes.c_int64(), ctypes.c_int64()
    for shape in [(0, 64, 64, 8), (4, 12, 64, 8), (4, 64, 60, 8), (4, 64, 0, 8), (4, 64, 64, 4), (4, 64, 64, 264),
                  (1 << 20, 512, 64, 8), (4, 1 << 15, 1 << 14, 8), (1 << 16, 64, 1 << 13, 8), (1, 8, 1 << 21, 256),
                  (1, 1 << 21, 64, 256)]:
        assert L.qlora_mx_workspace_bytes(*shape, ctypes.byref(f), ctypes.byref(b)) == qn.NF4_EINVAL, shape
    assert L.qlora_mx_workspace_bytes(4, 64, 72, 8, ctypes.byref(f), ctypes.byref(b)) == qn.NF4_OK
    wrong = [{"s": s} for s in BAD_STATES + [_mx(rows=32), _mx(cols=32)]]
    #     dt M  K   N   r  X      W      A      B      c  Y      Z      ws       bytes    stream
    ok = [0, 4, 64, 64, 8, 0x100, _mx(), 0x200, 0x300, C, 0x400, 0x500, 0x10000, 1 << 30, None]
    _refused(L.qlora_mx_linear_fwd, ok, [{0: 2}, {1: 0}, {2: 72}, {3: 72}, {4: 12}, {5: None}, {5: 0x108}, {7: None}, {7: 0x208},
                                         {8: None}, {8: 0x302}, {10: None}, {10: 0x404}, {11: 0x502}, {12: None},
                                         {12: 0x10010}, {13: 0}] + [{6: w["s"]} for w in wrong])
    a8 = ctypes.byref(qn._Act8(0x1000, 0x2000))
    #     dt grad M K   N   r  G      X      X8    Z      W      A      B      c  dX    dA     dB     ws       bytes    stream
    ok = [0, 1, 4, 64, 64, 8, 0x100, 0x110, None, 0x300, _mx(), 0x400, 0x500, C, None, 0x600, 0x700, 0x10000, 1 << 30, None]
    _refused(L.qlora_mx_linear_bwd, ok, [{0: 2}, {1: 2}, {1: 5}, {0: 1, 1: 0}, {6: None}, {6: 0x108}, {7: None}, {8: a8}, {7: 0x118},
                                         {7: None, 8: ctypes.byref(qn._Act8(None, 0x2000))}, {9: None}, {9: 0x302}, {11: None},
                                         {12: 0x508}, {14: 0x604}, {15: None}, {15: 0x608}, {16: None}, {17: None},
                                         {17: 0x10010}, {18: 0}] + [{10: w["s"]} for w in wrong])


def test_reference_by_hand():
    x = np.zeros((3, 40), dtype=np.float32)
    x[0, :9] = [4.0, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, -5.0, 7.0]     # scale 1; ties go to the even code
    x[0, 32:35] = [-3.0, 0.0, 2.0 ** -40]                               # the short last block, scale 1/2
    x[1, 5] = np.inf
    x[2, 0] = 2.0 ** -149
    codes, scales = oo.mxfp4_quantize(x)
    assert codes[0, :9].tolist() == [6, 0, 2, 8 + 2, 4, 4, 6, 8 + 6, 7]
    assert codes[0, 32:35].tolist() == [8 + 7, 0, 0] and scales.tolist() == [[127, 126], [255, 0], [0, 0]]
    v = oo.mxfp4_values(codes, scales, 40)
    assert v[0, :9].tolist() == [4, 0, 1, -1, 2, 2, 4, -4, 6] and v[0, 32] == -3.0
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all() and v[2, 0] == 0.0
    tiled = oo.mxfp4_tiled(scales)
    assert tiled.size == 256 and (tiled[0], tiled[64], tiled[4], tiled[68], tiled[8]) == (127, 126, 255, 0, 0)


def test_reference_is_the_nearest_value():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((40, 96)) * 10.0 ** rng.integers(-3, 3, size=(40, 1))
    codes, scales = oo.mxfp4_quantize(x)
    v, s = oo.mxfp4_values(codes, scales, 96), np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    grid = np.concatenate((oo.E2M1, -oo.E2M1))
    best = np.min(np.abs(np.clip(x / s, -6, 6)[:, :, None] - grid), axis=2) * s
    assert np.abs(np.abs(np.clip(x, -6 * s, 6 * s) - v) - best).max() <= 1e-12 * np.abs(x).max()
    top = np.abs(x).reshape(40, 3, 32).max(axis=2)
    scale = s[:, ::32]
    assert (4 * scale <= top).all() and (top < 8 * scale).all()


def test_reference_gradients_match_differences():
    """With values that four bits hold, so that quantising X changes nothing at the
    point itself: dX, dA and dB are the derivatives of X Wᵀ + c X A B."""
    rng = np.random.default_rng(4)
    M, K, N, r, c, h = 3, 8, 5, 2, 0.7, 1e-5
    X = rng.choice([-6.0, -1.5, 0.5, 2.0, 4.0], size=(M, K))
    X[:, 0] = 4.0
    W, A, B, G = (rng.standard_normal(s) for s in ((N, K), (K, r), (r, N), (M, N)))
    Y, Z = oo.mx_linear_forward(X, W, A, B, c)
    np.testing.assert_allclose(Y, X @ W.T + c * (X @ A @ B), rtol=1e-12)
    for v, g in zip((X, A, B), oo.mx_linear_backward(G, X, Z, W, A, B, c)):
        for i in np.ndindex(v.shape):
            at, d = v[i], []
            for s in (h, -h):
                v[i] = at + s
                d.append(np.sum(G * (X @ W.T + c * (X @ A @ B))))
            v[i] = at
            assert abs((d[0] - d[1]) / (2 * h) - g[i]) <= 1e-6 * (1 + abs(g[i]))


def test_wrappers_refuse_before_a_launch():
    torch = pytest.importorskip("torch")
    b = torch.bfloat16
    x = torch.zeros(8, 64, dtype=b)
    kept = qn.MXFP4(8, 64, torch.zeros(8 * 32, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8))
    for call in (lambda: qn.mxfp4_quantize(x), lambda: qn.mxfp4_quantize(x.double()), lambda: qn.mxfp4_dequantize(kept),
                 lambda: qn.mxfp4_matmul(kept, kept),
                 lambda: qn.qlora_mx_linear_fwd(x, kept, x[:, :8], x, C), lambda: qn.qlora_mx_linear_fwd(x.float(), kept, x, x, C),
                 lambda: qn.qlora_mx_linear_bwd(x, x, x, kept, x, x, C)):
        with pytest.raises(ValueError):
            call()


def test_workspaces_over_the_whole_range():
    for M in (1, 16, 17, 64, 129, 256, 700, 4096, 1 << 20):
        for K in (8, 72, 520, 4096, 1 << 16, 1 << 20):
            for N in (8, 264, 22016, 1 << 20):
                if M * K >= 1 << 29 or M * N >= 1 << 29 or K * N >= 1 << 29:
                    continue
                for r in (8, 256):
                    if K * r >= 1 << 29 or N * r >= 1 << 29:
                        continue
                    fwd, bwd = qn.qlora_mx_workspace_bytes(M, K, N, r)
                    assert 0 < fwd < 1 << 34 and 0 < bwd < 1 << 34, (M, K, N, r)
                assert 0 <= qn.mxfp4_matmul_workspace_bytes(M, N, K) < 1 << 34


def test_backward_without_z_says_so():
    """return_z=False keeps Z from the caller, and the backward does not form it again."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    kept = qn.MXFP4(8, 64, torch.zeros(8 * 32, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="Z is required"):
        qn.qlora_mx_linear_bwd(x[:, :8].contiguous(), x, None, kept, x.T.contiguous(), x[:, :8].contiguous(), C)
