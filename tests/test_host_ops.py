"""Host-side refusals of the operators around the NF4 layer, and their
references against formulas worked out by hand.  No GPU work is issued."""
import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo

C = ctypes.c_float(1.0)


def _a8(codes=0x1000, absmax=0x2000):
    return ctypes.byref(qn._Act8(codes, absmax))


def test_act8_refusals():
    L = qn.lib()
    ok = [0, 4, 64, 0x100, 64, _a8(), None]
    bad = [(0, 2), (0, -1), (1, 0), (2, 0), (2, 12), (3, None), (3, 0x108), (4, 56), (4, 68), (5, None),
           (5, _a8(codes=None)), (5, _a8(absmax=None)), (5, _a8(codes=0x1008)), (5, _a8(absmax=0x2001)),
           (1, 1 << 26), (4, 1 << 29)]
    for i, v in bad:
        args = list(ok)
        args[i] = v
        assert L.act8_encode(*args) == qn.NF4_EINVAL, (i, v)
        args[3], args[4], args[5] = args[5], args[3], args[4]      # decode: (in, X, ld)
        assert L.act8_decode(*args) == qn.NF4_EINVAL, (i, v)


def test_linear_bwd_ex_refusals():
    L = qn.lib()
    st = qn._State(64 * 64, 0x1000, 0x2000, 0x3000, 0x4000)
    #      dt grad M  K   N   r  G      X      X8     Z      W                 A      B      c  dX    dA     dB     ws       bytes    stream
    ok = [0, 1, 4, 64, 64, 8, 0x100, None, _a8(), 0x300, ctypes.byref(st), 0x400, 0x500, C, None, 0x600, 0x700, 0x10000, 1 << 30, None]
    bad = [{0: 2}, {1: 2}, {1: 5}, {0: 1, 1: 0}, {7: 0x100}, {8: None}, {9: None}, {8: _a8(codes=0x1004)}, {6: None},
           {15: None}, {16: 0x708}, {18: 0}, {3: 32}, {4: 32}, {17: 0x10010}, {14: 0x604}]
    for change in bad:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert L.qlora_linear_bwd_ex(*args) == qn.NF4_EINVAL, change


def test_act8_reference_by_hand():
    x = np.zeros((2, 72), dtype=np.float32)
    x[0, :5] = [127.0, 0.5, 1.5, -2.5, 126.5]     # ties go to the even code
    x[0, 64:67] = [-2.0, 1.0, 0.0]                # the short last block
    x[1, 3] = np.inf
    codes, absmax = oo.act8_encode(x)
    assert codes[0, :5].tolist() == [127, 0, 2, -2, 126]
    assert codes[0, 64:67].tolist() == [-127, 64, 0]          # 63.5 -> 64
    assert absmax[0].tolist() == [127.0, 2.0] and np.isnan(absmax[1, 0]) and absmax[1, 1] == 0.0
    back = oo.act8_decode(codes, absmax, "bf16")
    assert back[0, 0] == 127.0 and back[0, 64] == -2.0 and np.isnan(back[1, :64]).all() and (back[1, 64:] == 0).all()


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_act8_reference_keeps_the_largest_and_half_a_step(name):
    rng = np.random.default_rng(1)
    x = oo.round16(rng.standard_normal((50, 200)) * 10.0 ** rng.integers(-3, 3, size=(50, 1)), name)
    codes, absmax = oo.act8_encode(x)
    back = oo.act8_decode(codes, absmax, name)
    a = np.repeat(absmax, 64, axis=1)[:, :200]
    at = np.abs(x) == a
    np.testing.assert_array_equal(back[at], x[at])
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[name]
    assert (np.abs(back - x) <= a / 254 * (1 + 1e-6) + half * np.abs(x) + half * a / 254 + (2.0 ** -25 if name == "f16" else 0)).all()


def test_act8_wrappers_refuse_before_a_launch():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qn.act8_encode(x)                              # not a device tensor
    with pytest.raises(ValueError):
        qn.act8_encode(x.float())
    kept = qn.Act8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qn.act8_decode(kept)


def test_gated_refusals():
    L = qn.lib()
    i64 = ctypes.c_int64
    f, b = i64(), i64()
    for shape in [(0, 64, 64, 8), (4, 12, 64, 8), (4, 64, 96, 8), (4, 64, 0, 8), (4, 64, 64, 4), (4, 64, 64, 136),
                  (1 << 20, 64, 256, 8), (4, 1 << 15, 1 << 13, 8)]:
        assert L.qlora_gated_workspace_bytes(*shape, ctypes.byref(f), ctypes.byref(b)) == qn.NF4_EINVAL, shape
    assert L.qlora_gated_workspace_bytes(4, 64, 64, 8, ctypes.byref(f), ctypes.byref(b)) == qn.NF4_OK
    states = (qn._State * 2)(*[qn._State(64 * 64, 0x1000, 0x2000, 0x3000, 0x4000)] * 2)
    short = (qn._State * 2)(qn._State(64 * 64, 0x1000, 0x2000, 0x3000, 0x4000),
                            qn._State(64 * 32, 0x1000, 0x2000, 0x3000, 0x4000))
    #      dt act M  K   F   r  X      W       A      B      c  H      Z      GU    GU8   ws       bytes    stream
    ok = [0, 0, 4, 64, 64, 8, 0x100, states, 0x200, 0x300, C, 0x400, 0x500, None, None, 0x10000, 1 << 30, None]
    for change in [{0: 2}, {1: 2}, {1: -1}, {6: None}, {7: None}, {7: short}, {8: 0x208}, {11: None}, {12: 0x502},
                   {13: 0x600, 14: _a8()}, {13: 0x608}, {14: _a8(codes=0x1004)}, {15: None}, {15: 0x10080}, {16: 0},
                   {4: 96}, {5: 12}]:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert L.qlora_gated_fwd(*args) == qn.NF4_EINVAL, change
    #      dt act grad M  K   F   r  dH     X      X8    Z      GU     GU8   W       A      B      c  dX    dA     dB     ws       bytes    stream
    ok = [0, 0, 1, 4, 64, 64, 8, 0x100, 0x110, None, 0x120, 0x130, None, states, 0x200, 0x300, C, None, 0x400, 0x500, 0x10000, 1 << 30, None]
    for change in [{0: 2}, {1: 2}, {2: 2}, {7: None}, {8: None}, {9: _a8()}, {10: None}, {12: _a8()}, {13: short},
                   {8: None, 9: _a8(), 11: None}, {8: None, 9: _a8(absmax=None)}, {11: 0x132}, {17: 0x408}, {18: None},
                   {19: 0x504}, {20: 0x10010}, {21: 0}]:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert L.qlora_gated_bwd(*args) == qn.NF4_EINVAL, change


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_reference_gradients_match_differences(name):
    rng = np.random.default_rng(4)
    M, K, F, r, c, h = 3, 5, 4, 2, 0.7, 1e-5
    X, Wg, Wu = rng.standard_normal((M, K)), rng.standard_normal((K, F)), rng.standard_normal((K, F))
    A, B, dH = rng.standard_normal((K, 2 * r)), rng.standard_normal((r, 2 * F)), rng.standard_normal((M, F))
    _, Z, G, U = oo.gated_forward(X, Wg, Wu, A, B, c, name)
    grads = oo.gated_backward(dH, X, Z, G, U, Wg, Wu, A, B, c, name)
    for v, g in zip((X, A, B), grads):
        for i in np.ndindex(v.shape):
            at, d = v[i], []
            for s in (h, -h):
                v[i] = at + s
                d.append(np.sum(dH * oo.gated_forward(X, Wg, Wu, A, B, c, name)[0]))
            v[i] = at
            assert abs((d[0] - d[1]) / (2 * h) - g[i]) <= 1e-6 * (1 + abs(g[i]))


def test_head_reference_gradient_matches_differences():
    rng = np.random.default_rng(6)
    M, K, V, h = 4, 5, 7, 1e-6
    X, W, t, w = rng.standard_normal((M, K)), rng.standard_normal((V, K)), np.array([3, -100, 0, 6]), rng.random(M)
    loss, lse, dX = oo.head_loss(X, W, t, w)
    assert loss[1] == 0 and not dX[1].any() and np.isfinite(lse).all()
    for i in np.ndindex(X.shape):
        at, d = X[i], []
        for s in (h, -h):
            X[i] = at + s
            d.append(np.sum(oo.head_loss(X, W, t, w)[0]))
        X[i] = at
        assert abs((d[0] - d[1]) / (2 * h) - dX[i]) <= 1e-7


def test_head_refusals():
    L = qn.lib()
    n = ctypes.c_int64()
    for shape in [(0, 64, 10), (4, 12, 10), (4, 0, 10), (4, 64, 0), ((1 << 20) + 1, 64, 10), (1 << 20, 512, 10),
                  (4, (1 << 20) + 8, 10), (4, 64, (1 << 24) + 1)]:
        assert L.qlora_head_workspace_bytes(*shape, 1, ctypes.byref(n)) == qn.NF4_EINVAL, shape
    assert L.qlora_head_workspace_bytes(4, 64, 10, 1, ctypes.byref(n)) == qn.NF4_OK
    #     dt M  K   V   X      W      targets weights ignore loss   lse   dX     ws       bytes    stream
    ok = [0, 4, 64, 10, 0x100, 0x200, 0x300, None, -100, 0x400, None, 0x500, 0x10000, 1 << 30, None]
    for change in [{0: 2}, {1: 0}, {2: 12}, {3: 0}, {4: None}, {4: 0x108}, {5: None}, {6: None}, {6: 0x304}, {7: 0x302},
                   {9: None}, {9: 0x402}, {10: 0x602}, {11: 0x508}, {12: None}, {12: 0x10010}, {13: 16}]:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert L.qlora_head_loss(*args) == qn.NF4_EINVAL, change


def test_head_workspace_is_bounded_by_its_pieces():
    small = qn.qlora_head_workspace_bytes(4096, 4096, 32000)
    # twice the vocabulary costs no more probabilities, only the sums of the pieces
    large = qn.qlora_head_workspace_bytes(4096, 4096, 256000)
    assert small <= (256 << 20) + (32 << 20) and large <= small + 4096 * 4096 * 4 + (32 << 20)
    assert qn.qlora_head_workspace_bytes(4096, 4096, 256000, need_dx=False) < 128 << 20


def test_gated_and_head_wrappers_refuse_before_a_launch():
    torch = pytest.importorskip("torch")
    b = torch.bfloat16
    X, A, B, dH = (torch.zeros(*s, dtype=b) for s in ((4, 64), (64, 16), (8, 128), (4, 64)))
    state = qn.NF4State(64 * 64, *[torch.zeros(1)] * 4)
    for kw in ({"act": "relu"}, {"save": "4"}, {"save": 8}):
        with pytest.raises(ValueError, match="one of|save"):
            qn.qlora_gated_fwd(X, [state] * 2, A, B, C, 64, 64, **kw)
    with pytest.raises(ValueError, match="two states"):
        qn.qlora_gated_fwd(X, [state], A, B, C, 64, 64)
    with pytest.raises(ValueError, match="2r"):
        qn.qlora_gated_fwd(X, [state] * 2, A[:, :15], B, C, 64, 64)
    with pytest.raises(ValueError, match="compute type"):
        qn.qlora_gated_fwd(X.float(), [state] * 2, A, B, C, 64, 64)
    with pytest.raises(ValueError):                    # not device tensors
        qn.qlora_gated_fwd(X, [state] * 2, A, B, C, 64, 64)
    with pytest.raises(ValueError):
        qn.qlora_gated_bwd(dH, X, A, None, [state] * 2, A, B, C, 64, 64)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        qn.qlora_head_loss(X, torch.zeros(9, 64, dtype=b), t)
    with pytest.raises(ValueError, match="compute type"):
        qn.qlora_head_loss(X.float(), torch.zeros(9, 64), t)
    assert qn._grad_code(None, b) == (torch.float32, qn.NF4_AB_F32)
    assert qn._grad_code(b, b) == (b, qn.NF4_AB_BF16)
    with pytest.raises(ValueError, match="grad_dtype"):
        qn._grad_code(torch.float16, b)


def test_workspaces_over_the_whole_range():
    """Every size the calls take has a workspace size that is counted in whole,
    positive 64-bit bytes, also where the split partials are largest."""
    for M in (1, 16, 17, 64, 256, 257, 700, 4096, 1 << 20):
        for K in (8, 72, 520, 4096, 1 << 16, 1 << 20):
            if M * K >= 1 << 29:
                continue
            for V in (1, 300, 70000, 1 << 24):
                for need in (False, True):
                    n = qn.qlora_head_workspace_bytes(M, K, V, need)
                    # probabilities, sums of a piece, partials and a few values a row
                    assert 0 < n < max(256 << 20, M * 512) + M * K * 4 + (256 << 20) + M * 64 + (1 << 20) + M * V // 8 + 256 * M, (M, K, V)
            for F in (64, 704, 22016, 1 << 20):
                if K * 2 * F >= 1 << 29 or M * 2 * F >= 1 << 29 or 16 * F >= 1 << 29:
                    continue
                fwd, bwd = qn.qlora_gated_workspace_bytes(M, K, F, 8)
                assert 0 < fwd < 1 << 33 and 0 < bwd < 1 << 34, (M, K, F)
