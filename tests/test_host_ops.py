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
