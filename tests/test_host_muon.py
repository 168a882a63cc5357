"""Host-side refusals of the orthogonalised adapter step, and its reference against the
singular values.  No GPU work is issued."""
import ctypes
import math

import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _options(**kw):
    o = dict(lr=0.02, momentum=0.95, weight_decay=0.0, eps=1e-7, a=3.4, b=-4.7, c=2.0, steps=5, nesterov=1, scaling=1)
    o.update(kw)
    return ctypes.byref(qn._Muon(*o.values()))


def test_refusals():
    L = qn.lib()
    n = ctypes.c_int64()
    for shape in [(0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 4, 257), ((1 << 24) + 1, 4, 1), (1 << 22, 4, 128), (4, 1 << 22, 128)]:
        assert L.qlora_muon_workspace_bytes(*shape, ctypes.byref(n)) == qn.NF4_EINVAL, shape
    assert L.qlora_muon_workspace_bytes(7, 5, 3, ctypes.byref(n)) == qn.NF4_OK and n.value > 0
    #     pdt gdt K  N  r  A      B      dA     dB     mA     mB     MA    MB    options     ws       bytes    stream
    ok = [0, 1, 7, 5, 3, 0x102, 0x202, 0x304, 0x404, 0x504, 0x604, None, None, _options(), 0x10000, 1 << 30, None]
    bad = [{0: 2}, {1: 2}, {1: 3}, {0: 1, 1: 0}, {2: 0}, {3: 0}, {4: 0}, {4: 257}, {5: 0x103}, {6: 0x203}, {7: 0x302},
           {8: 0x402}, {9: 0x502}, {10: 0x602}, {11: 0x700}, {12: 0x700}, {11: 0x702, 12: 0x800}, {13: None}, {14: None},
           {14: 0x10080}, {15: 0}] + [{i: None} for i in range(5, 11)]
    for o in ({"lr": math.nan}, {"momentum": 1.0}, {"momentum": -0.1}, {"momentum": math.nan}, {"eps": 0.0}, {"eps": -1.0},
              {"weight_decay": math.inf}, {"a": math.nan}, {"b": math.inf}, {"c": math.nan}, {"steps": -1}, {"steps": 33},
              {"scaling": 3}, {"scaling": -1}):
        bad.append({13: _options(**o)})
    for change in bad:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert L.qlora_muon_step(*args) == qn.NF4_EINVAL, change
    # 16-bit gradients need 2 bytes' alignment alone, which is what is refused above for fp32's
    args = list(ok)
    args[1], args[7], args[4] = 0, 0x303, 3
    assert L.qlora_muon_step(*args) == qn.NF4_EINVAL


def test_wrapper_refuses_before_a_launch():
    torch = pytest.importorskip("torch")
    A, B = torch.zeros(8, 4, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    args = (A, B, A.float(), B.float(), A.float(), B.float(), 0.1)
    with pytest.raises(ValueError, match="scaling"):
        qn.qlora_muon_step(*args, scaling="adam")
    with pytest.raises(ValueError, match="device"):
        qn.qlora_muon_step(*args)
    with pytest.raises(ValueError, match="grad_dtype"):
        qn.qlora_muon_step(A, B, A.half(), B.half(), *args[4:])
    with pytest.raises(ValueError, match="compute type"):
        qn.qlora_muon_step(A.float(), *args[1:])


@pytest.mark.parametrize("shape", [(5, 5), (7, 3), (3, 11), (1, 4), (6, 1)])
def test_reference_changes_the_singular_values_alone(shape):
    rng = np.random.default_rng(3)
    u = rng.standard_normal(shape)
    left, sv, right = np.linalg.svd(u, full_matrices=False)
    sv = sv / np.sqrt(np.sum(sv * sv))
    for _ in range(5):
        sv = COEFFICIENTS[0] * sv + COEFFICIENTS[1] * sv ** 3 + COEFFICIENTS[2] * sv ** 5
    np.testing.assert_allclose(oo.newton_schulz(u, 5, COEFFICIENTS, 1e-7), (left * sv) @ right, atol=1e-10)


def test_reference_step_by_hand():
    # a single row of a single value: the iteration on 1 alone
    x = 1.0
    for _ in range(5):
        x = 3.4445 * x - 4.7750 * x ** 3 + 2.0315 * x ** 5
    p, m, o = oo.muon_step([[2.0]], [[4.0]], [[1.0]], 0.5, 0.75, True, 0.1, "spectral", 5, COEFFICIENTS, 1e-7)
    assert m[0, 0] == 0.75 + 0.25 * 4.0 and abs(o[0, 0] - x) < 1e-12 and abs(p[0, 0] - (2.0 * 0.95 - 0.5 * x)) < 1e-12
    _, m, o = oo.muon_step(np.ones((9, 4)), -np.ones((9, 4)), np.zeros((9, 4)), 0.1, 0.5, False, 0.0, "rms", 0, COEFFICIENTS, 1e-7)
    np.testing.assert_allclose(o, -1.0 / 6)
    p, _, _ = oo.muon_step(np.ones((9, 4)), -np.ones((9, 4)), np.zeros((9, 4)), 0.1, 0.5, False, 0.0, "rms", 0, COEFFICIENTS, 1e-7)
    np.testing.assert_allclose(p, 1 + 0.1 * 0.2 * 3 / 6)


def test_workspaces_over_the_whole_range():
    for K in (1, 17, 4096, 1 << 20, 1 << 24):
        for N in (1, 333, 22016, 1 << 24):
            for r in (1, 16, 31, 64, 65, 256):
                if K * r < 1 << 29 and N * r < 1 << 29:
                    assert 0 < qn.qlora_muon_workspace_bytes(K, N, r) < 1 << 34
