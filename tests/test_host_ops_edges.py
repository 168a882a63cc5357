"""References of the operators around the NF4 layer at infinite values, and
refusals and workspace sizes at the ends of their ranges.  No GPU work is issued."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo


def test_head_reference_with_infinite_logits():
    X = np.array([[1.0, 2.0], [-1.0, 2.0], [1.0, 0.5], [-1.0, 1.0]])
    W = np.array([[np.inf, 0.0], [1.0, 1.0], [0.0, -1.0]])
    # logits: row 0 (inf, 3, -2), row 1 (-inf, 1, -2), row 2 (inf, 1.5, -0.5), row 3 (-inf, 0, -1)
    with np.errstate(invalid="ignore"):
        loss, lse, dX = oo.head_loss(X, W, np.array([0, 0, 1, 1]))
    assert np.isnan(loss[0]) and np.isposinf(lse[0]) and np.isposinf(loss[1]) and np.isposinf(loss[2])
    np.testing.assert_allclose(lse[[1, 3]], [1 + np.log1p(np.exp(-3.0)), np.log1p(np.exp(-1.0))], rtol=1e-12)
    np.testing.assert_allclose(loss[3], np.log1p(np.exp(-1.0)), rtol=1e-12)


def test_fp16_checkpoints_round_alike_once_and_twice():
    """RNE_16(fl32(q step)) = RNE_16(q step) for every fp16 magnitude and code, so a
    kernel may convert the product directly."""
    a = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float32)
    step = (a / np.float32(127)).astype(np.float64)
    for q in range(1, 128):
        p = q * step          # exact: 7 and 24 bits
        with np.errstate(over="ignore"):
            np.testing.assert_array_equal(p.astype(np.float32).astype(np.float16), p.astype(np.float16))


def test_head_workspace_of_the_loss_alone():
    """Without the gradient nothing of size M x V is kept: bounds and sums of a piece
    (64 MiB, or a pair for each row and 128 of 256 columns), partials, a few values a row."""
    for M in (1, 333, 4096, 5003, 131072, 1 << 20):
        for K in (8, 256, 4096):
            if M * K >= 1 << 29:
                continue
            for V in (1, 50257, 128256, 1 << 24):
                n = qn.qlora_head_workspace_bytes(M, K, V, need_dx=False)
                assert n <= max(64 << 20, M * 16) + (256 << 20) + 64 * M + 4096, (M, K, V, n)
                assert n <= qn.qlora_head_workspace_bytes(M, K, V), (M, K, V)


def _host_tensors_pass(monkeypatch):
    """The wrappers' other checks on host tensors: no launch is reached."""
    def check(t, name, dtype=None):
        if not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
            raise ValueError(name)
    monkeypatch.setattr(qn, "_require_cuda", check)


def test_linear_backward_refuses_gradients_of_another_type_or_size(monkeypatch):
    """dA and dB are fp32 unless grad_dtype says otherwise: a 16-bit tensor would be
    written past its end."""
    torch = pytest.importorskip("torch")
    _host_tensors_pass(monkeypatch)
    b, M, K, N, r = torch.bfloat16, 4, 64, 128, 8
    z = lambda *s, t=b: torch.zeros(*s, dtype=t)
    state = qn.NF4State(K * N, *[torch.zeros(1)] * 4)
    f = torch.float32
    for kw in ({"dA": z(K, r)}, {"dB": z(r, N)}, {"dA": z(K, r - 1, t=f)}, {"dB": z(r, N // 2, t=f)}, {"dX": z(M, K, t=f)},
               {"dX": z(M - 1, K)}, {"dA": z(K, r), "grad_dtype": f}, {"dA": z(2 * K, r, t=f)[::2]}):
        with pytest.raises(ValueError, match="dA|dB|dX"):
            qn.qlora_linear_bwd(z(M, N), z(M, K), z(M, r), state, z(K, r), z(r, N), 1.0, K, N, **kw)


def _state(torch, K, N, single=False, **change):
    P = K * N
    n1, n2 = P // 64, (P // 64 + 255) // 256
    z = torch.zeros
    parts = {"codes": z(P // 2, dtype=torch.uint8), "qabsmax": z(n1, dtype=torch.int8), "absmax2": z(n2),
             "offset": z(1), "absmax": None}
    if single:
        parts |= {"qabsmax": None, "absmax2": None, "offset": None, "absmax": z(n1)}
    return qn.NF4State(P, **(parts | change))


def test_calls_refuse_states_that_are_not_their_weights(monkeypatch):
    """A tensor of a state that is too short, of another type, strided, missing or on
    another device would be read past its end."""
    torch = pytest.importorskip("torch")
    _host_tensors_pass(monkeypatch)
    b, M, K, F, r = torch.bfloat16, 4, 192, 128, 8
    z = lambda *s, t=b: torch.zeros(*s, dtype=t)
    X, A, B, dH, Z = z(M, K), z(K, 2 * r), z(r, 2 * F), z(M, F), z(M, 2 * r)
    good = _state(torch, K, F)
    n1 = K * F // 64
    assert good.check("x", X.device) is None and _state(torch, K, F, single=True).check("x", X.device) is None
    bad = [{"codes": z(K * F // 2 - 1, t=torch.uint8)}, {"codes": z(K * F // 2, t=torch.int8)}, {"qabsmax": None},
           {"qabsmax": z(n1 - 1, t=torch.int8)}, {"qabsmax": z(n1)}, {"absmax2": z(1)}, {"absmax2": z(4, t=torch.float32)[::2]},
           {"offset": z(0, t=torch.float32)}, {"offset": None}, {"absmax": z(n1 - 1, t=torch.float32)}, {"absmax": z(n1)},
           {"offset": torch.empty(1, device="meta")}]
    for change in bad:
        wrong = _state(torch, K, F, **change)
        for states in ([wrong, good], [good, wrong]):
            with pytest.raises(ValueError, match=r"states\[[01]\]"):
                qn.qlora_gated_fwd(X, states, A, B, 1.0, K, F)
            with pytest.raises(ValueError, match=r"states\[[01]\]"):
                qn.qlora_gated_bwd(dH, X, Z, None, states, A, B, 1.0, K, F)
        with pytest.raises(ValueError, match="state"):
            qn.qlora_linear_bwd(z(M, F), X, z(M, r), wrong, z(K, r), z(r, F), 1.0, K, F, grad_dtype=b)
    for ws in (z(1 << 20), z(1 << 20, t=torch.uint8)[::2], z(1, t=torch.uint8).expand(1 << 20)):
        with pytest.raises(ValueError, match="workspace"):
            qn._workspace(ws, 256, X.device)
