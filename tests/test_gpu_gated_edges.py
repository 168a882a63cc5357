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
