"""The head loss where its inputs are least kind: what lies behind them in
memory, infinite logits, long token lists."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from tests.gpu_util import host, say
from tests.test_gpu_head import _case, _compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,V", [(1, 64, 1), (3, 136, 129), (40, 520, 1000), (300, 264, 1024), (300, 264, 4099),
                                   (700, 2056, 1537), (1500, 8, 90001)])
def test_nothing_behind_the_inputs_is_used(M, K, V):
    """W and X are the first rows of larger matrices whose other rows are NaN:
    a value from behind either would meet a zero and still spoil a sum."""
    import torch
    say(f"head, NaN behind W M={M} K={K} V={V}")
    X, W, t, w = _case(M, K, V, "bf16", M + V)
    want = [host(v).copy() for v in qn.qlora_head_loss(X, W, t, weights=w)]
    big_w = torch.full((V + 300, K), float("nan"), dtype=W.dtype, device="cuda")
    big_x = torch.full((M + 300, K), float("nan"), dtype=W.dtype, device="cuda")
    big_w[:V], big_x[:M] = W, X
    got = qn.qlora_head_loss(big_x[:M], big_w[:V], t, weights=w)
    for g, v in zip(got, want):
        np.testing.assert_array_equal(host(g), v)
    rows = np.arange(min(M, 60))
    _compare(X, W, t, w, got, "bf16", rows)


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("K,V", [(136, 700), (2056, 700)])
def test_infinite_logits(K, V, name):
    """One entry of the head is +inf: its logit is +inf or -inf by the sign that a
    row has there.  Short K whole, long K summed from partials."""
    say(f"head, infinite logits K={K} {name}")
    M, v, col = 40, 5, 3
    X, W, t, _ = _case(M, K, V, name, 21)
    t[:] = (t.abs() * 7 + 11) % V
    t[t == v] = v + 1
    t[0:4] = v
    sign = np.where(np.arange(M) % 2 == 0, 1.0, -1.0)
    X[:, col] = X[:, col].abs().clamp(min=0.5)
    X[1::2, col] *= -1
    W[v, col] = float("inf")
    got = [host(g).astype(np.float64) for g in qn.qlora_head_loss(X, W, t)]
    alone = [host(g).astype(np.float64) for g in qn.qlora_head_loss(X, W, t, need_dx=False)[:2]]
    x, w64, tt = host(X).astype(np.float64), host(W).astype(np.float64), host(t)
    s = x @ np.delete(w64, v, axis=0).T
    top = s.max(axis=1)
    rest = np.log(np.exp(s - top[:, None]).sum(axis=1)) + top          # without the infinite one
    target = np.where(tt == v, sign * np.inf, (x * np.where(np.isinf(w64), 0, w64)[tt]).sum(axis=1))
    up, hit = sign > 0, tt == v
    tol = (K + 40) * 2.0 ** -24 * (np.abs(x) @ np.abs(np.delete(w64, v, axis=0)).T).max(axis=1) + 1e-5
    for loss, lse in (got[:2], alone):
        assert np.isnan(loss[up]).all() and not np.isfinite(lse[up]).any()
        assert np.isposinf(lse[up & hit]).all()
        assert np.isposinf(loss[~up & hit]).all()
        assert (np.abs(lse - rest)[~up] <= tol[~up]).all()
        fine = ~up & ~hit
        assert (np.abs(loss[fine] - (rest - target)[fine]) <= 2 * tol[fine]).all()
    assert np.isnan(got[2][up]).all()
    others = np.delete(got[2], col, axis=1)
    assert np.isfinite(others[~up]).all()


@pytest.mark.parametrize("M,K,V,name", [(40000, 16, 40007, "bf16"), (5003, 72, 300001, "f16")])
def test_loss_alone_in_pieces(M, K, V, name):
    """Many tokens: the bounds and sums of a piece end at 64 MiB, here two of them."""
    import torch
    say(f"head, loss alone in pieces M={M} V={V} {name}")
    X, W, t, w = _case(M, K, V, name, 12, lean=8.0)
    edge = np.concatenate((np.arange(0, V, V // 40), [V - 1]))
    t[:len(edge)] = torch.from_numpy(edge).cuda()
    got = qn.qlora_head_loss(X, W, t, weights=w, need_dx=False)
    _compare(X, W, t, w, got, name, np.arange(len(edge) + 20))
    _compare(X, W, t, w, got, name, np.arange(M - 40, M))
