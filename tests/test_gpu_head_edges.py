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
