"""The output head's cross entropy and its gradient on the GPU against the
64-bit reference.  Bounds are elementwise: an fp32 logit is off by at most
(K + 2) 2^-24 sum |x w| =: e, so lse by e and a few fp32 steps; a probability
by 2 e and one rounding to 16 bits (d = half a step), the result by another."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25}
F32 = 2.0 ** -24


def _torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _dev(x, name):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(_torch_type(name)).cuda()


def _case(M, K, V, name, seed, lean=4.0):
    import torch
    rng = np.random.default_rng(seed)
    W = _dev(rng.standard_normal((V, K)) / np.sqrt(K), name)
    t = rng.integers(0, V, size=M)
    X = _dev(rng.standard_normal((M, K)) + lean * rng.random((M, 1)) * host(W)[t], name)
    t[rng.random(M) < 0.3] = -100
    w = rng.random(M).astype(np.float32)
    return X, W, torch.from_numpy(t).cuda(), torch.from_numpy(w).cuda()


def _compare(X, W, t, w, got, name, rows=None, ignore=-100):
    x, W64, t, w = (host(v).astype(np.float64) if v is not None else None for v in (X, W, t, w))
    t = t.astype(np.int64)
    w = np.ones(len(t)) if w is None else w
    got = [None if g is None else host(g).astype(np.float64) for g in got]
    if rows is not None:
        x, t, w, got = x[rows], t[rows], w[rows], [None if g is None else g[rows] for g in got]
    K, V, d = x.shape[1], W64.shape[0], HALF[name]
    loss, lse, dX = oo.head_loss(x, W64, t, w, ignore)
    counted = t != ignore
    e = (K + 2) * F32 * (np.abs(x) @ np.abs(W64).T).max(axis=1)
    s_abs = np.abs(x @ W64.T).max(axis=1)
    # the bound's and the logarithm's fp32 steps, sums of V terms
    e_lse = e + 8 * F32 * (1 + s_abs) + (V / 64 + 64) * F32
    worst = {}

    def check(what, g, ref, bound):
        assert np.isfinite(g).all(), what
        worst[what] = float(np.max(np.abs(g - ref) / bound))
        assert worst[what] <= 1.0, (what, worst)

    check("lse", got[1], lse, e_lse + F32 * np.abs(lse))
    nll = np.where(counted, loss / np.where(w == 0, 1, w), 0)
    # softplus(u) with u off by 2 e_lse: its relative error is at most that too
    check("loss", got[0], loss, w * (2.02 * e_lse + 8 * F32) * np.minimum(1.0, nll * 1.5 + 1e-30) + 4 * F32 * np.abs(loss) + 1e-30)
    if got[2] is not None:
        s = x @ W64.T
        p = np.exp(s - lse[:, None])
        at = np.where(counted, t, 0)
        p[np.arange(len(t)), at] = 0.0
        rest = p.sum(axis=1)                       # 1 - p_t
        rel = 4.04 * e_lse + (V + 64) * F32 + 1e-6
        bound = (d + rel)[:, None] * (p @ np.abs(W64)) + (rel * rest)[:, None] * np.abs(W64[at])
        bound += 2.0 ** -37 * np.abs(W64).sum(axis=0)[None] if name == "f16" else 0.0
        bound = w[:, None] * bound * (1 + 2 * d) + d * np.abs(dX) + TINY[name] + 1e-30
        assert not got[2][~counted].any() and not got[0][~counted].any()
        check("dX", got[2], dX, bound)
    say(f"  worst error / bound {worst}")


SHAPES = [(1, 8, 1), (1, 64, 2), (3, 72, 63), (2, 4096, 130), (5, 264, 500), (17, 136, 1000), (256, 128, 256),
          (257, 1032, 513), (300, 520, 4099), (64, 4096, 2048), (700, 256, 3001), (130, 64, 20011)]


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,V", SHAPES)
def test_loss_and_gradient(M, K, V, name):
    say(f"head M={M} K={K} V={V} {name}")
    X, W, t, w = _case(M, K, V, name, M + K + V)
    got = qn.qlora_head_loss(X, W, t, weights=w)
    _compare(X, W, t, w, got, name)
    alone = qn.qlora_head_loss(X, W, t, weights=w, need_dx=False)
    assert alone[2] is None
    for g, h in zip(alone[:2], got[:2]):
        np.testing.assert_allclose(host(g), host(h), rtol=2e-6, atol=2e-6)
    _compare(X, W, t, None, qn.qlora_head_loss(X, W, t), name)


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_several_pieces(name):
    """P past 256 MiB: the vocabulary goes in pieces, with running sums."""
    M, K, V = 5003, 200, 60013
    say(f"head pieces {name}")
    X, W, t, w = _case(M, K, V, name, 11, lean=10.0)
    got = qn.qlora_head_loss(X, W, t, weights=w)
    rows = np.random.default_rng(0).choice(M, 150, replace=False)
    _compare(X, W, t, w, got, name, rows)
    # targets in every piece
    edge = np.concatenate((np.arange(0, V, V // 100), [V - 1]))
    t[:len(edge)] = __import__("torch").from_numpy(edge).cuda()
    _compare(X, W, t, w, qn.qlora_head_loss(X, W, t, weights=w), name, np.arange(len(edge)))


def test_head_past_4_gib():
    """V K past 2^31 elements: 64-bit offsets, several pieces for the loss alone."""
    import torch
    M, K, V = 3, 65536, 33000
    say("head, large W")
    gen = torch.Generator("cuda").manual_seed(2)
    W = torch.empty(V, K, dtype=torch.bfloat16, device="cuda")
    for i in range(0, V, 3000):
        n = min(3000, V - i)
        W[i:i + n] = (torch.randn(n, K, device="cuda", generator=gen) / K ** 0.5).bfloat16()
    X = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    t = torch.tensor([0, V - 1, 17000], device="cuda")
    s = torch.cat([X.double() @ W[i:i + 3000].double().T.contiguous() for i in range(0, V, 3000)], 1)
    lse = torch.logsumexp(s, 1)
    want = lse - s.gather(1, t[:, None])[:, 0]
    p = torch.exp(s - lse[:, None])
    dX = sum(p[:, i:i + 3000] @ W[i:i + 3000].double() for i in range(0, V, 3000)) - W[t].double()
    for need in (False, True):
        loss, l, g = qn.qlora_head_loss(X, W, t, need_dx=need)
        np.testing.assert_allclose(host(loss), want.cpu().numpy(), rtol=1e-5)
        np.testing.assert_allclose(host(l), lse.cpu().numpy(), rtol=1e-5)
    # two roundings of half a step each on sums whose terms are p W and W_t
    bound = 2.0 ** -8 * 1.1 * dX.abs() + 2.0 ** -8 * sum(p[:, i:i + 3000] @ W[i:i + 3000].double().abs() for i in range(0, V, 3000)) + 1e-5 * W[t].double().abs() + 1e-9
    assert bool(((g.double() - dX).abs() <= bound).all())


def test_nearly_certain_and_hopeless_targets():
    say("head extremes")
    import torch
    K, V = 64, 300
    rng = np.random.default_rng(5)
    W = _dev(rng.standard_normal((V, K)), "bf16")
    for gain in (0.5, 1.0, 3.0):        # target logits up to about +-200
        t = torch.arange(40, device="cuda")
        for sign in (1, -1):
            X = (sign * gain * W[:40].float()).bfloat16()
            _compare(X, W, t, None, qn.qlora_head_loss(X, W, t), "bf16")


@pytest.mark.parametrize("M,V", [(40, 700), (3, 129)])
def test_ignored_bad_and_non_finite_rows(M, V):
    import torch
    say("head masks")
    X, W, t, w = _case(M, 136, V, "bf16", 3)
    t.fill_(-100)
    loss, lse, dX = qn.qlora_head_loss(X, W, t, weights=w)
    assert not host(loss).any() and not host(dX).any() and np.isfinite(host(lse)).all()
    # an ignored row may hold anything; a bad target spoils its own row alone
    t[:] = torch.arange(M, device="cuda") % V
    want = [host(v).copy() for v in qn.qlora_head_loss(X, W, t, weights=w)]
    X2, t2 = X.clone(), t.clone()
    X2[0] = float("nan")
    t2[0], t2[1], t2[2] = -100, V, -7
    loss, lse, dX = (host(v) for v in qn.qlora_head_loss(X2, W, t2, weights=w))
    assert loss[0] == 0 and not dX[0].any()
    for r in (1, 2):
        assert np.isnan(loss[r]) and np.isnan(dX[r]).all()
        np.testing.assert_allclose(lse[r], want[1][r], rtol=1e-6)
    for g, h in zip((loss, lse, dX), want):
        np.testing.assert_array_equal(g[3:], h[3:])
    # another ignored index, one that is a vocabulary entry
    loss, _, dX = (host(v) for v in qn.qlora_head_loss(X, W, t, weights=w, ignore_index=5 % M))
    assert loss[5 % M] == 0 and not dX[5 % M].any()
    np.testing.assert_array_equal(np.delete(loss, 5 % M), np.delete(want[0], 5 % M))
    # a NaN in a counted row
    X2 = X.clone()
    X2[1, 4] = float("nan")
    loss, lse, dX = (host(v) for v in qn.qlora_head_loss(X2, W, t, weights=w))
    assert np.isnan(loss[1]) and np.isnan(dX[1]).all() and np.isfinite(np.delete(dX, 1, axis=0)).all()


def test_rows_behind_the_last_stay_and_calls_repeat():
    import torch
    say("head canaries")
    M, K, V = 70, 264, 1500
    X, W, t, w = _case(M, K, V, "bf16", 8)
    ws = torch.empty(qn.qlora_head_workspace_bytes(M, K, V), dtype=torch.uint8, device="cuda")
    ws.fill_(255)            # what a workspace holds does not matter
    outs = [torch.full((M + 2,), 7.0, device="cuda"), torch.full((M + 2,), 7.0, device="cuda"),
            torch.full((M + 2, K), 7.0, device="cuda").bfloat16()]
    call = lambda **kw: qn.qlora_head_loss(X, W, t, weights=w, loss=outs[0][:M], lse=outs[1][:M], dX=outs[2][:M],
                                           workspace=ws, **kw)
    call()
    want = [host(o).copy() for o in outs]
    assert all((o[M:] == 7.0).all() for o in want)
    _compare(X, W, t, w, [o[:M] for o in outs], "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for o in outs:
            o[:M] = 0
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for o, h in zip(outs, want):
            np.testing.assert_array_equal(host(o), h)


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("K", [64, 1032])
def test_rows_of_very_different_groups(K, name):
    """Vocabulary groups of 128 whose logits reach from a fraction to hundreds:
    bounds of one row's groups on both sides of where bf16 takes them as 0."""
    say(f"head groups K={K} {name}")
    M, V = 37, 1000
    rng = np.random.default_rng(K)
    gain = np.array([1.0, 0.05, 12.0, 40.0, 0.0, 3.0, 25.0, 1.0])[np.arange(V) // 128]
    W = rng.standard_normal((V, K)) / np.sqrt(K) * gain[:, None]
    # rows 0 .. 18: the large groups far below (every product negative)
    X = rng.standard_normal((M, K))
    W[256:512] = -np.abs(W[256:512])
    X[:19] = np.abs(X[:19])
    W, X = _dev(W, name), _dev(X, name)
    import torch
    t = torch.from_numpy(rng.integers(0, V, size=M)).cuda()
    t[3] = -100
    _compare(X, W, t, None, qn.qlora_head_loss(X, W, t), name)


def test_masks_of_a_split_reduction():
    """Few tiles and a long K: the logits come from partial sums."""
    import torch
    say("head masks, split")
    M, K, V = 40, 2056, 700
    X, W, t, w = _case(M, K, V, "bf16", 8)
    t[:] = torch.arange(M, device="cuda") % V
    want = [host(v).copy() for v in qn.qlora_head_loss(X, W, t, weights=w)]
    X2, t2 = X.clone(), t.clone()
    X2[0] = float("nan")
    t2[0], t2[1], t2[2] = -100, V, -7
    loss, lse, dX = (host(v) for v in qn.qlora_head_loss(X2, W, t2, weights=w))
    assert loss[0] == 0 and not dX[0].any()
    for r in (1, 2):
        assert np.isnan(loss[r]) and np.isnan(dX[r]).all()
        np.testing.assert_allclose(lse[r], want[1][r], rtol=1e-6)
    for g, h in zip((loss, lse, dX), want):
        np.testing.assert_array_equal(g[3:], h[3:])
    # the last columns of the last group, and a piece of one column
    t2[:] = V - 1
    _compare(X, W, t2, None, qn.qlora_head_loss(X, W, t2), "bf16")
    one = torch.zeros(M, dtype=torch.int64, device="cuda")
    loss, lse, dX = (host(v) for v in qn.qlora_head_loss(X, W[:1], one))
    assert not loss.any() and not dX.any()
