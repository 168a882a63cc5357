"""Plain CPU references (numpy, 64 bits) of the operators around the NF4
layer: 8-bit activation checkpoints, the gated feed-forward front with its
backward, and the output head's cross entropy with its gradient.  They share
no code with the GPU path."""
from __future__ import annotations

import numpy as np

ACT8_BLOCK = 64


def round16(x, dtype: str) -> np.ndarray:
    """Round to the 16-bit type ("bf16" or "f16"), as float32 values."""
    x = np.asarray(x, dtype=np.float32)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float32)
    u = np.ascontiguousarray(x).view(np.uint32)
    r = ((u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) >> np.uint32(16)) << np.uint32(16)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32).reshape(x.shape))


def act8_encode(x: np.ndarray):
    """Codes (int8, M x K) and block magnitudes (float32 values, M x nb) of a
    matrix of 16-bit values given as float32.  The quotients 127 x / a are
    compared with the half integers in integers scaled by powers of two, by
    way of float64, which holds 254 |x| and (2q + 1) a exactly."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    nb = -(-K // ACT8_BLOCK)
    codes = np.zeros((M, K), dtype=np.int8)
    absmax = np.zeros((M, nb), dtype=np.float32)
    for b in range(nb):
        blk = x[:, b * ACT8_BLOCK:(b + 1) * ACT8_BLOCK]
        a = np.max(np.abs(blk), axis=1)
        bad = ~np.all(np.isfinite(blk), axis=1)
        a_safe = np.where(bad | (a == 0), 1.0, a)
        v = np.where((bad | (a == 0))[:, None], 0.0, blk)
        q = np.floor(127.0 * np.abs(v) / a_safe[:, None])
        for _ in range(2):   # floor estimate -> exact nearest, ties to even
            low = (2 * q - 1) * a_safe[:, None] > 254.0 * np.abs(v)
            q = np.where(low, q - 1, q)
            high = (2 * q + 1) * a_safe[:, None] < 254.0 * np.abs(v)
            q = np.where(high, q + 1, q)
        tie = (2 * q + 1) * a_safe[:, None] == 254.0 * np.abs(v)
        q = np.where(tie & (q % 2 == 1), q + 1, q)
        codes[:, b * ACT8_BLOCK:(b + 1) * ACT8_BLOCK] = (np.sign(v) * q).astype(np.int8)
        absmax[:, b] = np.where(bad, np.nan, a)
    return codes, absmax


def act8_decode(codes: np.ndarray, absmax: np.ndarray, dtype: str) -> np.ndarray:
    step = (absmax.astype(np.float32) / np.float32(127.0)).astype(np.float32)
    step = np.repeat(step, ACT8_BLOCK, axis=1)[:, :codes.shape[1]]
    return round16(codes.astype(np.float32) * step, dtype)


def act(name: str, g: np.ndarray):
    """act(g) and act'(g) in float64: "silu" or "gelu" (its tanh form)."""
    g = np.asarray(g, dtype=np.float64)
    if name == "silu":
        p = np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))
        return g * p, p * (1.0 + g * (1.0 - p))
    k0, k1 = np.sqrt(2.0 / np.pi), 0.044715
    t = np.tanh(k0 * (g + k1 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k0 * (1.0 + 3.0 * k1 * g * g)


def gated_forward(X, Wg, Wu, A, B, c, name: str):
    """(H, Z, G, U) in float64.  A: K x 2r, B: r x 2F."""
    X, Wg, Wu, A, B = (np.asarray(v, dtype=np.float64) for v in (X, Wg, Wu, A, B))
    F, r = Wg.shape[1], B.shape[0]
    Z = X @ A
    G = X @ Wg + c * (Z[:, :r] @ B[:, :F])
    U = X @ Wu + c * (Z[:, r:] @ B[:, F:])
    return act(name, G)[0] * U, Z, G, U


def gated_backward(dH, X, Z, G, U, Wg, Wu, A, B, c, name: str):
    """(dX, dA, dB) in float64 from the kept X, Z, G, U."""
    dH, X, Z, G, U, Wg, Wu, A, B = (np.asarray(v, dtype=np.float64) for v in (dH, X, Z, G, U, Wg, Wu, A, B))
    F, r = Wg.shape[1], B.shape[0]
    f, df = act(name, G)
    dY = (dH * U * df, dH * f)
    dX, dA, dB = 0.0, [], []
    for i, W in enumerate((Wg, Wu)):
        Bi, Ai, Zi = B[:, i * F:(i + 1) * F], A[:, i * r:(i + 1) * r], Z[:, i * r:(i + 1) * r]
        dZ = c * (dY[i] @ Bi.T)
        dX = dX + dY[i] @ W.T + dZ @ Ai.T
        dA.append(X.T @ dZ)
        dB.append(c * (Zi.T @ dY[i]))
    return dX, np.hstack(dA), np.hstack(dB)


def head_loss(X, W, targets, weights=None, ignore_index: int = -100):
    """(loss, lse, dX) in float64: loss_m = w_m (lse_m - s_mt), 0 where ignored."""
    X, W = np.asarray(X, dtype=np.float64), np.asarray(W, dtype=np.float64)
    t = np.asarray(targets)
    M = X.shape[0]
    w = np.ones(M) if weights is None else np.asarray(weights, dtype=np.float64)
    counted = t != ignore_index
    w = np.where(counted, w, 0.0)
    s = X @ W.T
    top = s.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.exp(s - top)
    lse = np.where(np.isposinf(top[:, 0]), np.inf, np.log(e.sum(axis=1)) + top[:, 0])
    p = e / e.sum(axis=1, keepdims=True)
    at, row = np.where(counted, t, 0), np.arange(M)
    # lse - s_t = log(1 + sum_{v != t} e^{s_v - s_t}) and p_t - 1 = -sum_{v != t} p_v:
    # the differences themselves cancel to nothing where the target is nearly certain
    with np.errstate(over="ignore", invalid="ignore"):
        d = np.exp(s - s[row, at][:, None])
    d[row, at] = 0.0
    # (an infinite s_t: the difference as it stands, NaN for +inf and inf for -inf)
    near = np.where(np.isinf(s[row, at]), np.inf, d.sum(axis=1))
    with np.errstate(invalid="ignore"):
        nll = np.where(near < 1.0, np.log1p(np.minimum(near, 1.0)), lse - s[row, at])
    loss = np.where(counted, w * nll, 0.0)
    p[row, at] = 0.0
    p[row, at] = -p.sum(axis=1)
    dX = np.where(counted[:, None], (p * w[:, None]) @ W, 0.0)
    return loss, lse, dX
