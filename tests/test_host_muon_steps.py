"""How many steps the orthogonalised update may take: the iteration on the Gram matrix
against the one on the matrix itself, and the refusal past the last allowed count.  No
GPU work is issued."""
import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.test_host_muon import COEFFICIENTS, _options

# (coefficients, steps): the last count with |a|^(2 steps) <= 2^29, at most 32
LAST = [(COEFFICIENTS, 8), ((4.0, -6.8, 2.9), 7), ((2.0, -1.5, 0.5), 14), ((1.5, -0.5, 0.0), 24), ((1.0, 0.4, -0.4), 32)]


def _step(coefficients, steps):
    a, b, c = coefficients
    return qn.lib().qlora_muon_step(0, 1, 7, 5, 3, 0x102, 0x202, 0x304, 0x404, 0x504, 0x604, None, None,
                                    _options(a=a, b=b, c=c, steps=steps), 0x10000, 1 << 30, None)


@pytest.mark.parametrize("coefficients,last", LAST)
def test_steps_past_the_last_are_refused(coefficients, last):
    for steps in range(last + 1, 40):
        assert _step(coefficients, steps) == qn.NF4_EINVAL, steps
        # a's sign does not matter
        assert _step((-coefficients[0], *coefficients[1:]), steps) == qn.NF4_EINVAL, steps


def test_a_large_first_coefficient_is_refused_at_once():
    for a, last in ((2.0 ** 14.5 * 1.001, 0), (8.0, 4), (1e200, 0)):
        assert _step((a, -1.0, 0.0), last + 1) == qn.NF4_EINVAL


def _by_gram_matrix(u, steps, coefficients):
    """The kernels' iteration, in 64 bits: everything symmetric, stored from one half."""
    a, b, c = coefficients

    def symmetric(m):
        return np.triu(m) + np.triu(m, 1).T

    norm = np.sqrt(np.sum(u * u))
    G, Q = symmetric(u.T @ u / norm ** 2), np.eye(u.shape[1])
    for _ in range(steps):
        P = symmetric(a * np.eye(u.shape[1]) + b * G + c * (G @ G))
        Q = symmetric(Q @ P)
        G = symmetric(symmetric(G @ P) @ P)
    return u @ Q / norm


def directions():
    """Directions of low rank, exactly, and with singular values falling far."""
    rng = np.random.default_rng(4)
    whole = lambda *s: rng.integers(-3, 4, size=s).astype(np.float64)
    yield "rank 1", np.outer(whole(200) + 0.5, whole(16) + 0.5)
    yield "rank 4", whole(1000, 4) @ whole(4, 16)
    yield "rank 3 of 100", whole(700, 3) @ whole(3, 100)
    yield "wide", whole(17, 64)
    yield "wider", whole(8, 200)
    yield "equal columns", whole(300, 8).repeat(4, axis=1)
    for fall in (4, 8):
        left, _ = np.linalg.qr(rng.standard_normal((300, 32)))
        right, _ = np.linalg.qr(rng.standard_normal((32, 32)))
        yield f"falling to 1e-{fall}", (left * 10.0 ** np.linspace(0, -fall, 32)) @ right


@pytest.mark.parametrize("coefficients,last", LAST)
def test_the_gram_matrix_serves_as_long(coefficients, last):
    """The Gram matrix's rounding, a few 2^-53, grows by a^2 a step: below 2^-24 of the
    largest element up to the last count."""
    for name, u in directions():
        want = oo.newton_schulz(u, last, coefficients, 1e-7)
        got = _by_gram_matrix(u, last, coefficients)
        assert np.abs(got - want).max() <= 2.0 ** -24 * np.abs(want).max(), name


def test_and_no_longer():
    """Why there is a limit: null directions run away where the update itself stays small."""
    u = next(u for name, u in directions() if name == "rank 4")
    want = oo.newton_schulz(u, 20, COEFFICIENTS, 1e-7)
    assert np.abs(want).max() < 1.5
    with np.errstate(all="ignore"):
        got = _by_gram_matrix(u, 24, COEFFICIENTS)
    assert not np.abs(got).max() < 1.5
