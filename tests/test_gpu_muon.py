"""The orthogonalised adapter step on the GPU against its 64-bit reference.

With master copies at zero and lr = 1, weight decay 0, scaling None, the new master is
minus the orthogonalised update rounded once to fp32.  What the kernels add to that
rounding: u is rounded to fp32 (2^-24 of itself, twice: m and u), which moves the
update by what the iteration makes of such a change."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _dev(x, name):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(_torch_type(name)).cuda()


def _gradient(rng, rows, cols, fall=2.0):
    k = min(rows, cols)
    s = 10.0 ** np.linspace(0, -fall, k)
    return (rng.standard_normal((rows, k)) / np.sqrt(rows) * s) @ rng.standard_normal((k, cols)) / np.sqrt(cols)


class Case:
    def __init__(self, K, N, r, name, grad="f32", master=True, seed=0, fall=2.0):
        rng = np.random.default_rng(seed + K + N + r)
        self.K, self.N, self.r, self.name = K, N, r, name
        shapes = {"A": (K, r), "B": (r, N)}
        self.master = {n: _dev(rng.standard_normal(s) * 0.05, "f32") for n, s in shapes.items()} if master else {"A": None, "B": None}
        self.p = {n: _dev(host(self.master[n]) if master else rng.standard_normal(s) * 0.05, name) for n, s in shapes.items()}
        self.g = {n: _dev(_gradient(rng, *s, fall), grad) for n, s in shapes.items()}
        self.m = {n: _dev(_gradient(rng, *s, fall), "f32") for n, s in shapes.items()}

    def values(self):
        return {n: tuple(None if t is None else host(t).astype(np.float64) for t in (self.p[n], self.g[n], self.m[n], self.master[n]))
                for n in ("A", "B")}

    def step(self, lr, **kw):
        qn.qlora_muon_step(self.p["A"], self.p["B"], self.g["A"], self.g["B"], self.m["A"], self.m["B"], lr,
                           A_master=self.master["A"], B_master=self.master["B"], **kw)


def _moved(u, steps, eps, rel):
    """Bound, in every element, of what a relative change `rel` of u's elements does to
    the update: to first order the iteration's derivative, at most its largest slope
    sum of |a| + 3 |b| + 5 |c| per step for singular values up to 1.15, but no more than
    the slope a at each step for small ones; the observed largest is measured here by
    the change that random signs make in the reference, times 8 for the worst of many."""
    rng = np.random.default_rng(1)
    base = oo.newton_schulz(u, steps, COEFFICIENTS, eps)
    worst = 0.0
    for _ in range(2):
        other = oo.newton_schulz(u * (1 + 1e-6 * rng.choice([-1.0, 1.0], size=u.shape)), steps, COEFFICIENTS, eps)
        worst = max(worst, np.abs(other - base).max() / 1e-6)
    return 8 * worst * rel


def check(t, before, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scaling="spectral", steps=5, eps=1e-7):
    for n in ("A", "B"):
        p, g, m, master = before[n]
        full = p if master is None else master
        want, wm, x = oo.muon_step(full, g, m, lr, momentum, nesterov, weight_decay, scaling, steps, COEFFICIENTS, eps)
        got_m = host(t.m[n]).astype(np.float64)
        # momentum: one rounding of the exact sum
        assert (np.abs(got_m - wm) <= 2.0 ** -24 * np.abs(wm) * 1.01 + 1e-45).all(), n
        u = (1 - momentum) * g + momentum * wm if nesterov else wm
        factor = np.abs(lr) * {None: 1.0, "spectral": np.sqrt(max(1.0, x.shape[0] / x.shape[1])),
                               "rms": 0.2 * np.sqrt(max(x.shape))}[scaling]
        off = factor * _moved(u, steps, eps, 2.0 ** -23) + 1e-12
        got = host(t.p[n] if master is None else t.master[n]).astype(np.float64)
        d = HALF[t.name] if master is None else 2.0 ** -24
        tiny = 2.0 ** -25 if t.name == "f16" and master is None else 0.0
        worst = np.max(np.abs(got - want) / (1.01 * d * np.abs(want) + off + tiny))
        say(f"  {n}: worst error / bound {worst:.3f}, allowed beside the rounding {off:.2e}")
        assert worst <= 1.0, n
        if master is not None:
            rounded = host(t.p[n])
            np.testing.assert_array_equal(rounded, oo.round16(host(t.master[n]), t.name))


@pytest.mark.parametrize("K,N,r", [(1, 1, 1), (8, 8, 8), (64, 200, 1), (40, 24, 17), (300, 1000, 16), (1000, 77, 33),
                                   (17, 4096, 64), (4096, 2000, 64), (130, 500, 65), (700, 333, 128), (1500, 40, 200),
                                   (515, 1030, 256)])
def test_update_itself(K, N, r):
    import torch
    say(f"muon update K={K} N={N} r={r}")
    t = Case(K, N, r, "bf16")
    for n in ("A", "B"):
        t.master[n].zero_()
    before = t.values()
    t.step(1.0, scaling=None)
    check(t, before, 1.0, scaling=None)
    # what orthogonalised means: singular values near one where the direction has any
    if min(K, r) >= 8:
        sv = torch.linalg.svdvals(t.master["A"].double())
        assert 0.3 < float(sv[: min(K, r) // 2].min()) and float(sv.max()) < 1.3


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("grad", ["f32", "16"])
@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("K,N,r", [(72, 333, 24), (1024, 512, 64), (333, 72, 100)])
def test_steps(K, N, r, master, grad, name):
    say(f"muon step K={K} N={N} r={r} {name} grad {grad} master {master}")
    t = Case(K, N, r, name, name if grad == "16" else "f32", master)
    for kw in ({"lr": 0.02, "weight_decay": 0.1}, {"lr": 0.01, "nesterov": False, "scaling": "rms", "momentum": 0.0},
               {"lr": -0.02, "scaling": None, "momentum": 0.9, "steps": 2}):
        before = t.values()
        t.step(**kw)
        check(t, before, **kw)


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 7])
@pytest.mark.parametrize("r", [16, 80])
def test_numbers_of_steps(steps, r):
    say(f"muon {steps} steps, r={r}")
    t = Case(200, 150, r, "bf16")
    before = t.values()
    t.step(0.1, steps=steps)
    check(t, before, 0.1, steps=steps)


@pytest.mark.parametrize("r", [16, 72])
def test_zero_and_tiny_gradients(r):
    say(f"muon zero and tiny gradients r={r}")
    t = Case(120, 136, r, "bf16")
    for n in ("A", "B"):
        t.g[n].zero_()
        t.m[n].zero_()
    before = t.values()
    t.step(0.1, weight_decay=0.5)
    for n in ("A", "B"):
        np.testing.assert_array_equal(host(t.master[n]), (before[n][3] * (1 - 0.1 * 0.5)).astype(np.float32))
        assert not host(t.m[n]).any()
    # below eps the direction is divided by eps, not by its norm
    t = Case(120, 136, r, "bf16")
    for n in ("A", "B"):
        t.g[n].mul_(1e-9)
        t.m[n].mul_(1e-9)
    before = t.values()
    t.step(0.1, scaling=None)
    check(t, before, 0.1, scaling=None)


@pytest.mark.parametrize("r", [8, 100])
def test_directions_of_any_size_and_rank(r):
    say(f"muon ranks and sizes r={r}")
    for scale in (1e-15, 1e15):
        t = Case(200, 90, r, "bf16")
        for n in ("A", "B"):
            t.g[n].mul_(scale)
            t.m[n].mul_(scale)
        before = t.values()
        t.step(0.1, eps=1e-30)
        check(t, before, 0.1, eps=1e-30)
    # one direction alone: its singular value goes to near one, the others stay zero
    t = Case(200, 90, r, "bf16")
    for n in ("A", "B"):
        a = host(t.g[n])
        t.g[n].copy_(_dev(np.outer(a[:, 0], a[0]), "f32"))
        t.m[n].zero_()
        t.master[n].zero_()
    before = t.values()
    t.step(1.0, scaling=None)
    check(t, before, 1.0, scaling=None)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("r", [16, 80])
def test_what_is_not_finite_shows(r, bad):
    import torch
    say(f"muon with {bad} r={r}")
    t = Case(100, 130, r, "bf16")
    t.g["A"][3, 5] = bad
    t.step(0.1)
    assert torch.isnan(t.p["A"]).all() and torch.isnan(t.master["A"]).all()
    assert torch.isfinite(t.p["B"]).all()
    t2 = Case(100, 130, r, "bf16")
    t2.step(0.1)
    assert torch.equal(t.master["B"], t2.master["B"])


@pytest.mark.parametrize("K,N,r", [(1000, 77, 33), (64, 500, 64), (300, 130, 100)])
def test_unaligned_tensors_and_what_lies_around_them(K, N, r):
    """Tensors that start one element into their memory; their neighbours stay."""
    import torch
    say(f"muon unaligned K={K} N={N} r={r}")
    t, u = Case(K, N, r, "bf16"), Case(K, N, r, "bf16")
    around = []
    for d in (u.p, u.g, u.m, u.master):
        for n in ("A", "B"):
            v = d[n]
            buf = torch.full((v.numel() + 65,), 3.0, dtype=v.dtype, device="cuda")
            buf[1:1 + v.numel()].copy_(v.flatten())
            d[n] = buf[1:1 + v.numel()].view(v.shape)
            around.append((buf, v.numel()))
    n = qn.qlora_muon_workspace_bytes(K, N, r)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    t.step(0.1)
    u.step(0.1, workspace=ws[:n])
    assert (ws[n:] == 255).all()
    for d, e in ((t.p, u.p), (t.m, u.m), (t.master, u.master)):
        assert all(torch.equal(d[k], e[k]) for k in ("A", "B"))
    for buf, count in around:
        assert float(buf[0]) == 3.0 and (buf[1 + count:] == 3.0).all()


@pytest.mark.parametrize("r", [16, 64, 130])
def test_replayed_steps(r):
    """Three replays of a captured step, with eager work between, are three eager steps."""
    import torch
    say(f"muon graph r={r}")
    t, u = Case(700, 300, r, "bf16"), Case(700, 300, r, "bf16")
    before = {k: {n: d[n].clone() for n in ("A", "B")} for k, d in (("p", u.p), ("m", u.m), ("master", u.master))}
    g = torch.cuda.CUDAGraph()
    u.step(0.02)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        u.step(0.02)
    for k, d in (("p", u.p), ("m", u.m), ("master", u.master)):
        for n in ("A", "B"):
            d[n].copy_(before[k][n])
    for _ in range(3):
        t.step(0.02)
        g.replay()
        torch.cuda.synchronize()
        Case(40, 50, r, "f16").step(0.1)
        for d, e in ((t.p, u.p), (t.m, u.m), (t.master, u.master)):
            assert all(torch.equal(d[n], e[n]) for n in ("A", "B"))


def test_streams_at_once():
    import torch
    say("muon on three streams")
    shapes = [(700, 300, 16), (4096, 2000, 64), (300, 500, 100)]
    want = [Case(*s, "bf16") for s in shapes]
    for t in want:
        t.step(0.02)
    got = [Case(*s, "bf16") for s in shapes]
    torch.cuda.synchronize()
    for t in got:
        t.step(0.02, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for t, u in zip(want, got):
        assert all(torch.equal(t.master[n], u.master[n]) and torch.equal(t.m[n], u.m[n]) for n in ("A", "B"))


def test_longest_matrices():
    """2^24 - 1 rows of one rank: the update is the scaled direction."""
    import torch
    say("muon of the longest matrices")
    K = (1 << 24) - 1
    g = torch.Generator(device="cuda").manual_seed(3)
    A, B = torch.zeros(K, 1, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.randn(K, 1, generator=g, device="cuda"), torch.randn(1, K, generator=g, device="cuda")
    mA, mB, MA, MB = (torch.zeros_like(v) for v in (dA, dB, dA, dB))
    qn.qlora_muon_step(A, B, dA, dB, mA, mB, 1.0, scaling=None, A_master=MA, B_master=MB)
    x = 1.0
    for _ in range(5):
        x = COEFFICIENTS[0] * x + COEFFICIENTS[1] * x ** 3 + COEFFICIENTS[2] * x ** 5
    for d, M in ((dA, MA), (dB, MB)):
        want = -x * d.double() / d.double().square().sum().sqrt()
        assert float((M - want).abs().max()) <= 1e-6 * float(want.abs().max())


@pytest.mark.parametrize("r", [16, 80])
@pytest.mark.parametrize("eps", [2.2250738585072014e-308, 1e-200, 1e30])
def test_any_eps(r, eps):
    """Zeros stay zeros however small eps, whose square may be 0; a large one divides."""
    import torch
    say(f"muon eps={eps} r={r}")
    t = Case(90, 70, r, "bf16")
    for d in (t.g, t.m):
        for n in ("A", "B"):
            d[n].zero_()
    before = t.values()
    t.step(0.1, eps=eps)
    check(t, before, 0.1, eps=max(eps, 1e-150))
    t = Case(90, 70, r, "bf16")
    before = t.values()
    t.step(0.1, eps=eps)
    check(t, before, 0.1, eps=max(eps, 1e-150))


@pytest.mark.parametrize("K,N,r", [(11_300_000, 64, 33), (64, 11_300_000, 33), ((1 << 24) - 3, 100, 20), (100, (1 << 24) - 3, 20)])
def test_directions_past_two_gibibytes(K, N, r):
    """The direction, its rank filled up to a multiple of 16, takes more memory than its
    matrix: the last rows and columns are stepped like the first."""
    import torch
    say(f"muon of a direction past 2 GiB, {K} x {N}, rank {r}")
    gen = torch.Generator(device="cuda").manual_seed(9)
    shapes = ((K, r), (r, N))
    A, B = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in shapes)
    dA, dB = (torch.randn(*s, generator=gen, device="cuda") for s in shapes)
    mA, mB, MA, MB = (torch.zeros(*s, device="cuda") for s in shapes + shapes)
    qn.qlora_muon_step(A, B, dA, dB, mA, mB, 1.0, momentum=0.0, nesterov=False, scaling=None, A_master=MA, B_master=MB)
    a, b, c = COEFFICIENTS
    for U, M in ((dA, MA), (dB.T, MB.T)):
        n = U.shape[0]
        G = torch.zeros(r, r, dtype=torch.float64, device="cuda")
        for i in range(0, n, 1 << 20):
            x = U[i:i + (1 << 20)].double().contiguous()
            G += x.T.contiguous() @ x
        norm = float(G.trace()) ** 0.5
        G = host(G) / norm ** 2
        Q = np.eye(r)
        for _ in range(5):
            P = a * np.eye(r) + b * G + c * G @ G
            Q, G = Q @ P, P @ G @ P
        for part in (slice(0, 200), slice(n // 2, n // 2 + 200), slice(max(n - 200, 0), n)):
            want = -host(U[part]).astype(np.float64) @ Q / norm
            # u is the gradient itself; what is left are 64-bit sums and one rounding
            assert np.abs(host(M[part]) - want).max() <= 2.0 ** -24 * np.abs(want).max() * 1.01 + 1e-10 * np.abs(want).max()


@pytest.mark.parametrize("coefficients,steps", [(COEFFICIENTS, 8), ((2.0, -1.5, 0.5), 14), ((1.5, -0.5, 0.0), 24)])
@pytest.mark.parametrize("K,N,r,rank", [(200, 8, 16, 1), (17, 1000, 64, 4), (300, 40, 64, 0), (8, 700, 80, 3), (500, 130, 200, 2),
                                        (40, 300, 256, 0)])
def test_low_rank_directions_at_the_last_step(K, N, r, rank, coefficients, steps):
    """Whole numbers of that rank (0: pairs of equal columns of A, rows of B), or with fewer
    rows than the rank, so that the direction is exactly its gradient: what is left is one
    rounding to fp32 and the Gram matrix's, below 2^-24 of the largest element."""
    say(f"muon of rank {rank}: K={K} N={N} r={r}, {steps} steps")
    rng = np.random.default_rng(K + N + r)
    t = Case(K, N, r, "bf16")
    for n, (rows, cols) in (("A", (K, r)), ("B", (r, N))):
        k = rank or r // 2
        v = rng.integers(-3, 4, size=(rows if n == "A" else cols, k)).astype(np.float64)
        v = v @ rng.integers(-3, 4, size=(k, r)) if rank else v.repeat(2, axis=1)
        v[0, 0] += not v.any()
        t.g[n].copy_(_dev(v if n == "A" else v.T, "f32"))
        t.master[n].zero_()
    before = t.values()
    t.step(1.0, scaling=None, momentum=0.0, nesterov=False, steps=steps, coefficients=coefficients)
    for n in ("A", "B"):
        want = -oo.newton_schulz(before[n][1], steps, coefficients, 1e-7)
        got = host(t.master[n]).astype(np.float64)
        worst = np.abs(got - want).max() / np.abs(want).max() * 2.0 ** 24
        say(f"  {n}: off by {worst:.3f} x 2^-24 of the largest element")
        assert (np.abs(got - want) <= 1.01 * 2.0 ** -24 * (np.abs(want) + np.abs(want).max())).all(), n


def test_steps_past_the_last_are_refused():
    t = Case(100, 90, 16, "bf16")
    before = t.values()
    for kw in ({"steps": 9}, {"steps": 32}, {"steps": 33}, {"steps": 5, "coefficients": (8.0, -20.0, 13.0)}):
        with pytest.raises(qn.NF4Error):
            t.step(0.1, **kw)
    after = t.values()
    for n in ("A", "B"):
        for a, b in zip(before[n], after[n]):
            np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["gradient", "momentum"])
@pytest.mark.parametrize("r", [16, 64, 80])
@pytest.mark.parametrize("steps", [0, 1, 2])
def test_what_is_not_finite_shows_after_any_number_of_steps(steps, r, where, bad):
    """The whole matrix, without a step too, where an infinite norm alone would leave zeros."""
    import torch
    say(f"muon with {bad} in a {where}, {steps} steps, r={r}")
    t = Case(100, 130, r, "bf16")
    (t.g if where == "gradient" else t.m)["B"][5, 7] = bad
    t.step(0.1, steps=steps)
    assert torch.isnan(t.p["B"]).all() and torch.isnan(t.master["B"]).all()
    assert torch.isfinite(t.p["A"]).all() and torch.isfinite(t.m["A"]).all()


@pytest.mark.parametrize("scaling,a,b", [("spectral", 8.0, 1.0), ("rms", 0.2 * np.sqrt(1024.0), 0.2 * np.sqrt(400.0)), (None, 1.0, 1.0)])
def test_scalings_go_by_the_stored_rows_and_columns(scaling, a, b):
    """A is 1024 x 16, B 16 x 400: the factors as the header names them."""
    say(f"muon scaling {scaling}")
    steps = {}
    for s in (scaling, None):
        t = Case(1024, 400, 16, "bf16")
        for n in ("A", "B"):
            t.master[n].zero_()
        t.step(1.0, scaling=s)
        steps[s] = {n: host(t.master[n]).astype(np.float64) for n in ("A", "B")}
    for n, f in (("A", a), ("B", b)):
        # two roundings to fp32
        assert (np.abs(steps[scaling][n] - f * steps[None][n]) <= 2.02 * 2.0 ** -24 * f * np.abs(steps[None][n])).all(), n
