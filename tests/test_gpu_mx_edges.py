"""The MXFP4 calls at the ends of their ranges: products by tiles in whole numbers,
captured and replayed calls, two streams, workspaces full of NaN, memory behind the
outputs, the largest sizes; and a training step of the layer with its optimiser."""
import numpy as np
import pytest

import bit_nf4_quantized_10_amd as qn
from oracle import ops_oracle as oo
from tests.gpu_util import host, say
from tests.test_gpu_mx_linear import Case, check_backward, check_forward
from tests.test_gpu_mxfp4 import TYPES, _round, _state, _torch_type, _whole

pytestmark = pytest.mark.gpu
# one shape for each kernel and plan of the products: up to 16 rows, waves with chunks of
# their own, panels of 64 and 128 rows, tiles with and without a split, whole and ragged;
# dX decoding W, in one range and in several, and by the dense product (the last)
SHAPES = [(3, 520, 264, 16), (16, 4104, 4096, 64), (30, 1032, 520, 8), (50, 2056, 1000, 24), (100, 1032, 1336, 40),
          (300, 520, 2056, 16), (777, 264, 1336, 24), (1100, 1032, 2056, 24), (2100, 264, 1032, 256), (4000, 40, 4104, 8), (2600, 1032, 3400, 24)]


@pytest.mark.parametrize("M,N,K", [(1024, 2056, 8), (1030, 2064, 40), (1500, 1544, 256), (513, 4104, 264), (2048, 1032, 520),
                                   (1027, 2056, 776), (256, 8200, 1032), (65, 32776, 512), (4100, 520, 1544)])
def test_tiles_in_whole_numbers(M, N, K):
    """As the smaller products': fp32 sums are exact whatever their order."""
    say(f"mxfp4 tiles {M} x {N} x {K}")
    rng = np.random.default_rng(M + N + K)
    p, q = _whole(rng, M, K, -2, 2), _whole(rng, N, K, -2, 2)
    want = oo.mxfp4_values(*p, K) @ oo.mxfp4_values(*q, K).T
    P, Q = _state(*p, K), _state(*q, K)
    for name in TYPES:
        np.testing.assert_array_equal(host(qn.mxfp4_matmul(P, Q, _torch_type(name))), _round(want, name))


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,r", SHAPES)
def test_layer_of_every_plan(M, K, N, r, name):
    say(f"mx layer M={M} K={K} N={N} r={r} {name}")
    t = Case(M, K, N, r, name)
    Y, Z = t.forward()
    check_forward(t, Y, Z)
    check_backward(t, Z, *t.backward(Z), False)


@pytest.mark.parametrize("M,K,N,r", SHAPES)
def test_a_nan_block_of_the_weight_reaches_its_column_alone(M, K, N, r):
    import torch
    say(f"mx NaN block M={M} K={K} N={N}")
    t = Case(M, K, N, r, "bf16")
    clean, _ = t.forward()
    row, blk, chunks = 137 % N, (K // 32) // 2, -(-K // 512)
    t.W.scales[((row // 16) * chunks + blk // 16) * 256 + 4 * (16 * (blk % 4) + row % 16) + (blk % 16) // 4] = 255
    Y, _ = t.forward()
    rest = torch.arange(N, device="cuda") != row
    assert torch.isnan(Y[:, row]).all() and torch.equal(Y[:, rest], clean[:, rest])


def _guarded(shape, dtype):
    """A view of that shape in front of 512 sentinels, and the check that they stand."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), 7.0 if dtype.is_floating_point else 7, dtype=dtype, device="cuda")
    return buf[:n].view(shape), lambda: bool((buf[n:] == 7).all())


@pytest.mark.parametrize("M,K,N,r", SHAPES)
def test_workspaces_full_of_nan_and_memory_behind_the_outputs(M, K, N, r):
    import torch
    say(f"mx workspaces M={M} K={K} N={N} r={r}")
    t = Case(M, K, N, r, "bf16")
    Y, Z = t.forward()
    dX, dA, dB = t.backward(Z)
    fwd, bwd = qn.qlora_mx_workspace_bytes(M, K, N, r)
    guards = []

    def out(*shape, dtype=torch.bfloat16):
        v, stands = _guarded(shape, dtype)
        guards.append(stands)
        return v

    ws = torch.full((fwd + 512,), 255, dtype=torch.uint8, device="cuda")
    Y2, Z2 = t.forward(Y=out(M, N), Z=out(M, r), workspace=ws[:fwd])
    assert (ws[fwd:] == 255).all()
    ws = torch.full((bwd + 512,), 255, dtype=torch.uint8, device="cuda")
    got = t.backward(Z, dX=out(M, K), dA=out(K, r, dtype=torch.float32), dB=out(r, N, dtype=torch.float32), workspace=ws[:bwd])
    assert (ws[bwd:] == 255).all()
    for a, b in zip((Y, Z, dX, dA, dB), (Y2, Z2, *got)):
        assert torch.equal(a, b)
    codes, scales = qn.mxfp4_sizes(M, K)
    (c, cs), (s, ss) = _guarded((codes,), torch.uint8), _guarded((scales,), torch.uint8)
    P = qn.mxfp4_quantize(t.X, out=qn.MXFP4(M, K, c, s))
    n = qn.mxfp4_matmul_workspace_bytes(M, N, K)
    for dtype in (torch.bfloat16, torch.float32):
        ws = torch.full((max(n, 256) + 512,), 255, dtype=torch.uint8, device="cuda")
        C = qn.mxfp4_matmul(P, t.W, out=out(M, N, dtype=dtype), workspace=ws[:max(n, 256)])
        assert (ws[max(n, 256):] == 255).all()
        assert torch.equal(C, qn.mxfp4_matmul(P, t.W, dtype))
    assert cs() and ss() and all(g() for g in guards)


def _muon(t, seed=5):
    import torch
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() * 1e-3 for s in ((t.K, t.r), (t.r, t.N))]


@pytest.mark.parametrize("M,K,N,r", SHAPES)
def test_replayed_graph(M, K, N, r):
    """The whole step captured; three replays with eager work between them give the eager bits."""
    import torch
    say(f"mx graph M={M} K={K} N={N} r={r}")
    t = Case(M, K, N, r, "bf16")
    mA, mB = _muon(t)
    state = [v.clone() for v in (t.A, t.B, mA, mB)]

    def step():
        P = qn.mxfp4_quantize(t.X)
        C = qn.mxfp4_matmul(P, t.W, torch.bfloat16)
        back = qn.mxfp4_dequantize(P, torch.bfloat16)
        Y, Z = t.forward()
        dX, dA, dB = t.backward(Z)
        qn.qlora_muon_step(t.A, t.B, dA, dB, mA, mB, 0.02)
        return P.codes, P.scales, C, back, Y, Z, dX, dA, dB

    def bits(outs):
        return [host(v.view(torch.int16) if v.dtype == torch.bfloat16 else v).tobytes() for v in (*outs, t.A, t.B, mA, mB)]

    def restore():
        for v, s in zip((t.A, t.B, mA, mB), state):
            v.copy_(s)

    want = []
    for _ in range(3):
        want.append(bits(step()))
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    restore()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for k in range(3):
        for v in outs:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert bits(outs) == want[k], k
        t.forward()      # eager work in between


def test_two_streams_at_once():
    import torch
    say("mx on two streams")
    cases = [Case(100, 1032, 1336, 40, "bf16"), Case(1100, 520, 2056, 16, "f16"), Case(9, 4096, 2048, 64, "bf16")]
    want = []
    for t in cases:
        Y, Z = t.forward()
        want.append((Y, Z, *t.backward(Z)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for t, s in zip(cases, streams):
            Y, Z = t.forward(stream=s)
            got.append((Y, Z, *t.backward(Z, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_share_a_workspace():
    import torch
    say("mx: two graphs on one workspace")
    cases = [Case(100, 1032, 1336, 40, "bf16"), Case(1100, 520, 2056, 16, "bf16")]
    n = max(max(qn.qlora_mx_workspace_bytes(t.M, t.K, t.N, t.r)) for t in cases)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want, graphs, outs = [], [], []
    for t in cases:
        Y, Z = t.forward()
        want.append((Y, Z, *t.backward(Z)))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y, Z = t.forward(workspace=ws)
            outs.append((Y, Z, *t.backward(Z, workspace=ws)))
        graphs.append(g)
    for _ in range(3):
        ws.fill_(255)
        for g, o, w in zip(graphs, outs, want):
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_training_steps_together():
    """A K x N weight quantised, three steps of forward, backward and optimiser, each
    against the references on the values before it."""
    import torch
    say("mx training steps")
    t = Case(200, 520, 264, 16, "bf16")
    rng = np.random.default_rng(11)
    w = (rng.standard_normal((t.K, t.N)) / np.sqrt(t.K)).astype(np.float32)
    t.W = qn.mxfp4_quantize(torch.from_numpy(w).cuda(), transpose=True)
    t.w = oo.mxfp4_values(*oo.mxfp4_quantize(w.T), t.K)
    MA, MB, mA, mB = t.A.float(), t.B.float(), torch.zeros(t.K, t.r, device="cuda"), torch.zeros(t.r, t.N, device="cuda")
    for _ in range(3):
        t.a, t.b = (host(v).astype(np.float64) for v in (t.A, t.B))
        Y, Z = t.forward()
        check_forward(t, Y, Z)
        dX, dA, dB = t.backward(Z)
        check_backward(t, Z, dX, dA, dB, False)
        want = {}
        for n, p, g, m in (("A", MA, dA, mA), ("B", MB, dB, mB)):
            want[n] = oo.muon_step(host(p), host(g), host(m), 0.02, 0.95, True, 0.01, "spectral", 5, (3.4445, -4.7750, 2.0315), 1e-7)[0]
        qn.qlora_muon_step(t.A, t.B, dA, dB, mA, mB, 0.02, weight_decay=0.01, A_master=MA, B_master=MB)
        for n, p, q in (("A", MA, t.A), ("B", MB, t.B)):
            # the update's own tests bound it in detail; here within 2^-20 of its elements' scale
            assert np.abs(host(p) - want[n]).max() <= 2.0 ** -20 * (1 + np.abs(want[n]).max())
            np.testing.assert_array_equal(host(q), oo.round16(host(p), "bf16"))


def test_largest_matrices():
    """Just under 2^29 elements each way: rows and blocks at the end are the right ones."""
    import torch
    say("mxfp4 of the largest matrix")
    rows, cols = 65528, 8184
    X = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    X.copy_(torch.arange(rows, device="cuda")[:, None] % 251 - 125)
    X.mul_(((torch.arange(cols, device="cuda") % 13) - 6).to(torch.bfloat16)[None, :])
    chunks = -(-cols // 512)
    kept = qn.mxfp4_quantize(X)
    for i in (0, 17, 32767, 32768, rows - 1):
        x = host(X[i:i + 1])
        codes, scales = oo.mxfp4_quantize(x)
        got = host(kept.codes).reshape(rows, -1)[i] if i == 0 else host(kept.codes.view(rows, -1)[i])
        np.testing.assert_array_equal(got, (codes[0, 0::2] | codes[0, 1::2] << 4))
        b = np.arange(scales.shape[1])
        at = ((i // 16) * chunks + b // 16) * 256 + 4 * (16 * (b % 4) + i % 16) + (b % 16) // 4
        np.testing.assert_array_equal(host(kept.scales[torch.from_numpy(at).cuda()]), scales[0])
    back = qn.mxfp4_dequantize(kept, torch.bfloat16)
    for i in (5, rows - 1):
        np.testing.assert_array_equal(host(back[i]), oo.mxfp4_values(*oo.mxfp4_quantize(host(X[i:i + 1])), cols)[0])
    del back
    # the other way round: the same matrix as columns
    across = qn.mxfp4_quantize(X.T.contiguous(), transpose=True)
    assert torch.equal(across.codes, kept.codes) and torch.equal(across.scales, kept.scales)
    back = qn.mxfp4_dequantize(across, torch.bfloat16, transpose=True)
    assert torch.equal(back[:, rows - 8:], qn.mxfp4_dequantize(kept, torch.bfloat16)[rows - 8:].T)


def test_largest_product():
    import torch
    say("mxfp4 product of nearly 2^29 outputs")
    rng = np.random.default_rng(3)
    M, N, K = 65528, 8184, 40
    p, q = _whole(rng, M, K, -2, 2), _whole(rng, N, K, -2, 2)
    C = qn.mxfp4_matmul(_state(*p, K), _state(*q, K), torch.float32)
    v, w = oo.mxfp4_values(*p, K), oo.mxfp4_values(*q, K)
    for i in (0, 255, 256, 32768, M - 1):
        np.testing.assert_array_equal(host(C[i]), (v[i] @ w.T).astype(np.float32))
    np.testing.assert_array_equal(host(C[:, N - 1]), (v @ w[N - 1]).astype(np.float32))


@pytest.mark.parametrize("M", [1, 20])
def test_widest_layer(M):
    import torch
    say(f"mx layer of 2^24 - 8 columns, {M} rows")
    K, N, r = 8, (1 << 24) - 8, 8
    rng = np.random.default_rng(7)
    codes, scales = _whole(rng, N, K, 0, 0)
    W = _state(codes, scales, K)
    X = torch.from_numpy(rng.choice([-2.0, -1.0, 0.0, 1.0, 2.0], size=(M, K)).astype(np.float32))
    A = torch.zeros(K, r)
    A[0, 0] = 1.0
    B = torch.from_numpy(rng.integers(-2, 3, size=(r, N)).astype(np.float32))
    Y, Z = qn.qlora_mx_linear_fwd(X.bfloat16().cuda(), W, A.bfloat16().cuda(), B.bfloat16().cuda(), 1.0)
    w = oo.mxfp4_values(codes, scales, K)
    for n in (slice(0, 600), slice(N // 2, N // 2 + 600), slice(N - 600, N)):
        want = X.numpy().astype(np.float64) @ w[n].T + X.numpy()[:, :1].astype(np.float64) * B.numpy()[:1, n]
        np.testing.assert_array_equal(host(Y[:, n]), oo.round16(want, "bf16"))


@pytest.mark.parametrize("M,N,K", [(262144, 8, 1032), (131072, 16, 1032), (65536, 32, 2056)])
def test_many_rows_of_few_columns(M, N, K):
    """Whole numbers throughout: X of -2 .. 2, one 1 a column of A, c B of -2 .. 2."""
    import torch
    say(f"mx layer of {M} rows, {N} columns")
    r = 256
    rng = np.random.default_rng(M + N)
    codes, scales = _whole(rng, N, K, 0, 0)
    W, w = _state(codes, scales, K), oo.mxfp4_values(codes, scales, K)
    X = torch.randint(-2, 3, (M, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    a = np.zeros((K, r), dtype=np.float32)
    a[rng.integers(0, K, size=r), np.arange(r)] = 1.0
    b = rng.integers(-2, 3, size=(r, N)).astype(np.float32)
    A, B = (torch.from_numpy(v).bfloat16().cuda() for v in (a, b))
    Y, Z = qn.qlora_mx_linear_fwd(X, W, A, B, 1.0)
    for rows in (slice(0, 300), slice(M // 2 - 150, M // 2 + 150), slice(M - 300, M)):
        x = host(X[rows]).astype(np.float64)
        np.testing.assert_array_equal(host(Z[rows]), x @ a)
        np.testing.assert_array_equal(host(Y[rows]), oo.round16(x @ w.T + x @ a @ b, "bf16"))


@pytest.mark.parametrize("M,K,N,r", [((1 << 20), 8, 8, 8), ((1 << 20), 24, 40, 16), (1, 8, (1 << 24) - 8, 8), (40, 16, 1 << 22, 16),
                                     (1, (1 << 22), 8, 8), (700, (1 << 19) + 8, 8, 8)])
def test_longest_sides_in_whole_numbers(M, K, N, r):
    """Forward and backward with one side at the end of its range.  A and B hold a 1 a row
    or column at most, G few elements, so that every sum is exact and Z and dZ are whole
    numbers of at most eight bits."""
    import torch
    say(f"mx layer M={M} K={K} N={N} r={r}")
    rng = np.random.default_rng(M % 1000 + K % 1000 + N % 1000)
    gen = torch.Generator(device="cuda").manual_seed(2)
    codes, scales = _whole(rng, N, K, 0, 0)
    W, w = _state(codes, scales, K), torch.from_numpy(oo.mxfp4_values(codes, scales, K)).cuda()

    def sparse(rows, cols, count, high):
        v = torch.zeros(rows * cols, dtype=torch.float64, device="cuda")
        at = torch.randint(0, rows * cols, (count,), device="cuda", generator=gen)
        v[at] = torch.randint(-high, high + 1, (count,), device="cuda", generator=gen).double()
        return v.view(rows, cols)

    x = torch.randint(-2, 3, (M, K), device="cuda", generator=gen).double() if K < 1 << 12 else sparse(M, K, 60 * M, 2)
    x[:, :1] = 2.0       # every row's first block has scale 1/2; the others hold -2 .. 2 too
    a, b, g = sparse(K, r, 64, 1), sparse(r, N, min(r * N, 4096), 1), sparse(M, N, min(M * N // 2 + 1, 30 * max(1, M // 100)), 1)
    X, A, B, G = (v.bfloat16() for v in (x, a, b, g))
    Y, Z = qn.qlora_mx_linear_fwd(X, W, A, B, 1.0)
    z = x @ a
    assert float(z.abs().max()) <= 256
    assert torch.equal(Z.double(), z)
    for i in range(0, N, 1 << 18):
        n = slice(i, i + (1 << 18))
        for j in range(0, M, 1 << 18):
            m = slice(j, j + (1 << 18))
            want = x[m] @ w[n].T.contiguous() + z[m] @ b[:, n].contiguous()
            assert torch.equal(Y[m, n], want.float().bfloat16())
    dX, dA, dB = qn.qlora_mx_linear_bwd(G, X, Z, W, A, B, 1.0)
    dz = g @ b.T.contiguous()
    assert float(dz.abs().max()) <= 256
    assert torch.equal(dA.double(), x.T.contiguous() @ dz)
    assert torch.equal(dB.double(), z.T.contiguous() @ g)
    assert torch.equal(dX, (g @ w + dz @ a.T.contiguous()).float().bfloat16())


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_gradient_of_a_where_few_channels_are_large(name):
    """dA comes from dZ before its rounding: two 16-bit parts hold it within half a step
    of half a step."""
    import torch
    from tests.test_gpu_mx_linear import F32, HALF, TINY, close
    say(f"mx dA with large channels {name}")
    t = Case(300, 520, 264, 16, name)
    t.X[:, 7] *= 40.0
    t.X[:, 300] *= 100.0
    t.x = host(t.X).astype(np.float64)
    Y, Z = t.forward()
    dX, dA, dB = t.backward(Z, need_dx=False)
    _, want, _ = oo.mx_linear_backward(t.g, t.x, host(Z).astype(np.float64), t.w, t.a, t.b, t.c)
    dz = abs(t.c) * np.abs(t.g @ t.b.T)
    near = HALF[name] ** 2 * dz + 1.01 * abs(t.c) * t.N * F32 * (np.abs(t.g) @ np.abs(t.b).T) + TINY[name]
    close(dA, want, 1.01 * (np.abs(t.x).T @ near) + 2 * t.M * F32 * (np.abs(t.x).T @ dz), "dA")
