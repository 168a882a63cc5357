"""Python binding of the MI355X QLoRA NF4 library (libqlora_nf4.so).

Argument marshalling only: every step of the path runs in the HIP kernels
behind the C ABI declared in include/qlora_nf4.h.  PyTorch provides device
memory and the current stream.  There is no CPU fallback: if the library is
not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqlora_nf4.so")

NF4_OK, NF4_EINVAL, NF4_ENONFINITE, NF4_EPADDING, NF4_EHIP = 0, 1, 2, 4, 8
NF4_OUT_F32, NF4_OUT_BF16, NF4_OUT_F16 = 0, 1, 2
NF4_COMPUTE_BF16, NF4_COMPUTE_F16 = 0, 1
KERNEL_IDS = {
    "quant_pass1": 0, "quant_mean": 1, "quant_pass2": 2, "dequant": 3, "lora_down": 4,
    "fwd_gemm": 5, "fwd_gemv": 6, "bwd_dz": 7, "bwd_dx": 8, "bwd_colsum": 9, "dequant_bf16": 10,
    "reduce": 11, "merge": 12, "sgd": 13, "act8_encode": 14, "act8_decode": 15, "gated_fwd": 16, "gated_dy": 17,
    "head_logits": 18, "head_rows": 19, "head_dx": 20,
}
C_FUNCTIONS = [
    "nf4_sizes", "nf4_quantize", "nf4_dequantize", "qlora_workspace_bytes",
    "qlora_linear_fwd", "qlora_linear_bwd", "nf4_status_read", "qlora_timer_enable",
    "qlora_timer_read", "qlora_merge", "qlora_sgd_step", "qlora_grouped_workspace_bytes",
    "qlora_grouped_fwd", "qlora_grouped_bwd", "qlora_linear_fwd_dt", "qlora_linear_bwd_dt", "qlora_sgd_step_dt",
    "qlora_linear_fwd_noalloc", "qlora_grouped_fwd_dt", "qlora_grouped_bwd_dt",
    "act8_encode", "act8_decode", "qlora_linear_bwd_ex",
    "qlora_gated_workspace_bytes", "qlora_gated_fwd", "qlora_gated_bwd", "qlora_head_workspace_bytes", "qlora_head_loss",
    "nf4_error_string",
]
NF4_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class NF4Error(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: error {code}")
        self.code = code


class _State(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("codes", ctypes.c_void_p), ("qabsmax", ctypes.c_void_p),
                ("absmax2", ctypes.c_void_p), ("offset", ctypes.c_void_p), ("absmax", ctypes.c_void_p)]


class _Act8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_nf4_quantized_10_amd.build_lib`")
        # PyTorch brings its own HIP and HSA runtimes.  Loaded first, they
        # satisfy this library's libamdhip64 dependency, so the process holds
        # one HSA runtime; loaded the other way round, the process ends up
        # with two, and the second cannot reach the GPU.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, i32p = ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p
        sp = ctypes.POINTER(_State)
        L.nf4_sizes.argtypes = [i64] + [ctypes.POINTER(i64)] * 4
        L.nf4_quantize.argtypes = [vp, sp, vp, i64, i32p, vp]
        L.nf4_dequantize.argtypes = [sp, vp, ctypes.c_int, i32p, vp]
        L.qlora_workspace_bytes.argtypes = [i64, i64, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.qlora_linear_fwd.argtypes = [i64, i64, i64, i64, vp, sp, vp, vp, ctypes.c_float, vp, vp, vp, i64, vp]
        L.qlora_linear_bwd.argtypes = [i64, i64, i64, i64, vp, vp, vp, sp, vp, vp, ctypes.c_float,
                                       vp, vp, vp, vp, i64, vp]
        L.nf4_status_read.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
        L.qlora_timer_enable.argtypes = [ctypes.c_int, ctypes.c_int]
        L.qlora_timer_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)]
        L.qlora_merge.argtypes = [i64, i64, i64, sp, vp, vp, ctypes.c_int, ctypes.c_float, vp, vp]
        L.qlora_sgd_step.argtypes = [i64, i64, i64, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]
        i64p = ctypes.POINTER(i64)
        L.qlora_grouped_workspace_bytes.argtypes = [i64, i64, ctypes.c_int, i64p, i64, i64p, i64p]
        L.qlora_grouped_fwd.argtypes = [i64, i64, ctypes.c_int, i64p, i64, vp, sp, vp, vp, ctypes.c_float,
                                        vp, vp, vp, i64, vp]
        L.qlora_grouped_bwd.argtypes = [i64, i64, ctypes.c_int, i64p, i64, vp, vp, vp, sp, vp, vp, ctypes.c_float,
                                        vp, vp, vp, vp, i64, vp]
        L.qlora_linear_fwd_dt.argtypes = [ctypes.c_int] + L.qlora_linear_fwd.argtypes
        L.qlora_linear_bwd_dt.argtypes = [ctypes.c_int] + L.qlora_linear_bwd.argtypes
        L.qlora_sgd_step_dt.argtypes = [ctypes.c_int] + L.qlora_sgd_step.argtypes
        L.qlora_linear_fwd_noalloc.argtypes = [i64, i64, i64, i64, vp, sp, vp, vp, ctypes.c_float, vp, vp, vp]
        L.qlora_grouped_fwd_dt.argtypes = [ctypes.c_int] + L.qlora_grouped_fwd.argtypes
        L.qlora_grouped_bwd_dt.argtypes = [ctypes.c_int] + L.qlora_grouped_bwd.argtypes
        a8 = ctypes.POINTER(_Act8)
        L.act8_encode.argtypes = [ctypes.c_int, i64, i64, vp, i64, a8, vp]
        L.act8_decode.argtypes = [ctypes.c_int, i64, i64, a8, vp, i64, vp]
        L.qlora_linear_bwd_ex.argtypes = [ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, vp, vp, a8, vp, sp, vp, vp,
                                          ctypes.c_float, vp, vp, vp, vp, i64, vp]
        L.qlora_gated_workspace_bytes.argtypes = L.qlora_workspace_bytes.argtypes
        L.qlora_gated_fwd.argtypes = [ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, vp, sp, vp, vp, ctypes.c_float,
                                      vp, vp, vp, a8, vp, i64, vp]
        L.qlora_gated_bwd.argtypes = [ctypes.c_int] * 3 + [i64, i64, i64, i64, vp, vp, a8, vp, vp, a8, sp, vp, vp,
                                                           ctypes.c_float, vp, vp, vp, vp, i64, vp]
        L.qlora_head_workspace_bytes.argtypes = [i64, i64, i64, ctypes.c_int, i64p]
        L.qlora_head_loss.argtypes = [ctypes.c_int, i64, i64, i64, vp, vp, vp, vp, i64, vp, vp, vp, vp, i64, vp]
        L.nf4_error_string.argtypes = [ctypes.c_int]
        L.nf4_error_string.restype = ctypes.c_char_p
        for name in C_FUNCTIONS[:-1]:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int, what: str) -> None:
    if rc != NF4_OK:
        raise NF4Error(rc, f"{what} ({lib().nf4_error_string(rc).decode()})")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _require_cuda(t, name: str, dtype=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


class _on:
    """The scope in which a call on tensor t allocates and launches: t's
    device current and, where one is given, `stream` current, so that outputs
    and workspaces belong to the stream that the kernels run on.  Yields that
    stream's handle.  The other tensors must be on the same device."""
    __slots__ = ("device", "stream", "scope")

    def __init__(self, t, stream=None, *others):
        self.device = d = t.device
        for o in others:
            if o is not None and o.device != d:
                raise ValueError(f"tensors on {d} and {o.device}")
        if stream is not None and stream.device != d:
            raise ValueError(f"tensors on {d}, stream on {stream.device}")
        self.stream = stream
        self.scope = None

    def __enter__(self):
        import torch
        if self.stream is not None:
            self.scope = torch.cuda.stream(self.stream)
        elif self.device.index != torch._C._cuda_getDevice():
            self.scope = torch.cuda.device(self.device)
        if self.scope is not None:
            self.scope.__enter__()
        # the handle of torch.cuda.current_stream(), without making a Stream of it
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *e):
        if self.scope is not None:
            self.scope.__exit__(*e)


def _require_shape(t, name: str, *shape) -> None:
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {' x '.join(map(str, shape))}, got {tuple(t.shape)}")


@dataclass
class Act8:
    """An M x K matrix of activations kept in 8 bits (device tensors): int8
    codes and, per row and block of 64 columns, the largest magnitude in the
    activations' 16-bit type.  Made by act8_encode."""
    codes: "torch.Tensor"     # int8, M x K
    absmax: "torch.Tensor"    # bf16 or fp16, M x ceil(K / 64)

    @property
    def shape(self):
        return self.codes.shape

    @property
    def dtype(self):
        return self.absmax.dtype

    @property
    def device(self):
        return self.codes.device

    def c_struct(self) -> _Act8:
        return _Act8(self.codes.data_ptr(), self.absmax.data_ptr())

    def check(self, name: str) -> None:
        import torch
        _require_cuda(self.codes, f"{name}.codes", torch.int8)
        if self.codes.dim() != 2:
            raise ValueError(f"{name}.codes must be a matrix")
        _require_cuda(self.absmax, f"{name}.absmax", _compute_dtype(self.absmax))
        _require_shape(self.absmax, f"{name}.absmax", self.codes.shape[0], (self.codes.shape[1] + 63) // 64)
        if self.absmax.device != self.codes.device:
            raise ValueError(f"{name}'s tensors must be on one device")


def empty_act8(rows: int, cols: int, dtype, device="cuda") -> Act8:
    import torch
    return Act8(torch.empty(rows, cols, dtype=torch.int8, device=device),
                torch.empty(rows, (cols + 63) // 64, dtype=dtype, device=device))


def _require_matrix(t, name: str) -> int:
    """A device matrix of the compute types whose rows are contiguous; returns
    its row stride."""
    _compute_dtype(t)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() == 2 and t.is_contiguous():
        return t.shape[1]
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def act8_encode(X, out: Act8 | None = None, stream=None) -> Act8:
    """Keep the bf16 or fp16 matrix X (M x K, K % 8 == 0; rows may be strided
    by a multiple of 8 elements) in 8 bits."""
    ld = _require_matrix(X, "X")
    M, K = X.shape
    if out is not None:
        out.check("out")
        _require_shape(out.codes, "out.codes", M, K)
        _require_cuda(out.absmax, "out.absmax", X.dtype)
    with _on(X, stream, None if out is None else out.codes) as s:
        if out is None:
            out = empty_act8(M, K, X.dtype, X.device)
        st = out.c_struct()
        _check(lib().act8_encode(_COMPUTE[X.dtype], M, K, X.data_ptr(), ld, ctypes.byref(st), s), "act8_encode")
    return out


def act8_decode(kept: Act8, out=None, stream=None):
    """The M x K values that `kept` stands for, in its 16-bit type."""
    import torch
    kept.check("kept")
    M, K = kept.shape
    ld = K
    if out is not None:
        if out.dtype != kept.dtype:
            raise ValueError(f"out must be {kept.dtype}, got {out.dtype}")
        ld = _require_matrix(out, "out")
        _require_shape(out, "out", M, K)
    with _on(kept.codes, stream, out) as s:
        if out is None:
            out = torch.empty(M, K, dtype=kept.dtype, device=kept.device)
        st = kept.c_struct()
        _check(lib().act8_decode(_COMPUTE[kept.dtype], M, K, ctypes.byref(st), out.data_ptr(), ld, s), "act8_decode")
    return out


@dataclass
class NF4State:
    """Frozen NF4 state of one weight tensor (device tensors).  Double
    quantized: qabsmax / absmax2 / offset set, absmax None.  Single level
    (double quantization off): absmax set, the other three None."""
    numel: int
    codes: "torch.Tensor"             # uint8[ceil(P/2)]
    qabsmax: "torch.Tensor | None"    # int8[n1]
    absmax2: "torch.Tensor | None"    # float32[n2]
    offset: "torch.Tensor | None"     # float32[1]
    absmax: "torch.Tensor | None" = None   # float32[n1]

    @property
    def double_quant(self) -> bool:
        return self.absmax is None

    def c_struct(self) -> _State:
        return _State(self.numel, self.codes.data_ptr(), _ptr(self.qabsmax), _ptr(self.absmax2),
                      _ptr(self.offset), _ptr(self.absmax))

    def check(self, name: str, device) -> None:
        """Raises where a tensor is not what numel weights need, on `device`."""
        n1 = (self.numel + 63) // 64
        _require_part(self.codes, name, "codes", "torch.uint8", (self.numel + 1) // 2, device)
        if self.absmax is None:
            _require_part(self.qabsmax, name, "qabsmax", "torch.int8", n1, device)
            _require_part(self.absmax2, name, "absmax2", "torch.float32", (n1 + 255) // 256, device)
            _require_part(self.offset, name, "offset", "torch.float32", 1, device)
        else:
            _require_part(self.absmax, name, "absmax", "torch.float32", n1, device)


def _require_part(t, name: str, part: str, dtype: str, count: int, device) -> None:
    if t is None or t.device != device or str(t.dtype) != dtype or t.numel() < count or not t.is_contiguous():
        raise ValueError(f"{name}.{part} must be {count} contiguous {dtype} on {device}")


def nf4_sizes(numel: int) -> dict:
    out = [ctypes.c_int64() for _ in range(4)]
    _check(lib().nf4_sizes(numel, *[ctypes.byref(o) for o in out]), "nf4_sizes")
    return dict(zip(("code_bytes", "n1", "n2", "quant_workspace_bytes"), (o.value for o in out)))


def empty_state(numel: int, device="cuda", double_quant: bool = True) -> NF4State:
    import torch
    s = nf4_sizes(numel)
    codes = torch.empty(s["code_bytes"], dtype=torch.uint8, device=device)
    if not double_quant:
        return NF4State(numel, codes, None, None, None, torch.empty(s["n1"], dtype=torch.float32, device=device))
    return NF4State(numel, codes,
                    torch.empty(s["n1"], dtype=torch.int8, device=device),
                    torch.empty(s["n2"], dtype=torch.float32, device=device),
                    torch.empty(1, dtype=torch.float32, device=device))


def nf4_quantize(W, state: NF4State | None = None, workspace=None, status=None, stream=None,
                 double_quant: bool = True):
    """Encode fp32 weights (any shape, flattened row-major) into an NF4State
    (single level when double_quant is False or the given state has absmax).
    Returns (state, status) where status is the device int32 status word."""
    import torch
    _require_cuda(W, "W", torch.float32)
    P = W.numel()
    if state is None:
        state = empty_state(P, W.device, double_quant)
    sizes = nf4_sizes(P)
    if workspace is None:
        workspace = torch.empty(sizes["quant_workspace_bytes"], dtype=torch.uint8, device=W.device)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=W.device)
    st = state.c_struct()
    _check(lib().nf4_quantize(W.data_ptr(), ctypes.byref(st), workspace.data_ptr(), workspace.numel(),
                              status.data_ptr(), _stream(stream)), "nf4_quantize")
    return state, status


def nf4_dequantize(state: NF4State, out_dtype: str = "bf16", out=None, status=None, stream=None):
    """ŵ as fp32 ("fp32"), bf16 ("bf16") or fp16 ("f16")."""
    import torch
    dt, code = {"bf16": (torch.bfloat16, NF4_OUT_BF16), "f16": (torch.float16, NF4_OUT_F16),
                "fp32": (torch.float32, NF4_OUT_F32)}[out_dtype]
    if out is None:
        out = torch.empty(state.numel, dtype=dt, device=state.codes.device)
    st = state.c_struct()
    _check(lib().nf4_dequantize(ctypes.byref(st), out.data_ptr(), code, _ptr(status), _stream(stream)),
           "nf4_dequantize")
    return out


def _group_args(states, Ns):
    g = len(Ns)
    if len(states) != g or not 1 <= g <= 8:
        raise ValueError("one state per member, 1 to 8 members")
    return g, (ctypes.c_int64 * g)(*Ns), (_State * g)(*[s.c_struct() for s in states])


def qlora_grouped_workspace_bytes(M: int, K: int, Ns, r: int) -> tuple[int, int]:
    f, b = ctypes.c_int64(), ctypes.c_int64()
    arr = (ctypes.c_int64 * len(Ns))(*Ns)
    _check(lib().qlora_grouped_workspace_bytes(M, K, len(Ns), arr, r, ctypes.byref(f), ctypes.byref(b)),
           "qlora_grouped_workspace_bytes")
    return f.value, b.value


def qlora_grouped_fwd(X, states, A, B, c: float, K: int, Ns, Y=None, Z=None, workspace=None, stream=None):
    """Members sharing X, side by side: A = [A_i] (K x g r), B = [B_i] (r x sum N),
    returns (Y = [Y_i] (M x sum N), Z = [Z_i] (M x g r)).  The compute type is
    X's dtype (bf16 or fp16); A, B, Y and Z share it."""
    import torch
    g, Narr, Sarr = _group_args(states, Ns)
    M = X.shape[0]
    r = A.shape[1] // g
    Ntot = sum(Ns)
    dt = _compute_dtype(X)
    for t, n in ((X, "X"), (A, "A"), (B, "B")):
        _require_cuda(t, n, dt)
    if Y is None:
        Y = torch.empty(M, Ntot, dtype=dt, device=X.device)
    if Z is None:
        Z = torch.empty(M, g * r, dtype=dt, device=X.device)
    _require_cuda(Y, "Y", dt)
    _require_cuda(Z, "Z", dt)
    if workspace is None:
        workspace = torch.empty(max(qlora_grouped_workspace_bytes(M, K, Ns, r)[0], 256), dtype=torch.uint8,
                                device=X.device)
    _check(lib().qlora_grouped_fwd_dt(_COMPUTE[dt], M, K, g, Narr, r, X.data_ptr(), Sarr, A.data_ptr(),
                                      B.data_ptr(), ctypes.c_float(c), Y.data_ptr(), Z.data_ptr(),
                                      workspace.data_ptr(), workspace.numel(), _stream(stream)),
           "qlora_grouped_fwd_dt")
    return Y, Z


def qlora_grouped_bwd(G, X, Z, states, A, B, c: float, K: int, Ns, need_dx: bool = True, dX=None, dA=None,
                      dB=None, workspace=None, stream=None):
    """Returns (dX or None, dA = [dA_i] (K x g r fp32), dB = [dB_i] (r x sum N fp32)).
    The compute type is X's dtype (bf16 or fp16); G, Z, A, B and dX share it."""
    import torch
    g, Narr, Sarr = _group_args(states, Ns)
    M = X.shape[0]
    r = A.shape[1] // g
    Ntot = sum(Ns)
    dt = _compute_dtype(X)
    for t, n in ((G, "G"), (X, "X"), (Z, "Z"), (A, "A"), (B, "B")):
        _require_cuda(t, n, dt)
    if need_dx and dX is None:
        dX = torch.empty(M, K, dtype=dt, device=X.device)
    if need_dx:
        _require_cuda(dX, "dX", dt)
    if dA is None:
        dA = torch.empty(K, g * r, dtype=torch.float32, device=X.device)
    if dB is None:
        dB = torch.empty(r, Ntot, dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(max(qlora_grouped_workspace_bytes(M, K, Ns, r)[1], 256), dtype=torch.uint8,
                                device=X.device)
    _check(lib().qlora_grouped_bwd_dt(_COMPUTE[dt], M, K, g, Narr, r, G.data_ptr(), X.data_ptr(), Z.data_ptr(),
                                      Sarr, A.data_ptr(), B.data_ptr(), ctypes.c_float(c),
                                      dX.data_ptr() if need_dx else None, dA.data_ptr(), dB.data_ptr(),
                                      workspace.data_ptr(), workspace.numel(), _stream(stream)),
           "qlora_grouped_bwd_dt")
    return (dX if need_dx else None), dA, dB


NF4_AB_BF16, NF4_AB_F32, NF4_AB_F16 = 0, 1, 2


class _ComputeMap(dict):
    """torch dtype -> NF4_COMPUTE_* code (torch is imported lazily)."""

    def __missing__(self, dt):
        import torch
        self.update({torch.bfloat16: NF4_COMPUTE_BF16, torch.float16: NF4_COMPUTE_F16})
        return dict.__getitem__(self, dt)


_COMPUTE = _ComputeMap()


def _compute_dtype(X):
    dt = X.dtype
    if dt not in _COMPUTE:
        import torch
        if dt not in (torch.bfloat16, torch.float16):
            raise ValueError(f"the compute type is bf16 or fp16, got {dt}")
    return dt


def qlora_merge(state: NF4State, A, B, c: float, K: int, N: int, out=None, stream=None):
    """W' = fl32(ŵ + c A B) as a K*N fp32 tensor (A: K x r, B: r x N, both
    bf16 or both fp32); pass it to nf4_quantize to re-quantize."""
    import torch
    r = A.shape[1]
    if A.dtype != B.dtype or A.dtype not in (torch.bfloat16, torch.float32, torch.float16):
        raise ValueError("A and B must both be bf16, both fp16 or both fp32")
    for t, n in ((A, "A"), (B, "B")):
        _require_cuda(t, n, A.dtype)
    if tuple(A.shape) != (K, r) or tuple(B.shape) != (r, N):
        raise ValueError("A must be K x r and B r x N")
    if out is None:
        out = torch.empty(K * N, dtype=torch.float32, device=A.device)
    st = state.c_struct()
    _check(lib().qlora_merge(K, N, r, ctypes.byref(st), A.data_ptr(), B.data_ptr(),
                             {torch.float32: NF4_AB_F32, torch.float16: NF4_AB_F16}.get(A.dtype, NF4_AB_BF16),
                             ctypes.c_float(c),
                             out.data_ptr(), _stream(stream)), "qlora_merge")
    return out


def qlora_merge_requantize(state: NF4State, A, B, c: float, K: int, N: int, stream=None):
    """Merge, then re-quantize: returns (new NF4State, device status word)."""
    return nf4_quantize(qlora_merge(state, A, B, c, K, N, stream=stream), stream=stream)


def qlora_sgd_step(A, B, dA, dB, lr: float, A_master=None, B_master=None, stream=None) -> None:
    """In-place SGD step on the bf16 or fp16 adapter (optionally through fp32 masters)."""
    import torch
    K, r = A.shape
    N = B.shape[1]
    pdt = _compute_dtype(A)
    for t, n, dt in ((A, "A", pdt), (B, "B", pdt), (dA, "dA", torch.float32),
                     (dB, "dB", torch.float32)):
        _require_cuda(t, n, dt)
    for m, n in ((A_master, "A_master"), (B_master, "B_master")):
        if m is not None:
            _require_cuda(m, n, torch.float32)
    _check(lib().qlora_sgd_step_dt(_COMPUTE[pdt], K, N, r, A.data_ptr(), B.data_ptr(), dA.data_ptr(),
                                   dB.data_ptr(), ctypes.c_float(lr), _ptr(A_master), _ptr(B_master),
                                   _stream(stream)), "qlora_sgd_step_dt")


def nf4_status_read(status, stream=None) -> int:
    v = ctypes.c_int32()
    _check(lib().nf4_status_read(status.data_ptr(), ctypes.byref(v), _stream(stream)), "nf4_status_read")
    return v.value


def qlora_workspace_bytes(M: int, K: int, N: int, r: int) -> tuple[int, int]:
    f, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().qlora_workspace_bytes(M, K, N, r, ctypes.byref(f), ctypes.byref(b)), "qlora_workspace_bytes")
    return f.value, b.value


def qlora_linear_fwd(X, state: NF4State, A, B, c: float, K: int, N: int, Y=None, Z=None,
                     workspace=None, stream=None, return_z: bool = True):
    """Y = X Ŵ + c (X A) B.  X: M x K, A: K x r, B: r x N, all bf16 or all fp16
    (the compute type).  Returns (Y, Z); with return_z=False and no Z given,
    Z stays in the workspace and (Y, None) is returned."""
    import torch
    M, r = X.shape[0], A.shape[1]
    dt = _compute_dtype(X)
    for t, n in ((X, "X"), (A, "A"), (B, "B")):
        _require_cuda(t, n, dt)
    if Y is None:
        Y = torch.empty(M, N, dtype=dt, device=X.device)
    if Z is None and return_z:
        Z = torch.empty(M, r, dtype=dt, device=X.device)
    if workspace is None:
        workspace = torch.empty(max(qlora_workspace_bytes(M, K, N, r)[0], 256), dtype=torch.uint8,
                                device=X.device)
    st = state.c_struct()
    _check(lib().qlora_linear_fwd_dt(_COMPUTE[dt], M, K, N, r, X.data_ptr(), ctypes.byref(st), A.data_ptr(),
                                     B.data_ptr(), float(c), Y.data_ptr(), _ptr(Z), workspace.data_ptr(),
                                     workspace.numel(), _stream(stream)), "qlora_linear_fwd_dt")
    return Y, Z


def qlora_linear_fwd_noalloc(X, state: NF4State, A, B, c: float, K: int, N: int, Y, Z=None, stream=None):
    """qlora_linear_fwd (bf16) with the library's own device scratch instead
    of a workspace: allocates nothing.  Y (and Z, if given) must be passed
    in.  Shapes whose forward workspace exceeds NF4_NOALLOC_SCRATCH_BYTES
    are rejected.  Returns (Y, Z)."""
    import torch
    M, r = X.shape[0], A.shape[1]
    for t, n in ((X, "X"), (A, "A"), (B, "B"), (Y, "Y")):
        _require_cuda(t, n, torch.bfloat16)
    if Z is not None:
        _require_cuda(Z, "Z", torch.bfloat16)
    st = state.c_struct()
    _check(lib().qlora_linear_fwd_noalloc(M, K, N, r, X.data_ptr(), ctypes.byref(st), A.data_ptr(), B.data_ptr(),
                                          float(c), Y.data_ptr(), _ptr(Z), _stream(stream)),
           "qlora_linear_fwd_noalloc")
    return Y, Z


def qlora_linear_bwd(G, X, Z, state: NF4State, A, B, c: float, K: int, N: int, need_dx: bool = True,
                     dX=None, dA=None, dB=None, workspace=None, stream=None, grad_dtype=None):
    """dZ = c G Bᵀ, dA = Xᵀ dZ, dB = c Zᵀ G, dX = G Ŵᵀ + dZ Aᵀ.  Returns (dX, dA, dB).
    Z = None recomputes Z = X A in the workspace.  X may be an Act8 (kept in 8
    bits; Z is then required).  grad_dtype: of dA and dB, float32 (the default)
    or X's dtype."""
    import torch
    if isinstance(X, Act8) or grad_dtype not in (None, torch.float32):
        return _linear_bwd_ex(G, X, Z, state, A, B, c, K, N, need_dx, dX, dA, dB, workspace, stream, grad_dtype)
    M, r = X.shape[0], A.shape[1]
    dt = _compute_dtype(X)
    for t, n in ((G, "G"), (X, "X"), (Z, "Z"), (A, "A"), (B, "B")):
        if t is not None or n != "Z":
            _require_cuda(t, n, dt)
    for t, n, odt, count in ((dX if need_dx else None, "dX", dt, M * K), (dA, "dA", torch.float32, K * r),
                             (dB, "dB", torch.float32, r * N)):
        if t is not None:
            _require_cuda(t, n, odt)
            if t.numel() < count:
                raise ValueError(f"{n} must hold {count} elements, got {t.numel()}")
    if need_dx and dX is None:
        dX = torch.empty(M, K, dtype=dt, device=X.device)
    if dA is None:
        dA = torch.empty(K, r, dtype=torch.float32, device=X.device)
    if dB is None:
        dB = torch.empty(r, N, dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(max(qlora_workspace_bytes(M, K, N, r)[1], 256), dtype=torch.uint8,
                                device=X.device)
    st = state.c_struct()
    _check(lib().qlora_linear_bwd_dt(_COMPUTE[dt], M, K, N, r, G.data_ptr(), X.data_ptr(), _ptr(Z),
                                     ctypes.byref(st), A.data_ptr(), B.data_ptr(), float(c),
                                     _ptr(dX if need_dx else None), dA.data_ptr(), dB.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), _stream(stream)), "qlora_linear_bwd_dt")
    return (dX if need_dx else None), dA, dB


def _grad_code(grad_dtype, dt) -> tuple:
    """(torch dtype, NF4_AB_* code) of adapter gradients for compute type dt."""
    import torch
    if grad_dtype in (None, torch.float32):
        return torch.float32, NF4_AB_F32
    if grad_dtype != dt:
        raise ValueError(f"grad_dtype is float32 or the compute type {dt}, got {grad_dtype}")
    return dt, NF4_AB_F16 if dt == torch.float16 else NF4_AB_BF16


def _out(t, name: str, dtype, device, *shape):
    """A given output, checked, or a new one."""
    import torch
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    _require_cuda(t, name, dtype)
    _require_shape(t, name, *shape)
    return t


def _workspace(workspace, need: int, device):
    import torch
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")
    return workspace


def _kept_or_dense(X, M: int, K: int, name: str):
    """(device pointer or None, _Act8 or None) of an input given in 16 or 8 bits."""
    if isinstance(X, Act8):
        X.check(name)
        _require_shape(X.codes, f"{name}.codes", M, K)
        return None, X.c_struct()
    _require_shape(X, name, M, K)
    return X.data_ptr(), None


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _linear_bwd_ex(G, X, Z, state, A, B, c, K, N, need_dx, dX, dA, dB, workspace, stream, grad_dtype):
    M, r = X.shape[0], A.shape[1]
    dt = _compute_dtype(X)
    for t, n, shape in ((G, "G", (M, N)), (Z, "Z", (M, r)), (A, "A", (K, r)), (B, "B", (r, N))):
        if t is not None or n != "Z":
            _require_cuda(t, n, dt)
            _require_shape(t, n, *shape)
    if not isinstance(X, Act8):
        _require_cuda(X, "X", dt)
    elif Z is None:
        raise ValueError("Z is required where X is kept in 8 bits")
    xp, x8 = _kept_or_dense(X, M, K, "X")
    gdt, gcode = _grad_code(grad_dtype, dt)
    state.check("state", G.device)
    with _on(G, stream, X, Z, A, B, dX, dA, dB, workspace) as s:
        dX = _out(dX, "dX", dt, G.device, M, K) if need_dx else None
        dA = _out(dA, "dA", gdt, G.device, K, r)
        dB = _out(dB, "dB", gdt, G.device, r, N)
        ws = _workspace(workspace, qlora_workspace_bytes(M, K, N, r)[1], G.device)
        st = state.c_struct()
        _check(lib().qlora_linear_bwd_ex(_COMPUTE[dt], gcode, M, K, N, r, G.data_ptr(), xp, _ref(x8), _ptr(Z),
                                         ctypes.byref(st), A.data_ptr(), B.data_ptr(), float(c), _ptr(dX),
                                         dA.data_ptr(), dB.data_ptr(), ws.data_ptr(), ws.numel(), s),
               "qlora_linear_bwd_ex")
    return dX, dA, dB


NF4_ACT_SILU, NF4_ACT_GELU = 0, 1
_ACTS = {"silu": NF4_ACT_SILU, "gelu": NF4_ACT_GELU}


def qlora_gated_workspace_bytes(M: int, K: int, F: int, r: int) -> tuple[int, int]:
    f, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().qlora_gated_workspace_bytes(M, K, F, r, ctypes.byref(f), ctypes.byref(b)),
           "qlora_gated_workspace_bytes")
    return f.value, b.value


def _gated_args(X, states, A, B, K: int, F: int, act: str):
    """Checks shared by the gated calls: (M, r, compute dtype, states array, act code)."""
    if act not in _ACTS:
        raise ValueError(f"act is one of {sorted(_ACTS)}, got {act!r}")
    if len(states) != 2:
        raise ValueError("two states: the gate's weight and the up weight")
    M, r2 = X.shape[0], A.shape[1]
    dt = _compute_dtype(X)
    if r2 % 2:
        raise ValueError("A must be K x 2r: the gate's adapter and the up adapter side by side")
    _require_cuda(A, "A", dt)
    _require_cuda(B, "B", dt)
    _require_shape(A, "A", K, r2)
    _require_shape(B, "B", r2 // 2, 2 * F)
    for i, state in enumerate(states):
        state.check(f"states[{i}]", A.device)
    return M, r2 // 2, dt, (_State * 2)(*[s.c_struct() for s in states]), _ACTS[act]


def _gated_kept(saved, M: int, F: int, dt):
    """(GU pointer or None, _Act8 or None) of a gated forward's kept pair."""
    if saved is None:
        return None, None
    if saved.dtype != dt:
        raise ValueError(f"saved must be of {dt}, got {saved.dtype}")
    if not isinstance(saved, Act8):
        _require_cuda(saved, "saved")
    return _kept_or_dense(saved, M, 2 * F, "saved")


def qlora_gated_fwd(X, states, A, B, c: float, K: int, F: int, act: str = "silu", save: str = "none", H=None, Z=None,
                    saved=None, workspace=None, stream=None, return_z: bool = True):
    """H = act(G) * U with G = X Ŵ0 + c Zg Bg, U = X Ŵ1 + c Zu Bu, [Zg | Zu] = X A.
    X: M x K, A = [Ag | Au] (K x 2r), B = [Bg | Bu] (r x 2F), all bf16 or all
    fp16; states: the gate's and the up weight (K x F).  save: what is kept of
    [G | U] (M x 2F) for the backward: "none", "16" (a tensor) or "8" (an
    Act8); a given `saved` of either kind is filled instead.  Returns
    (H, Z, saved); with return_z=False and no Z given, Z is None."""
    if save not in ("none", "16", "8"):
        raise ValueError(f'save is "none", "16" or "8", got {save!r}')
    M, r, dt, st, code = _gated_args(X, states, A, B, K, F, act)
    _require_cuda(X, "X", dt)
    _require_shape(X, "X", M, K)
    import torch
    with _on(X, stream, A, B, H, Z, saved, workspace) as s:
        H = _out(H, "H", dt, X.device, M, F)
        if Z is not None or return_z:
            Z = _out(Z, "Z", dt, X.device, M, 2 * r)
        if saved is None and save == "16":
            saved = torch.empty(M, 2 * F, dtype=dt, device=X.device)
        elif saved is None and save == "8":
            saved = empty_act8(M, 2 * F, dt, X.device)
        gu, gu8 = _gated_kept(saved, M, F, dt)
        ws = _workspace(workspace, qlora_gated_workspace_bytes(M, K, F, r)[0], X.device)
        _check(lib().qlora_gated_fwd(_COMPUTE[dt], code, M, K, F, r, X.data_ptr(), st, A.data_ptr(), B.data_ptr(),
                                     float(c), H.data_ptr(), _ptr(Z), gu, _ref(gu8), ws.data_ptr(), ws.numel(), s),
               "qlora_gated_fwd")
    return H, Z, saved


def qlora_gated_bwd(dH, X, Z, saved, states, A, B, c: float, K: int, F: int, act: str = "silu", need_dx: bool = True,
                    grad_dtype=None, dX=None, dA=None, dB=None, workspace=None, stream=None):
    """Backward of qlora_gated_fwd given dH (M x F): (dX or None, dA (K x 2r),
    dB (r x 2F)).  saved: the forward's (None: G and U are computed again from
    X).  X may be an Act8 where saved is given.  grad_dtype: of dA and
    dB, float32 (the default) or X's dtype."""
    M, r, dt, st, code = _gated_args(X, states, A, B, K, F, act)
    for t, n, shape in ((dH, "dH", (M, F)), (Z, "Z", (M, 2 * r))):
        _require_cuda(t, n, dt)
        _require_shape(t, n, *shape)
    if not isinstance(X, Act8):
        _require_cuda(X, "X", dt)
    elif saved is None:
        raise ValueError("saved is required where X is kept in 8 bits")
    xp, x8 = _kept_or_dense(X, M, K, "X")
    gu, gu8 = _gated_kept(saved, M, F, dt)
    gdt, gcode = _grad_code(grad_dtype, dt)
    with _on(dH, stream, X, Z, saved, A, B, dX, dA, dB, workspace) as s:
        dX = _out(dX, "dX", dt, dH.device, M, K) if need_dx else None
        dA = _out(dA, "dA", gdt, dH.device, K, 2 * r)
        dB = _out(dB, "dB", gdt, dH.device, r, 2 * F)
        ws = _workspace(workspace, qlora_gated_workspace_bytes(M, K, F, r)[1], dH.device)
        _check(lib().qlora_gated_bwd(_COMPUTE[dt], code, gcode, M, K, F, r, dH.data_ptr(), xp, _ref(x8), Z.data_ptr(),
                                     gu, _ref(gu8), st, A.data_ptr(), B.data_ptr(), float(c), _ptr(dX), dA.data_ptr(),
                                     dB.data_ptr(), ws.data_ptr(), ws.numel(), s), "qlora_gated_bwd")
    return dX, dA, dB


def qlora_head_workspace_bytes(M: int, K: int, V: int, need_dx: bool = True) -> int:
    b = ctypes.c_int64()
    _check(lib().qlora_head_workspace_bytes(M, K, V, int(need_dx), ctypes.byref(b)), "qlora_head_workspace_bytes")
    return b.value


def qlora_head_loss(X, W, targets, weights=None, need_dx: bool = True, ignore_index: int = -100, loss=None, lse=None,
                    dX=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits X Wᵀ per token, and its gradient,
    without keeping the logits: (loss (M, fp32), lse (M, fp32), dX (M x K) or
    None).  X: M x K and the frozen head W: V x K, both bf16 or both fp16;
    targets: M int64, ignore_index where a token carries no loss; weights: M
    fp32 factors of the tokens' losses and gradients (None: 1; a mean over n
    tokens is 1/n)."""
    import torch
    dt = _compute_dtype(X)
    M, K = X.shape
    V = W.shape[0]
    _require_cuda(X, "X", dt)
    _require_cuda(W, "W", dt)
    _require_shape(W, "W", V, K)
    _require_cuda(targets, "targets", torch.int64)
    _require_shape(targets, "targets", M)
    if weights is not None:
        _require_cuda(weights, "weights", torch.float32)
        _require_shape(weights, "weights", M)
    with _on(X, stream, W, targets, weights, loss, lse, dX, workspace) as s:
        loss = _out(loss, "loss", torch.float32, X.device, M)
        lse = _out(lse, "lse", torch.float32, X.device, M)
        dX = _out(dX, "dX", dt, X.device, M, K) if need_dx else None
        ws = _workspace(workspace, qlora_head_workspace_bytes(M, K, V, need_dx), X.device)
        _check(lib().qlora_head_loss(_COMPUTE[dt], M, K, V, X.data_ptr(), W.data_ptr(), targets.data_ptr(),
                                     _ptr(weights), ignore_index, loss.data_ptr(), lse.data_ptr(), _ptr(dX),
                                     ws.data_ptr(), ws.numel(), s), "qlora_head_loss")
    return loss, lse, dX


def qlora_timer_enable(kernel: str, enable: bool = True) -> None:
    _check(lib().qlora_timer_enable(KERNEL_IDS[kernel], int(enable)), "qlora_timer_enable")


def qlora_timer_read(kernel: str) -> tuple[float, int]:
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check(lib().qlora_timer_read(KERNEL_IDS[kernel], ctypes.byref(ms), ctypes.byref(n)), "qlora_timer_read")
    return ms.value, n.value
