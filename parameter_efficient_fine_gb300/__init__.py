"""DoRA weight-norm and compose hot path for GB300 (sm_103a).

Thin ctypes binding over libdora.so (include/dora.h).  Every function here only
marshals arguments -- shapes from tensor sizes, raw device pointers, the
current torch stream -- and calls the C entry point of the same name; all
arithmetic runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "DoraError",
    "load_library",
    "library_path",
    "dora_status_str",
    "dora_norm_factored_workspace",
    "dora_norm_factored",
    "dora_row_sumsq_bf16",
    "dora_norm_factored_bf16_workspace",
    "dora_norm_factored_bf16",
    "dora_norm_factored_bwd_workspace",
    "dora_norm_factored_bwd",
    "dora_compose_fwd",
    "dora_compose_fused_workspace",
    "dora_compose_lora_fwd",
    "dora_compose_lora_fwd_bf16",
    "dora_linear_fwd",
    "dora_compose_bwd_workspace",
    "dora_compose_bwd",
    "dora_compose_bwd_noalloc",
    "dora_q8_store",
    "dora_q8_load",
    "dora_compose_fwd_q8",
    "dora_compose_bwd_q8_workspace",
    "dora_compose_bwd_q8",
    "dora_lora_grad_q8_workspace",
    "dora_lora_grad_q8",
    "dora_matmul_q8_workspace",
    "dora_matmul_q8",
    "dora_matmul_q8_t_workspace",
    "dora_matmul_q8_t",
    "dora_q4_store",
    "dora_q4_load",
    "dora_matmul_q4_workspace",
    "dora_matmul_q4",
    "dora_matmul_q4_t_workspace",
    "dora_matmul_q4_t",
    "dora_expert_sort",
    "dora_expert_send",
    "dora_expert_return",
    "dora_expert_return_bwd",
    "dora_expert_clear",
    "dora_device_error",
    "dora_kernel_launches",
    "dora_test_stall_loads",
    "dora_test_fused_pairs",
    "DORA_F32",
    "DORA_BF16",
]

DORA_F32 = 0
DORA_BF16 = 1

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "lib", "libdora.so")
_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_int = ctypes.c_int

_SIGNATURES = {
    "dora_status_str": (ctypes.c_char_p, [_int]),
    "dora_norm_factored_workspace": (_sz, [_i64, _i64, _i64]),
    "dora_norm_factored": (_int, [_vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "dora_row_sumsq_bf16": (_int, [_vp, _i64, _i64, _vp, _vp]),
    "dora_norm_factored_bf16_workspace": (_sz, [_i64, _i64, _i64]),
    "dora_norm_factored_bf16": (_int, [_vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "dora_norm_factored_bwd_workspace": (_sz, [_i64, _i64, _i64]),
    "dora_norm_factored_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "dora_compose_fwd": (_int, [_int, _vp, _vp, _vp, _f32, _i64, _i64, _vp, _vp]),
    "dora_compose_fused_workspace": (_sz, [_i64, _i64]),
    "dora_compose_lora_fwd": (_int, [_vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_compose_lora_fwd_bf16": (_int, [_vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp]),
    "dora_linear_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_compose_bwd_workspace": (_sz, [_i64, _i64]),
    "dora_compose_bwd": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "dora_compose_bwd_noalloc": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _vp, _vp, _vp, _vp]),
    "dora_q8_store": (_int, [_int, _vp, _i64, _i64, _int, _vp, _vp, _vp]),
    "dora_q8_load": (_int, [_int, _vp, _vp, _i64, _i64, _int, _vp, _vp]),
    "dora_compose_fwd_q8": (_int, [_int, _vp, _vp, _vp, _f32, _i64, _i64, _vp, _vp, _vp, _vp]),
    "dora_compose_bwd_q8_workspace": (_sz, [_i64, _i64]),
    "dora_compose_bwd_q8": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "dora_lora_grad_q8_workspace": (_sz, [_i64, _i64, _i64]),
    "dora_lora_grad_q8": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_matmul_q8_workspace": (_sz, [_i64, _i64, _i64]),
    "dora_matmul_q8": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_matmul_q8_t_workspace": (_sz, [_i64, _i64, _i64]),
    "dora_matmul_q8_t": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_q4_store": (_int, [_int, _vp, _i64, _i64, _vp, _vp, _vp]),
    "dora_q4_load": (_int, [_int, _vp, _vp, _i64, _i64, _vp, _vp]),
    "dora_matmul_q4_workspace": (_sz, [_i64, _i64, _i64, _i64]),
    "dora_matmul_q4": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_matmul_q4_t_workspace": (_sz, [_i64, _i64, _i64, _i64]),
    "dora_matmul_q4_t": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "dora_expert_sort": (_int, [_int, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "dora_expert_send": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]),
    "dora_expert_return": (_int, [_int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]),
    "dora_expert_clear": (_int, [_int, _vp, _vp, _i64, _i64, _i64, _vp]),
    "dora_expert_return_bwd": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp]),
    "dora_device_error": (_int, [ctypes.POINTER(_int)]),
    "dora_kernel_launches": (ctypes.c_uint64, []),
    "dora_test_stall_loads": (_int, [_int, ctypes.c_uint64]),
    "dora_test_fused_pairs": (_int, [_int]),
}


class DoraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {load_library().dora_status_str(status).decode()}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libdora.so (built by __graft_entry__.build()); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libdora.so not built ({_LIB_PATH}); run __graft_entry__.build() first")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(x) -> int:
    if getattr(x, "is_cuda", False):
        return x.data_ptr()
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    # every pointer of the C ABI is a device pointer: a host tensor would hand
    # a host address to the kernels
    raise ValueError(f"libdora takes CUDA tensors (device memory); got one on {getattr(x, 'device', type(x))}")


_raw_stream = None   # torch's lookup of a device's current stream, as a raw handle
_cuda = None         # torch.cuda, once torch is here
_TYPES = ()          # torch's bfloat16, float32, int32, once torch is here
_ACTS = {}           # torch dtype -> dora_dtype


def _stream(stream, device=None) -> int:
    global _raw_stream
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _raw_stream is None:
        import torch
        # the raw handle where torch gives it: building a Stream object takes 3 us a call
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    if device is None:
        import torch
        device = torch.cuda.current_device()
    return _raw_stream(device)


def _types():
    """torch.bfloat16, torch.float32, torch.int32.  An import statement in each call would
    take as long as all its comparisons."""
    global _TYPES
    import torch
    _TYPES = (torch.bfloat16, torch.float32, torch.int32)
    return _TYPES


def _act(t) -> int:
    act = _ACTS.get(t.dtype)
    if act is None:
        import torch
        _ACTS.update({torch.float32: DORA_F32, torch.bfloat16: DORA_BF16})
        act = _ACTS.get(t.dtype)
    if act is None:
        raise TypeError(f"activation dtype {t.dtype} not supported (float32 or bfloat16)")
    return act


def _check(name: str, st: int) -> None:
    if st != 0:
        raise DoraError(name, st)


def dora_status_str(status: int) -> str:
    return load_library().dora_status_str(status).decode()


def dora_norm_factored_workspace(out: int, inp: int, r: int) -> int:
    return int(load_library().dora_norm_factored_workspace(out, inp, r))


def dora_compose_bwd_workspace(T: int, out: int) -> int:
    return int(load_library().dora_compose_bwd_workspace(T, out))


def dora_norm_factored(W0, A, B, m, s: float, norm, g, workspace, stream=None) -> None:
    """norm[i] = ||W0_i + s (B A)_i||, g = m / norm (see include/dora.h)."""
    out, inp = W0.shape
    r = A.shape[0]
    st = load_library().dora_norm_factored(
        _ptr(W0), _ptr(A), _ptr(B), _ptr(m), float(s), out, inp, r, _ptr(norm), _ptr(g),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dora_norm_factored", st)


def dora_row_sumsq_bf16(W0, n0sq, stream=None) -> None:
    """n0sq[i] = sum_j W0[i, j]^2 for a bfloat16 W0 (see include/dora.h)."""
    rows, cols = W0.shape
    _check("dora_row_sumsq_bf16",
           load_library().dora_row_sumsq_bf16(_ptr(W0), rows, cols, _ptr(n0sq), _stream(stream)))


def dora_norm_factored_bf16_workspace(out: int, inp: int, r: int) -> int:
    return int(load_library().dora_norm_factored_bf16_workspace(out, inp, r))


def dora_norm_factored_bf16(W0, A, B, m, n0sq, s: float, norm, g, workspace, stream=None) -> None:
    """dora_norm_factored for bfloat16 W0, A, B with the base term from n0sq (see include/dora.h)."""
    out, inp = W0.shape
    r = A.shape[0]
    st = load_library().dora_norm_factored_bf16(
        _ptr(W0), _ptr(A), _ptr(B), _ptr(m), _ptr(n0sq), float(s), out, inp, r, _ptr(norm), _ptr(g),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dora_norm_factored_bf16", st)


def dora_norm_factored_bwd_workspace(out: int, inp: int, r: int) -> int:
    return int(load_library().dora_norm_factored_bwd_workspace(out, inp, r))


def dora_norm_factored_bwd(W0, A, B, norm, g, d_mag, s: float, dA, dB, workspace, stream=None) -> None:
    """dA, dB: the gradient that flows through the row norm (see include/dora.h)."""
    out, inp = W0.shape
    r = A.shape[0]
    st = load_library().dora_norm_factored_bwd(
        _ptr(W0), _ptr(A), _ptr(B), _ptr(norm), _ptr(g), _ptr(d_mag), float(s), out, inp, r, _ptr(dA), _ptr(dB),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dora_norm_factored_bwd", st)


def dora_compose_fwd(base, lora, g, s: float, y, stream=None) -> None:
    """y = base + (g-1)*base + g*s*lora (see include/dora.h)."""
    T, out = base.shape
    st = load_library().dora_compose_fwd(_act(base), _ptr(base), _ptr(lora), _ptr(g), float(s), T, out,
                                         _ptr(y), _stream(stream))
    _check("dora_compose_fwd", st)


def dora_compose_fused_workspace(out: int, r: int) -> int:
    return int(load_library().dora_compose_fused_workspace(out, r))


def dora_compose_lora_fwd(base, xa, B, g, s: float, y, workspace, stream=None) -> None:
    """y = base + (g-1) base + g s (xa B^T), lora formed in the kernel (see include/dora.h)."""
    T, out = base.shape
    r = xa.shape[1]
    st = load_library().dora_compose_lora_fwd(
        _ptr(base), _ptr(xa), _ptr(B), _ptr(g), float(s), T, out, r, _ptr(y),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dora_compose_lora_fwd", st)


def dora_compose_lora_fwd_bf16(base, xa, B, g, s: float, y, stream=None) -> None:
    """y = base + (g-1) base + g s (xa B^T) for a bf16 B: one product, s applied to
    the accumulator (see include/dora.h)."""
    T, out = base.shape
    r = xa.shape[1]
    st = load_library().dora_compose_lora_fwd_bf16(
        _ptr(base), _ptr(xa), _ptr(B), _ptr(g), float(s), T, out, r, _ptr(y), _stream(stream))
    _check("dora_compose_lora_fwd_bf16", st)


def dora_linear_fwd(x, W0, xa, B, g, s: float, y, workspace, stream=None) -> None:
    """y = g (x W0^T + s xa B^T) as one GEMM with the compose in its epilogue (see include/dora.h)."""
    T, inp = x.shape
    out = W0.shape[0]
    r = xa.shape[1]
    st = load_library().dora_linear_fwd(
        _ptr(x), _ptr(W0), _ptr(xa), _ptr(B), _ptr(g), float(s), T, inp, out, r, _ptr(y),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dora_linear_fwd", st)


def dora_compose_bwd(grad_out, base, lora, g, norm, s: float, d_base, d_lora, d_mag, workspace,
                     stream=None) -> None:
    """d_base = g*dy, d_lora = s*g*dy, d_mag = sum_t dy*(base+s*lora)/norm (see include/dora.h)."""
    T, out = grad_out.shape
    st = load_library().dora_compose_bwd(
        _act(grad_out), _ptr(grad_out), _ptr(base), _ptr(lora), _ptr(g), _ptr(norm), float(s), T, out,
        _ptr(d_base), _ptr(d_lora), _ptr(d_mag), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dora_compose_bwd", st)


def dora_compose_bwd_noalloc(grad_out, base, lora, g, norm, s: float, d_base, d_lora, d_mag,
                             stream=None) -> None:
    """dora_compose_bwd without a workspace, for callers that cannot allocate
    device memory where they run the backward: the partial sums use the
    library's fixed device scratch array (see include/dora.h; calls that
    overlap on the GPU race on that array)."""
    T, out = grad_out.shape
    st = load_library().dora_compose_bwd_noalloc(
        _act(grad_out), _ptr(grad_out), _ptr(base), _ptr(lora), _ptr(g), _ptr(norm), float(s), T, out,
        _ptr(d_base), _ptr(d_lora), _ptr(d_mag), _stream(stream))
    _check("dora_compose_bwd_noalloc", st)


def _q8(name: str, rows: int, cols: int, block_rows: int, q, scale) -> None:
    """The shapes of an 8-bit form; the C ABI sees only the matrix's."""
    if q.element_size() != 1 or scale.element_size() != 1:
        raise TypeError(f"{name}: the 8-bit form is bytes, got {q.dtype} and {scale.dtype}")
    if block_rows != 1 and block_rows != 128:      # the C int would take it modulo 2^32
        raise ValueError(f"{name}: 1 or 128 rows a scale, got {block_rows}")
    if q.shape != (rows, cols) or scale.shape != (-(-rows // block_rows), -(-cols // 128)):
        raise ValueError(f"{name}: 8-bit form of [{rows}, {cols}] with {block_rows} rows a scale: "
                         f"got q {tuple(q.shape)}, scale {tuple(scale.shape)}")


def _addresses(name: str, stream, *ts) -> list[int]:
    """Device addresses of a call's tensors, which are dense and in the memory of
    the current device, as the kernels run there; then the stream's handle."""
    global _cuda
    here = None
    for t in ts:
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensors must be contiguous (row-major)")
        d = t.get_device()
        if d != here:
            if d < 0:
                raise ValueError(f"libdora takes CUDA tensors (device memory); got one on {t.device}")
            if _cuda is None:
                import torch
                _cuda = torch.cuda
            here = _cuda.current_device()
            if d != here:
                raise ValueError(f"{name}: a tensor on cuda:{d}, but the current device is cuda:{here}")
    return [t.data_ptr() for t in ts] + [_stream(stream, here)]


def _same(name: str, shape, dtype, *ts) -> None:
    for t in ts:
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")


def dora_q8_store(x, block_rows: int, q, scale, stream=None) -> None:
    """x [rows, cols] into its 8-bit form: q bytes and a scale per block_rows (1 or
    128) x 128 elements (see include/dora.h)."""
    rows, cols = x.shape
    _q8("dora_q8_store", rows, cols, block_rows, q, scale)
    act = _act(x)
    px, pq, psc, cs = _addresses("dora_q8_store", stream, x, q, scale)
    st = load_library().dora_q8_store(act, px, rows, cols, block_rows, pq, psc, cs)
    _check("dora_q8_store", st)


def dora_q8_load(q, scale, block_rows: int, x, stream=None) -> None:
    """The values of an 8-bit form into x (see include/dora.h)."""
    rows, cols = x.shape
    _q8("dora_q8_load", rows, cols, block_rows, q, scale)
    act = _act(x)
    px, pq, psc, cs = _addresses("dora_q8_load", stream, x, q, scale)
    st = load_library().dora_q8_load(act, pq, psc, rows, cols, block_rows, px, cs)
    _check("dora_q8_load", st)


def dora_compose_fwd_q8(base, lora, g, s: float, y, q, scale, stream=None) -> None:
    """dora_compose_fwd that also keeps v = base + s lora in 8 bits (see include/dora.h)."""
    T, out = base.shape
    import torch
    _same("dora_compose_fwd_q8", base.shape, base.dtype, lora, y)
    _same("dora_compose_fwd_q8", (out,), torch.float32, g)
    _q8("dora_compose_fwd_q8", T, out, 1, q, scale)
    act = _act(base)
    pb, pl, pg, py, pq, psc, cs = _addresses("dora_compose_fwd_q8", stream, base, lora, g, y, q, scale)
    st = load_library().dora_compose_fwd_q8(act, pb, pl, pg, float(s), T, out, py, pq, psc, cs)
    _check("dora_compose_fwd_q8", st)


def dora_compose_bwd_q8_workspace(T: int, out: int) -> int:
    return int(load_library().dora_compose_bwd_q8_workspace(T, out))


def dora_compose_bwd_q8(grad_out, q, scale, g, norm, s: float, d_base, d_lora, d_mag, workspace, stream=None) -> None:
    """dora_compose_bwd with d_mag from the 8-bit v of dora_compose_fwd_q8 (see include/dora.h)."""
    T, out = grad_out.shape
    import torch
    _same("dora_compose_bwd_q8", grad_out.shape, grad_out.dtype, d_base, d_lora)
    _same("dora_compose_bwd_q8", (out,), torch.float32, g, norm, d_mag)
    _q8("dora_compose_bwd_q8", T, out, 1, q, scale)
    act = _act(grad_out)
    pws, pd, pq, psc, pg, pn, pdb, pdl, pdm, cs = _addresses("dora_compose_bwd_q8", stream, workspace, grad_out, q, scale,
                                                             g, norm, d_base, d_lora, d_mag)
    st = load_library().dora_compose_bwd_q8(act, pd, pq, psc, pg, pn, float(s), T, out, pdb, pdl, pdm, pws,
                                            workspace.numel() * workspace.element_size(), cs)
    _check("dora_compose_bwd_q8", st)


def dora_lora_grad_q8_workspace(T: int, inp: int, r: int) -> int:
    return int(load_library().dora_lora_grad_q8_workspace(T, inp, r))


def dora_lora_grad_q8(dxa, xq, xscale, dA, workspace, stream=None) -> None:
    """dA = dxa^T x from the 8-bit x (see include/dora.h)."""
    import torch
    T, r = dxa.shape
    inp = xq.shape[1]
    _same("dora_lora_grad_q8", (T, r), torch.bfloat16, dxa)
    _same("dora_lora_grad_q8", (r, inp), torch.float32, dA)
    _q8("dora_lora_grad_q8", T, inp, 1, xq, xscale)
    pws, pd, pq, psc, pa, cs = _addresses("dora_lora_grad_q8", stream, workspace, dxa, xq, xscale, dA)
    st = load_library().dora_lora_grad_q8(pd, pq, psc, T, inp, r, pa, pws,
                                          workspace.numel() * workspace.element_size(), cs)
    _check("dora_lora_grad_q8", st)


def dora_matmul_q8_workspace(T: int, out: int, inp: int) -> int:
    return int(load_library().dora_matmul_q8_workspace(T, out, inp))


def dora_matmul_q8_t_workspace(T: int, out: int, inp: int) -> int:
    return int(load_library().dora_matmul_q8_t_workspace(T, out, inp))


def _matmul_q8(name: str, q, scale, wq, wscale, y, workspace, stream, out_side: bool) -> None:
    import torch
    out, inp = wq.shape
    T = q.shape[0]
    _q8(name, T, inp if out_side else out, 1, q, scale)
    _q8(name, out, inp, 128, wq, wscale)
    _same(name, (T, out if out_side else inp), torch.bfloat16, y)
    pq, psc, pw, pwsc, py, cs = _addresses(name, stream, q, scale, wq, wscale, y)
    st = getattr(load_library(), name)(pq, psc, pw, pwsc, T, out, inp, py, _ptr(workspace),
                                       0 if workspace is None else workspace.numel() * workspace.element_size(),
                                       cs)
    _check(name, st)


def dora_matmul_q8(xq, xscale, wq, wscale, y, workspace=None, stream=None) -> None:
    """y = x W^T for x and W in 8 bits (see include/dora.h)."""
    _matmul_q8("dora_matmul_q8", xq, xscale, wq, wscale, y, workspace, stream, True)


def dora_matmul_q8_t(dyq, dyscale, wq, wscale, dx, workspace=None, stream=None) -> None:
    """dx = dy W for dy and the same W in 8 bits (see include/dora.h)."""
    _matmul_q8("dora_matmul_q8_t", dyq, dyscale, wq, wscale, dx, workspace, stream, False)


def _q4(name: str, shape, q, scale) -> None:
    """The shapes of a 4-bit form of a matrix or of a stack of them; the C ABI sees only
    the matrix's."""
    if q.element_size() != 1 or scale.element_size() != 1:
        raise TypeError(f"{name}: the 4-bit form is bytes, got {q.dtype} and {scale.dtype}")
    *lead, cols = shape
    if not lead:
        raise ValueError(f"{name}: a matrix or a stack of them, got {tuple(shape)}")
    if cols % 32:
        raise ValueError(f"{name}: the 4-bit form has rows of whole groups of 32 columns, got {cols}")
    if q.shape != (*lead, cols // 2) or scale.shape != (*lead, cols // 32):
        raise ValueError(f"{name}: 4-bit form of {list(shape)}: got q {tuple(q.shape)}, scale {tuple(scale.shape)}")


def dora_q4_store(x, q, scale, stream=None) -> None:
    """x [..., rows, cols] into its 4-bit form: two E2M1 values a byte and a scale per
    32 columns of a row (see include/dora.h)."""
    shape = x.shape
    _q4("dora_q4_store", shape, q, scale)
    act = _act(x)
    px, pq, psc, cs = _addresses("dora_q4_store", stream, x, q, scale)
    _check("dora_q4_store", load_library().dora_q4_store(act, px, shape[:-1].numel(), shape[-1], pq, psc, cs))


def dora_q4_load(q, scale, x, stream=None) -> None:
    """The values of a 4-bit form into x (see include/dora.h)."""
    shape = x.shape
    _q4("dora_q4_load", shape, q, scale)
    act = _act(x)
    px, pq, psc, cs = _addresses("dora_q4_load", stream, x, q, scale)
    _check("dora_q4_load", load_library().dora_q4_load(act, pq, psc, shape[:-1].numel(), shape[-1], px, cs))


def dora_matmul_q4_workspace(T: int, out: int, inp: int, experts: int = 1) -> int:
    return int(load_library().dora_matmul_q4_workspace(T, out, inp, experts))


def dora_matmul_q4_t_workspace(T: int, out: int, inp: int, experts: int = 1) -> int:
    return int(load_library().dora_matmul_q4_t_workspace(T, out, inp, experts))


def _matmul_q4_sizes(name: str, x, wq, wscale, offsets, out_side: bool) -> tuple[int, int, int, int, int]:
    """T, out, in, the result's columns and the number of experts of a product's operands."""
    bf16, _, i32 = _TYPES or _types()
    xs, ws = x.shape, wq.shape
    if len(ws) != (2 if offsets is None else 3):
        raise ValueError(f"{name}: a weight [out, in / 2], or with offsets a stack [experts, out, in / 2], got {tuple(ws)}")
    if len(xs) != 2:
        raise ValueError(f"{name}: rows [T, {'in' if out_side else 'out'}], got {tuple(xs)}")
    T, out, inp = xs[0], ws[-2], 2 * ws[-1]
    k, n = (inp, out) if out_side else (out, inp)
    if inp % 32 or wscale.shape != (*ws[:-1], inp // 32) or wq.element_size() != 1 or wscale.element_size() != 1:
        _q4(name, (*ws[:-1], inp), wq, wscale)
    if xs[1] != k or x.dtype != bf16:
        _same(name, (T, k), bf16, x)
    if offsets is None:
        return T, out, inp, n, 1
    _same(name, (ws[0] + 1,), i32, offsets)
    return T, out, inp, n, ws[0]


def _matmul_q4(name: str, x, wq, wscale, y, offsets, workspace, stream, out_side: bool) -> None:
    T, out, inp, n, experts = _matmul_q4_sizes(name, x, wq, wscale, offsets, out_side)
    _same(name, (T, n), _TYPES[0], y)
    nbytes = 0
    ts = [x, wq, wscale, y]
    if offsets is not None:
        ts.append(offsets)
    if workspace is not None:
        nbytes = workspace.numel() * workspace.element_size()
        ts.append(workspace)
    px, pw, psc, py, *more, cs = _addresses(name, stream, *ts)
    poff = more.pop(0) if offsets is not None else 0
    st = getattr(load_library(), name)(px, poff, pw, psc, T, out, inp, experts, py, more[0] if more else 0, nbytes, cs)
    if st:
        _check(name, st)


def dora_matmul_q4(x, wq, wscale, y, offsets=None, workspace=None, stream=None) -> None:
    """y = x W^T for a bfloat16 x and W in 4 bits; with offsets, W is a stack and rows
    offsets[e] to offsets[e + 1] of x meet W[e] (see include/dora.h)."""
    _matmul_q4("dora_matmul_q4", x, wq, wscale, y, offsets, workspace, stream, True)


def dora_matmul_q4_t(dy, wq, wscale, dx, offsets=None, workspace=None, stream=None) -> None:
    """dx = dy W for the same W (see include/dora.h)."""
    _matmul_q4("dora_matmul_q4_t", dy, wq, wscale, dx, offsets, workspace, stream, False)


def _expert_sort_sizes(expert, experts: int) -> tuple[int, int]:
    i32 = (_TYPES or _types())[2]
    if expert.dtype != i32:
        import torch
        if expert.dtype != torch.int64:
            raise TypeError(f"dora_expert_sort: expert is int32 or int64, got {expert.dtype}")
    if not 1 <= experts <= 4096:
        raise ValueError(f"dora_expert_sort: 1 to 4096 experts, got {experts}")
    if len(expert.shape) != 2:
        raise ValueError(f"dora_expert_sort: expert is [T, k], got {tuple(expert.shape)}")
    return expert.shape


def dora_expert_sort(expert, experts: int, order, inverse, offsets, stream=None) -> None:
    """The entries of expert [T, k] sorted by expert, stably: order, its inverse and
    where each expert's begin (see include/dora.h)."""
    T, k = _expert_sort_sizes(expert, experts)
    i32 = _TYPES[2]
    _same("dora_expert_sort", (T * k,), i32, order)
    _same("dora_expert_sort", (T, k), i32, inverse)
    _same("dora_expert_sort", (experts + 1,), i32, offsets)
    pe, po, pi, pf, cs = _addresses("dora_expert_sort", stream, expert, order, inverse, offsets)
    _check("dora_expert_sort", load_library().dora_expert_sort(expert.element_size(), pe, T, k, experts, po, pi, pf, cs))


def _routed(name: str, x, xs, inverse, offsets) -> tuple[int, int, int, int]:
    """T, k, cols and the number of experts of tokens x [T, cols] and their rows xs [T k, cols]."""
    i32 = (_TYPES or _types())[2]
    if len(inverse.shape) != 2 or len(x.shape) != 2:
        raise ValueError(f"{name}: tokens [T, cols] and inverse [T, k], got {tuple(x.shape)} and {tuple(inverse.shape)}")
    T, k = inverse.shape
    cols, so = x.shape[1], offsets.shape
    experts = so[0] - 1
    if len(so) != 1 or not 1 <= experts <= 4096:
        raise ValueError(f"{name}: offsets are [experts + 1], 1 to 4096 experts, got {tuple(so)}")
    if inverse.dtype != i32 or offsets.dtype != i32 or x.shape != (T, cols) or xs.shape != (T * k, cols) or xs.dtype != x.dtype:
        _same(name, (T, k), i32, inverse)
        _same(name, (experts + 1,), i32, offsets)
        _same(name, (T, cols), x.dtype, x)
        _same(name, (T * k, cols), x.dtype, xs)
    return T, k, cols, experts


def dora_expert_send(x, inverse, offsets, xs, stream=None) -> None:
    """xs[inverse[t, j]] = x[t], the tokens' rows sorted by expert (see include/dora.h)."""
    T, k, cols, experts = _routed("dora_expert_send", x, xs, inverse, offsets)
    act = _act(x)
    px, ps, pi, pf, cs = _addresses("dora_expert_send", stream, x, xs, inverse, offsets)
    _check("dora_expert_send", load_library().dora_expert_send(act, px, pi, pf, T, k, cols, experts, ps, cs))


def dora_expert_return(ys, inverse, offsets, weight, y, stream=None) -> None:
    """y[t] = sum_j weight[t, j] ys[inverse[t, j]]; weight None: every one 1 (see include/dora.h)."""
    T, k, cols, experts = _routed("dora_expert_return", y, ys, inverse, offsets)
    act = _act(y)
    ts = [ys, y, inverse, offsets]
    if weight is not None:
        _same("dora_expert_return", (T, k), _TYPES[1], weight)
        ts.append(weight)
    ps, py, pi, pf, *pw, cs = _addresses("dora_expert_return", stream, *ts)
    _check("dora_expert_return",
           load_library().dora_expert_return(act, ps, pi, pf, pw[0] if pw else 0, T, k, cols, experts, py, cs))


def dora_expert_return_bwd(dy, ys, inverse, offsets, weight, d_ys, d_weight, stream=None) -> None:
    """d_ys[inverse[t, j]] = weight[t, j] dy[t], d_weight[t, j] = <dy[t], ys[inverse[t, j]]> (see include/dora.h)."""
    T, k, cols, experts = _routed("dora_expert_return_bwd", dy, ys, inverse, offsets)
    _same("dora_expert_return_bwd", (T * k, cols), dy.dtype, d_ys)
    _same("dora_expert_return_bwd", (T, k), _TYPES[1], weight, d_weight)
    act = _act(dy)
    pd, ps, pi, pf, pw, pds, pdw, cs = _addresses("dora_expert_return_bwd", stream, dy, ys, inverse, offsets, weight,
                                                  d_ys, d_weight)
    _check("dora_expert_return_bwd",
           load_library().dora_expert_return_bwd(act, pd, ps, pi, pf, pw, T, k, cols, experts, pds, pdw, cs))


def dora_expert_clear(x, offsets, stream=None) -> None:
    """Zeros in the rows of x [rows, cols] that no expert has (see include/dora.h)."""
    rows, cols = x.shape
    experts = offsets.shape[0] - 1
    _same("dora_expert_clear", (experts + 1,), (_TYPES or _types())[2], offsets)
    if not 1 <= experts <= 4096:
        raise ValueError(f"dora_expert_clear: offsets are [experts + 1], 1 to 4096 experts, got {tuple(offsets.shape)}")
    act = _act(x)
    px, pf, cs = _addresses("dora_expert_clear", stream, x, offsets)
    _check("dora_expert_clear", load_library().dora_expert_clear(act, px, pf, rows, cols, experts, cs))


def dora_device_error() -> int:
    """Reads and clears the device error word (synchronises the device)."""
    code = _int(0)
    st = load_library().dora_device_error(ctypes.byref(code))
    if st not in (0, 8):
        raise DoraError("dora_device_error", st)
    return int(code.value)


def dora_kernel_launches() -> int:
    return int(load_library().dora_kernel_launches())


def dora_test_stall_loads(on: bool, wait_limit_ns: int = 0) -> None:
    """Testing hook: make later norm calls' bounded waits expire (see include/dora.h)."""
    _check("dora_test_stall_loads", load_library().dora_test_stall_loads(1 if on else 0, int(wait_limit_ns)))


def dora_test_fused_pairs(allow: bool) -> None:
    """Testing hook: run the fused kernels as single CTAs when False (see include/dora.h)."""
    _check("dora_test_fused_pairs", load_library().dora_test_fused_pairs(1 if allow else 0))
