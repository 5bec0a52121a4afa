"""GB300-native (sm_103a) W8A8 block-FP8 matmul.

    C[m,n] = cast_out( sum_g a_s[m,g] * b_s[n/128,g] * sum_{k in g} A[m,k] * B[n,k] )

("feat: optimize w8a8 block fp8 matmul for Hopper", FlagGems-vllm PR #693,
Description and Numerical safety.)  The compute runs in the hand-written CUDA
kernels of the shared library built from ``csrc/``; this package only
marshals arguments to its C ABI (``include/w8a8_block_fp8.h``) and uses
PyTorch for device memory and streams.  Loading is lazy, so that the seeded
input generator ``synth`` can be imported without the library.
"""
from __future__ import annotations

from . import _binding
from ._binding import (  # noqa: F401
    EXPORTED, W8A8Error, W8A8_OK, W8A8_ERR_INVALID_ARG, W8A8_ERR_UNSUPPORTED, W8A8_ERR_CUDA,
    W8A8_ERR_DEVICE_TIMEOUT, W8A8_ERR_WORKSPACE, W8A8_ERR_NO_DEVICE, W8A8_ERR_DEVICE_BOUNDS,
    W8A8_OUT_BF16,
    W8A8_OUT_FP16, W8A8_OUT_FP32, W8A8_VARIANT_AUTO, W8A8_VARIANT_TILED, W8A8_VARIANT_SWAPAB,
    W8A8_VARIANT_SPLITK, W8A8_VARIANT_SPLITK_CLUSTER, W8A8_VARIANT_SMALLM, W8A8_VARIANT_TILED_PAIR,
    W8A8_VARIANT_GENERIC, w8a8_block_fp8_matmul_strided,
    _opts_address, _stream, check, library_path, load_library,
    w8a8_abi_version, w8a8_debug_bounds_build, w8a8_env_config, debug_bounds_requested,
    w8a8_block_fp8_host_staging_size, w8a8_block_fp8_matmul, w8a8_block_fp8_matmul_ex,
    w8a8_block_fp8_matmul_host, w8a8_block_fp8_plan, w8a8_block_fp8_workspace_size,
    w8a8_block_fp8_matmul_splitk_noalloc, W8A8_NOALLOC_SCRATCH_BYTES,
    w8a8_quantize_fp8_per_token_group, W8A8_IN_BF16, W8A8_IN_FP16, W8A8_IN_FP32,
    w8a8_block_fp8_grouped_matmul_masked, w8a8_block_fp8_grouped_matmul_contiguous,
    w8a8_block_fp8_grouped_matmul_ragged, W8A8_RAGGED_MAX_EXPERTS,
    w8a8_int8_matmul, w8a8_int8_workspace_size, W8A8_INT8_MAX_K, w8a8_quantize_int8_per_token,
    w8a8_sandwich_norm, W8A8_NORM_SAME, W8A8_NORM_FP8, W8A8_NORM_INT8, W8A8_NORM_MAX_D,
    w8a8_launch_floor_kernel, w8a8_block_fp8_quant_matmul,
    w8a8_block_fp8_quant_matmul_workspace_size,
    w8a8_get_device_status, w8a8_last_error, w8a8_options, w8a8_shutdown, w8a8_status_string,
)

_OUT_CODES = {"bf16": W8A8_OUT_BF16, "fp16": W8A8_OUT_FP16, "fp32": W8A8_OUT_FP32}


def out_code(dtype) -> int:
    """W8A8_OUT_* code of a torch dtype or of 'bf16' / 'fp16' / 'fp32'."""
    if isinstance(dtype, str):
        return _OUT_CODES[dtype]
    import torch
    return {torch.bfloat16: W8A8_OUT_BF16, torch.float16: W8A8_OUT_FP16,
            torch.float32: W8A8_OUT_FP32}[dtype]


def options(**kw) -> w8a8_options:
    """A w8a8_options with the given fields set (the rest zero = defaults)."""
    o = w8a8_options()
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def matmul(A, a_s, B, b_s, out_dtype="bf16", out=None, stream=None, block_n=128, block_k=128,
           **opts):
    """C = A B^T with block de-quantisation, on CUDA tensors.

    A: uint8 or float8_e4m3fn [M, K]; a_s: float32 [M, ceil(K/block_k)]; B:
    uint8 or float8_e4m3fn [N, K]; b_s: float32 [ceil(N/block_n),
    ceil(K/block_k)].  Every tensor needs unit stride along its last dimension;
    its row stride is passed through (views of larger buffers work).  ``out``
    (a preallocated [M, N] tensor) is optional; keyword options map to
    w8a8_options fields.  Raises W8A8Error on a non-zero status.
    """
    import torch
    M, K = A.shape
    N = B.shape[0]
    code = out_code(out_dtype)
    if out is None:
        tdt = {W8A8_OUT_BF16: torch.bfloat16, W8A8_OUT_FP16: torch.float16,
               W8A8_OUT_FP32: torch.float32}[code]
        out = torch.empty((M, N), dtype=tdt, device=A.device)

    def ld(t):
        if t.dim() != 2 or (t.size(1) > 1 and t.stride(1) != 1):
            raise W8A8Error(W8A8_ERR_UNSUPPORTED, "each row must be contiguous (unit stride)")
        return t.stride(0) if t.size(0) > 1 else t.size(1)

    st = w8a8_block_fp8_matmul_strided(A, ld(A), a_s, ld(a_s), B, ld(B), b_s, ld(b_s), out,
                                       ld(out), M, N, K, block_n, block_k, code, stream,
                                       options(**opts) if opts else None)
    check(st)
    return out


def quantize_fp8_per_token_group(X, group_size=128, A=None, a_s=None, stream=None):
    """Per-token-group E4M3 quantisation of a CUDA tensor X [M, K] (bf16, fp16
    or fp32): returns (A uint8 [M, K], a_s float32 [M, ceil(K/128)]), the
    matmul's activation operand and its scales.  ``A`` / ``a_s`` may be
    preallocated.  Raises W8A8Error on a non-zero status."""
    import torch
    M, K = X.shape
    code = {torch.bfloat16: W8A8_IN_BF16, torch.float16: W8A8_IN_FP16,
            torch.float32: W8A8_IN_FP32}.get(X.dtype)
    if code is None:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"unsupported input dtype {X.dtype}")
    if A is None:
        A = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    if a_s is None:
        a_s = torch.empty((M, (K + group_size - 1) // group_size), dtype=torch.float32,
                          device=X.device)
    for t in (X, A, a_s):
        if not t.is_contiguous():
            raise W8A8Error(W8A8_ERR_UNSUPPORTED, "tensors must be contiguous row-major")
    check(w8a8_quantize_fp8_per_token_group(X, code, A, a_s, M, K, group_size, stream))
    return A, a_s


def _out_tensor(shape, code, device):
    import torch
    tdt = {W8A8_OUT_BF16: torch.bfloat16, W8A8_OUT_FP16: torch.float16,
           W8A8_OUT_FP32: torch.float32}[code]
    return torch.empty(shape, dtype=tdt, device=device)


def grouped_matmul_masked(A, a_s, B, b_s, masked_m, out_dtype="bf16", out=None, stream=None,
                          **opts):
    """Grouped matmul, masked layout, on CUDA tensors: A [E, max_m, K], a_s
    [E, max_m, K/128], B [E, N, K], b_s [E, ceil(N/128), K/128], masked_m int32
    [E].  Returns C [E, max_m, N]; rows at or past masked_m[e] are unspecified."""
    E, max_m, K = A.shape
    N = B.shape[1]
    code = out_code(out_dtype)
    if out is None:
        out = _out_tensor((E, max_m, N), code, A.device)
    for t in (A, a_s, B, b_s, out, masked_m):
        if not t.is_contiguous():
            raise W8A8Error(W8A8_ERR_UNSUPPORTED, "tensors must be contiguous row-major")
    check(w8a8_block_fp8_grouped_matmul_masked(A, a_s, B, b_s, out, masked_m, E, max_m, N, K,
                                               128, 128, code, stream,
                                               options(**opts) if opts else None))
    return out


def grouped_matmul_contiguous(A, a_s, B, b_s, m_indices, out_dtype="bf16", out=None,
                              stream=None, **opts):
    """Grouped matmul, contiguous layout, on CUDA tensors: A [M, K], a_s [M,
    K/128], B [E, N, K], b_s [E, ceil(N/128), K/128], m_indices int32 [M] (the
    expert of each row, -1 = padding; each aligned 128-row block holds one
    expert).  Returns C [M, N]; padding rows are unspecified."""
    M, K = A.shape
    E, N = B.shape[0], B.shape[1]
    code = out_code(out_dtype)
    if out is None:
        out = _out_tensor((M, N), code, A.device)
    for t in (A, a_s, B, b_s, out, m_indices):
        if not t.is_contiguous():
            raise W8A8Error(W8A8_ERR_UNSUPPORTED, "tensors must be contiguous row-major")
    check(w8a8_block_fp8_grouped_matmul_contiguous(A, a_s, B, b_s, out, m_indices, M, E, N, K,
                                                   128, 128, code, stream,
                                                   options(**opts) if opts else None))
    return out


def quant_matmul(X, B, b_s, out_dtype="bf16", out=None, stream=None, **opts):
    """C = matmul(quantize_fp8_per_token_group(X), B) on CUDA tensors: X [M, K]
    bf16/fp16/fp32, B uint8/float8_e4m3fn [N, K], b_s float32 [ceil(N/128),
    K/128].  One fused launch for decode sizes, the quantiser then the matmul
    above them (see w8a8_block_fp8_quant_matmul).  Same bits as the two calls
    in sequence."""
    import torch
    M, K = X.shape
    N = B.shape[0]
    code = out_code(out_dtype)
    xk = {torch.bfloat16: W8A8_IN_BF16, torch.float16: W8A8_IN_FP16,
          torch.float32: W8A8_IN_FP32}.get(X.dtype)
    if xk is None:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"unsupported activation dtype {X.dtype}")
    if out is None:
        out = _out_tensor((M, N), code, X.device)
    for t in (X, B, b_s, out):
        if not t.is_contiguous():
            raise W8A8Error(W8A8_ERR_UNSUPPORTED, "tensors must be contiguous row-major")
    check(w8a8_block_fp8_quant_matmul(X, xk, B, b_s, out, M, N, K, 128, 128, code, stream,
                                      options(**opts) if opts else None))
    return out


def _want(t, shape, name):
    if t.shape != shape:
        raise W8A8Error(W8A8_ERR_INVALID_ARG,
                        f"{name} has shape {tuple(t.shape)}, want {tuple(shape)}")


def _dense(t, name):
    if not t.is_contiguous():
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, f"{name} must be contiguous")


class _Dtypes:
    """torch's dtypes that the wrappers below compare with (torch is imported late)."""

    def __init__(self):
        import torch
        self.f32, self.i32, self.i8 = torch.float32, torch.int32, torch.int8
        self.e4m3 = (torch.float8_e4m3fn, torch.uint8)
        self.out = {W8A8_OUT_BF16: torch.bfloat16, W8A8_OUT_FP16: torch.float16,
                    W8A8_OUT_FP32: torch.float32}
        self.fast = (self.i8, self.f32, *(self.out[c] for c in sorted(self.out)))   # see pycall.c


_dtypes = None


def _load_dtypes():
    global _dtypes
    _dtypes = _Dtypes()
    return _dtypes


def _typed(t, wanted, name):
    """Refuse a tensor whose elements the kernels would take for another type."""
    if t.dtype not in wanted:
        raise W8A8Error(W8A8_ERR_INVALID_ARG,
                        f"{name} must be {' or '.join(str(w) for w in wanted)}, not {t.dtype}")


def _one_gpu(*tensors):
    """Refuse tensors (None: not given) whose addresses the kernels cannot use together."""
    ext = _binding._pycall
    if ext is not None and ext.one_gpu(*tensors):
        return
    devices = {t.get_device() for t in tensors if t is not None}
    if len(devices) > 1 or -1 in devices:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, "tensors must be on one CUDA device, not on " +
                        ", ".join(sorted({str(t.device) for t in tensors if t is not None})))


def _rows(t):
    """Row stride of a 2-D tensor whose rows are contiguous, 0 for a dense one."""
    if t.is_contiguous():
        return 0
    if t.size(1) > 1 and t.stride(1) != 1:
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, "each row must be contiguous (unit stride)")
    if t.size(0) > 1 and t.stride(0) < t.size(1):
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, "rows must not overlap")
    return t.stride(0) if t.size(0) > 1 else 0


class _Codes(dict):
    """W8A8_IN_* codes by torch dtype; filled at the first use (torch is imported late)."""

    def __missing__(self, dtype):
        import torch
        if not self:
            self.update({torch.bfloat16: W8A8_IN_BF16, torch.float16: W8A8_IN_FP16,
                         torch.float32: W8A8_IN_FP32})
            if dtype in self:
                return self[dtype]
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"unsupported input dtype {dtype}")


_in_codes = _Codes()

# The wrappers below stand before kernels of a few microseconds, so their checks
# are written out in line and they call the library without the marshalling
# functions between (a sandwich_norm call took 9.3 us of host time with them, and takes
# 4.8 with its outputs given, which the extension module checks: see csrc/pycall.c).


def grouped_matmul_ragged(A, a_s, B, b_s, offsets, out_dtype="bf16", out=None, stream=None,
                          **opts):
    """Grouped matmul, ragged layout, on CUDA tensors: A [M, K] and B [E, N, K] uint8 or
    float8_e4m3fn, a_s [M, ceil(K/128)] and b_s [E, ceil(N/128), ceil(K/128)] float32,
    offsets int32 [E + 1] (expert e's rows are offsets[e] .. offsets[e+1]-1; read on
    the device).  Returns C [M, N]; rows of no expert are left as they are in ``out``
    (of out_dtype; unspecified without it)."""
    M, K = A.shape
    E, N, Kb = B.shape
    code = out_code(out_dtype)
    G = (K + 127) // 128
    if Kb != K:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"B has {Kb} columns, A {K}")
    if a_s.shape != (M, G) or b_s.shape != (E, (N + 127) // 128, G) or offsets.shape != (E + 1,):
        _want(a_s, (M, G), "a_s")
        _want(b_s, (E, (N + 127) // 128, G), "b_s")
        _want(offsets, (E + 1,), "offsets")
    if out is None:
        out = _out_tensor((M, N), code, A.device)
    elif out.shape != (M, N):
        _want(out, (M, N), "out")
    if not (A.is_contiguous() and a_s.is_contiguous() and B.is_contiguous() and
            b_s.is_contiguous() and out.is_contiguous() and offsets.is_contiguous()):
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, "tensors must be contiguous row-major")
    types = _dtypes or _load_dtypes()
    if (offsets.dtype is not types.i32 or a_s.dtype is not types.f32 or
            b_s.dtype is not types.f32 or A.dtype not in types.e4m3 or
            B.dtype not in types.e4m3 or out.dtype is not types.out[code]):
        _typed(offsets, (types.i32,), "offsets")
        _typed(a_s, (types.f32,), "a_s")
        _typed(b_s, (types.f32,), "b_s")
        _typed(A, types.e4m3, "A")
        _typed(B, types.e4m3, "B")
        _typed(out, (types.out[code],), "out")
    _one_gpu(A, a_s, B, b_s, offsets, out)
    o = options(**opts) if opts else None
    st = load_library().w8a8_block_fp8_grouped_matmul_ragged(
        A.data_ptr(), a_s.data_ptr(), B.data_ptr(), b_s.data_ptr(), out.data_ptr(),
        offsets.data_ptr(), M, E, N, K, 128, 128, code, _stream(stream), _opts_address(o))
    if st:
        check(st)
    return out


def int8_matmul(A, a_s, B, b_s, out_dtype="bf16", out=None, stream=None, **opts):
    """C[m,n] = a_s[m] b_s[n] sum_k A[m,k] B[n,k] on CUDA tensors: A int8 [M, K], a_s
    float32 [M], B int8 [N, K], b_s float32 [N]; the sum is exact.  A, B and ``out``
    (of out_dtype) need unit stride along their last dimension only.  Keyword options
    map to w8a8_options fields.  Raises W8A8Error on a non-zero status."""
    code, lib, types = out_code(out_dtype), load_library(), _dtypes or _load_dtypes()
    if out is not None and not opts and lib.int8_tensors is not None:
        st = lib.int8_tensors(A, a_s, B, b_s, out, code, types.fast,
                              stream if stream is None else _stream(stream))
        if st == 0:
            return out
        if st is not None:
            check(st)
    M, K = A.shape
    N = B.shape[0]
    _typed(A, (types.i8,), "A")
    _typed(B, (types.i8,), "B")
    if B.shape != (N, K) or a_s.shape != (M,) or b_s.shape != (N,):
        _want(B, (N, K), "B")
        _want(a_s, (M,), "a_s")
        _want(b_s, (N,), "b_s")
    if out is None:
        out = _out_tensor((M, N), code, A.device)
    elif out.shape != (M, N) or out.dtype is not types.out[code]:
        _want(out, (M, N), "out")
        _typed(out, (types.out[code],), "out")
    if not (a_s.is_contiguous() and b_s.is_contiguous()):
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, "scales must be contiguous")
    if a_s.dtype is not types.f32 or b_s.dtype is not types.f32:
        _typed(a_s, (types.f32,), "a_s")
        _typed(b_s, (types.f32,), "b_s")
    ld_a, ld_b, ld_c = _rows(A), _rows(B), _rows(out)
    _one_gpu(A, a_s, B, b_s, out)
    o = options(**opts) if opts else None
    st = lib.w8a8_int8_matmul(
        A.data_ptr(), ld_a, a_s.data_ptr(), B.data_ptr(), ld_b, b_s.data_ptr(),
        out.data_ptr(), ld_c, M, N, K, code, _stream(stream), _opts_address(o))
    if st:
        check(st)
    return out


def quantize_int8_per_token(X, A=None, a_s=None, stream=None):
    """Per-token INT8 quantisation of a CUDA tensor X [M, K] (bf16, fp16 or fp32, unit
    stride along K): returns (A int8 [M, K], a_s float32 [M]), the INT8 matmul's
    activation operand.  ``A`` / ``a_s`` may be preallocated."""
    lib, types = load_library(), _dtypes or _load_dtypes()
    if A is not None and a_s is not None and lib.quant_tensors is not None:
        st = lib.quant_tensors(X, A, a_s, _in_codes, types.fast,
                               stream if stream is None else _stream(stream))
        if st == 0:
            return A, a_s
        if st is not None:
            check(st)
    shape = X.shape
    M, K = shape
    code = _in_codes[X.dtype]
    if A is None or a_s is None:
        import torch
    if A is None:
        A = torch.empty(shape, dtype=torch.int8, device=X.device)
    elif A.shape != shape or A.dtype is not types.i8:
        _want(A, shape, "A")
        _typed(A, (types.i8,), "A")
    if a_s is None:
        a_s = torch.empty(M, dtype=torch.float32, device=X.device)
    elif a_s.shape != (M,) or a_s.dtype is not types.f32 or not a_s.is_contiguous():
        _want(a_s, (M,), "a_s")
        _typed(a_s, (types.f32,), "a_s")
        _dense(a_s, "a_s")
    ld_x, ld_a = _rows(X), _rows(A)
    _one_gpu(X, A, a_s)
    st = lib.w8a8_quantize_int8_per_token(
        X.data_ptr(), code, ld_x, A.data_ptr(), ld_a, a_s.data_ptr(), M, K, _stream(stream))
    if st:
        check(st)
    return A, a_s


_NORM_KINDS = {"same": W8A8_NORM_SAME, "fp8": W8A8_NORM_FP8, "int8": W8A8_NORM_INT8}


def _norm_weight(t, dtype, D=None):
    """Why a norm's weight (or gate, without D) is refused."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, "weights and gate must be contiguous, of h's dtype")
    _want(t, (D,), "a norm's weight")


def sandwich_norm(h, x, w_post=None, w_pre=None, gate=None, gate_rows=None, res_scale=1.0,
                  eps=1e-6, out="same", x_out=None, y_out=None, scales_out=None, stream=None):
    """The norms around a block, fused with its gate and residual, on CUDA tensors:

        u = h / rms(h) * w_post;  r = res_scale * x + gate * u;  y = r / rms(r) * w_pre

    h, x [M, D]; w_post, w_pre [D] (None: no norm); gate [R, D], row m // gate_rows for
    token m (default: R equal runs of tokens), or [D] for all, or None.  Returns (r, y),
    r in x's type; with out="fp8" (E4M3 codes and one float32 scale per 128 columns) or
    "int8" (one scale per row) (r, codes, scales).  x_out may be x itself.  Raises W8A8Error
    on a non-zero status."""
    kind, lib, types = _NORM_KINDS[out], load_library(), _dtypes or _load_dtypes()
    if x_out is not None and y_out is not None and lib.norm_tensors is not None:
        st = lib.norm_tensors(h, x, w_post, w_pre, gate, gate_rows, res_scale, eps, kind, x_out, y_out,
                              scales_out, _in_codes, types.fast,
                              stream if stream is None else _stream(stream))
        if st == 0:
            return (x_out, y_out) if not kind else (x_out, y_out, scales_out)
        if st is not None:
            check(st)
    shape = h.shape
    M, D = shape
    dtype, xtype = h.dtype, x.dtype
    hk = _in_codes[dtype]
    if x.shape != shape:
        _want(x, shape, "x")
    if x_out is None or y_out is None or scales_out is None and kind:
        import torch            # not on the way of a call with its outputs (0.1 us)
    if x_out is None:
        x_out = torch.empty(shape, dtype=xtype, device=x.device)
    elif x_out.shape != shape or x_out.dtype is not xtype:
        _want(x_out, shape, "x_out")
        raise W8A8Error(W8A8_ERR_INVALID_ARG, "x_out must have x's dtype")
    if y_out is None:
        y_out = torch.empty(shape, device=h.device, dtype=(dtype, torch.uint8, torch.int8)[kind])
    elif y_out.shape != shape or (y_out.element_size() != 1 if kind else y_out.dtype is not dtype):
        _want(y_out, shape, "y_out")
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"y_out of {y_out.dtype} for out={out!r}")
    scales = None
    if kind:
        s_shape = (M, (D + 127) // 128) if kind == W8A8_NORM_FP8 else (M,)
        if scales_out is None:
            scales_out = torch.empty(s_shape, dtype=torch.float32, device=h.device)
        elif (scales_out.shape != s_shape or scales_out.dtype is not types.f32 or
              not scales_out.is_contiguous()):
            _want(scales_out, s_shape, "scales_out")
            _typed(scales_out, (types.f32,), "scales_out")
            _dense(scales_out, "scales_out")
        scales = scales_out.data_ptr()
    width = (D,)
    post = pre = gates = None
    if w_post is not None:
        if w_post.dtype is not dtype or not w_post.is_contiguous() or w_post.shape != width:
            _norm_weight(w_post, dtype, D)
        post = w_post.data_ptr()
    if w_pre is not None:
        if w_pre.dtype is not dtype or not w_pre.is_contiguous() or w_pre.shape != width:
            _norm_weight(w_pre, dtype, D)
        pre = w_pre.data_ptr()
    if gate is not None:
        if gate.dtype is not dtype or not gate.is_contiguous():
            _norm_weight(gate, dtype)
        gates = gate.data_ptr()
        g_shape = gate.shape
        if len(g_shape) not in (1, 2):
            raise W8A8Error(W8A8_ERR_INVALID_ARG,
                            f"gate must be [{D}] or [rows, {D}], not {list(g_shape)}")
        R = g_shape[0] if len(g_shape) == 2 else 1
        if gate_rows is None:
            gate_rows = max(1, -(-M // max(R, 1)))
        if g_shape[-1] != D or gate_rows < 1 or R * gate_rows < M:
            raise W8A8Error(W8A8_ERR_INVALID_ARG,
                            f"gate of {tuple(g_shape)} for {M} rows of {D}, {gate_rows} to a gate")
    ld_h, ld_x, ld_xo, ld_y = _rows(h), _rows(x), _rows(x_out), _rows(y_out)
    _one_gpu(h, x, x_out, y_out, w_post, w_pre, gate, scales_out if kind else None)
    st = lib.w8a8_sandwich_norm(
        h.data_ptr(), hk, ld_h, x.data_ptr(), _in_codes[xtype], ld_x, post, gates,
        gate_rows or 1, pre, res_scale, eps, x_out.data_ptr(), ld_xo, y_out.data_ptr(), scales,
        kind, ld_y, M, D, _stream(stream))
    if st:
        check(st)
    return (x_out, y_out) if not kind else (x_out, y_out, scales_out)
