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
    w8a8_route_experts, w8a8_route_workspace_size, W8A8_SCORE_SOFTMAX, W8A8_SCORE_SIGMOID,
    w8a8_group_rows, w8a8_group_workspace_size, W8A8_GROUPS_MAX, W8A8_ROUTE_MAX_K,
    W8A8_ROUTE_MAX_GROUPS, w8a8_combine_experts, w8a8_adapter_matmul,
    w8a8_adapter_workspace_size, W8A8_ADAPTER_MAX_R,
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
        self.u8, self.bool = torch.uint8, torch.bool
        self.routing = (self.i32, self.f32, self.bool, self.u8)        # see pycall.c
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


def _on_stream(stream):
    """Where a call's own tensors are allocated: on the stream that uses them, so that
    their memory is not handed on before it has passed the call."""
    import contextlib

    import torch
    if stream is None or not torch.cuda.is_available():
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _here(t, *others):
    """Refuse tensors that are not all on the current GPU, whose stream the call takes."""
    _one_gpu(t, *others)
    if t.get_device() >= 0:
        import torch
        if t.get_device() != torch.cuda.current_device():
            raise W8A8Error(W8A8_ERR_INVALID_ARG, f"tensors on {t.device}, which is not the current device")


def _given(t, shape, dtype, name):
    """Refuse a tensor that is not dense, of this shape and type."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        _want(t, shape, name)
        _typed(t, (dtype,), name)
        _dense(t, name)


def _outputs(out, specs, device):
    """The caller's output tensors, checked, or new ones: specs of (name, shape, dtype)."""
    if out is None:
        import torch
        return tuple(torch.empty(shape, dtype=dtype, device=device) for _, shape, dtype in specs)
    if len(out) != len(specs):
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"out has {len(out)} tensors, want {len(specs)}")
    for t, (name, shape, dtype) in zip(out, specs):
        _given(t, shape, dtype, name)
    return tuple(out)


def _workspace(size, device):
    """(tensor, address) of device scratch; the tensor lives to the end of the call."""
    if not size:
        return None, None
    import torch
    t = torch.empty(size, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


def _number(v, name, low=1, high=2 ** 31 - 1):
    """v as a whole number, refused out of range: the C calls take it in 32 bits."""
    import operator
    try:
        v = operator.index(v)
    except TypeError:
        v = None
    if v is None or not low <= v <= high:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"{name}: want a whole number from {low} to {high}")
    return v


_SCORES = {"softmax": W8A8_SCORE_SOFTMAX, "sigmoid": W8A8_SCORE_SIGMOID}


def route_experts(logits, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=2,
                  renormalize=True, scale=1.0, valid=None, out=None, stream=None):
    """Each token's experts and their weights, and the (token, choice) pairs in the experts'
    order, on CUDA tensors.

    logits bf16, fp16 or fp32 [T, E]; scores are their softmax or sigmoid, and with bias
    (float32 [E]) added they rank the experts; of the ``groups`` runs of neighbouring experts
    the ``top_groups`` with the largest sums of their ``group_top`` (1 or 2) best are open.
    Weights are scale * the top_k chosen experts' scores (without the bias), divided by
    their sum with ``renormalize``.  ``valid`` (bool or uint8 [T]): False for padding, whose
    tokens get no expert.  Returns (ids int32 [T, top_k], weights float32 [T, top_k],
    order int32 [T * top_k], offsets int32 [E + 1], rows int32 [T, top_k]): grouped_matmul_ragged
    takes rows order // top_k of the activations by offsets, combine_experts takes rows and
    weights.  ``out``: those five, preallocated.  Raises W8A8Error on a non-zero status."""
    lib, types = load_library(), _dtypes or _load_dtypes()
    code = _SCORES.get(scoring)
    if code is None:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"scoring {scoring!r}: want 'softmax' or 'sigmoid'")
    if lib.route_tensors is not None:
        st = lib.route_tensors(logits, top_k, code, bias, groups, top_groups, group_top, renormalize, scale, valid,
                               out, _in_codes, types.routing, stream if stream is None else _stream(stream))
        if type(st) is tuple:
            return st
        if st == 0:
            return out
        if st is not None:
            check(st)
    if logits.dim() != 2:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"logits must be [tokens, experts], not {list(logits.shape)}")
    T, E = logits.shape
    kind = _in_codes[logits.dtype]
    if not isinstance(top_k, int) or top_k < 1 or top_k > W8A8_ROUTE_MAX_K:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"top_k of {top_k}: want 1 to {W8A8_ROUTE_MAX_K}")
    groups, top_groups = _number(groups, "groups"), _number(top_groups, "top_groups")
    group_top = _number(group_top, "group_top")
    if bias is not None:
        _given(bias, (E,), types.f32, "bias")
    if valid is not None:
        _typed(valid, (types.bool, types.u8), "valid")
        _given(valid, (T,), valid.dtype, "valid")
    ld = _rows(logits)
    with _on_stream(stream):
        outs = _outputs(out, (("ids", (T, top_k), types.i32), ("weights", (T, top_k), types.f32),
                              ("order", (T * top_k,), types.i32), ("offsets", (E + 1,), types.i32),
                              ("rows", (T, top_k), types.i32)), logits.device)
        _here(logits, bias, valid, *outs)
        size = lib.w8a8_route_workspace_size(T, E, top_k)
        keep, scratch = _workspace(size, logits.device)
    st = lib.w8a8_route_experts(
        logits.data_ptr(), kind, ld, None if bias is None else bias.data_ptr(),
        None if valid is None else valid.data_ptr(), T, E, top_k, code, groups, top_groups, group_top,
        1 if renormalize else 0, scale, *(t.data_ptr() for t in outs), scratch, size, _stream(stream))
    if st:
        check(st)
    return outs


def group_rows(ids, groups, out=None, stream=None):
    """The places of ``ids`` (int32 CUDA tensor of n values, of any dense shape) sorted by
    value, stable: returns (order int32 [n], offsets int32 [groups + 1]): group g's are
    order[offsets[g]] .. order[offsets[g + 1] - 1], and those of no group (values outside
    0 .. groups - 1) come last.  ``out``: both, preallocated."""
    lib, types = load_library(), _dtypes or _load_dtypes()
    if lib.group_tensors is not None:
        st = lib.group_tensors(ids, groups, out, types.routing, stream if stream is None else _stream(stream))
        if type(st) is tuple:
            return st
        if st == 0:
            return out
        if st is not None:
            check(st)
    n = ids.numel()
    _given(ids, ids.shape, types.i32, "ids")
    groups = _number(groups, "groups")
    if groups > W8A8_GROUPS_MAX:        # (before offsets of that size are made)
        raise W8A8Error(W8A8_ERR_UNSUPPORTED, f"{groups} groups: at most {W8A8_GROUPS_MAX}")
    with _on_stream(stream):
        outs = _outputs(out, (("order", (n,), types.i32), ("offsets", (groups + 1,), types.i32)), ids.device)
        _here(ids, *outs)
        size = lib.w8a8_group_workspace_size(n, groups)
        keep, scratch = _workspace(size, ids.device)
    st = lib.w8a8_group_rows(ids.data_ptr(), n, groups, outs[0].data_ptr(), outs[1].data_ptr(), None, scratch, size,
                             _stream(stream))
    if st:
        check(st)
    return outs


def combine_experts(Y, rows, weights, add=None, out_dtype=None, out=None, stream=None):
    """out[t] = add[t] + sum_j weights[t, j] * Y[rows[t, j]] on CUDA tensors: Y [M, D] bf16, fp16
    or fp32 in the experts' order, rows int32 and weights float32 [T, k] from route_experts;
    rows outside Y (-1) are left out.  add [T, D] of the output's type, which is Y's or fp32
    (``out_dtype``, or ``out``'s); ``out`` may be ``add``.  Raises W8A8Error on a non-zero
    status."""
    lib, types = load_library(), _dtypes or _load_dtypes()
    if lib.combine_tensors is not None and (out is None or out_dtype is None):
        st = lib.combine_tensors(Y, rows, weights, add,
                                 out if out_dtype is None else types.out[out_code(out_dtype)], _in_codes,
                                 types.routing, stream if stream is None else _stream(stream))
        if type(st) is int:
            if st == 0:
                return out
            check(st)
        elif st is not None:
            return st
    if Y.dim() != 2 or rows.dim() != 2:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, f"Y must be [rows, columns] and rows [tokens, choices], not "
                                              f"{list(Y.shape)} and {list(rows.shape)}")
    (M, D), (T, k) = Y.shape, rows.shape
    kind = _in_codes[Y.dtype]
    _given(rows, (T, k), types.i32, "rows")
    _given(weights, (T, k), types.f32, "weights")
    dtype = types.out[out_code(out_dtype)] if out_dtype is not None else Y.dtype if out is None else out.dtype
    with _on_stream(stream):
        if out is None:
            import torch
            out = torch.empty((T, D), dtype=dtype, device=Y.device)
        _want(out, (T, D), "out")
        _typed(out, (dtype,), "out")
        if add is not None:
            _want(add, (T, D), "add")
            _typed(add, (dtype,), "add")
        ld_y, ld_out, ld_add = _rows(Y), _rows(out), 0 if add is None else _rows(add)
        _here(Y, rows, weights, add, out)
    st = lib.w8a8_combine_experts(Y.data_ptr(), kind, ld_y, M, rows.data_ptr(), weights.data_ptr(),
                                  None if add is None else add.data_ptr(), ld_add, out.data_ptr(), _in_codes[dtype],
                                  ld_out, T, k, D, _stream(stream))
    if st:
        check(st)
    return out


def adapter_matmul(x, A, B, order, offsets, base, scales=None, out=None, stream=None,
                   variant=W8A8_VARIANT_AUTO):
    """out[t] = base[t] + scales[l] * (x[t] A[l]^T) B[l]^T on CUDA tensors, l the adapter of row
    t: low-rank adapters of many requests beside the projection that made ``base``.

    x [T, K] bf16 or fp16; A [L, r, K] and B [L, N, r] of its type; order int32 [T] and
    offsets int32 [L + 1] from group_rows(the rows' adapters, L); base [T, N] of x's type or
    fp32; scales float32 [L] (None: 1).  Rows without an adapter are base's.  ``out`` may be
    ``base``, whose rows without an adapter are then not touched.  variant: W8A8_VARIANT_AUTO,
    _SMALLM or _TILED (see the header).  Raises W8A8Error on a non-zero status."""
    lib, types = load_library(), _dtypes or _load_dtypes()
    if not variant and lib.adapter_tensors is not None:
        st = lib.adapter_tensors(x, A, B, order, offsets, base, scales, out, _in_codes, types.routing,
                                 stream if stream is None else _stream(stream))
        if type(st) is int:
            if st == 0:
                return out
            check(st)
        elif st is not None:
            return st
    variant = _number(variant, "variant", 0) if variant else W8A8_VARIANT_AUTO
    if x.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise W8A8Error(W8A8_ERR_INVALID_ARG, "x must be [rows, K], A [adapters, r, K] and B [adapters, N, r]")
    T, K = x.shape
    L, r, _ = A.shape
    N = B.shape[1]
    kind = _in_codes[x.dtype]
    _given(A, (L, r, K), x.dtype, "A")
    _given(B, (L, N, r), x.dtype, "B")
    _given(order, (T,), types.i32, "order")
    _given(offsets, (L + 1,), types.i32, "offsets")
    if scales is not None:
        _given(scales, (L,), types.f32, "scales")
    _want(base, (T, N), "base")
    with _on_stream(stream):
        if out is None:
            import torch
            out = torch.empty((T, N), dtype=base.dtype, device=base.device)
        _want(out, (T, N), "out")
        _typed(out, (base.dtype,), "out")
        ld_x, ld_base, ld_out = _rows(x), _rows(base), _rows(out)
        _here(x, A, B, order, offsets, base, scales, out)
        size = lib.w8a8_adapter_workspace_size(T, L, r, K, variant)
        keep, scratch = _workspace(size, x.device)
    st = lib.w8a8_adapter_matmul(x.data_ptr(), kind, ld_x, A.data_ptr(), B.data_ptr(), order.data_ptr(),
                                 offsets.data_ptr(), None if scales is None else scales.data_ptr(), base.data_ptr(),
                                 ld_base, out.data_ptr(), _in_codes[base.dtype], ld_out, T, L, r, K, N, variant,
                                 scratch, size, _stream(stream))
    if st:
        check(st)
    return out
