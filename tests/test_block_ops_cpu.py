"""Refusals of the ragged, INT8 and norm entry points: every one comes before any
CUDA call, so they are checked without a GPU, by status and message."""
import ctypes

import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8
from block_scaled_fp8_w8a8_gb300 import _binding, build

OK, ARG, UNS = w8.W8A8_OK, w8.W8A8_ERR_INVALID_ARG, w8.W8A8_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return w8.load_library()


def ragged(M=8, E=2, N=128, K=256, out=0, bn=128, bk=128, opts=None, **ptr):
    p = dict(A=256, a_s=256, B=256, b_s=256, C=256, off=256)
    p.update(ptr)
    return w8.w8a8_block_fp8_grouped_matmul_ragged(p["A"], p["a_s"], p["B"], p["b_s"], p["C"], p["off"], M, E, N, K,
                                                   bn, bk, out, 0, opts)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(N=-8), ARG), (dict(E=-1), ARG), (dict(E=0), ARG), (dict(out=3), ARG),
    (dict(A=0), ARG), (dict(off=0), ARG), (dict(C=0), ARG), (dict(M=0), OK), (dict(bn=64), UNS), (dict(K=250), UNS),
    (dict(K=8), UNS), (dict(N=132), UNS), (dict(N=130, out=2), UNS), (dict(A=264), UNS), (dict(off=258), UNS),
    (dict(E=w8.W8A8_RAGGED_MAX_EXPERTS + 1), UNS), (dict(M=1 << 31), UNS), (dict(M=(1 << 31) - 1, N=1 << 20), UNS),
    (dict(opts=w8.options(variant=w8.W8A8_VARIANT_SWAPAB)), UNS),
    (dict(opts=w8.options(variant=99)), ARG), (dict(opts=w8.options(wait_limit_cycles=5)), ARG),
])
def test_ragged(kw, status):
    assert ragged(**kw) == status
    assert (w8.w8a8_last_error() != "") == (status != OK)


def int8(M=4, N=8, K=16, out=0, lda=0, ldb=0, ldc=0, opts=None, **ptr):
    p = dict(A=256, a_s=256, B=256, b_s=256, C=256)
    p.update(ptr)
    return w8.w8a8_int8_matmul(p["A"], lda, p["a_s"], p["B"], ldb, p["b_s"], p["C"], ldc, M, N, K, out, 0, opts)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=-1), ARG), (dict(out=-1), ARG), (dict(lda=15), ARG),
    (dict(ldb=1), ARG), (dict(ldc=7), ARG), (dict(A=0), ARG), (dict(b_s=0), ARG), (dict(C=0), ARG), (dict(M=0), OK),
    (dict(N=0, C=0), OK), (dict(K=w8.W8A8_INT8_MAX_K + 1), UNS), (dict(C=257), UNS), (dict(C=258, out=2), UNS),
    (dict(a_s=258), UNS), (dict(M=1 << 31), UNS), (dict(opts=w8.options(variant=w8.W8A8_VARIANT_SPLITK)), UNS),
    (dict(opts=w8.options(stages=9)), ARG),
])
def test_int8(kw, status):
    assert int8(**kw) == status


def test_int8_workspace_size():
    size = w8.w8a8_int8_workspace_size
    assert size(-1, 8, 8) == 0 and size(0, 8, 8) == 0 and size(4, 8, w8.W8A8_INT8_MAX_K + 1) == 0
    # large problems are cut: the workspace does not grow with M without end
    assert size(1 << 20, 4096, 4096) == size(1 << 22, 4096, 4096) < 1 << 30


def quant(M=4, K=16, kind=0, ld_x=0, ld_a=0, X=256, A=256, s=256):
    return w8.w8a8_quantize_int8_per_token(X, kind, ld_x, A, ld_a, s, M, K, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(K=-1), ARG), (dict(kind=3), ARG), (dict(ld_x=15), ARG), (dict(ld_a=3), ARG),
    (dict(X=0), ARG), (dict(s=0), ARG), (dict(M=0), OK), (dict(K=0), OK), (dict(X=257), UNS), (dict(s=258), UNS),
    (dict(X=258, kind=2), UNS), (dict(K=(1 << 30) + 1), UNS), (dict(M=1 << 31), UNS),
])
def test_quantiser(kw, status):
    assert quant(**kw) == status


def norm(M=4, D=32, hk=0, xk=0, ld_h=0, ld_x=0, gate=0, gate_rows=1, ld_xo=0, kind=0, ld_y=0, **ptr):
    p = dict(h=256, x=256, w_post=256, w_pre=256, x_out=256, y=256, s=256)
    p.update(ptr)
    return w8.w8a8_sandwich_norm(p["h"], hk, ld_h, p["x"], xk, ld_x, p["w_post"], gate, gate_rows, p["w_pre"], 1.0,
                                 1e-6, p["x_out"], ld_xo, p["y"], p["s"], kind, ld_y, M, D, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ARG), (dict(D=-1), ARG), (dict(hk=3), ARG), (dict(xk=-1), ARG), (dict(kind=3), ARG),
    (dict(gate=256, gate_rows=0), ARG), (dict(ld_h=31), ARG), (dict(ld_y=1), ARG), (dict(h=0), ARG), (dict(y=0), ARG),
    (dict(kind=1, s=0), ARG), (dict(M=0), OK), (dict(D=0), OK), (dict(hk=0, xk=1), UNS), (dict(hk=2, xk=0), UNS),
    (dict(D=w8.W8A8_NORM_MAX_D + 1), UNS), (dict(M=1 << 31), UNS), (dict(h=257), UNS), (dict(s=258, kind=2), UNS),
    (dict(kind=1, D=24), UNS), (dict(kind=1, h=258), UNS), (dict(kind=1, ld_x=33), UNS),
])
def test_norm(kw, status):
    assert norm(**kw) == status


def test_python_wrappers_refuse_shapes_and_types():
    e8 = lambda *s: torch.zeros(s, dtype=torch.int8)  # noqa: E731
    f = torch.zeros
    for call in (
        lambda: w8.int8_matmul(e8(4, 16).float(), f(4), e8(8, 16), f(8)),
        lambda: w8.int8_matmul(e8(4, 16), f(5), e8(8, 16), f(8)),
        lambda: w8.int8_matmul(e8(4, 16), f(4), e8(8, 17), f(8)),
        lambda: w8.int8_matmul(e8(16, 4).t(), f(4), e8(8, 16), f(8)),
        lambda: w8.int8_matmul(e8(4, 16), f(4), e8(8, 16), f(8), out=f(4, 9)),
        lambda: w8.quantize_int8_per_token(e8(4, 16)),
        lambda: w8.quantize_int8_per_token(f(4, 16), A=e8(4, 15)),
        lambda: w8.grouped_matmul_ragged(e8(4, 128), f(4, 1), e8(2, 8, 128), f(2, 1, 1), torch.zeros(2, dtype=torch.int32)),
        lambda: w8.grouped_matmul_ragged(e8(4, 128), f(4, 2), e8(2, 8, 128), f(2, 1, 1), torch.zeros(3, dtype=torch.int32)),
        lambda: w8.grouped_matmul_ragged(e8(4, 128), f(4, 1), e8(2, 8, 64), f(2, 1, 1), torch.zeros(3, dtype=torch.int32)),
        lambda: w8.sandwich_norm(f(4, 8), f(4, 9)),
        lambda: w8.sandwich_norm(f(4, 8), f(4, 8), w_post=f(9)),
        lambda: w8.sandwich_norm(f(4, 8), f(4, 8), w_pre=f(8).half()),
        lambda: w8.sandwich_norm(f(4, 8), f(4, 8), gate=f(1, 8), gate_rows=2),
        lambda: w8.sandwich_norm(f(4, 8), f(4, 8), x_out=f(4, 8).half()),
        lambda: w8.sandwich_norm(f(8, 4).t(), f(4, 8)),
        lambda: w8.sandwich_norm(f(1, 8).expand(4, 8), f(4, 8)),
        lambda: w8.sandwich_norm(f(4, 8), f(4, 8), y_out=torch.zeros(4, 8, dtype=torch.int8)),
        lambda: w8.sandwich_norm(f(4, 16), f(4, 16), out="fp8", y_out=f(4, 16)),
        lambda: w8.int8_matmul(e8(1, 16).expand(4, 16), f(4), e8(8, 16), f(8)),
    ):
        with pytest.raises(w8.W8A8Error):
            call()


def test_sandwich_norm_refuses_the_same_with_its_outputs_given():
    f, h = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    good = dict(h=f(4, 8), x=f(4, 8), x_out=f(4, 8), y_out=f(4, 8))
    e4, i8 = torch.zeros(4, 8, dtype=torch.float8_e4m3fn), torch.zeros(4, 8, dtype=torch.int8)
    for bad in (dict(x=f(4, 9)), dict(h=f(5, 8)), dict(x_out=f(4, 9)), dict(y_out=f(3, 8)), dict(x_out=h(4, 8)),
                dict(y_out=h(4, 8)), dict(w_post=f(9)), dict(w_post=h(8)), dict(w_pre=f(1, 8)), dict(w_pre=h(8)),
                dict(w_pre=f(16)[::2]), dict(gate=f(1, 8), gate_rows=2), dict(gate=f(2, 9)), dict(gate=h(8)),
                dict(gate=f(8), gate_rows=3), dict(gate=f(0, 8)), dict(gate=f(4, 8), gate_rows=0),
                dict(out="fp8", y_out=f(4, 8)), dict(out="fp8", y_out=e4, scales_out=f(4)),
                dict(out="int8", y_out=i8, scales_out=f(4, 1)), dict(h=f(8, 4).t()), dict(x=f(1, 8).expand(4, 8)),
                dict(h=torch.zeros(4, 8, dtype=torch.int32))):
        with pytest.raises(w8.W8A8Error) as e:
            w8.sandwich_norm(**dict(good, **bad))
        assert e.value.status in (ARG, UNS), (bad, e.value)


def test_int8_calls_refuse_the_same_with_their_outputs_given():
    e8, f = lambda *s: torch.zeros(s, dtype=torch.int8), torch.zeros  # noqa: E731
    good = dict(A=e8(4, 16), a_s=f(4), B=e8(8, 16), b_s=f(8), out=f(4, 8))
    for bad in (dict(A=f(4, 16)), dict(B=f(8, 16)), dict(A=e8(4, 17)), dict(B=e8(8, 15)), dict(a_s=f(5)), dict(b_s=f(7)),
                dict(a_s=f(8)[::2]), dict(out=f(4, 9)), dict(A=e8(16, 4).t()), dict(a_s=f(4, 1))):
        with pytest.raises(w8.W8A8Error) as e:
            w8.int8_matmul(**dict(good, **bad), out_dtype="fp32")
        assert e.value.status in (ARG, UNS), (bad, e.value)
    good = dict(X=f(4, 16), A=e8(4, 16), a_s=f(4))
    for bad in (dict(X=e8(4, 16)), dict(X=f(4, 17)), dict(A=e8(5, 16)), dict(a_s=f(4, 1)), dict(a_s=f(8)[::2]),
                dict(X=f(16, 4).t())):
        with pytest.raises(w8.W8A8Error) as e:
            w8.quantize_int8_per_token(**dict(good, **bad))
        assert e.value.status in (ARG, UNS), (bad, e.value)


@pytest.fixture(params=["python", "extension"])
def reached(request, monkeypatch):
    """The calls that reach the library's functions, which are stood in for; with the
    wrappers' checks in Python alone, and with those of the extension module before them."""
    hits, real = [], w8.load_library()

    def enter(*args):
        hits.append(args)
        return 0

    if request.param == "python":
        lib = type("Library", (), dict.fromkeys(("norm_tensors", "int8_tensors", "quant_tensors")))()
        for name in _binding._PYCALL:
            setattr(lib, name, enter)
        monkeypatch.setattr(w8, "load_library", lambda: lib)
        yield hits
        return
    if real.norm_tensors is None:
        pytest.skip("no extension module")
    entry = ctypes.CFUNCTYPE(ctypes.c_int)(enter)
    real.norm_tensors.__self__.bind(*[ctypes.cast(entry, ctypes.c_void_p).value] * 4)
    yield hits
    _binding._bind_pycall(ctypes.CDLL(w8.library_path()))


def refused(call, good, bad, reached):
    """The call with `bad` in the place of good arguments is refused for what it names
    (the first of `bad`, or the text that follows it) and does not reach the library."""
    kw, says = bad if isinstance(bad, tuple) else (bad, next(iter(bad)) + " must be")
    with pytest.raises(w8.W8A8Error, match=says) as e:
        call(**dict(good, **kw))
    assert e.value.status in (ARG, UNS), (bad, e.value)
    assert not reached, bad


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def test_ragged_refuses_elements_of_another_type(reached):
    u8, i32 = torch.uint8, torch.int32
    good = dict(A=z(4, 128, dtype=u8), a_s=z(4, 1), B=z(2, 8, 128, dtype=torch.float8_e4m3fn), b_s=z(2, 1, 1),
                offsets=z(3, dtype=i32), out_dtype="bf16", out=z(4, 8, dtype=torch.bfloat16), stream=0)
    for bad in (dict(offsets=z(3, dtype=torch.int64)), dict(offsets=z(3)), dict(a_s=z(4, 1, dtype=torch.bfloat16)),
                dict(b_s=z(2, 1, 1, dtype=torch.float64)), dict(A=z(4, 128, dtype=torch.bfloat16)),
                dict(A=z(4, 128, dtype=torch.int8)), dict(B=z(2, 8, 128, dtype=torch.float16)),
                dict(B=z(2, 8, 128, dtype=torch.float8_e5m2)), dict(out=z(4, 8)), dict(out=z(4, 8, dtype=torch.float16)),
                dict(out=good["out"], out_dtype="fp32"), dict(out=good["out"], out_dtype=torch.float16)):
        refused(w8.grouped_matmul_ragged, good, bad, reached)


def test_int8_matmul_refuses_elements_of_another_type(reached):
    i8, bf16 = torch.int8, torch.bfloat16
    good = dict(A=z(4, 16, dtype=i8), a_s=z(4), B=z(8, 16, dtype=i8), b_s=z(8), out_dtype="fp32", out=z(4, 8), stream=0)
    for given in (good, dict(good, out=None)):
        for bad in (dict(a_s=z(4, dtype=bf16)), dict(b_s=z(8, dtype=torch.float64)), dict(A=z(4, 16, dtype=torch.uint8)),
                    dict(B=z(8, 16, dtype=torch.uint8)), dict(out=z(4, 8, dtype=bf16)),
                    (dict(out_dtype="bf16", out=good["out"]), "out must be"),
                    (dict(out_dtype="bf16", out=z(4, 8, dtype=torch.float16)), "out must be")):
            refused(w8.int8_matmul, given, bad, reached)


def test_quantiser_refuses_outputs_of_another_type(reached):
    good = dict(X=z(4, 16), A=z(4, 16, dtype=torch.int8), a_s=z(4), stream=0)
    for bad in (dict(A=z(4, 16, dtype=torch.uint8)), dict(A=z(4, 16)), dict(a_s=z(4, dtype=torch.bfloat16)),
                dict(a_s=z(4, dtype=torch.float64))):
        refused(w8.quantize_int8_per_token, good, bad, reached)
        other = "a_s" if "A" in bad else "A"
        refused(w8.quantize_int8_per_token, dict(good, **{other: None}), bad, reached)


def test_sandwich_norm_refuses_scales_of_another_type(reached):
    for out, code, shape in (("fp8", torch.float8_e4m3fn, (4, 2)), ("int8", torch.int8, (4,))):
        good = dict(h=z(4, 144), x=z(4, 144), x_out=z(4, 144), y_out=z(4, 144, dtype=code), out=out, stream=0)
        for kw in (good, dict(good, x_out=None)):
            for dtype in (torch.bfloat16, torch.float64, torch.int32):
                refused(w8.sandwich_norm, kw, dict(scales_out=z(*shape, dtype=dtype)), reached)


def test_tensors_off_the_gpu_do_not_reach_the_library(reached):
    i8, u8, says = torch.int8, torch.uint8, "one CUDA device, not on cpu"
    for given in (True, False):
        for call, good in (
            (w8.grouped_matmul_ragged, dict(
                A=z(4, 128, dtype=u8), a_s=z(4, 1), B=z(2, 8, 128, dtype=u8), b_s=z(2, 1, 1),
                offsets=z(3, dtype=torch.int32), out_dtype="fp32", out=z(4, 8) if given else None)),
            (w8.int8_matmul, dict(A=z(4, 16, dtype=i8), a_s=z(4), B=z(8, 16, dtype=i8), b_s=z(8), out_dtype="fp32",
                                  out=z(4, 8) if given else None)),
            (w8.quantize_int8_per_token, dict(X=z(4, 16), **(dict(A=z(4, 16, dtype=i8), a_s=z(4)) if given else {}))),
            (w8.sandwich_norm, dict(h=z(4, 16), x=z(4, 16), w_post=z(16), w_pre=z(16), gate=z(16),
                                    **(dict(x_out=z(4, 16), y_out=z(4, 16)) if given else {}))),
        ):
            refused(call, good, (dict(stream=0), says), reached)


def test_sandwich_norm_refuses_a_gate_of_other_than_one_or_two_dimensions(reached, monkeypatch):
    """(A gate [B, 1, D] of an adaptive norm is not one row for all tokens.)"""
    monkeypatch.setattr(w8, "_one_gpu", lambda *tensors: None)      # these are on the host
    w8.sandwich_norm(z(12, 16), z(12, 16), gate=z(4, 16), stream=0)
    assert len(reached) == 1
    reached.clear()
    for outs in (dict(x_out=z(12, 16), y_out=z(12, 16)), {}):
        good = dict(h=z(12, 16), x=z(12, 16), stream=0, **outs)
        for shape in ((4, 1, 16), (1, 1, 16), (2, 2, 3, 16), ()):
            for rows in (None, 3, 12):
                refused(w8.sandwich_norm, good, dict(gate=z(*shape), gate_rows=rows), reached)
