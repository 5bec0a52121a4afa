"""Refusals of the routing, grouping, combining and adapter calls: every one comes before any
CUDA call, so they are checked without a GPU, by status and message."""
import ctypes

import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8
from block_scaled_fp8_w8a8_gb300 import _binding, build

OK, ARG, UNS, WS = w8.W8A8_OK, w8.W8A8_ERR_INVALID_ARG, w8.W8A8_ERR_UNSUPPORTED, w8.W8A8_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return w8.load_library()


def route(T=4, E=64, k=4, dtype=0, ld=0, scoring=0, groups=1, top_groups=1, group_top=1, **ptr):
    p = dict(x=256, bias=0, valid=0, ids=256, w=256, order=256, off=256, rows=256, ws=0, size=0)
    p.update(ptr)
    return w8.w8a8_route_experts(p["x"], dtype, ld, p["bias"], p["valid"], T, E, k, scoring, groups, top_groups, group_top,
                                 1, 1.0, p["ids"], p["w"], p["order"], p["off"], p["rows"], p["ws"], p["size"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(E=-4), ARG), (dict(k=0), ARG), (dict(k=65), ARG), (dict(dtype=3), ARG),
    (dict(scoring=2), ARG), (dict(scoring=-1), ARG), (dict(groups=0), ARG), (dict(groups=3), ARG),
    (dict(groups=4, top_groups=5), ARG), (dict(groups=4, top_groups=0), ARG), (dict(group_top=3), ARG),
    (dict(group_top=0), ARG), (dict(groups=64, top_groups=8, group_top=2), ARG), (dict(groups=32, top_groups=1, k=3), ARG),
    (dict(ld=63), ARG), (dict(x=0), ARG), (dict(ids=0), ARG), (dict(w=0), ARG), (dict(order=0), ARG), (dict(off=0), ARG),
    (dict(rows=0), ARG), (dict(T=0, off=0), ARG), (dict(E=w8.W8A8_GROUPS_MAX + 1), UNS), (dict(k=33), UNS),
    (dict(groups=64, top_groups=64), UNS), (dict(T=1 << 29), UNS), (dict(x=257), UNS), (dict(x=258, dtype=2), UNS),
    (dict(bias=258), UNS), (dict(ids=258), UNS), (dict(rows=258), UNS), (dict(T=100000), WS),
    (dict(T=100000, ws=256, size=16), WS), (dict(T=100000, ws=258, size=1 << 30), WS),
])
def test_route(kw, status):
    assert route(**kw) == status
    assert w8.w8a8_last_error() != ""


def test_workspace_sizes():
    size = w8.w8a8_route_workspace_size
    assert size(64, 256, 8) == 0 and size(0, 256, 8) == 0 and size(16384, 256, 8) > 0
    for bad in ((-1, 256, 8), (64, 0, 8), (1 << 20, w8.W8A8_GROUPS_MAX + 1, 8), (1 << 20, 256, 0), (1 << 30, 256, 8)):
        assert size(*bad) == 0
    size = w8.w8a8_group_workspace_size
    assert size(16384, 64) == 0 and size(1 << 20, 64) >= 4 << 20
    assert size(-1, 4) == size(1 << 20, 0) == size(1 << 31, 4) == size(1 << 20, w8.W8A8_GROUPS_MAX + 1) == 0


    size = w8.w8a8_adapter_workspace_size
    assert size(64, 32, 16, 4096) == 0 and size(16384, 16, 64, 4096) >= 16384 * 64 * 4
    assert size(64, 32, 16, 4096, w8.W8A8_VARIANT_TILED) > 0 and size(16384, 16, 64, 4096, w8.W8A8_VARIANT_SMALLM) == 0
    for bad in ((0, 1, 16, 64), (4096, 0, 16, 64), (4096, 1, 0, 64), (4096, 1, 16, 0), (1 << 28, 1, 16, 64),
                (4096, 1, w8.W8A8_ADAPTER_MAX_R + 1, 64), (4096, w8.W8A8_GROUPS_MAX + 1, 16, 64)):
        assert size(*bad) == 0


def group(n=8, groups=4, **ptr):
    p = dict(ids=256, order=256, off=256, rows=0, ws=0, size=0)
    p.update(ptr)
    return w8.w8a8_group_rows(p["ids"], n, groups, p["order"], p["off"], p["rows"], p["ws"], p["size"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(groups=0), ARG), (dict(groups=w8.W8A8_GROUPS_MAX + 1), UNS), (dict(n=1 << 31), UNS),
    (dict(ids=0), ARG), (dict(order=0), ARG), (dict(off=0), ARG), (dict(n=0, off=0), ARG), (dict(ids=257), UNS),
    (dict(rows=258), UNS), (dict(n=1 << 20), WS), (dict(n=1 << 20, ws=256, size=4096), WS),
])
def test_group_rows(kw, status):
    assert group(**kw) == status


def combine(M=8, T=4, k=2, D=32, dtype=0, out_dtype=0, ld_y=0, ld_add=0, ld_out=0, **ptr):
    p = dict(Y=256, rows=256, w=256, add=0, out=256)
    p.update(ptr)
    return w8.w8a8_combine_experts(p["Y"], dtype, ld_y, M, p["rows"], p["w"], p["add"], ld_add, p["out"], out_dtype, ld_out,
                                   T, k, D, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(k=-1), ARG), (dict(D=-1), ARG), (dict(M=-1), ARG), (dict(dtype=3), ARG), (dict(out_dtype=-1), ARG),
    (dict(dtype=0, out_dtype=1), UNS), (dict(dtype=2, out_dtype=0), UNS), (dict(ld_y=31), ARG), (dict(ld_add=1), ARG),
    (dict(ld_out=31), ARG), (dict(T=0), OK), (dict(D=0), OK), (dict(Y=0), ARG), (dict(rows=0), ARG), (dict(w=0), ARG),
    (dict(out=0), ARG), (dict(D=(1 << 24) + 1), UNS), (dict(T=1 << 31), UNS), (dict(k=(1 << 20) + 1), UNS),
    (dict(Y=257), UNS), (dict(out=257), UNS), (dict(out=258, out_dtype=2), UNS), (dict(add=257), UNS), (dict(w=258), UNS),
])
def test_combine(kw, status):
    assert combine(**kw) == status


def test_combine_in_place_of_an_addend_of_another_stride():
    assert combine(add=256, ld_add=64, ld_out=40) == ARG
    assert "add's place" in w8.w8a8_last_error()


def adapters(T=4, L=2, r=16, K=64, N=32, dtype=0, out_dtype=0, ld_x=0, ld_base=0, ld_out=0, variant=0, **ptr):
    p = dict(x=256, A=256, B=256, order=256, off=256, scales=0, base=256, out=512, ws=0, size=0)
    p.update(ptr)
    return w8.w8a8_adapter_matmul(p["x"], dtype, ld_x, p["A"], p["B"], p["order"], p["off"], p["scales"], p["base"], ld_base,
                                  p["out"], out_dtype, ld_out, T, L, r, K, N, variant, p["ws"], p["size"], 0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(L=-1), ARG), (dict(r=-1), ARG), (dict(K=-1), ARG), (dict(N=-1), ARG), (dict(dtype=3), ARG),
    (dict(out_dtype=3), ARG), (dict(dtype=2, out_dtype=2), UNS), (dict(dtype=0, out_dtype=1), UNS),
    (dict(dtype=1, out_dtype=0), UNS), (dict(ld_x=63), ARG), (dict(ld_base=31), ARG), (dict(ld_out=31), ARG),
    (dict(out=256, ld_out=40), ARG), (dict(T=0), OK), (dict(N=0), OK), (dict(x=0), ARG), (dict(A=0), ARG), (dict(B=0), ARG),
    (dict(order=0), ARG), (dict(off=0), ARG), (dict(base=0), ARG), (dict(out=0), ARG), (dict(L=w8.W8A8_GROUPS_MAX + 1), UNS),
    (dict(r=w8.W8A8_ADAPTER_MAX_R + 1), UNS), (dict(T=1 << 28), UNS), (dict(K=(1 << 24) + 1), UNS), (dict(x=257), UNS),
    (dict(base=258, out_dtype=2), UNS), (dict(scales=258), UNS), (dict(order=257), UNS), (dict(T=4096), WS),
    (dict(T=4096, ws=256, size=4096), WS), (dict(T=4096, ws=264, size=1 << 30), WS),
    (dict(variant=-1), ARG), (dict(variant=8), ARG), (dict(variant=w8.W8A8_VARIANT_SWAPAB), UNS),
    (dict(variant=w8.W8A8_VARIANT_TILED), WS), (dict(variant=w8.W8A8_VARIANT_TILED, r=12), UNS),
    (dict(variant=w8.W8A8_VARIANT_TILED, r=136), UNS), (dict(variant=w8.W8A8_VARIANT_TILED, K=66), UNS),
    (dict(variant=w8.W8A8_VARIANT_TILED, K=56), UNS), (dict(variant=w8.W8A8_VARIANT_TILED, N=36), UNS),
    (dict(variant=w8.W8A8_VARIANT_TILED, x=264), UNS), (dict(variant=w8.W8A8_VARIANT_TILED, ld_x=65), UNS),
    (dict(variant=w8.W8A8_VARIANT_TILED, L=0), UNS),
])
def test_adapters(kw, status):
    assert adapters(**kw) == status


# ---------------------------------------------------------------- Python


@pytest.fixture(params=["python", "extension"])
def reached(request, monkeypatch):
    """The calls that reach the library's functions, which are stood in for; with the wrappers'
    checks in Python alone, and with those of the extension module before them."""
    hits, real = [], w8.load_library()

    def enter(*args):
        hits.append(args)
        return 0

    if request.param == "python":
        lib = type("Library", (), dict.fromkeys(_binding._ROUTING_TENSORS))()
        for name in _binding._PYCALL_ROUTING:
            setattr(lib, name, enter)
        monkeypatch.setattr(w8, "load_library", lambda: lib)
        yield hits
        return
    if real.route_tensors is None:
        pytest.skip("no extension module")
    entry = ctypes.CFUNCTYPE(ctypes.c_int)(enter)
    real.route_tensors.__self__.bind_routing(*[ctypes.cast(entry, ctypes.c_void_p).value] * 7)
    yield hits
    _binding._bind_pycall(ctypes.CDLL(w8.library_path()))


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


I32, BF16 = torch.int32, torch.bfloat16


def route_outs():
    return z(4, 2, dtype=I32), z(4, 2), z(8, dtype=I32), z(9, dtype=I32), z(4, 2, dtype=I32)


GOOD = {
    "route_experts": (dict(logits=z(4, 8), top_k=2, bias=z(8), valid=z(4, dtype=torch.bool), out=route_outs(), stream=0), [
        dict(logits=z(4, 8, dtype=torch.float64)), dict(logits=z(4, 8, dtype=I32)), dict(logits=z(8)), dict(logits=z(8, 4).t()),
        dict(logits=z(1, 8).expand(4, 8)), dict(top_k=0), dict(top_k=33), dict(top_k=2.0), dict(scoring="tanh"),
        dict(bias=z(7)), dict(bias=z(8, dtype=BF16)), dict(bias=z(1, 8)), dict(bias=z(16)[::2]), dict(valid=z(3, dtype=torch.bool)),
        dict(valid=z(4)), dict(valid=z(4, 1, dtype=torch.bool)), dict(valid=z(8, dtype=torch.bool)[::2]), dict(out=route_outs()[:4]),
        *[dict(out=tuple(z(*t.shape, dtype=torch.int64) if i == j else t for i, t in enumerate(route_outs()))) for j in range(5)],
        *[dict(out=tuple(z(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype) if i == j else t for i, t in enumerate(route_outs())))
          for j in range(5)],
        dict(out=tuple(z(2, 4, dtype=t.dtype).t() if i == 0 else t for i, t in enumerate(route_outs()))),
    ]),
    "group_rows": (dict(ids=z(6, dtype=I32), groups=3, out=(z(6, dtype=I32), z(4, dtype=I32)), stream=0), [
        dict(ids=z(6, dtype=torch.int64)), dict(ids=z(6)), dict(ids=z(12, dtype=I32)[::2]), dict(ids=z(5, dtype=I32)),
        dict(groups=4), dict(out=(z(6, dtype=I32),)), dict(out=(z(6), z(4, dtype=I32))),
        dict(out=(z(6, dtype=I32), z(3, dtype=I32))), dict(out=(z(6, dtype=I32), z(4, dtype=torch.int64))),
    ]),
    "combine_experts": (dict(Y=z(9, 16), rows=z(4, 2, dtype=I32), weights=z(4, 2), add=z(4, 16), out=z(4, 16), stream=0), [
        dict(Y=z(9, 16, dtype=torch.float64)), dict(Y=z(9)), dict(Y=z(9, 17)), dict(Y=z(16, 9).t()),
        dict(rows=z(4, 2, dtype=torch.int64)), dict(rows=z(8, dtype=I32)), dict(rows=z(5, 2, dtype=I32)),
        dict(rows=z(4, 4, dtype=I32)[:, ::2]), dict(weights=z(4, 3)), dict(weights=z(4, 2, dtype=BF16)), dict(add=z(4, 15)),
        dict(add=z(4, 16, dtype=BF16)), dict(out=z(5, 16)), dict(out=z(4, 16, dtype=BF16)), dict(out=z(1, 16).expand(4, 16)),
        dict(out_dtype="bf16"),
    ]),
    "adapter_matmul": (dict(x=z(4, 8, dtype=BF16), A=z(2, 3, 8, dtype=BF16), B=z(2, 16, 3, dtype=BF16), order=z(4, dtype=I32),
                            offsets=z(3, dtype=I32), base=z(4, 16), scales=z(2), out=z(4, 16), stream=0), [
        dict(x=z(4, 8, dtype=torch.float64)), dict(x=z(4, 9, dtype=BF16)), dict(x=z(4, 8, dtype=torch.float16)), dict(x=z(8, dtype=BF16)),
        dict(A=z(2, 3, 9, dtype=BF16)), dict(A=z(2, 3, 8)), dict(A=z(6, 8, dtype=BF16)), dict(A=z(3, 3, 8, dtype=BF16)),
        dict(A=z(2, 8, 3, dtype=BF16).transpose(1, 2)), dict(B=z(2, 16, 4, dtype=BF16)), dict(B=z(1, 16, 3, dtype=BF16)),
        dict(B=z(2, 3, 16, dtype=BF16).transpose(1, 2)), dict(order=z(5, dtype=I32)), dict(order=z(4, dtype=torch.int64)),
        dict(offsets=z(4, dtype=I32)), dict(offsets=z(3)), dict(base=z(4, 15)), dict(base=z(4, 16, dtype=BF16)),
        dict(scales=z(3)), dict(scales=z(2, dtype=BF16)), dict(scales=z(4)[::2]), dict(out=z(4, 17)), dict(out=z(4, 16, dtype=BF16)),
        dict(out=z(1, 16).expand(4, 16)),
    ]),
}


@pytest.mark.parametrize("name", GOOD)
def test_wrappers_refuse_shapes_types_and_strides(name, reached):
    good, bads = GOOD[name]
    for bad in bads:
        for given in (good, {k: v for k, v in good.items() if k != "out"}):
            if given is not good and ("out" in bad or (name == "group_rows" and ("groups" in bad or bad["ids"].shape == (5,)))
                                      or "out_dtype" in bad or (name, list(bad)) == ("adapter_matmul", ["base"]) and bad["base"].shape == (4, 16)
                                      or name == "combine_experts" and bad.get("Y", z()).shape == (9, 17) and "add" not in given):
                continue
            with pytest.raises(w8.W8A8Error) as e:
                getattr(w8, name)(**dict(given, **bad))
            assert e.value.status in (ARG, UNS), (bad, e.value)
            assert not [h for h in reached if len(h) > 3], bad      # (sizes may be asked for)


@pytest.mark.parametrize("name", GOOD)
def test_tensors_off_the_gpu_do_not_reach_the_library(name, reached):
    good, _ = GOOD[name]
    for given in (good, {k: v for k, v in good.items() if k != "out"}):
        with pytest.raises(w8.W8A8Error, match="one CUDA device, not on cpu"):
            getattr(w8, name)(**given)
        assert not [h for h in reached if len(h) > 3]


# ---------------------------------------------------------------- operands of sizes that are zero


@pytest.mark.parametrize("kw", [dict(K=0, B=0), dict(K=0, B=0, x=0, A=0), dict(K=0, B=0, N=1), dict(K=0, B=0, out_dtype=2),
                                dict(K=0, B=0, T=5000, r=64)])
def test_adapters_without_columns_of_x_still_read_b(kw):
    """B [L, N, r] does not depend on K: it is read where there are adapters of some rank."""
    assert adapters(**kw) == ARG
    assert "null pointer" in w8.w8a8_last_error()


# ---------------------------------------------------------------- numbers that the C calls take in 32 bits


@pytest.mark.parametrize("kw", [dict(groups=2 ** 32 + 1), dict(groups=2 ** 31), dict(groups=-2 ** 32), dict(groups=0), dict(groups=1.0),
                                dict(groups=4, top_groups=2 ** 32 + 2), dict(groups=4, top_groups=2 ** 40), dict(groups=2, group_top=2 ** 32 + 1),
                                dict(groups=2, group_top=0), dict(groups=2, group_top=None)])
def test_routing_refuses_numbers_of_groups_out_of_range(kw, reached):
    """They would be cut to 32 bits on their way to the library: 2^32 + 1 groups to one."""
    with pytest.raises(w8.W8A8Error, match=list(kw)[-1]) as e:
        w8.route_experts(z(4, 8), 2, **kw)
    assert e.value.status == ARG and not [h for h in reached if len(h) > 3]


@pytest.mark.parametrize("variant", [2 ** 32, 2 ** 32 + w8.W8A8_VARIANT_SMALLM, -1, 2 ** 31, 1.5, "tiled"])
def test_adapters_refuse_a_variant_out_of_range(variant, reached):
    with pytest.raises(w8.W8A8Error, match="variant") as e:
        w8.adapter_matmul(**dict(GOOD["adapter_matmul"][0], variant=variant))
    assert e.value.status == ARG and not [h for h in reached if len(h) > 3]


@pytest.mark.parametrize("groups", [2 ** 32 + 3, 2 ** 63, 0, -1, 1025, 3.0])
def test_grouping_refuses_numbers_of_groups_out_of_range(groups, reached):
    with pytest.raises(w8.W8A8Error, match="groups"):
        w8.group_rows(z(6, dtype=I32), groups)
    assert not [h for h in reached if len(h) > 3]
