"""GPU: the routing, grouping, sum and adapter kernels in the debug-bounds build, which checks
every index and TMA box: no check fires and the bits are the release build's, over the forms that a
size, stride, type or tie can choose."""
import os
import subprocess
import sys

import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8
from block_scaled_fp8_w8a8_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SMALL, TILED = w8.W8A8_VARIANT_SMALLM, w8.W8A8_VARIANT_TILED


def wide(t, shift, pad):
    """t as a view of wider rows, one more of them on either side."""
    big = torch.zeros(t.shape[0] + 2, shift + t.shape[1] + pad, device="cuda", dtype=t.dtype)
    big[1:-1, shift:shift + t.shape[1]] = t
    return big[1:-1, shift:shift + t.shape[1]]


def run(seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    out = {}

    def route(name, x, k, **kw):
        for part, t in zip(("ids", "weights", "order", "offsets", "rows"), w8.route_experts(x, k, **kw)):
            out[f"route {name} {part}"] = t

    for T, E, k, groups, top, group_top in ((0, 9, 2, 1, 1, 1), (1, 1, 1, 1, 1, 1), (7, 31, 31, 1, 1, 1), (40, 250, 8, 2, 1, 2),
                                            (300, 160, 6, 8, 3, 1), (513, 1024, 32, 32, 9, 2), (5000, 60, 5, 5, 2, 2),
                                            (9000, 1000, 3, 4, 2, 2), (600, 96, 4, 3, 2, 1)):
        for dtype in (F32, BF16, F16):
            for scoring in ("softmax", "sigmoid"):
                x = (2 * rn(T, E)).to(dtype)
                route(f"{T}x{E} {dtype} {scoring}", x, k, scoring=scoring, groups=groups, top_groups=top, group_top=group_top)
                route(f"{T}x{E} {dtype} {scoring} biased", x, k, scoring=scoring, bias=8 + rn(E) / 8, groups=groups,
                      top_groups=top, group_top=group_top, valid=rn(T) < 1, renormalize=False)
                if T:
                    route(f"{T}x{E} {dtype} {scoring} strided", wide(x, 3, 2), k, scoring=scoring, groups=groups,
                          top_groups=top, group_top=group_top)
    for E, groups in ((256, 8), (100, 4), (1024, 1)):       # ties: in 64 bits one after the other
        for bias in (None, torch.zeros(E, device="cuda")):
            route(f"ties {E} {bias is None}", torch.zeros(90, E, device="cuda"), 8, scoring="sigmoid", bias=bias, groups=groups,
                  top_groups=max(1, groups // 2))
            route(f"near {E} {bias is None}", -90 - rn(90, E).abs() / 1e6, 8, bias=bias, groups=groups,
                  top_groups=max(1, groups // 2))
    for n, L in ((0, 1), (1, 1), (65536, 1024), (65600, 300), (300001, 7)):
        ids = ints(-2, L + 2, n)
        out[f"group {n} order"], out[f"group {n} offsets"] = w8.group_rows(ids, L)
    for T, k, D, M in ((1, 8, 4096, 8), (300, 1, 1936, 300), (300, 2, 160, 90), (2000, 1, 512, 2000), (5, 17, 2050, 40),
                       (130, 6, 1537, 200), (3000, 1, 70, 3000), (3000, 2, 33, 3), (4, 0, 100, 5), (2, 3, 1, 1), (3, 2, 24, 0)):
        for dtype, kind in ((BF16, BF16), (F16, F32), (F32, F32)):
            Y, rows, w, add = rn(M, D).to(dtype), ints(-1, M + 1, T, k), rn(T, k), rn(T, D).to(kind)
            code = {BF16: "bf16", F32: "fp32"}[kind]
            out[f"sum {T} {k} {D} {dtype}"] = w8.combine_experts(Y, rows, w, add=add, out_dtype=code)
            out[f"sum {T} {k} {D} {dtype} strided"] = w8.combine_experts(wide(Y, 1, 2), rows, w, out=wide(add, 3, 1))
    for T, L, K, N, r, variant in ((1, 1, 64, 64, 16, SMALL), (3, 2, 1, 1, 1, SMALL), (33, 2, 2048, 160, 256, SMALL),
                                   (40, 3, 1000, 1537, 24, SMALL), (6, 3, 0, 32, 8, SMALL), (6, 3, 64, 32, 0, SMALL),
                                   (2, 0, 64, 32, 8, SMALL), (300, 40, 520, 264, 64, SMALL), (9, 1024, 64, 32, 4, SMALL),
                                   (32, 1, 64, 8, 8, TILED), (257, 1, 72, 136, 72, TILED), (1000, 3, 1000, 1032, 40, TILED),
                                   (400, 3, 2048, 64, 104, TILED), (640, 20, 256, 200, 128, TILED), (5000, 4, 512, 264, 48, TILED)):
        for dtype, kind in ((BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)):
            ids = ints(-1, max(L, 1), T) if L else torch.full((T,), -1, dtype=torch.int32, device="cuda")
            order, offsets = w8.group_rows(ids, L) if L else (torch.arange(T, dtype=torch.int32, device="cuda"),
                                                              torch.zeros(1, dtype=torch.int32, device="cuda"))
            x, a, b, base = rn(T, K).to(dtype), rn(L, r, K).to(dtype), rn(L, N, r).to(dtype), rn(T, N).to(kind)
            name = f"adapters {T} {K} {N} {r} {dtype} {kind}"
            out[name] = w8.adapter_matmul(x, a, b, order, offsets, base, scales=rn(L), variant=variant)
            place = base.clone()
            out[name + " in place"] = w8.adapter_matmul(x, a, b, order, offsets, place, out=place, variant=variant)
            out[name + " strided"] = w8.adapter_matmul(wide(x, 8, 8), a, b, order, offsets, wide(base, 8, 8), variant=variant)
            if T >= 30 and L:      # entries that name no row, offsets out of order and range
                bad = order.clone()
                bad[3], bad[20] = -5, 2 ** 30
                # (rows that are skipped are not written)
                out[name + " order"] = w8.adapter_matmul(x, a, b, bad, offsets, base, out=base.clone(), variant=variant)
                wrong = offsets.clone()
                wrong[0], wrong[-1] = -1, 2 ** 31 - 1
                w8.adapter_matmul(x, a, b, order, wrong, base, variant=variant)
    torch.cuda.synchronize()
    return {k: v.cpu().contiguous() for k, v in out.items()}


CHILD = r"""
import sys, torch
import block_scaled_fp8_w8a8_gb300 as w8
sys.path.insert(0, sys.argv[2])
from test_gpu_routing_bounds import run
assert w8.w8a8_debug_bounds_build() == 1
torch.save({"out": run(), "status": w8.w8a8_get_device_status()}, sys.argv[1])
"""


def bits(t):
    return t.view(torch.uint8).numpy().tobytes() if t.numel() else b""


def test_no_check_fires_and_the_bits_are_the_release_builds(tmp_path):
    build.build(debug_bounds=True)
    path = str(tmp_path / "res.pt")
    env = {k: v for k, v in os.environ.items() if not k.startswith("W8A8_")}
    env["W8A8_DEBUG_BOUNDS"] = "1"
    r = subprocess.run([sys.executable, "-c", CHILD, path, os.path.dirname(os.path.abspath(__file__))], env=env,
                       capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = torch.load(path)
    assert res["status"][0] == w8.W8A8_OK, hex(res["status"][1])
    want = run()
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
    assert want.keys() == res["out"].keys()
    for k, v in want.items():
        assert bits(res["out"][k]) == bits(v), k
