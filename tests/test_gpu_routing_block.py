"""GPU: routing, the experts' products, their weighted sum and the requests' adapters
run together -- as the example runs them, captured into graphs, and in the
debug-bounds build."""
import os
import subprocess
import sys

import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8
from block_scaled_fp8_w8a8_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import moe_block  # noqa: E402


@pytest.mark.parametrize("tokens", [1, 6, 77, 2600])
def test_the_block_with_adapters_against_fp64(tokens):
    """Quantising an activation to E4M3 moves it by at most 2^-4 of itself and to INT8
    by 2^-8 of its row's largest; the block's four 8-bit products average such
    errors over their columns, the adapters' product and the experts' sum round once
    each (2^-8), and the norms keep relative errors."""
    w = moe_block.make_weights(seed=tokens, top_k=3)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    attn = torch.randn(tokens, 512, generator=g, device="cuda").bfloat16()
    x = 2 * torch.randn(tokens, 512, generator=g, device="cuda")
    which = torch.randint(-1, 4, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    adapters = moe_block.make_adapters(which, L=4, seed=tokens)
    r, codes, scales = moe_block.forward(w, attn, x, adapters)
    want_r, want_y = moe_block.reference(w, attn, x, adapters)
    assert (r - want_r).norm() <= 2.0 ** -4 * want_r.norm()
    assert (codes.double() * scales[:, None] - want_y).norm() <= 2.0 ** -4 * want_y.norm()
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


def chain(d):
    """Adapters into a projection's output, routing, the experts' ragged product of the
    routed rows, their weighted sum onto the projection's output."""
    order, offsets = w8.group_rows(d["of_token"], 3)
    h = w8.adapter_matmul(d["x"], d["a"], d["b"], order, offsets, d["base"], scales=d["scales"])
    _, weights, order, offsets, rows = w8.route_experts(d["logits"], 2, "sigmoid", bias=d["bias"], groups=4, top_groups=2,
                                                        scale=2.5, valid=d["valid"])
    q, s = w8.quantize_fp8_per_token_group(h)
    y = w8.grouped_matmul_ragged(q[order // 2], s[order // 2], d["w"], d["w_s"], offsets, "bf16")
    return h, weights, rows, w8.combine_experts(y, rows, weights, add=h)


def chain_inputs(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(of_token=torch.randint(-1, 3, (T,), generator=g, device="cuda", dtype=torch.int32),
                x=rn(T, 192).bfloat16(), a=rn(3, 16, 192).bfloat16(), b=rn(3, 256, 16).bfloat16(),
                base=rn(T, 256).bfloat16(), scales=rn(3), logits=rn(T, 16), bias=rn(16) / 8, valid=rn(T) < 1.5,
                w=(rn(16, 256, 256) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn), w_s=rn(16, 2, 2).abs() / 1000)


@pytest.mark.parametrize("T", [1, 50, 700])
def test_the_chain_against_fp64_and_padding(T):
    d = chain_inputs(T, T)
    h, weights, rows, out = chain(d)
    f = lambda t: t.double()  # noqa: E731
    q, s = w8.quantize_fp8_per_token_group(h)
    act = f(q.view(torch.float8_e4m3fn)) * f(s).repeat_interleave(128, 1)
    w = f(d["w"]) * f(d["w_s"]).repeat_interleave(128, 1).repeat_interleave(128, 2)
    scores = f(d["logits"]).sigmoid()
    ranked = scores + f(d["bias"])
    best = ranked.view(T, 4, 4).topk(2, 2)[0].sum(2).topk(2, 1)[1]
    closed = torch.ones(T, 4, dtype=torch.bool, device="cuda").scatter_(1, best, False)
    ids = ranked.masked_fill(closed.repeat_interleave(4, 1), -torch.inf).topk(2, 1)[1]
    wt = scores.gather(1, ids)
    wt = 2.5 * wt / wt.sum(1, keepdim=True)
    y = torch.einsum("tk,tjnk->tjn", act, w[ids])
    want = f(h) + torch.where(d["valid"][:, None], (y * wt[:, :, None]).sum(1), 0.0)
    # y and out round to bf16; the rest is fp32, and the sum over 256 columns of an 8-bit
    # product (in order, 2^-24 each) is far below either
    bound = 2.0 ** -8 * ((y.abs() * wt[:, :, None]).sum(1) * 1.01 + want.abs()) * 1.01 + 1e-3 * 2.0 ** -8
    products = torch.einsum("tk,tjnk->tjn", act.abs(), w[ids].abs()).mul(wt[:, :, None]).sum(1)
    assert ((f(out) - want).abs() <= bound + 300 * 2.0 ** -24 * products).all()
    off = ~d["valid"]
    assert (rows[off] == -1).all() and (weights[off] == 0).all() and torch.equal(out[off], h[off])


def test_the_chain_in_two_graphs_over_new_inputs():
    """Two graphs of one chain replayed side by side give a plain call's bits."""
    a, b = chain_inputs(130, 1), chain_inputs(300, 2)
    chain(a), chain(b)                      # everything is loaded before the capture
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], []
    for d in (a, b):
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            outs.append(chain(d))
        graphs.append(graph), streams.append(s)
    for seed in (11, 12, 13):
        for d, T in ((a, 130), (b, 300)):
            for k, v in chain_inputs(T, seed).items():
                d[k].copy_(v)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for d, got in zip((a, b), outs):
            for x, y in zip(got, chain(d)):
                assert torch.equal(x, y)
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


def run_all(seed=1):
    """Every kernel of the operators once or more, on sizes with ragged ends."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    out = {}
    for T, E, k, kw in ((1, 16, 2, {}), (77, 250, 8, dict(scoring="sigmoid")), (3000, 64, 4, dict(groups=8, top_groups=3)),
                        (70000, 8, 2, {})):
        for name, t in zip(("ids", "weights", "order", "offsets", "rows"), w8.route_experts(rn(T, E), k, **kw)):
            out[f"route{T}_{name}"] = t
    for n, L in ((0, 3), (700, 5), (200000, 1000)):
        ids = torch.randint(-1, L, (n,), generator=g, device="cuda", dtype=torch.int32)
        out[f"group{n}_order"], out[f"group{n}_offsets"] = w8.group_rows(ids, L)
    for T, k, D, dtype in ((5, 2, 512, torch.bfloat16), (130, 6, 1537, torch.float16), (130, 6, 515, torch.float32)):
        Y = rn(T * k, D).to(dtype)
        rows = torch.randint(-1, T * k, (T, k), generator=g, device="cuda", dtype=torch.int32)
        out[f"sum{D}"] = w8.combine_experts(Y, rows, rn(T, k), add=rn(T, D).to(dtype))
    for T, L, r, K, N, dtype, variant in ((1, 2, 16, 512, 264, torch.bfloat16, w8.W8A8_VARIANT_SMALLM),
                                          (90, 5, 40, 259, 131, torch.float16, w8.W8A8_VARIANT_SMALLM),
                                          (700, 3, 64, 640, 328, torch.bfloat16, w8.W8A8_VARIANT_TILED),
                                          (300, 3, 120, 520, 264, torch.float16, w8.W8A8_VARIANT_TILED)):
        for kind in (dtype, torch.float32):
            ids = torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=torch.int32)
            order, offsets = w8.group_rows(ids, L)
            out[f"adapters{T}_{kind}"] = w8.adapter_matmul(rn(T, K).to(dtype), rn(L, r, K).to(dtype), rn(L, N, r).to(dtype),
                                                           order, offsets, rn(T, N).to(kind), scales=rn(L),
                                                           variant=variant)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in out.items()}


CHILD = r"""
import sys, torch
import block_scaled_fp8_w8a8_gb300 as w8
sys.path.insert(0, sys.argv[2])
from test_gpu_routing_block import run_all
assert w8.w8a8_debug_bounds_build() == 1
torch.save({"out": run_all(), "status": w8.w8a8_get_device_status()}, sys.argv[1])
"""


def test_debug_bounds_build(tmp_path):
    """The build that checks every index finds none outside its buffer and gives the
    release build's bits."""
    build.build(debug_bounds=True)
    path = str(tmp_path / "res.pt")
    env = {k: v for k, v in os.environ.items() if not k.startswith("W8A8_")}
    env["W8A8_DEBUG_BOUNDS"] = "1"
    r = subprocess.run([sys.executable, "-c", CHILD, path, os.path.dirname(os.path.abspath(__file__))], env=env,
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = torch.load(path)
    assert res["status"][0] == w8.W8A8_OK, hex(res["status"][1])
    for k, v in run_all().items():
        assert torch.equal(res["out"][k], v), k
