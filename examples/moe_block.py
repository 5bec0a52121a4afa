"""The second half of a transformer block with norms around its parts, in 8 bits:

    attention output --INT8 projection, requests' adapters--> post-norm, residual,
    pre-norm --FP8--> routing, experts (ragged grouped matmuls, SwiGLU between),
    their weighted sum --> post-norm, gate, residual, pre-norm --INT8--> the next
    block's operand

One token and a long prompt take the same path: the routing stays on the device,
the experts' rows need no padding, and each norm writes the 8-bit operand that
the next matmul reads.

    python examples/moe_block.py            # checks against fp64, prints times
"""
from __future__ import annotations

import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_w8a8_gb300 as w8  # noqa: E402

EPS = 1e-6


@dataclasses.dataclass
class Weights:
    w_o: torch.Tensor         # int8 [D, D] and one scale per output channel
    w_o_s: torch.Tensor
    router: torch.Tensor      # fp32 [E, D]
    up: torch.Tensor          # E4M3 [E, 2 F, D] (gate rows, then up rows) and block scales
    up_s: torch.Tensor
    down: torch.Tensor        # E4M3 [E, D, F] and block scales
    down_s: torch.Tensor
    norms: list               # bf16 [D]: attention post, experts' pre, experts' post, next pre
    gate: torch.Tensor        # bf16 [D], on the experts' output
    top_k: int = 2


@dataclasses.dataclass
class Adapters:
    """Low-rank adapters beside w_o: L of them, and one (or none, -1) for each token."""
    a: torch.Tensor           # bf16 [L, r, D]
    b: torch.Tensor           # bf16 [L, D, r]
    scales: torch.Tensor      # fp32 [L]
    of_token: torch.Tensor    # int32 [T]


def make_weights(D=512, F=256, E=8, top_k=2, seed=0, device="cuda") -> Weights:
    g = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    rnd = lambda *s: torch.rand(s, generator=g, device=device) + 0.5  # noqa: E731

    def fp8(n, k):
        codes = (rn(E, n, k) * 112).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return codes, rnd(E, -(-n // 128), -(-k // 128)) / (112 * k ** 0.5)

    w_o = (rn(D, D) * 32).round_().clamp_(-127, 127).to(torch.int8)
    up, up_s = fp8(2 * F, D)
    down, down_s = fp8(D, F)
    return Weights(w_o, rnd(D) / (32 * D ** 0.5), rn(E, D) / D ** 0.5, up, up_s, down, down_s,
                   [(1 + 0.1 * rn(D)).bfloat16() for _ in range(4)], (0.5 * rn(D)).bfloat16(), top_k)


def make_adapters(of_token: torch.Tensor, L=3, r=16, D=512, seed=0) -> Adapters:
    g = torch.Generator(device=of_token.device).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=of_token.device)  # noqa: E731
    return Adapters((rn(L, r, D) / D ** 0.5).bfloat16(), (rn(L, D, r) / r ** 0.5).bfloat16(), rn(L).abs(), of_token)


def route(y: torch.Tensor, router: torch.Tensor, top_k: int):
    """Each token's experts and weights, and the rows in the experts' order: (order
    of the T * top_k (token, choice) pairs, offsets [E + 1], where each pair's row is
    [T, top_k], weights [T, top_k])."""
    _, weights, order, offsets, rows = w8.route_experts(y @ router.t(), top_k)
    return order, offsets, rows, weights


def dequantise(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """E4M3 codes with a scale per 128 columns, as fp32."""
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1)[:, :codes.shape[1]]


def project(w: Weights, attn: torch.Tensor, adapters: Adapters | None = None) -> torch.Tensor:
    """The attention's output through w_o and each token's adapter."""
    a, a_s = w8.quantize_int8_per_token(attn)
    h = w8.int8_matmul(a, a_s, w.w_o, w.w_o_s, "bf16")
    if adapters is not None:
        order, offsets = w8.group_rows(adapters.of_token, adapters.a.shape[0])
        w8.adapter_matmul(attn, adapters.a, adapters.b, order, offsets, h, adapters.scales, out=h)
    return h


def forward(w: Weights, attn: torch.Tensor, x: torch.Tensor, adapters: Adapters | None = None):
    """attn bf16 [T, D] (the attention's output), x fp32 [T, D] (the residual stream):
    returns (the new residual stream, INT8 codes and scales of the next block's input)."""
    h = project(w, attn, adapters)
    x, q, q_s = w8.sandwich_norm(h, x, w.norms[0], w.norms[1], eps=EPS, out="fp8")
    order, offsets, rows, weights = route(dequantise(q, q_s), w.router, w.top_k)
    token = order // w.top_k
    gu = w8.grouped_matmul_ragged(q[token], q_s[token], w.up, w.up_s, offsets, "bf16")
    gate, up = gu.chunk(2, 1)
    f, f_s = w8.quantize_fp8_per_token_group((torch.nn.functional.silu(gate) * up).contiguous())
    out = w8.grouped_matmul_ragged(f, f_s, w.down, w.down_s, offsets, "bf16")
    moe = w8.combine_experts(out, rows, weights)
    return w8.sandwich_norm(moe, x, w.norms[2], w.norms[3], gate=w.gate, eps=EPS, out="int8")


def reference(w: Weights, attn: torch.Tensor, x: torch.Tensor, adapters: Adapters | None = None):
    """The same block in fp64 with the weights' values and unquantised activations; the
    routing is taken from the 8-bit path (near-ties may fall either way)."""
    d = lambda t: t.double()  # noqa: E731
    rms = lambda t: t / (t.square().mean(1, keepdim=True) + EPS).sqrt()  # noqa: E731
    h = d(attn) @ (d(w.w_o) * d(w.w_o_s)[:, None]).t()
    if adapters is not None:
        for i in range(adapters.a.shape[0]):
            mine = adapters.of_token == i
            h[mine] += d(adapters.scales[i]) * (d(attn[mine]) @ d(adapters.a[i]).t() @ d(adapters.b[i]).t())
    x1 = d(x) + rms(h) * d(w.norms[0])
    y = rms(x1) * d(w.norms[1])
    _, q, q_s = w8.sandwich_norm(project(w, attn, adapters), x, w.norms[0], w.norms[1], eps=EPS, out="fp8")
    order, offsets, _, weights = route(dequantise(q, q_s), w.router, w.top_k)
    off = offsets.tolist()
    blocks = lambda s, n, k: d(s).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]  # noqa: E731
    out = torch.zeros(order.shape[0], x.shape[1], dtype=torch.float64, device=x.device)
    for e in range(len(off) - 1):
        rows = order[off[e]:off[e + 1]]
        if rows.numel():
            up = d(w.up[e]) * blocks(w.up_s[e], *w.up[e].shape)
            down = d(w.down[e]) * blocks(w.down_s[e], *w.down[e].shape)
            gate, u = (y[rows // w.top_k] @ up.t()).chunk(2, 1)
            out[rows] = (torch.nn.functional.silu(gate) * u) @ down.t()
    moe = (out.view(-1, w.top_k, x.shape[1]) * d(weights)[:, :, None]).sum(1)
    x2 = x1 + d(w.gate) * rms(moe) * d(w.norms[2])
    return x2, rms(x2) * d(w.norms[3])


def main():
    w = make_weights(D=1024, F=512, E=32, top_k=4)
    for tokens in (1, 7, 64, 1000):
        g = torch.Generator(device="cuda").manual_seed(tokens)
        attn = torch.randn(tokens, 1024, generator=g, device="cuda").bfloat16()
        x = 2 * torch.randn(tokens, 1024, generator=g, device="cuda")
        which = torch.randint(-1, 3, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        adapters = make_adapters(which, D=1024)
        r, codes, scales = forward(w, attn, x, adapters)
        want_r, want_y = reference(w, attn, x, adapters)
        err = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            forward(w, attn, x, adapters)
        end.record()
        torch.cuda.synchronize()
        print(f"{tokens:5d} tokens: {start.elapsed_time(end) * 50:8.1f} us, error of the residual stream "
              f"{err(r, want_r):.2e}, of the next input {err(codes.double() * scales[:, None], want_y):.2e}")


if __name__ == "__main__":
    main()
