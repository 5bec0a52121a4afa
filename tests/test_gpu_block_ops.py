"""GPU: the ragged, INT8 and norm operators together -- the example that runs them as
a block, calls from several threads, and their kernels in the debug-bounds build."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8
from block_scaled_fp8_w8a8_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import moe_block  # noqa: E402


@pytest.mark.parametrize("tokens", [1, 5, 64, 333])
def test_the_block_against_fp64(tokens):
    """Quantising an activation to E4M3 moves it by at most 2^-4 of itself and to INT8
    by 2^-8 of its row's largest; the block's four 8-bit products average such
    errors over their columns, and the norms keep relative errors."""
    w = moe_block.make_weights(seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    attn = torch.randn(tokens, 512, generator=g, device="cuda").bfloat16()
    x = 2 * torch.randn(tokens, 512, generator=g, device="cuda")
    r, codes, scales = moe_block.forward(w, attn, x)
    want_r, want_y = moe_block.reference(w, attn, x)
    assert (r - want_r).norm() <= 2.0 ** -4 * want_r.norm()
    assert (codes.double() * scales[:, None] - want_y).norm() <= 2.0 ** -4 * want_y.norm()
    # the same tokens one by one give the same rows (routing and sums are per token)
    if tokens <= 5:
        for i in range(tokens):
            ri, ci, si = moe_block.forward(w, attn[i:i + 1], x[i:i + 1])
            assert (ri - r[i]).abs().max() <= 2.0 ** -6 * r[i].abs().max()


def test_threads_on_their_own_streams():
    """Four host threads, each with its own stream, data and library workspace."""
    errors = []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g = torch.Generator(device="cuda").manual_seed(seed)
                A = torch.randint(-128, 128, (400 + seed, 600), generator=g, device="cuda", dtype=torch.int8)
                B = torch.randint(-128, 128, (520, 600), generator=g, device="cuda", dtype=torch.int8)
                a, b = (torch.rand(n, generator=g, device="cuda") for n in (400 + seed, 520))
                want = ((A.double() @ B.double().t()).float() * a[:, None] * b)
                h = torch.randn(50 + seed, 777, generator=g, device="cuda")
                r0, y0 = w8.sandwich_norm(h, h)
                for v in (w8.W8A8_VARIANT_AUTO, w8.W8A8_VARIANT_SMALLM, w8.W8A8_VARIANT_TILED,
                          w8.W8A8_VARIANT_TILED_PAIR) * 5:
                    assert torch.equal(w8.int8_matmul(A, a, B, b, "fp32", variant=v), want)
                    r, y = w8.sandwich_norm(h, h)
                    assert torch.equal(r, r0) and torch.equal(y, y0)
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors[0]
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


@pytest.mark.parametrize("grown", [True, False])
def test_threads_on_one_stream(grown):
    """Four host threads whose calls share a stream and so the library's workspace, which
    each of the calls fills by one launch and reads by the next; with the workspace as
    large as the largest call needs it before the first, and growing between them."""
    M, N, K = (600, 300, 130, 900), (520, 300, 900, 264), (600, 1040, 300, 2000)
    stream, errors, start = torch.cuda.Stream(), [], threading.Barrier(4)
    x = []
    for i in range(4):
        g = torch.Generator(device="cuda").manual_seed(i)
        A, B = (torch.randint(-128, 128, (n, K[i]), generator=g, device="cuda", dtype=torch.int8) for n in (M[i], N[i]))
        a, b = (torch.rand(n, generator=g, device="cuda") for n in (M[i], N[i]))
        X = torch.randn(M[i], 512, generator=g, device="cuda")
        W = (torch.randn(512, 512, generator=g, device="cuda") * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)
        W_s = torch.rand(4, 4, generator=g, device="cuda")
        x.append((A, a, B, b, X, W, W_s, (A.double() @ B.double().t()).float() * a[:, None] * b,
                  w8.matmul(*w8.quantize_fp8_per_token_group(X), W, W_s, "fp32")))
    torch.cuda.synchronize()
    if grown:
        big = torch.ones(3000, 3000, device="cuda", dtype=torch.int8)
        w8.int8_matmul(big, torch.ones(3000, device="cuda"), big, torch.ones(3000, device="cuda"), stream=stream,
                       variant=w8.W8A8_VARIANT_TILED)

    def work(i):
        try:
            A, a, B, b, X, W, W_s, want, want8 = x[i]
            got = []
            start.wait()
            with torch.cuda.stream(stream):
                for r in range(30):
                    v = (w8.W8A8_VARIANT_TILED, w8.W8A8_VARIANT_TILED_PAIR)[r % 2]
                    got.append((w8.int8_matmul(A, a, B, b, "fp32", variant=v), want))
                    if r % 3 == 0:      # quantiser and product, the codes in the workspace
                        got.append((w8.quant_matmul(X, W, W_s, "fp32"), want8))
            stream.synchronize()
            for C, ref in got:
                assert torch.equal(C, ref)
        except Exception as e:      # noqa: BLE001
            errors.append((i, repr(e)))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in ts) and not errors, errors
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


def test_a_tensor_on_the_host_among_others_is_refused():
    """Each argument in turn, with the outputs given and without."""
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i8, u8 = torch.int8, torch.uint8
    for call, args, outs in (
        (w8.grouped_matmul_ragged, dict(A=z(4, 128, dtype=u8), a_s=z(4, 1), B=z(2, 8, 128, dtype=u8), b_s=z(2, 1, 1),
                                        offsets=z(3, dtype=torch.int32)), dict(out=z(4, 8, dtype=torch.bfloat16))),
        (w8.int8_matmul, dict(A=z(4, 16, dtype=i8), a_s=z(4), B=z(8, 16, dtype=i8), b_s=z(8)),
         dict(out=z(4, 8, dtype=torch.bfloat16))),
        (w8.quantize_int8_per_token, dict(X=z(4, 16)), dict(A=z(4, 16, dtype=i8), a_s=z(4))),
        (w8.sandwich_norm, dict(h=z(4, 16), x=z(4, 16), w_post=z(16), w_pre=z(16), gate=z(16), out="int8"),
         dict(x_out=z(4, 16), y_out=z(4, 16, dtype=i8), scales_out=z(4))),
    ):
        for good in (args, {**args, **outs}):
            call(**good)
            for name, t in good.items():
                if torch.is_tensor(t):
                    with pytest.raises(w8.W8A8Error, match="one CUDA device") as e:
                        call(**{**good, name: t.cpu()})
                    assert e.value.status == w8.W8A8_ERR_INVALID_ARG
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


def run_all(seed=1):
    """Every kernel of the three operators once or more, on sizes with ragged ends."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    out = {}
    A, B = ((rn(*s) * 90).clamp_(-448, 448).to(torch.float8_e4m3fn) for s in ((230, 400), (5, 264, 400)))
    off = torch.tensor([3, 40, 40, 173, 200, 229], dtype=torch.int32, device="cuda")
    for bn in (128, 256):
        C = torch.zeros(230, 264, device="cuda")
        out[f"ragged{bn}"] = w8.grouped_matmul_ragged(A, rn(230, 4).abs(), B, rn(5, 3, 4).abs(), off, "fp32", out=C,
                                                      block_n_tile=bn)
    for split in (1, 2):
        C = torch.zeros(230, 264, device="cuda")
        out[f"ragged_few{split}"] = w8.grouped_matmul_ragged(A, rn(230, 4).abs(), B, rn(5, 3, 4).abs(), off, "fp32",
                                                             out=C, m_tile=32, split_k=split)
    for name, M, N, K, v in (("small8", 3, 50, 200, 5), ("small32", 29, 130, 333, 5), ("mid", 100, 200, 520, 2),
                             ("tiled", 300, 200, 520, 1), ("pair", 300, 300, 515, 6)):
        out["int8_" + name] = w8.int8_matmul(i8(M, K), rn(M), i8(N, K), rn(N), "fp32", variant=v)
    for M, K in ((5, 77), (9, 4096), (2, 17000)):
        out[f"quant{K}"], out[f"quant_s{K}"] = w8.quantize_int8_per_token(rn(M, K))
    for M, D, kind in ((5, 77, "same"), (700, 4096, "fp8"), (350, 1537, "int8"), (3, 528, "fp8"), (2, 16400, "int8"),
                       (310, 5001, "same"), (2, 10000, "same")):
        got = w8.sandwich_norm(rn(M, D).bfloat16(), rn(M, D), rn(D).bfloat16(), rn(D).bfloat16(), out=kind,
                               gate=rn(-(-M // 3), D).bfloat16(), gate_rows=3)
        for j, t in enumerate(got):
            out[f"norm{M}_{D}_{j}"] = t
    torch.cuda.synchronize()
    return {k: v.cpu().view(torch.uint8) if v.element_size() == 1 else v.cpu() for k, v in out.items()}


CHILD = r"""
import sys, torch
import block_scaled_fp8_w8a8_gb300 as w8
sys.path.insert(0, sys.argv[2])
from test_gpu_block_ops import run_all
assert w8.w8a8_debug_bounds_build() == 1
res = {"out": run_all(), "status": w8.w8a8_get_device_status()}
x = torch.randint(-128, 128, (300, 520), device="cuda", dtype=torch.int8)
s = torch.ones(300, device="cuda")
A = torch.zeros(64, 256, dtype=torch.uint8, device="cuda")
B = torch.zeros(2, 128, 256, dtype=torch.uint8, device="cuda")
off = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
o = dict(debug_bad_index=1, wait_limit_cycles=2_000_000)
res["bad"] = []
for call in (lambda k: w8.int8_matmul(x, s, x, s, variant=1, **k), lambda k: w8.int8_matmul(x, s, x, s, variant=6, **k),
             lambda k: w8.grouped_matmul_ragged(A, torch.ones(64, 2, device="cuda"), B,
                                                torch.ones(2, 1, 2, device="cuda"), off, **k)):
    call(o)
    bad = w8.w8a8_get_device_status()
    call({})
    res["bad"].append((bad, w8.w8a8_get_device_status()))
torch.save(res, sys.argv[1])
"""


def test_debug_bounds_build(tmp_path):
    """The build that checks every index finds none outside its buffer and gives the
    release build's bits; an index moved outside is caught, and the next call is right."""
    build.build(debug_bounds=True)
    path = str(tmp_path / "res.pt")
    env = {k: v for k, v in os.environ.items() if not k.startswith("W8A8_")}
    env["W8A8_DEBUG_BOUNDS"] = "1"
    r = subprocess.run([sys.executable, "-c", CHILD, path, os.path.dirname(os.path.abspath(__file__))], env=env,
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = torch.load(path)
    assert res["status"][0] == w8.W8A8_OK, hex(res["status"][1])
    want = run_all()
    for k, v in want.items():
        assert torch.equal(res["out"][k], v), k
    for bad, after in res["bad"]:
        assert bad[0] == w8.W8A8_ERR_DEVICE_BOUNDS and (bad[1] >> 8) & 0xFF == 20, hex(bad[1])
        assert after[0] == w8.W8A8_OK
