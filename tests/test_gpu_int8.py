"""GPU: the INT8 matmul and its per-token quantiser.

The sum of the products is a whole number and exact, and what follows is three
fp32 roundings in a fixed order, so the matmul's results are compared bit for
bit: fp32(sum) * a_s * b_s, then the cast.  The quantiser's quotients are
correctly rounded fp32 ones: its codes and scales are compared bit for bit too."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8

pytestmark = pytest.mark.gpu

OUT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(M, N, K, seed, lo=-128, hi=127):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = lambda *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    rnd = lambda n: 1e-3 * (0.1 + torch.rand(n, generator=g, device="cuda"))  # noqa: E731
    return codes(M, K), rnd(M), codes(N, K), rnd(N)


def reference(A, a_s, B, b_s, out):
    """Sums in fp64 (whole numbers below 2^53: exact), then the fp32 steps."""
    s = (A.double() @ B.double().t()).float()
    return (s * a_s[:, None] * b_s).to(OUT[out])


def assert_same(got, want, what=""):
    bad = (got != want).sum().item()
    assert bad == 0, f"{what}: {bad} of {want.numel()} differ"


SIZES = [(1, 1, 1), (1, 128, 64), (3, 64, 16), (7, 130, 100), (16, 512, 256), (33, 1537, 1000), (64, 256, 4096),
         (100, 96, 513), (128, 128, 512), (129, 257, 1040), (257, 1000, 777), (300, 520, 2048), (1025, 768, 320),
         (2048, 1536, 1024)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_parity(M, N, K, out):
    x = make(M, N, K, seed=M + N + K)
    C = w8.int8_matmul(*x, out)
    torch.cuda.synchronize()
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
    assert_same(C, reference(*x, out), f"{M} {N} {K} {out}")


VARIANTS = [w8.W8A8_VARIANT_SMALLM, w8.W8A8_VARIANT_SWAPAB, w8.W8A8_VARIANT_TILED, w8.W8A8_VARIANT_TILED_PAIR]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 48, 8192), (9, 40, 5000), (20, 100, 2048), (130, 70, 64), (40, 70, 65), (300, 520, 1100), (513, 768, 2048),
                                   (5003, 100, 1040)])
def test_forced_kernels(M, N, K, variant):
    x = make(M, N, K, seed=3)
    for grid in (0, 4):
        C = w8.int8_matmul(*x, "fp32", variant=variant, grid_limit=grid)
        assert_same(C, reference(*x, "fp32"), f"{variant} {grid}")


@pytest.mark.parametrize("M", [1, 11, 30])
@pytest.mark.parametrize("N,K", [(4865, 64), (15001, 700), (33000, 1100), (10000, 4096)])
def test_more_weight_rows_than_ctas(M, N, K):
    """A CTA of the small-M kernel walks several tiles and starts the next
    one's loads while it finishes one."""
    x = make(M, N, K, seed=N + M)
    assert_same(w8.int8_matmul(*x, "fp32", variant=w8.W8A8_VARIANT_SMALLM), reference(*x, "fp32"))


@pytest.mark.parametrize("K", [512, 513, 4096, 20000, w8.W8A8_INT8_MAX_K])
@pytest.mark.parametrize("M", [2, 40, 130])
def test_largest_sums_are_exact(M, K):
    """Every product 2^14, the most any can be: the accumulators and their
    running total reach their limits; one operand off by one shows a lost unit."""
    A = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    B = torch.full((136, K), -128, dtype=torch.int8, device="cuda")
    A[1, K // 2], B[5, K - 1] = 127, -127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    s = (A.double() @ B.double().t())
    C = w8.int8_matmul(A, one(M), B, one(136), "fp32")
    assert_same(C, s.float())
    for variant in VARIANTS:
        try:
            C = w8.int8_matmul(A, one(M), B, one(136), "fp32", variant=variant)
        except w8.W8A8Error:
            assert variant == w8.W8A8_VARIANT_SWAPAB and K > 8 * 512
            continue
        assert_same(C, s.float())


@pytest.mark.parametrize("M,opts,most", [(2, {}, 65536), (40, {}, 65536), (130, {}, 65536), (256, {}, 65536),
                                         (300, dict(m_tile=256), 8192), (100, dict(m_tile=64, split_k=2), 8192),
                                         (40, dict(m_tile=48, split_k=1), 4096), (40, dict(m_tile=16, split_k=3), 24576)])
def test_longest_sums_of_the_some_hundred_token_form(M, opts, most):
    """K up to 512 * split_k * (512 / m_tile rounded up to 32), and no more."""
    for K in (most - 1, most):
        x = make(M, 136, K, seed=M)
        assert_same(w8.int8_matmul(*x, "fp32", variant=w8.W8A8_VARIANT_SWAPAB, **opts), reference(*x, "fp32"))
    x = make(M, 136, most + 1, seed=M)
    with pytest.raises(w8.W8A8Error) as e:
        w8.int8_matmul(*x, variant=w8.W8A8_VARIANT_SWAPAB, **opts)
    assert e.value.status == w8.W8A8_ERR_UNSUPPORTED
    assert_same(w8.int8_matmul(*x, "fp32"), reference(*x, "fp32"))


def test_every_unit_of_a_large_sum_counts():
    """Sums around 2^23 whose last units differ, read through scales of one."""
    K = 1024
    A = torch.full((64, K), 127, dtype=torch.int8, device="cuda")
    B = torch.full((128, K), 64, dtype=torch.int8, device="cuda")
    B[:, 0] = torch.arange(128, device="cuda", dtype=torch.int8)
    A[:, 0] = torch.arange(64, device="cuda", dtype=torch.int8) - 32
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    assert_same(w8.int8_matmul(A, one(64), B, one(128), "fp32"), (A.double() @ B.double().t()).float())


def test_strided_and_misaligned_operands_and_memory_around_c():
    for off, pad in ((0, 16), (4, 4), (1, 3), (0, 0)):
        M, N, K = (37, 83, 200) if off != 4 else (91, 83, 200)
        a = torch.randint(-128, 128, (off + (M + 1) * (K + pad),), device="cuda", dtype=torch.int8)
        b = torch.randint(-128, 128, (off + (N + 1) * (K + pad),), device="cuda", dtype=torch.int8)
        A = a[off:off + M * (K + pad)].view(M, K + pad)[:, :K]
        B = b[off:off + N * (K + pad)].view(N, K + pad)[:, :K]
        a_s, b_s = torch.rand(M + 1, device="cuda")[1:], torch.rand(N + 1, device="cuda")[1:]
        for out in ("bf16", "fp32"):
            buf = torch.full(((M + 2) * (N + pad) + 64,), 7.0, dtype=OUT[out], device="cuda")
            C = buf[off:off + M * (N + pad)].view(M, N + pad)[:, :N]
            w8.int8_matmul(A, a_s, B, b_s, out, out=C)
            assert_same(C, reference(A, a_s, B, b_s, out))
            C.fill_(7.0)
            assert (buf == 7).all()


def test_no_columns_gives_zeros_and_no_rows_nothing():
    z = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")  # noqa: E731
    C = w8.int8_matmul(z(3, 0), torch.ones(3, device="cuda"), z(5, 0), torch.ones(5, device="cuda"), "fp32",
                       out=torch.full((3, 5), 9.0, device="cuda"))
    assert (C == 0).all()
    assert w8.int8_matmul(z(0, 8), torch.ones(0, device="cuda"), z(5, 8), torch.ones(5, device="cuda")).shape == (0, 5)


@pytest.mark.parametrize("variant", [w8.W8A8_VARIANT_TILED, w8.W8A8_VARIANT_TILED_PAIR])
def test_more_rows_than_the_workspace_holds(variant):
    """A's rows go through the workspace in pieces (2048 rows of this K), the last one short."""
    M, N, K = 4123, 136, 131000
    A, a_s, B, b_s = make(M, N, K, seed=31)
    assert w8.w8a8_int8_workspace_size(M, N, K) == w8.w8a8_int8_workspace_size(2 * M, N, K)
    want = torch.cat([reference(A[i:i + 1000], a_s[i:i + 1000], B, b_s, "fp32") for i in range(0, M, 1000)])
    for pad in (0, 3):          # rows of C on 16-byte boundaries, and not
        wide = torch.full((M + 1, N + pad), 7.0, device="cuda")
        C = w8.int8_matmul(A, a_s, B, b_s, "fp32", out=wide[:M, :N], variant=variant)
        assert_same(C, want)
        assert (wide[M] == 7).all() and (wide[:, N:] == 7).all()


def test_callers_workspace_and_capture():
    x = make(200, 300, 700, seed=4)
    need = w8.w8a8_int8_workspace_size(200, 300, 700)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    C = torch.zeros(200, 300, dtype=torch.bfloat16, device="cuda")
    opts = dict(workspace_dev=ws.data_ptr(), workspace_bytes=need, variant=w8.W8A8_VARIANT_TILED)
    w8.int8_matmul(*x, out=C, stream=s, **opts)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w8.int8_matmul(*x, out=C, stream=s, **opts)
    x[0].copy_(make(200, 300, 700, seed=5)[0])
    g.replay()
    torch.cuda.synchronize()
    assert_same(C, reference(*x, "bf16"))
    with pytest.raises(w8.W8A8Error) as e:
        w8.int8_matmul(*x, **dict(opts, workspace_bytes=need - 256))
    assert e.value.status == w8.W8A8_ERR_WORKSPACE


def test_a_captured_call_keeps_its_workspace():
    """A graph that holds the library's workspace, replayed after a call on the same
    stream needed a larger one, and after a timeout made the library drop its
    workspaces.  (A split-K product of the FP8 matmul, whose counters lie there too,
    is captured with it.)"""
    s = torch.cuda.Stream()
    x, y = make(100, 300, 700, seed=21), make(1500, 1400, 2000, seed=22)
    A, a_s = w8.quantize_fp8_per_token_group(torch.randn(40, 2048, device="cuda"))
    B, b_s = torch.randn(512, 2048, device="cuda").to(torch.float8_e4m3fn), torch.rand(4, 16, device="cuda")
    C, D = torch.zeros(100, 300, device="cuda"), torch.zeros(40, 512, device="cuda")
    torch.cuda.synchronize()

    def step():
        w8.int8_matmul(*x, "fp32", out=C, stream=s, variant=w8.W8A8_VARIANT_TILED)
        w8.matmul(A, a_s, B, b_s, "fp32", out=D, stream=s, variant=w8.W8A8_VARIANT_SPLITK, split_k=4)

    step()
    s.synchronize()
    want = D.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()

    def replay_is_right(seed):
        x[0].copy_(make(100, 300, 700, seed=seed)[0])
        C.zero_(), D.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
        assert_same(C, reference(*x, "fp32"))
        assert torch.equal(D, want)

    def large():
        return w8.int8_matmul(*y, "fp32", stream=s, variant=w8.W8A8_VARIANT_TILED)

    E = large()
    replay_is_right(23)
    assert_same(E, reference(*y, "fp32"))
    w8.int8_matmul(*y, stream=s, variant=w8.W8A8_VARIANT_TILED, debug_skip_load=2, wait_limit_cycles=2_000_000)
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_ERR_DEVICE_TIMEOUT
    replay_is_right(24)
    E = large()
    s.synchronize()
    assert_same(E, reference(*y, "fp32"))
    replay_is_right(25)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    x = make(300, 520, 1100, seed=6)
    for variant in (w8.W8A8_VARIANT_SWAPAB, w8.W8A8_VARIANT_TILED, w8.W8A8_VARIANT_TILED_PAIR):
        w8.int8_matmul(*x, variant=variant, debug_skip_load=2, wait_limit_cycles=2_000_000)
        assert w8.w8a8_get_device_status()[0] == w8.W8A8_ERR_DEVICE_TIMEOUT
        assert_same(w8.int8_matmul(*x, variant=variant), reference(*x, "bf16"))
        assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


def quant_reference(X):
    x = X.float().cpu().numpy()
    s = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
    s[s == 0] = 1
    q = np.clip(np.rint(x / s[:, None]), -127, 127).astype(np.int8)
    return q, s


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 64), (33, 512), (9, 513), (17, 1000), (65, 4096), (2, 16384),
                                 (2, 16392), (3, 20001), (8000, 640), (1300, 4096), (1300, 4104), (700, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantiser(M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M * K)
    X = torch.randn((M, K), generator=g, device="cuda")
    X[:, K // 2] *= 40
    X[0] = 0 if M > 1 else X[0]
    X = X.to(OUT[dtype])
    q, s = w8.quantize_int8_per_token(X)
    want_q, want_s = quant_reference(X)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), want_q)


def test_quantiser_extremes_and_strides():
    """Rows of tiny, huge and tied values; rows of a wider buffer."""
    X = torch.zeros(6, 264, device="cuda")
    X[0] = 1e-44
    X[1, :3] = torch.tensor([3e38, -3e38, 1e38])
    X[2] = torch.arange(264, device="cuda") - 127.5                 # quotients in halves
    X[3, 5] = 1e-45
    X[4] = torch.arange(264, device="cuda") * 2.0 ** -130
    wide = torch.randn(6, 300, device="cuda")
    wide[:, 8:272] = X
    for src in (X, wide[:, 8:272], wide[:, 7:271]):
        out = torch.full((6, 280), 9, dtype=torch.int8, device="cuda")
        q, s = w8.quantize_int8_per_token(src, A=out[:, 3:267])
        want_q, want_s = quant_reference(src)
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert (out[:, :3] == 9).all() and (out[:, 267:] == 9).all()


@pytest.mark.parametrize("M,K", [(5, 1), (6, 64), (9, 513), (5, 4096), (4, 16384), (3, 20001), (3, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantiser_of_rows_that_are_not_finite(M, K, dtype):
    """NaN and infinity show in their row's scale, wherever they stand, and leave the
    other rows as they are; the row's products are NaN."""
    for at in {0, K // 2, K - 1}:
        X = torch.randn(M, K, device="cuda").to(OUT[dtype])
        want_q, want_s = quant_reference(X)
        X[0, at], X[1, at] = float("nan"), -float("inf")
        q, s = w8.quantize_int8_per_token(X)
        assert torch.isnan(s[0]) and s[1] == float("inf") and (q[:2] == 0).all()
        assert np.array_equal(s[2:].cpu().numpy(), want_s[2:]) and np.array_equal(q[2:].cpu().numpy(), want_q[2:])
        C = w8.int8_matmul(q, s, *make(1, 24, K, seed=K)[2:], "fp32")
        assert torch.isnan(C[:2]).all() and torch.isfinite(C[2:]).all()


def test_from_activations():
    """Quantise and multiply, back to back on a side stream."""
    X = torch.randn(77, 1000, device="cuda", dtype=torch.bfloat16)
    _, _, B, b_s = make(1, 400, 1000, seed=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    A, a_s = w8.quantize_int8_per_token(X, stream=s)
    C = w8.int8_matmul(A, a_s, B, b_s, "fp16", stream=s)
    s.synchronize()
    q, sc = quant_reference(X)
    assert_same(C, reference(torch.from_numpy(q).cuda(), torch.from_numpy(sc).cuda(), B, b_s, "fp16"))


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_given_outputs_hold_what_new_ones_would(out):
    X = torch.randn(9, 200, device="cuda", dtype=torch.float16)
    B, b_s = make(1, 70, 200, seed=12)[2:]
    A, a_s = w8.quantize_int8_per_token(X)
    A2, s2 = torch.empty_like(A), torch.empty_like(a_s)
    assert all(a is b for a, b in zip(w8.quantize_int8_per_token(X, A=A2, a_s=s2), (A2, s2)))
    assert torch.equal(A, A2) and torch.equal(a_s, s2)
    C = torch.empty(9, 70, dtype=OUT[out], device="cuda")
    assert w8.int8_matmul(A, a_s, B, b_s, out, out=C) is C
    assert_same(C, w8.int8_matmul(A, a_s, B, b_s, out))
