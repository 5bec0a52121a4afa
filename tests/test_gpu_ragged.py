"""GPU: the ragged grouped matmul against a plain fp64 implementation.

Bound per element, from the arithmetic: every product of two E4M3 values is
exact, an element's sum has at most K fp32 additions inside its groups and one
fp32 FMA per group (after one rounding of the scale product), so the fp32 result
is within (K + 2 G + 2) 2^-24 of the sum of the terms' magnitudes; the cast adds
half an ulp (2^-8 relative for bf16, 2^-11 for fp16, plus 2^-25 below fp16's
normal range)."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8

pytestmark = pytest.mark.gpu

OUT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_ULP = {n: torch.finfo(t).eps / 2 for n, t in OUT.items()}


def make(counts, N, K, seed, start=0, tail=0):
    """Inputs with counts[e] rows per expert, `start` and `tail` rows of no expert."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, G = len(counts), -(-K // 128)
    M = start + sum(counts) + tail
    codes = lambda *s: (torch.randn(s, generator=g, device="cuda") * 120).clamp_(-448, 448).to(  # noqa: E731
        torch.float8_e4m3fn).view(torch.uint8)
    rnd = lambda *s: 0.01 * (0.25 + torch.rand(s, generator=g, device="cuda"))  # noqa: E731
    offsets = torch.tensor(np.cumsum([start] + list(counts)), dtype=torch.int32, device="cuda")
    return codes(M, K), rnd(M, G), codes(E, N, K), rnd(E, -(-N // 128), G), offsets


def reference(A, a_s, B, b_s, offsets):
    """(C, sum of the terms' magnitudes) in fp64; rows of no expert are NaN."""
    off = offsets.tolist()
    K, N = A.shape[1], B.shape[1]
    kg, nb = torch.arange(K, device="cuda") // 128, torch.arange(N, device="cuda") // 128
    a = A.view(torch.float8_e4m3fn).double() * a_s.double()[:, kg]
    C = torch.full((A.shape[0], N), float("nan"), dtype=torch.float64, device="cuda")
    S = C.clone()
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        w = B[e].view(torch.float8_e4m3fn).double() * b_s[e].double()[nb][:, kg]
        C[lo:hi] = a[lo:hi] @ w.t()
        S[lo:hi] = a[lo:hi].abs() @ w.abs().t()
    return C, S


def assert_right(got, x, out, what=""):
    C, S = reference(*x)
    K = x[0].shape[1]
    rows = ~torch.isnan(C[:, 0]) if C.shape[1] else torch.zeros(0, dtype=torch.bool)
    bound = HALF_ULP[out] * C.abs() + (2.0 ** -25 if out == "fp16" else 0.0) + \
        (K + 2 * (-(-K // 128)) + 2) * 2.0 ** -24 * S * (1 + HALF_ULP[out])
    err = (got.double() - C).abs()
    bad = ~(err <= bound) & rows[:, None]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements outside the bound"


CASES = [
    # counts, N, K, options
    ([1], 128, 16, {}),
    ([0, 0, 5, 0], 256, 256, {}),
    ([31, 32, 33, 0, 127, 128, 129, 1], 264, 528, {}),
    ([300, 0, 7, 256, 63], 520, 1088, {}),
    ([300, 0, 7, 256, 63], 520, 1088, dict(block_n_tile=256)),
    ([40] * 37, 136, 384, dict(block_n_tile=128)),
    ([2, 1, 0, 3] * 64, 512, 1024, {}),
    ([1000, 0, 1, 2000], 1536, 640, dict(block_n_tile=256)),
    ([64, 65], 1024, 4096, dict(grid_limit=3)),
    ([5] * 1024, 128, 128, {}),
    ([5, 0, 3], 256, 1024, dict(split_k=8)),
    ([130, 2], 128, 640, dict(split_k=4)),
    ([33] * 3, 264, 4096, dict(split_k=2)),
    ([1, 0, 0, 0, 1], 360, 3552, {}),
    ([7], 1000, 272, {}),
]


@pytest.mark.parametrize("counts,N,K,opts", CASES)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_parity(counts, N, K, opts, out):
    x = make(counts, N, K, seed=N + K)
    C = w8.grouped_matmul_ragged(*x, out, **opts)
    torch.cuda.synchronize()
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
    assert_right(C, x, out, f"{len(counts)} experts N={N} K={K} {opts} {out}")


FEW = [
    # counts, N, K: 32-row tiles, whole and split over K
    ([1], 8, 16),
    ([0, 31, 32, 33, 0, 64, 65, 1], 264, 528),
    ([2, 1, 0, 3] * 64, 520, 1040),
    ([200, 0, 9, 100], 136, 1088),
    ([1] * 700, 384, 256),
    ([5, 0, 3], 1000, 4096),
]


@pytest.mark.parametrize("counts,N,K", FEW)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_tiles_of_32_rows(counts, N, K, out):
    x = make(counts, N, K, seed=N + K + 1, start=3, tail=5)
    M = x[0].shape[0]
    for opts in (dict(), dict(split_k=1), dict(grid_limit=5)):
        C = torch.full((M, N), 7.0, dtype=OUT[out], device="cuda")
        w8.grouped_matmul_ragged(*x, out, out=C, m_tile=32, **opts)
        torch.cuda.synchronize()
        assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
        assert_right(C, x, out, f"{opts}")
        assert (C[:3] == 7).all() and (C[M - 5:] == 7).all()


def test_a_wait_that_runs_out_in_tiles_of_32_rows():
    x = make([5, 6], 256, 1024, seed=11)
    for opts in (dict(split_k=1, debug_skip_load=3), dict(split_k=4, debug_skip_load=1)):
        w8.grouped_matmul_ragged(*x, m_tile=32, wait_limit_cycles=2_000_000, **opts)
        assert w8.w8a8_get_device_status()[0] == w8.W8A8_ERR_DEVICE_TIMEOUT
        C = w8.grouped_matmul_ragged(*x, m_tile=32)
        torch.cuda.synchronize()
        assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
        assert_right(C, x, "bf16")


def test_equals_the_plain_matmul_per_expert():
    """Every expert's rows carry the bits of a plain call on them alone."""
    counts = [70, 0, 129, 3]
    x = make(counts, 256, 512, seed=2)
    C = w8.grouped_matmul_ragged(*x, "fp32", split_k=1)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            want = w8.matmul(x[0][lo:lo + n], x[1][lo:lo + n], x[2][e], x[3][e], "fp32",
                             variant=w8.W8A8_VARIANT_TILED)
            assert torch.equal(C[lo:lo + n], want), e
        lo += n


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_rows_of_no_expert_and_memory_around_c_stay_as_they_are(out):
    x = make([33, 0, 60], 264, 256, seed=5, start=7, tail=40)
    M, N = x[0].shape[0], 264
    big = torch.full((M * N + 4096,), 7.0, dtype=OUT[out], device="cuda")
    C = big[2048:2048 + M * N].view(M, N)
    w8.grouped_matmul_ragged(*x, out, out=C)
    torch.cuda.synchronize()
    assert (big[:2048] == 7).all() and (big[2048 + M * N:] == 7).all()
    assert (C[:7] == 7).all() and (C[100:] == 7).all()
    assert_right(C, x, out)


def test_nan_rows_stay_in_their_rows():
    """A row of NaN codes, and NaN weights of an expert, reach their own results only."""
    x = make([20, 30, 10], 256, 256, seed=6)
    x[0][25] = 0x7F
    x[2][2, 3] = 0x7F
    C = w8.grouped_matmul_ragged(*x, "fp32")
    assert torch.isnan(C[25]).all() and torch.isnan(C[50:, 3]).all()
    C[25] = 0
    C[50:, 3] = 0
    assert not torch.isnan(C).any()


@pytest.mark.parametrize("offsets", [[0, 200, 50, 300], [-5, 10, 20, 1 << 30], [400, 500, 600, 700],
                                     [10, 10, 10, 10], [250, 0, 0, 0]])
def test_offsets_out_of_order_or_range_stay_in_bounds(offsets):
    x = make([100, 100, 50], 128, 256, seed=7)
    M, N = 250, 128
    big = torch.full((M * N + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    w8.grouped_matmul_ragged(*x[:4], off, out=big[2048:2048 + M * N].view(M, N))
    torch.cuda.synchronize()
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
    assert (big[:2048] == 3).all() and (big[2048 + M * N:] == 3).all()


def test_routing_changes_under_graph_replay():
    x = make([40, 0, 24], 256, 512, seed=8)
    C = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w8.grouped_matmul_ragged(*x, out=C, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w8.grouped_matmul_ragged(*x, out=C, stream=s)
    for off in ([0, 40, 40, 64], [0, 0, 0, 64], [0, 1, 63, 64]):
        x[4].copy_(torch.tensor(off, dtype=torch.int32))
        C.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert_right(C, x, "bf16", str(off))


def test_pdl_behind_the_quantiser_and_the_same_bits_every_time():
    x = make([5, 0, 90, 33], 512, 1024, seed=9)
    X = torch.randn(128, 1024, device="cuda", dtype=torch.bfloat16)
    want = None
    A, a_s = torch.empty_like(x[0]), torch.empty_like(x[1])
    for _ in range(20):
        A.zero_()
        w8.quantize_fp8_per_token_group(X, A=A, a_s=a_s)
        C = w8.grouped_matmul_ragged(A, a_s, *x[2:], "bf16")
        want = C if want is None else want
        assert torch.equal(C, want)
    assert_right(want, (A, a_s, *x[2:]), "bf16")


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    x = make([50, 60], 256, 1024, seed=10)
    w8.grouped_matmul_ragged(*x, debug_skip_load=3, split_k=1, wait_limit_cycles=2_000_000)
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_ERR_DEVICE_TIMEOUT
    w8.grouped_matmul_ragged(*x, debug_skip_load=1, wait_limit_cycles=2_000_000)
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_ERR_DEVICE_TIMEOUT
    C = w8.grouped_matmul_ragged(*x)
    torch.cuda.synchronize()
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK
    assert_right(C, x, "bf16")


def test_options_outside_the_kernels_are_refused():
    x = make([5, 6], 256, 1024, seed=12)
    many = make([1] * 200, 512, 1024, seed=13)
    for args, opts in ((x, dict(m_tile=64)), (x, dict(m_tile=32, block_n_tile=256)), (x, dict(block_n_tile=192)),
                       (x, dict(m_tile=128, split_k=2)), (x, dict(split_k=3)), (x, dict(split_k=16)),
                       (many, dict(split_k=8)), (x, dict(block_n_tile=256, split_k=2))):
        with pytest.raises(w8.W8A8Error) as e:
            w8.grouped_matmul_ragged(*args, **opts)
        assert e.value.status == w8.W8A8_ERR_UNSUPPORTED, (opts, e.value)
