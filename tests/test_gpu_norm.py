"""GPU: the sandwich norm against a plain fp64 implementation.

Bounds, from the arithmetic.  A thread sums at most 16 squares (56 where a row is
held in shared memory) before 10 levels of a tree, so a mean of squares is
within 70 2^-24 of its value; its reciprocal square root within half of that and
2 ulp; each product adds a rounding.  So u is within 48 2^-24 of its value, r
within 48 2^-24 of |res_scale x| + |gate u|, and y = w r / rms(r), whose own norm
repeats that, within 96 2^-24 of w (|res_scale x| + |gate u|) / rms(r).  The cast
adds half an ulp."""
import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
EPS = 1e-6


def make(M, D, dtype="bf16", resid=None, gate_rows=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + D)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dt, rt = DT[dtype], DT[resid or dtype]
    k = dict(h=rn(M, D).to(dt), x=(3 * rn(M, D)).to(rt), w_post=(1 + 0.2 * rn(D)).to(dt),
             w_pre=(1 + 0.2 * rn(D)).to(dt), res_scale=0.75)
    if gate_rows:
        k.update(gate=rn(-(-M // gate_rows), D).to(dt), gate_rows=gate_rows)
    return k


def reference(h, x, w_post=None, w_pre=None, gate=None, gate_rows=None, res_scale=1.0):
    """r, y and the bounds of their fp32 errors, in fp64."""
    h, x = h.double(), x.double()
    M = h.shape[0]
    u = h
    if w_post is not None:
        u = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * w_post.double()
    if gate is not None:
        u = u * gate.double().reshape(-1, h.shape[1])[torch.arange(M, device="cuda") // gate_rows]
    r = res_scale * x + u
    size = (res_scale * x).abs() + u.abs()
    y, ybound = r, 48 * 2.0 ** -24 * size
    if w_pre is not None:
        k = w_pre.double() / (r.square().mean(1, keepdim=True) + EPS).sqrt()
        y, ybound = r * k, 96 * 2.0 ** -24 * size * k.abs()
    return r, y, 48 * 2.0 ** -24 * size, ybound


def assert_near(got, want, bound, what):
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134
    err = (got.double() - want).abs()
    bad = ~(err <= HALF_ULP[got.dtype] * (want.abs() + bound) + bound + tiny)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound"


def check(k, r, y, what=""):
    want_r, want_y, rb, yb = reference(**k)
    assert_near(r, want_r, rb, what + " r")
    assert_near(y, want_y, yb, what + " y")


SHAPES = [(1, 1), (1, 8), (5, 7), (3, 64), (130, 75), (33, 512), (9, 513), (4, 520), (17, 1537), (64, 4096), (7, 5000),
          (2, 16384), (3, 16385), (2, 16392), (1, 57344)]


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("dtype,resid", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                         ("fp32", "fp32")])
def test_parity(M, D, dtype, resid):
    for gate_rows in (0, 1, 3, M):
        k = make(M, D, dtype, resid, gate_rows)
        r, y = w8.sandwich_norm(**k, eps=EPS)
        check(k, r, y, f"{M} {D} gate_rows={gate_rows}")


@pytest.mark.parametrize("D", [72, 777, 17000])
def test_parts_left_out(D):
    """Without either norm, without the gate, in every combination."""
    for drop in (["w_post"], ["w_pre"], ["w_post", "w_pre"], ["w_post", "gate"], ["w_post", "w_pre", "gate"]):
        k = make(6, D, "bf16", "fp32", gate_rows=2)
        for name in drop:
            k[name] = None
        if "gate" in drop:
            k.pop("gate_rows")
        r, y = w8.sandwich_norm(**k, eps=EPS)
        check(k, r, y, str(drop))


@pytest.mark.parametrize("M,D", [(1, 16), (3, 128), (5, 144), (33, 512), (7, 4096), (3, 8208), (2, 16400), (1, 57344)])
@pytest.mark.parametrize("dtype,resid", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_codes_are_the_quantisers(M, D, dtype, resid):
    """FP8 and INT8 codes and scales are, bit for bit, those of the stand-alone
    quantisers on the fp32 y (which an fp32 h gives through out='same')."""
    k = make(M, D, dtype, resid, gate_rows=2)
    k["h"][0] = 0
    k["x"][0] = 0
    full = dict(k, h=k["h"].float(), x=k["x"].float(), w_post=k["w_post"].float(), w_pre=k["w_pre"].float(),
                gate=k["gate"].float())
    _, y = w8.sandwich_norm(**full, eps=EPS)
    r, q, s = w8.sandwich_norm(**k, eps=EPS, out="fp8")
    want_q, want_s = w8.quantize_fp8_per_token_group(y)
    assert torch.equal(s, want_s) and torch.equal(q, want_q)
    r8, q8, s8 = w8.sandwich_norm(**k, eps=EPS, out="int8")
    want_q, want_s = w8.quantize_int8_per_token(y)
    assert torch.equal(s8, want_s) and torch.equal(q8, want_q)
    assert torch.equal(r, r8)
    assert_near(r, *[reference(**k)[i] for i in (0, 2)], "r")


def test_int8_codes_of_odd_rows():
    k = make(5, 1537, "bf16", "bf16")
    full = {n: (v.float() if torch.is_tensor(v) else v) for n, v in k.items()}
    _, y = w8.sandwich_norm(**full, eps=EPS)
    _, q, s = w8.sandwich_norm(**k, eps=EPS, out="int8")
    want_q, want_s = w8.quantize_int8_per_token(y)
    assert torch.equal(s, want_s) and torch.equal(q, want_q)


@pytest.mark.parametrize("D", [256, 250, 16640])
def test_in_place_gives_the_same_bits(D):
    k = make(9, D, "bf16", "bf16", gate_rows=9)
    r, y = w8.sandwich_norm(**k, eps=EPS)
    x, h = k["x"].clone(), k["h"].clone()
    w8.sandwich_norm(**dict(k, x=x, h=h), eps=EPS, x_out=x, y_out=h)
    assert torch.equal(x, r) and torch.equal(h, y)


@pytest.mark.parametrize("pad", [16, 3])
def test_strides_and_memory_around_the_outputs(pad):
    M, D = 6, 272
    k = make(M, D, "fp16", "fp32")
    wide = lambda t: torch.nn.functional.pad(t, (0, pad))[:, :D]  # noqa: E731
    r, y = w8.sandwich_norm(**k, eps=EPS)
    ro = torch.full((M + 1, D + pad), 7.0, device="cuda")
    yo = torch.full((M + 1, D + pad), 7.0, device="cuda", dtype=torch.float16)
    w8.sandwich_norm(**dict(k, h=wide(k["h"]), x=wide(k["x"])), eps=EPS, x_out=ro[:M, :D], y_out=yo[:M, :D])
    check(k, ro[:M, :D], yo[:M, :D])
    for t in (ro, yo):
        assert (t[M:] == 7).all() and (t[:, D:] == 7).all()


def test_zero_rows_and_non_finite_values():
    """A zero row stays zero; NaN and infinity stay in their rows."""
    k = make(4, 640, "bf16", "bf16")
    k["h"][0] = 0
    k["x"][0] = 0
    k["h"][1, 5] = float("nan")
    k["x"][2, 7] = float("inf")
    r, y = w8.sandwich_norm(**k, eps=EPS)
    assert (r[0] == 0).all() and (y[0] == 0).all()
    assert torch.isnan(r[1]).all() and torch.isnan(y[1]).all()
    assert r[2, 7] == float("inf") and torch.isnan(y[2, 7])
    sub = {n: (v[3:4] if n in "hx" else v) for n, v in k.items()}
    check(sub, r[3:4], y[3:4])


@pytest.mark.parametrize("M,D", [(6, 75), (6, 640), (5, 1537), (4, 17000), (4, 17001), (2500, 1024), (700, 4096),
                                 (2500, 1032), (400, 1537), (350, 12003)])
@pytest.mark.parametrize("dtype,resid", [("bf16", "fp32"), ("fp32", "fp32")])
def test_int8_scales_of_rows_that_are_not_finite(M, D, dtype, resid):
    """One NaN or infinity in a row of y (without norms it stays alone) shows in the
    row's scale; the rows around it are as they were."""
    for norms in ((), ("w_post", "w_pre")):
        k = make(M, D, dtype, resid)
        for n in ("w_post", "w_pre"):
            if n not in norms:
                k[n] = None
        _, q0, s0 = w8.sandwich_norm(**k, eps=EPS, out="int8")
        for at in (0, D - 1):
            h, x = k["h"].clone(), k["x"].clone()
            h[1, at], x[M - 1, at] = float("nan"), float("inf")
            _, q, s = w8.sandwich_norm(**dict(k, h=h, x=x), eps=EPS, out="int8")
            assert torch.isnan(s[1]) and (torch.isnan(s[M - 1]) if norms else s[M - 1] == float("inf"))
            assert (q[1] == 0).all() and (q[M - 1] == 0).all()
            rest = [i for i in range(M) if i not in (1, M - 1)]
            assert torch.equal(q[rest], q0[rest]) and torch.equal(s[rest], s0[rest])


def test_many_rows_on_a_side_stream_and_in_a_graph():
    k = make(3000, 264, "bf16", "fp32", gate_rows=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r, y = torch.empty_like(k["x"]), torch.empty_like(k["h"])
    w8.sandwich_norm(**k, eps=EPS, x_out=r, y_out=y, stream=s)
    s.synchronize()
    check(k, r, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w8.sandwich_norm(**k, eps=EPS, x_out=r, y_out=y, stream=s)
    k["h"].mul_(0.5)
    k["x"].add_(1.0)
    g.replay()
    torch.cuda.synchronize()
    check(k, r, y)


@pytest.mark.parametrize("M,D", [(2500, 1024), (1000, 2056), (701, 4096), (333, 8192), (5000, 1032), (8000, 640), (400, 1537), (305, 3943),
                                 (310, 6001), (304, 12003), (333, 4095), (4100, 517)])
@pytest.mark.parametrize("dtype,resid", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_many_long_rows(M, D, dtype, resid):
    """Enough rows for the persistent kernel; its codes are those of few rows at a time."""
    for gate_rows, drop in ((M, ()), (100, ()), (1, ("w_post",)), (0, ("w_post", "w_pre")), (0, ("w_pre",))):
        k = make(M, D, dtype, resid, gate_rows)
        for n in drop:
            k[n] = None
        r, y = w8.sandwich_norm(**k, eps=EPS)
        check(k, r, y, f"{gate_rows} {drop}")
    k = make(M, D, dtype, resid)
    for out in ("fp8", "int8") if D % 16 == 0 else ("int8",):
        r, q, s = w8.sandwich_norm(**k, eps=EPS, out=out)
        for lo in (0, M // 2, M - 8):
            few = dict(k, h=k["h"][lo:lo + 8], x=k["x"][lo:lo + 8])
            r1, q1, s1 = w8.sandwich_norm(**few, eps=EPS, out=out)
            assert_near(r[lo:lo + 8], r1.double(), reference(**few)[2] + r1.double().abs() * HALF_ULP[r1.dtype], out)
            scale = s1 if out == "fp8" else s1[:, None]
            got = s[lo:lo + 8] if out == "fp8" else s[lo:lo + 8, None]
            assert ((got - scale).abs() <= 2.0 ** -16 * scale).all()
            view = torch.float8_e4m3fn if out == "fp8" else torch.int8
            a, b = q[lo:lo + 8].view(view).float(), q1.view(view).float()
            # a code may differ by one step where y lies at the edge of two
            step = torch.maximum(b.abs() / 8, torch.full_like(b, 2.0 ** -9)) if out == "fp8" else 1.0
            assert ((a - b).abs() <= step).all() and (a != b).float().mean() < 1e-3
    x = k["x"].clone()
    w8.sandwich_norm(**dict(k, x=x), eps=EPS, x_out=x)
    assert torch.equal(x, w8.sandwich_norm(**k, eps=EPS)[0])


def test_empty():
    for M, D in ((0, 64), (3, 0)):
        r, y = w8.sandwich_norm(torch.empty(M, D, device="cuda"), torch.empty(M, D, device="cuda"))
        assert r.shape == (M, D) and y.shape == (M, D)


@pytest.mark.parametrize("out", ["same", "fp8", "int8"])
@pytest.mark.parametrize("gate", [None, (1, None), (4, 3), "flat"])
def test_given_outputs_hold_what_new_ones_would(out, gate):
    M, D = 10, 304
    g = torch.Generator(device="cuda").manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    k = dict(h=rn(M, D), x=rn(M, D).float(), w_post=rn(D), w_pre=rn(D), out=out, res_scale=0.5, eps=EPS)
    if gate == "flat":
        k["gate"] = rn(D)
    elif gate:
        k.update(gate=rn(gate[0], D), gate_rows=gate[1])
    want = w8.sandwich_norm(**k)
    given = [torch.empty_like(t) for t in want]
    got = w8.sandwich_norm(**k, x_out=given[0], y_out=given[1], scales_out=given[2] if len(given) > 2 else None)
    assert len(got) == len(want) and all(a is b for a, b in zip(got, given))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
