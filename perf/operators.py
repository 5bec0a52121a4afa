"""Timed cases of the 8-bit block operators: the ragged grouped FP8 matmul, the
INT8 matmul with per-token and per-channel scales, and the sandwich norm.

``own = False`` computes each operator in elementary torch operations in fp32;
``own = True`` calls this package's kernels.  ``exact`` evaluates the
definitions in fp64, on its own code path.

    ragged   C[i,n] = cast(sum_g a_s[i,g] b_s[e,n/128,g] sum_{k in g} A[i,k] B[e,n,k]),
             e = the expert with offsets[e] <= i < offsets[e+1]
    int8     C[m,n] = cast(a_s[m] b_s[n] sum_k A[m,k] B[n,k]), the sum over whole numbers;
             from activations: a_s[m] = max_k |X[m,k]| / 127, A = round(X / a_s)
    norm     r = res_scale x + gate * (w_post h / rms(h)),  y = w_pre r / rms(r);
             y in the input's type, or as E4M3 codes with one scale per 128 columns
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # One token of a mixture-of-experts layer: 8 of 256 experts, one row each.
        dict(name="ragged_token", op="ragged", rows=8, experts=256, N=1536, K=4096, out="bf16", skew=0.0),
        # A decode batch of 64 tokens x 8: nearly every expert is read, for a row or a few.
        dict(name="ragged_decode", op="ragged", rows=512, experts=256, N=1536, K=4096, out="bf16", skew=0.5),
        # A small layer in a short prompt: odd row counts, crowded and empty experts, K of 8.5 scale groups.
        dict(name="ragged_odd", op="ragged", rows=1013, experts=16, N=520, K=1088, out="fp16", skew=1.5),
        # Prefill of 2048 tokens x 8 over 64 experts.
        dict(name="ragged_prefill", op="ragged", rows=16384, experts=64, N=4096, K=4096, out="bf16", skew=0.5),
        # One decoded token through a projection, codes and scales in hand.
        dict(name="int8_token", op="int8", M=1, N=4096, K=4096, out="bf16", src="codes"),
        # A decode batch through a wide projection, from its bf16 activations.
        dict(name="int8_decode", op="int8", M=32, N=8192, K=1024, out="bf16", src="bf16"),
        # A chunk of a prompt, odd in every size.
        dict(name="int8_odd", op="int8", M=257, N=1537, K=1000, out="fp16", src="codes"),
        # Prefill, from bf16 activations.
        dict(name="int8_prefill", op="int8", M=16384, N=4096, K=4096, out="bf16", src="bf16"),
        # One decoded token between two blocks.
        dict(name="norm_token", op="norm", M=1, D=4096, dtype="bf16", resid="bf16", gate_rows=1, out="same"),
        # A decode batch into an FP8 block, residual stream kept in fp32.
        dict(name="norm_decode_fp8", op="norm", M=64, D=4096, dtype="bf16", resid="fp32", gate_rows=0, out="fp8"),
        # Packed sequences of 100 tokens with a gate each, odd width.
        dict(name="norm_odd", op="norm", M=1111, D=1537, dtype="fp16", resid="fp16", gate_rows=100, out="same"),
        # Prefill into an FP8 block: both norms, one gate vector, codes and scales out.
        dict(name="norm_prefill_fp8", op="norm", M=16384, D=4096, dtype="bf16", resid="bf16", gate_rows=16384,
             out="fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ragged", "int8", "norm"])
    if op == "ragged":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 16384), experts=_log(rng, 4, 256), N=8 * _log(rng, 16, 512),
                     K=16 * _log(rng, 16, 256), out=rng.choice(["bf16", "fp16", "fp32"]),
                     skew=round(rng.uniform(0, 1.5), 2))
            if c["experts"] * c["N"] * c["K"] <= 1.6e9:
                return c
    if op == "int8":
        while True:
            c = dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 64, 8192), K=_log(rng, 64, 4096),
                     out=rng.choice(["bf16", "fp16", "fp32"]), src=rng.choice(["codes", "bf16", "fp16"]))
            if rng.random() < 0.75:     # most layers are wide in whole 16-byte rows
                c["N"], c["K"] = -(-c["N"] // 16) * 16, -(-c["K"] // 16) * 16
            if c["M"] * c["N"] * c["K"] <= 16384 * 4096 * 4096:
                return c
    while True:
        c = dict(op=op, M=_log(rng, 1, 16384), D=_log(rng, 64, 16384), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 resid="same", gate_rows=0, out=rng.choice(["same", "fp8"]))
        if c["out"] == "fp8" or rng.random() < 0.5:
            c["D"] = -(-c["D"] // 16) * 16
        c["resid"] = rng.choice([c["dtype"], "fp32"])
        c["gate_rows"] = rng.choice([0, 1, c["M"], _log(rng, 1, c["M"])])
        if c["M"] * c["D"] <= 16384 * 4096:
            return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _counts(case, seed):
    """Rows of each expert: a routing with popularities (e+1)^-skew in random order."""
    g = torch.Generator().manual_seed(seed)
    E = case["experts"]
    p = torch.arange(1, E + 1, dtype=torch.float64).pow(-case["skew"])[torch.randperm(E, generator=g)]
    if case["rows"] <= E and case["skew"] == 0:     # one token's choices are distinct
        ids = torch.randperm(E, generator=g)[:case["rows"]]
    else:
        ids = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(ids, minlength=E)


def _codes(shape, sigma, g):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * sigma).clamp_(-448, 448).to(
        torch.float8_e4m3fn)


def prepare(case, seed):
    g = _gen(seed)
    rnd = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    out = DTYPES.get(case["out"])
    s = dict(case)
    if case["op"] == "ragged":
        M, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        G, NB = -(-K // 128), -(-N // 128)
        counts = _counts(case, seed)
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        offsets[1:] = counts.cumsum(0)
        s.update(A=_codes((M, K), 166.0, g), a_s=0.006 * (0.5 + rnd(M, G)),
                 B=torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda"),
                 b_s=0.0002 * (0.5 + rnd(E, NB, G)), offsets=offsets.cuda(),
                 C=torch.empty((M, N), dtype=out, device="cuda"),
                 active=counts.nonzero()[:, 0].cuda(), longest=int(counts.max()))
        s["B"].copy_(_codes((E, N, K), 112.0, g))
    elif case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        s.update(B=(torch.randn((N, K), generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8),
                 b_s=0.0006 * (0.5 + rnd(N)), C=torch.empty((M, N), dtype=out, device="cuda"))
        if case["src"] == "codes":
            s.update(A=(torch.randn((M, K), generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8),
                     a_s=0.03 * (0.5 + rnd(M)))
        else:   # a few channels of an activation stand out
            X = torch.randn((M, K), generator=g, device="cuda") * torch.where(rnd(K) < 0.01, 8.0, 1.0)
            s.update(X=X.to(DTYPES[case["src"]]), A=torch.empty((M, K), dtype=torch.int8, device="cuda"),
                     a_s=torch.empty(M, device="cuda"))
    else:
        M, D, dt, rt = case["M"], case["D"], DTYPES[case["dtype"]], DTYPES[case["resid"]]
        randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
        s.update(h=(0.7 * randn(M, D)).to(dt), x=(2.0 * randn(M, D) * torch.where(rnd(D) < 0.01, 20.0, 1.0)).to(rt),
                 w_post=(1 + 0.1 * randn(D)).to(dt), w_pre=(1 + 0.1 * randn(D)).to(dt), res_scale=0.8, gate=None,
                 r=torch.empty((M, D), dtype=rt, device="cuda"))
        if case["gate_rows"]:
            s["gate"] = (0.5 * randn(-(-M // case["gate_rows"]), D)).to(dt)
        if case["out"] == "fp8":
            s.update(y=torch.empty((M, D), dtype=torch.float8_e4m3fn, device="cuda"),
                     y_s=torch.empty((M, -(-D // 128)), device="cuda"))
        else:
            s.update(y=torch.empty((M, D), dtype=dt, device="cuda"), y_s=None)
    return s


def run(s):
    if own:
        import block_scaled_fp8_w8a8_gb300 as w8
        if s["op"] == "ragged":
            return w8.grouped_matmul_ragged(s["A"], s["a_s"], s["B"], s["b_s"], s["offsets"], s["out"], out=s["C"])
        if s["op"] == "int8":
            if s["src"] != "codes":
                w8.quantize_int8_per_token(s["X"], A=s["A"], a_s=s["a_s"])
            return w8.int8_matmul(s["A"], s["a_s"], s["B"], s["b_s"], s["out"], out=s["C"])
        return w8.sandwich_norm(s["h"], s["x"], s["w_post"], s["w_pre"], gate=s["gate"],
                                gate_rows=s["gate_rows"] or None, res_scale=s["res_scale"], eps=EPS, out=s["out"],
                                x_out=s["r"], y_out=s["y"], scales_out=s["y_s"])
    return {"ragged": _plain_ragged, "int8": _plain_int8, "norm": _plain_norm}[s["op"]](s)


def _spread(scales, block, size, dim):
    return scales.repeat_interleave(block, dim).narrow(dim, 0, size)


def _plain_ragged(s):
    """The experts that have rows, each with its rows padded to the longest's count, as one batched product."""
    M, N, K = s["rows"], s["N"], s["K"]
    a = s["A"].float() * _spread(s["a_s"], 128, K, 1)
    w = s["B"][s["active"]].float() * _spread(_spread(s["b_s"][s["active"]], 128, K, 2), 128, N, 1)
    row = s["offsets"][:-1].long()[s["active"]][:, None] + torch.arange(s["longest"], device="cuda")
    inside = row < s["offsets"][1:].long()[s["active"]][:, None]
    c = torch.bmm(a[row.clamp(max=M - 1)], w.transpose(1, 2))
    # each padding row goes to a spare row after the last
    out = torch.empty((M + 1, N), dtype=DTYPES[s["out"]], device="cuda")
    out[torch.where(inside, row, M)] = c.to(out.dtype)
    return out[:M]


def _plain_int8(s):
    A, a_s = s["A"], s["a_s"]
    if s["src"] != "codes":
        X = s["X"].float()
        amax = X.abs().amax(1)
        a_s = amax / torch.full_like(amax, 127.0)
        a_s = torch.where(a_s == 0, torch.ones_like(a_s), a_s)
        A = (X / a_s[:, None]).round().clamp(-127, 127)
    c = A.float() @ s["B"].float().t()
    return (c * a_s[:, None] * s["b_s"]).to(DTYPES[s["out"]])


def _plain_norm(s):
    h, x = s["h"].float(), s["x"].float()
    u = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float().repeat_interleave(s["gate_rows"], 0)[:s["M"]]
    r = s["res_scale"] * x + u
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    r = r.to(s["x"].dtype)
    if s["out"] != "fp8":
        return r, y.to(s["h"].dtype)
    D = s["D"]
    G = -(-D // 128)
    yg = torch.nn.functional.pad(y, (0, G * 128 - D)).view(-1, G, 128)
    amax = yg.abs().amax(2)
    scale = amax / torch.full_like(amax, 448.0)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (yg / scale[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return r, q.view(-1, G * 128)[:, :D], scale


def work(case):
    if case["op"] == "ragged":
        # What the routing reads of the weights depends on the seed: the expected number of experts with a row.
        M, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        G, NB, ob = -(-K // 128), -(-N // 128), DTYPES[case["out"]].itemsize
        if case["skew"] == 0 and M <= E:
            live = M
        else:
            p = [(e + 1) ** -case["skew"] for e in range(E)]
            live = sum(1 - (1 - x / sum(p)) ** M for x in p)
        return {"bytes": live * (N * K + 4 * NB * G) + M * (K + 4 * G + N * ob) + 4 * (E + 1),
                "flops": 2.0 * M * N * K}
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K + 4 * M if case["src"] == "codes" else 2 * M * K
        return {"bytes": a + N * K + 4 * N + M * N * DTYPES[case["out"]].itemsize, "flops": 2.0 * M * N * K}
    M, D = case["M"], case["D"]
    hb, xb = DTYPES[case["dtype"]].itemsize, DTYPES[case["resid"]].itemsize
    y = M * D + 4 * M * -(-D // 128) if case["out"] == "fp8" else M * D * hb
    gate = -(-M // case["gate_rows"]) * D * hb if case["gate_rows"] else 0
    return {"bytes": M * D * (hb + 2 * xb) + y + 2 * D * hb + gate, "flops": 12.0 * M * D}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "ragged":
        off = s["offsets"].tolist()
        C = torch.zeros((case["rows"], case["N"]), dtype=f64, device="cuda")
        kg = torch.arange(case["K"], device="cuda") // 128
        nb = torch.arange(case["N"], device="cuda") // 128
        for e in range(case["experts"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                a = s["A"][lo:hi].to(f64) * s["a_s"][lo:hi].to(f64)[:, kg]
                C[lo:hi] = a @ (s["B"][e].to(f64) * s["b_s"][e].to(f64)[nb][:, kg]).t()
        return C
    if case["op"] == "int8":
        if case["src"] == "codes":
            A, a_s = s["A"].to(f64), s["a_s"].to(f64)
        else:
            X = s["X"].to(f64)
            a_s = X.abs().max(1).values / 127
            a_s[a_s == 0] = 1
            A = torch.round(X / a_s[:, None])
        return torch.einsum("mk,nk->mn", A, s["B"].to(f64)) * torch.outer(a_s, s["b_s"].to(f64))
    h, x = s["h"].to(f64), s["x"].to(f64)
    u = s["w_post"].to(f64) * h / torch.sqrt((h * h).sum(1, keepdim=True) / case["D"] + EPS)
    if s["gate"] is not None:
        u *= s["gate"].to(f64)[torch.arange(case["M"], device="cuda") // case["gate_rows"]]
    r = x * s["res_scale"] + u
    y = s["w_pre"].to(f64) * r / torch.sqrt((r * r).sum(1, keepdim=True) / case["D"] + EPS)
    if case["out"] != "fp8":
        return r, y
    codes, scales = [], []
    for part in y.split(128, 1):
        sc = part.abs().max(1, keepdim=True).values / 448
        sc[sc == 0] = 1
        codes.append((part / sc).clamp(-448, 448).float().to(torch.float8_e4m3fn).to(f64))
        scales.append(sc)
    return r, torch.cat(codes, 1), torch.cat(scales, 1)
