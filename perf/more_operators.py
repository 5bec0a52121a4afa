"""Timed cases of what stands around the 8-bit products: the routing of tokens to
experts, the sum of the experts' rows, and low-rank adapters beside a projection.

``own = False`` computes each operator in elementary torch operations (scores that
are compared in fp64, the rest in fp32); ``own = True`` calls this package's kernels.
``exact`` evaluates the definitions in fp64, on its own code path.

    route     s = softmax(l) or sigmoid(l), c = s + bias; of the groups of neighbouring experts the
              top_groups with the largest sums of their group_top best c stay; ids = the top_k largest
              c of what stays, weights = their s, renormalised.  Then the pairs (token, choice) in the
              experts' order: order[p] the pair in place p, offsets [E + 1], rows[t, j] the pair's
              place.  A token that is not valid: ids and rows -1, weights 0, its pairs after all others
    combine   out[t] = add[t] + sum_j weights[t, j] * Y[rows[t, j]], rows of -1 left out
    adapters  out[t] = base[t] + scales[l] (x[t] A[l]^T) B[l]^T, l the adapter of row t; rows without
              one (id -1) are base's
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One decoded token: biased sigmoid scores, 4 of 8 groups.
        dict(name="route_token", op="route", T=1, E=256, k=8, scoring="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, dtype="fp32", masked=0.0),
        # A decode batch padded to the size of its captured graph, bf16 logits (with ties).
        dict(name="route_decode", op="route", T=64, E=256, k=8, scoring="softmax", bias=False, groups=1, top_groups=1,
             group_top=2, dtype="bf16", masked=0.1),
        # A chunk of a prompt, groups by their best expert, odd sizes.
        dict(name="route_odd", op="route", T=1013, E=160, k=6, scoring="softmax", bias=True, groups=8, top_groups=3,
             group_top=1, dtype="fp16", masked=0.02),
        # Prefill.
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, scoring="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, dtype="fp32", masked=0.0),
        # One decoded token: the sum of its 8 experts' rows.
        dict(name="combine_token", op="combine", T=1, k=8, D=4096, dtype="bf16", out="bf16", add=False, masked=0.0),
        # A chunk of a prompt beside a shared expert, odd width.
        dict(name="combine_odd", op="combine", T=1013, k=6, D=1537, dtype="fp16", out="fp16", add=True, masked=0.02),
        # Prefill beside a shared expert.
        dict(name="combine_prefill", op="combine", T=16384, k=8, D=4096, dtype="bf16", out="bf16", add=True, masked=0.0),
        # One decoded token with an adapter, the rows' grouping in hand.
        dict(name="adapters_token", op="adapters", T=1, L=8, K=4096, N=4096, r=16, dtype="bf16", out="bf16", none=0.0,
             skew=0.0, run=1, grouped=True),
        # A decode batch of 64 requests over 32 adapters, some without one; the step's first projection, which groups the rows.
        dict(name="adapters_decode", op="adapters", T=64, L=32, K=4096, N=4096, r=64, dtype="bf16", out="bf16", none=0.2,
             skew=0.8, run=1, grouped=False),
        # Short prompts, odd in every size.
        dict(name="adapters_odd", op="adapters", T=257, L=7, K=1000, N=1537, r=24, dtype="fp16", out="fp16", none=0.1,
             skew=0.5, run=19, grouped=False),
        # A chunk of several prompts into a wide projection, sums kept in fp32.
        dict(name="adapters_chunk", op="adapters", T=2048, L=16, K=1024, N=8192, r=32, dtype="bf16", out="fp32", none=0.1,
             skew=0.5, run=128, grouped=True),
        # Prefill of prompts of some 1000 tokens.
        dict(name="adapters_prefill", op="adapters", T=16384, L=16, K=4096, N=4096, r=64, dtype="bf16", out="bf16", none=0.1,
             skew=0.5, run=1000, grouped=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine", "adapters"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * _log(rng, max(2, 16 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        k = min(_log(rng, 1, 16), top_groups * (E // groups))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.6, groups=groups, top_groups=top_groups,
                    group_top=min(rng.choice([1, 2]), E // groups), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    masked=rng.choice([0.0, 0.0, round(rng.uniform(0, 0.5), 2)]))
    if op == "combine":
        while True:
            c = dict(op=op, T=_log(rng, 1, 16384), k=_log(rng, 1, 16), D=_log(rng, 64, 16384),
                     dtype=rng.choice(["bf16", "fp16", "fp32"]), out="", add=rng.random() < 0.5,
                     masked=rng.choice([0.0, round(rng.uniform(0, 0.5), 2)]))
            if rng.random() < 0.75:     # most layers are wide in whole 16-byte rows
                c["D"] = -(-c["D"] // 16) * 16
            c["out"] = rng.choice([c["dtype"], "fp32"])
            if c["T"] * c["k"] * c["D"] * DTYPES[c["dtype"]].itemsize <= 2 ** 30:
                return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 16384), L=_log(rng, 1, 64), K=_log(rng, 64, 8192), N=_log(rng, 64, 8192),
                 r=_log(rng, 4, 128), dtype=rng.choice(["bf16", "fp16"]), out="", none=rng.choice([0.0, 0.1, 0.5]),
                 skew=round(rng.uniform(0, 1.5), 2), run=_log(rng, 1, 2000), grouped=rng.random() < 0.5)
        if rng.random() < 0.75:         # most layers are wide in whole 16-byte rows
            c["K"], c["N"] = -(-c["K"] // 16) * 16, -(-c["N"] // 16) * 16
            c["r"] = -(-c["r"] // 8) * 8
        c["out"] = rng.choice([c["dtype"], c["dtype"], "fp32"])
        if c["T"] * (c["K"] + c["N"]) * c["r"] <= 16384 * 8192 * 64 and c["T"] * (c["K"] + c["N"]) <= 16384 * 8192:
            return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    rnd = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case)
    T, dt = case["T"], DTYPES[case["dtype"]]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        # what a router gives: some experts are liked by many tokens, and the bias pulls against that
        liked = 0.5 * randn(E)
        s.update(logits=(1.5 * randn(T, E) + liked).to(dt), valid=None, scale=2.5 if case["scoring"] == "sigmoid" else 1.0,
                 b=(0.05 * randn(E) - 0.1 * liked if case["scoring"] == "sigmoid" else 0.01 * rnd(E)) if case["bias"] else None,
                 outs=(ints(T, k), torch.empty((T, k), device="cuda"), ints(T * k), ints(E + 1), ints(T, k)))
        if case["masked"]:
            s["valid"] = rnd(T) >= case["masked"]
    elif case["op"] == "combine":
        k, D, ot = case["k"], case["D"], DTYPES[case["out"]]
        valid = rnd(T) >= case["masked"]
        # places of the pairs in the experts' order, those of invalid tokens after all others
        place = rnd(T, k).where(valid[:, None], 2.0).view(-1).argsort().argsort().view(T, k).int()
        weights = rnd(T, k) + 0.1
        s.update(Y=torch.empty((T * k, D), dtype=dt, device="cuda"), rows=place.where(valid[:, None], -1),
                 weights=(2.5 * weights / weights.sum(1, keepdim=True)).where(valid[:, None], 0.0),
                 plus=randn(T, D).to(ot) if case["add"] else None, C=torch.empty((T, D), dtype=ot, device="cuda"))
        for part in s["Y"].split(1 << 14):
            part.copy_(randn(*part.shape))
    else:
        L, K, N, r, ot = case["L"], case["K"], case["N"], case["r"], DTYPES[case["out"]]
        # runs of rows of one request, adapters of popularity (l + 1)^-skew
        runs = -(-T // case["run"])
        p = torch.arange(1, L + 1, dtype=torch.float64, device="cuda").pow(-case["skew"])
        ids = torch.multinomial(p, runs, replacement=True, generator=g)
        ids = ids.where(rnd(runs) >= case["none"], -1).repeat_interleave(case["run"])[:T].int()
        group = ids.where(ids >= 0, L)
        offsets = ints(L + 1)
        offsets[0] = 0
        offsets[1:] = torch.bincount(group, minlength=L + 1)[:L].cumsum(0)
        live = torch.unique(ids[ids >= 0]).long()
        s.update(x=randn(T, K).to(dt), A=(randn(L, r, K) / K ** 0.5).to(dt), B=(randn(L, N, r) / r ** 0.5).to(dt),
                 scales=0.5 + rnd(L), base=randn(T, N).to(ot), C=torch.empty((T, N), dtype=ot, device="cuda"), ids=ids,
                 order=torch.argsort(group, stable=True).int(), offsets=offsets, live=live,
                 longest=int((offsets[1:] - offsets[:-1]).max()))
    return s


def run(s):
    if own:
        import block_scaled_fp8_w8a8_gb300 as w8
        if s["op"] == "route":
            return w8.route_experts(s["logits"], s["k"], s["scoring"], bias=s["b"], groups=s["groups"],
                                    top_groups=s["top_groups"], group_top=s["group_top"], scale=s["scale"],
                                    valid=s["valid"], out=s["outs"])
        if s["op"] == "combine":
            return w8.combine_experts(s["Y"], s["rows"], s["weights"], add=s["plus"], out=s["C"])
        order, offsets = s["order"], s["offsets"]
        if not s["grouped"]:
            order, offsets = w8.group_rows(s["ids"], s["L"])
        return w8.adapter_matmul(s["x"], s["A"], s["B"], order, offsets, s["base"], scales=s["scales"], out=s["C"])
    return {"route": _plain_route, "combine": _plain_combine, "adapters": _plain_adapters}[s["op"]](s)


def _plain_group(ids, groups):
    """Stable order of flat ids, -1 last: (order, offsets, place of each)."""
    order = torch.sort(torch.where(ids < 0, groups, ids), stable=True).indices
    offsets = (ids[None, :] == torch.arange(groups, device="cuda")[:, None]).sum(1).cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    return order.int(), torch.nn.functional.pad(offsets, (1, 0)).int(), place.int()


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    logits = s["logits"].double()       # experts are compared: fp32 scores could swap two of them
    if s["scoring"] == "softmax":
        e = (logits - logits.amax(1, keepdim=True)).exp()
        scores = e / e.sum(1, keepdim=True)
    else:
        scores = 1 / (1 + (-logits).exp())
    choice = scores if s["b"] is None else scores + s["b"].double()
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        rank = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, rank, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    weights = scores.gather(1, ids)
    weights = weights / weights.sum(1, keepdim=True) * s["scale"]
    if s["valid"] is not None:
        ids = torch.where(s["valid"][:, None], ids, -1)
        weights = torch.where(s["valid"][:, None], weights, 0.0)
    order, offsets, place = _plain_group(ids.reshape(-1), E)
    return ids.int(), weights.float(), order, offsets, torch.where(ids < 0, -1, place.view(T, k))


def _plain_combine(s):
    rows = s["rows"].long()
    w = torch.where(rows >= 0, s["weights"], 0.0)
    out = (s["Y"][rows.clamp(min=0)].float() * w[:, :, None]).sum(1)
    if s["plus"] is not None:
        out = out + s["plus"].float()
    return out.to(s["C"].dtype)


def _plain_adapters(s):
    """The adapters that have rows, each with its rows padded to the longest's count, as batched products."""
    T, live = s["T"], s["live"]
    order, offsets = s["order"], s["offsets"]
    if not s["grouped"]:
        order, offsets, _ = _plain_group(s["ids"], s["L"])
    out = torch.empty((T + 1, s["N"]), dtype=s["C"].dtype, device="cuda")   # a spare row for the padding
    out[:T] = s["base"]
    place = offsets[:-1].long()[live][:, None] + torch.arange(s["longest"], device="cuda")
    inside = place < offsets[1:].long()[live][:, None]
    row = order.long()[place.clamp(max=T - 1)]
    h = torch.bmm(s["x"][row].float(), s["A"][live].float().transpose(1, 2))
    d = torch.bmm(h * s["scales"][live][:, None, None], s["B"][live].float().transpose(1, 2))
    out[torch.where(inside, row, T)] = (d + s["base"][row].float()).to(out.dtype)
    return out[:T]


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * DTYPES[case["dtype"]].itemsize + 16 * T * k + 4 * (E + 1) + 4 * E * case["bias"],
                "flops": 8.0 * T * E}
    if case["op"] == "combine":
        k, D, ob = case["k"], case["D"], DTYPES[case["out"]].itemsize
        some = T * (1 - case["masked"])
        return {"bytes": some * k * D * DTYPES[case["dtype"]].itemsize + T * D * ob * (1 + case["add"]) + 8 * T * k,
                "flops": 2.0 * some * k * D}
    # Which adapters have rows depends on the seed: the expected number.
    L, K, N, r, ob = case["L"], case["K"], case["N"], case["r"], DTYPES[case["out"]].itemsize
    p = [(i + 1) ** -case["skew"] for i in range(L)]
    runs = -(-T // case["run"])
    live = sum(1 - (1 - (1 - case["none"]) * x / sum(p)) ** runs for x in p)
    some = T * (1 - case["none"])
    return {"bytes": live * r * (K + N) * 2 + some * K * 2 + 2 * T * N * ob + 4 * T + 4 * (L + 1) + 4 * live,
            "flops": 2.0 * some * r * (K + N)}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "route":
        import numpy as np
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        x = s["logits"].to(f64).cpu().numpy()
        if case["scoring"] == "softmax":
            p = np.exp(x - np.max(x, axis=1)[:, None])
            p /= p.sum(axis=1)[:, None]
        else:
            p = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        c = p + (s["b"].to(f64).cpu().numpy() if case["bias"] else 0)
        if G > 1:
            value = np.partition(c.reshape(T, G, E // G), E // G - case["group_top"], axis=2)
            value = value[:, :, E // G - case["group_top"]:].sum(axis=2)
            out = np.argsort(-value, axis=1, kind="stable")[:, case["top_groups"]:]
            closed = np.zeros((T, G), dtype=bool)
            np.put_along_axis(closed, out, True, axis=1)
            c = np.where(np.repeat(closed, E // G, axis=1), -np.inf, c)
        ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(p, ids, axis=1)
        w = s["scale"] * w / w.sum(axis=1)[:, None]
        if s["valid"] is not None:
            gone = ~s["valid"].cpu().numpy()
            ids[gone], w[gone] = E, 0
        flat = ids.reshape(-1)
        order = np.argsort(flat, kind="stable")
        rows = np.empty(flat.size, dtype=np.int64)
        rows[order] = np.arange(flat.size)
        rows[flat == E] = -1
        offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E)[:E])])
        whole = lambda a, *shape: torch.from_numpy(a.reshape(shape)).int().cuda()  # noqa: E731
        return (whole(np.where(ids == E, -1, ids), T, k), torch.from_numpy(w).cuda(), whole(order, T * k),
                whole(offsets, E + 1), whole(rows, T, k))
    if case["op"] == "combine":
        out = torch.zeros(s["C"].shape, dtype=f64, device="cuda")
        if s["plus"] is not None:
            out += s["plus"]
        for j in range(case["k"]):
            there = (s["rows"][:, j] >= 0).nonzero()[:, 0]
            out[there] += s["Y"][s["rows"][there, j].long()].to(f64) * s["weights"][there, j].to(f64)[:, None]
        return out
    out = s["base"].to(f64)
    for l in range(case["L"]):  # noqa: E741
        t = (s["ids"] == l).nonzero()[:, 0]
        if t.numel():
            out[t] += s["scales"][l].to(f64) * (s["x"][t].to(f64) @ s["A"][l].to(f64).t() @ s["B"][l].to(f64).t())
    return out
