"""GPU: routing of tokens to experts, the sort of rows by group, the sum of the experts'
rows and the low-rank adapters, each against its definition in 64 bits."""
import math
import threading

import numpy as np
import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def smallest(dtype):
    """The smallest subnormal number."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ok():
    assert w8.w8a8_get_device_status()[0] == w8.W8A8_OK


# ---------------------------------------------------------------- the sort


def sorted_pairs(ids, groups):
    """(order, offsets, rows) of flat ids by numpy's stable sort; outside [0, groups): last."""
    ids = np.asarray(ids).reshape(-1)
    bins = np.where((ids < 0) | (ids >= groups), groups, ids).astype(np.int64)
    order = np.argsort(bins, kind="stable")
    rows = np.empty(ids.size, dtype=np.int64)
    rows[order] = np.arange(ids.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(bins, minlength=groups + 1)[:groups])])
    return order, offsets, np.where(bins == groups, -1, rows)


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 511, 513, 4097, 65536, 65537, 300001])
@pytest.mark.parametrize("groups", [1, 5, 256, 1024])
def test_group_rows(n, groups):
    g = gen(n + groups)
    for low, high in ((0, groups), (-2, groups + 2), (groups // 2, groups // 2 + 1)):
        ids = torch.randint(low, high, (n,), generator=g, device="cuda", dtype=torch.int32)
        order, offsets = w8.group_rows(ids, groups)
        want = sorted_pairs(ids.cpu().numpy(), groups)
        assert np.array_equal(order.cpu().numpy(), want[0])
        assert np.array_equal(offsets.cpu().numpy(), want[1])


def test_group_rows_far_ids_and_shapes():
    ids = torch.tensor([[5, -1, 2 ** 31 - 1], [-2 ** 31, 0, 5]], dtype=torch.int32, device="cuda")
    order, offsets = w8.group_rows(ids, 6)
    assert order.tolist() == [4, 0, 5, 1, 2, 3]
    assert offsets.tolist() == [0, 1, 1, 1, 1, 1, 3]
    out = (torch.full((6,), -7, dtype=torch.int32, device="cuda"), torch.full((7,), -7, dtype=torch.int32, device="cuda"))
    assert w8.group_rows(ids.view(-1), 6, out=out) is out
    assert out[0].tolist() == order.tolist() and out[1].tolist() == offsets.tolist()
    rows = torch.empty(6, dtype=torch.int32, device="cuda")
    assert w8.w8a8_group_rows(ids, 6, 6, out[0], out[1], rows) == w8.W8A8_OK
    assert rows.tolist() == [1, -1, -1, -1, 0, 2]


# ---------------------------------------------------------------- routing


def route_reference(logits, k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True,
                    scale=1.0, valid=None):
    """The definition, token by token."""
    x = logits.double().cpu().numpy()
    T, E = x.shape
    b = None if bias is None else bias.double().cpu().numpy()
    size = E // groups
    ids, weights = np.full((T, k), -1), np.zeros((T, k))
    with np.errstate(all="ignore"):
        for t in range(T):
            if valid is not None and not valid[t]:
                continue
            if scoring == "sigmoid":
                s = 1 / (1 + np.exp(-x[t]))
            else:
                top = np.nanmax(x[t]) if not np.isnan(x[t]).all() else 0.0
                e = np.exp(x[t] - (0.0 if top == -np.inf else top))
                s = e / e.sum() if e.sum() != 0 else e
            c = s if b is None else s + b
            rank = x[t] if b is None else c         # scores have the logits' order

            def first(v, n):
                """The n largest of v, NaN above all, ties to the lower index."""
                return np.lexsort((np.arange(v.size), -np.where(np.isnan(v), 0, v), ~np.isnan(v)))[:n]

            open_ = np.arange(E)
            if groups > 1:
                by = (rank if group_top == 1 else c).reshape(groups, size)
                value = np.array([row[first(row, group_top)].sum() for row in by])
                kept = np.sort(first(value, top_groups))
                open_ = (kept[:, None] * size + np.arange(size)).reshape(-1)
            ids[t] = open_[first(rank[open_], k)]
            w = s[ids[t]]
            if renormalize:
                if scoring == "softmax":        # from the logits, where scores underflow
                    l = x[t][ids[t]]
                    w = np.exp(l - l.max()) if l.max() > -np.inf else np.zeros(k)
                    w = w if not np.isnan(s).any() else w * np.nan
                else:                           # 1 / (1 + exp(-l)) over exp(r), which 64 bits hold
                    l = x[t][ids[t]]
                    r = min(0.0, l.max()) if l.max() > -np.inf else 0.0
                    w = np.exp(np.minimum(l, 0) - r) / (1 + np.exp(-np.abs(l)))
                w = w / w.sum() if w.sum() != 0 else w * 0
            weights[t] = scale * w
    return ids, weights


def weight_tolerance(logits, k, scoring, renormalize):
    """Relative: an exponential is off by 2 units of 2^-23 and by its argument's rounding, at
    most |x| 2^-24; the quotient has two such sums, of k terms, and three roundings.  Without
    renormalisation the sum over all experts is of faster exponentials: below 31 units (the
    kernel's bound)."""
    x = logits.double()
    far = float(torch.where(x.isfinite(), x, 0.0).abs().max()) if x.numel() else 0.0
    t = 2 * (2 * 2.0 ** -23 + 2 * far * 2.0 ** -24) + (k + 3) * 2.0 ** -24
    return t if renormalize or scoring == "sigmoid" else t + 31 * 2.0 ** -23


def check_route(logits, k, **kw):
    got = [t.cpu().numpy() for t in w8.route_experts(logits, k, **kw)]
    want_ids, want_w = route_reference(logits, k, **{a: v for a, v in kw.items() if a not in ("out", "stream")})
    ids, weights, order, offsets, rows = got
    assert np.array_equal(ids, want_ids), np.argwhere(ids != want_ids)[:4]
    tol = weight_tolerance(logits, k, kw.get("scoring", "softmax"), kw.get("renormalize", True))
    assert np.array_equal(np.isnan(weights), np.isnan(want_w))
    fine = ~np.isnan(want_w)
    # 2^-126: below it fp32 has fewer bits
    assert (np.abs(weights - want_w)[fine] <= tol * np.abs(want_w)[fine] + 2.0 ** -126).all()
    want = sorted_pairs(ids, logits.shape[1])
    assert np.array_equal(order, want[0]) and np.array_equal(offsets, want[1])
    assert np.array_equal(rows.reshape(-1), want[2])
    ok()
    return got


SHAPES = [  # T, E, k, groups, top_groups, group_top
    (0, 8, 2, 1, 1, 2), (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 7, 7, 1, 1, 1), (5, 33, 32, 1, 1, 1),
    (64, 256, 8, 1, 1, 1), (65, 64, 6, 8, 3, 1), (33, 160, 6, 8, 3, 2), (70, 152, 5, 8, 2, 2), (17, 96, 4, 3, 2, 1),
    (9, 1024, 32, 32, 7, 2), (40, 512, 3, 16, 5, 2), (513, 128, 8, 4, 2, 2), (1500, 72, 6, 1, 1, 1), (12, 60, 20, 5, 2, 2),
    (10, 31, 2, 31, 4, 1),
]


@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route(T, E, k, groups, top_groups, group_top, scoring, biased):
    for seed, (dtype, renormalize, masked) in enumerate((("fp32", True, False), ("bf16", False, True), ("fp16", True, True),
                                                         ("bf16", True, False))):
        g = gen(100 * T + E + seed)
        logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(DT[dtype])
        bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
        valid = torch.rand(T, generator=g, device="cuda") < 0.7 if masked else None
        check_route(logits, k, scoring=scoring, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                    renormalize=renormalize, scale=1.5, valid=valid)


@pytest.mark.parametrize("T,E,k,groups", [(131073, 1023, 32, 31), (140000, 1024, 32, 1), (1 << 20, 3, 1, 3), (300000, 33, 7, 1)])
def test_route_as_many_as_its_shared_memory_holds(T, E, k, groups):
    """Without a bias the scores' order is the logits', compared here as numbers (those of one
    value may stand in any order in torch.topk)."""
    g = gen(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, weights, order, offsets, rows = w8.route_experts(logits, k, "sigmoid", groups=groups, top_groups=groups, group_top=1)
    top = logits.topk(k, 1).values
    assert torch.equal(logits.gather(1, ids.long()), top)
    s = top.double().sigmoid()
    # 4 roundings of a score, k of the sum, one quotient
    assert ((weights - s / s.sum(1, keepdim=True)).abs() <= (k + 8) * 2.0 ** -24).all()
    pairs = torch.sort(ids.flatten(), stable=True)
    assert torch.equal(order, pairs.indices.int())
    assert torch.equal(offsets[1:].long(), torch.bincount(ids.flatten(), minlength=E).cumsum(0)) and offsets[0] == 0
    assert torch.equal(rows.flatten()[order.long()], torch.arange(T * k, device="cuda", dtype=torch.int32))
    ok()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", ["none", "zero", "levels"])
def test_route_ties_go_to_the_lower_index(scoring, bias):
    g = gen(3)
    for E, groups in ((64, 1), (96, 8), (256, 8)):
        logits = torch.randint(-2, 3, (90, E), generator=g, device="cuda").float()
        logits[:3] = 0.5
        b = {"none": None, "zero": torch.zeros(E, device="cuda"),
             "levels": 0.25 * torch.randint(0, 2, (E,), generator=g, device="cuda").float()}[bias]
        check_route(logits, 5, scoring=scoring, bias=b, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 1, 1, 8), (256, 8, 4, 8), (152, 8, 2, 6), (40, 1, 1, 32)])
def test_route_scores_nearer_than_their_rounding(scoring, E, groups, top_groups, k):
    """Biases that take the scores away but for their own rounding: the fp32 sums of score
    and bias do not tell the experts apart, scores in 64 bits do."""
    g = gen(E + groups)
    row = torch.randn(E, generator=g, device="cuda")
    s = torch.sigmoid(row.double()) if scoring == "sigmoid" else torch.softmax(row.double(), 0)
    logits = row[None, :].expand(20, E).contiguous()
    check_route(logits, k, scoring=scoring, bias=(0.5 - s).float(), groups=groups, top_groups=top_groups)


def test_route_masked_and_not_finite_logits():
    g = gen(5)
    inf = math.inf
    for scoring in ("softmax", "sigmoid"):
        for biased in (False, True):
            x = torch.randn(24, 64, generator=g, device="cuda")
            x[0] = -inf                             # nothing left
            x[1, 3:] = -inf                         # three left for five choices
            x[2] = torch.finfo(torch.float32).min   # the type's lowest value everywhere
            x[3, 10:] = torch.finfo(torch.float32).min
            x[4, ::2] = -inf
            x[5] = -100.0                           # sigmoid scores near fp32's smallest numbers
            x[5, 7], x[5, 20] = -98.5, -99.0
            x[6, 11] = math.nan
            x[7] = math.nan
            if scoring == "sigmoid":
                x[8, 5] = inf
            x[9] = 300.0
            bias = 0.05 * torch.randn(64, generator=g, device="cuda") if biased else None
            for groups, top_groups, group_top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
                rows = [i for i in range(24) if not (scoring == "sigmoid" and i == 5)]
                check_route(x[rows], 5, scoring=scoring, bias=bias, groups=groups, top_groups=top_groups,
                            group_top=group_top)
    # an infinity makes softmax weights NaN, and is chosen first without a bias
    x = torch.randn(2, 64, generator=g, device="cuda")
    x[0, 9] = inf
    ids, weights, *_ = w8.route_experts(x, 4)
    assert ids[0, 0] == 9 and weights[0].isnan().all() and weights[1].isfinite().all()
    # small scores keep their ratios when renormalised
    x = torch.full((1, 64), -200.0, device="cuda")
    x[0, 7], x[0, 20] = -99.0, -98.0
    ids, weights, *_ = w8.route_experts(x, 2, "sigmoid")
    assert ids.tolist() == [[20, 7]]
    e = math.exp(-1.0)
    assert (weights.cpu().double() - torch.tensor([[1 / (1 + e), e / (1 + e)]]).double()).abs().max() < 2.0 ** -20
    # a bias of -infinity ranks last, and is chosen where nothing else is open
    bias = torch.zeros(64, device="cuda")
    bias[8:] = -inf
    check_route(torch.randn(7, 64, generator=g, device="cuda"), 10, bias=bias, scoring="sigmoid")
    check_route(torch.randn(7, 64, generator=g, device="cuda"), 10, bias=bias, groups=8, top_groups=2)


def test_route_strided_logits_given_outputs_and_streams():
    g = gen(8)
    wide = torch.randn(70, 300, generator=g, device="cuda")
    view = wide[:, 7:263]
    got = check_route(view, 8, scoring="sigmoid")
    outs = tuple(torch.empty_like(torch.from_numpy(t)).cuda() for t in got)
    for logits in (view, view.contiguous()):
        assert w8.route_experts(logits, 8, "sigmoid", out=outs) is outs
        for a, b in zip(outs, got):
            assert np.array_equal(a.cpu().numpy(), b)
    valid = torch.rand(70, generator=g, device="cuda") < 0.5
    assert torch.equal(w8.route_experts(view, 8, valid=valid)[0], w8.route_experts(view, 8, valid=valid.byte())[0])
    side = torch.cuda.Stream()
    logits = torch.randn(3000, 256, generator=g, device="cuda")
    want = w8.route_experts(logits, 8)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = w8.route_experts(logits, 8)
    b = w8.route_experts(logits, 8, stream=side)
    c = w8.route_experts(logits, 8, stream=side.cuda_stream)
    side.synchronize()
    for t in (a, b, c):
        assert all(torch.equal(u, v) for u, v in zip(t, want))


def test_captured_routing_is_replayed_over_new_logits_and_two_graphs_at_once():
    """Each captured call has its own scratch: two graphs replayed on two streams at a time."""
    g = gen(11)
    x = [torch.randn(2000, 256, generator=g, device="cuda") for _ in range(2)]
    w8.route_experts(x[0], 8)
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w8.route_experts(x[i], 8, "sigmoid", groups=8, top_groups=4) +
                        w8.group_rows(torch.zeros(70000, dtype=torch.int32, device="cuda"), 3))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            x[i].copy_(torch.randn(2000, 256, generator=g, device="cuda"))
        want = [w8.route_experts(v, 8, "sigmoid", groups=8, top_groups=4) for v in x]
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
            assert outs[i][6].tolist() == [0, 70000, 70000, 70000]
    ok()


# ---------------------------------------------------------------- the experts' rows


def check_combine(Y, rows, weights, add=None, **kw):
    got = w8.combine_experts(Y, rows, weights, add=add, **kw)
    there = (rows >= 0) & (rows < Y.shape[0])
    y = Y.double()[rows.clamp(0, max(Y.shape[0] - 1, 0)).long()] if Y.shape[0] else torch.zeros(*rows.shape, Y.shape[1],
                                                                                               device="cuda").double()
    y = torch.where(there[:, :, None], y, 0.0)
    w = torch.where(there, weights.double(), 0.0)[:, :, None]
    plus = torch.zeros(got.shape, device="cuda").double() if add is None else add.double()
    want, size = plus + (w * y).sum(1), plus.abs() + (w * y).abs().sum(1)
    # k roundings of partial sums, then the output's
    bound = rows.shape[1] * 2.0 ** -24 * size + HALF_STEP[got.dtype] * (want.abs() + 2.0 ** -10 * size)
    assert got.shape == want.shape
    assert ((got.double() - want).abs() <= bound + smallest(got.dtype)).all()
    ok()
    return got


@pytest.mark.parametrize("T,k,D,M", [(1, 8, 4096, 8), (1, 1, 1, 1), (5, 3, 7, 11), (33, 6, 1537, 200), (17, 9, 64, 100),
                                     (3, 17, 2050, 40), (250, 2, 520, 500), (4, 0, 100, 5), (0, 4, 64, 4), (2, 4, 16400, 8)])
@pytest.mark.parametrize("dtype,out", [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "fp32"), ("fp16", "fp32")])
def test_combine(T, k, D, M, dtype, out):
    g = gen(T + k + D)
    Y = torch.randn(M, D, generator=g, device="cuda").to(DT[dtype])
    rows = torch.randint(-1, M + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand(T, k, generator=g, device="cuda")
    add = torch.randn(T, D, generator=g, device="cuda").to(DT[out or dtype])
    for a in (None, add):
        got = check_combine(Y, rows, weights, add=a, out_dtype=out)
        given = torch.empty_like(got)
        assert w8.combine_experts(Y, rows, weights, add=a, out=given) is given
        assert torch.equal(given, got)
    assert w8.combine_experts(Y, rows, weights, add=add, out=add) is add     # in place
    assert torch.equal(add, got)


def test_combine_leaves_out_what_has_no_row():
    """Neither a NaN in a row that nothing names nor a NaN weight without a row is seen."""
    Y = torch.full((6, 48), math.nan, device="cuda")
    Y[2], Y[4] = 1.0, 2.0
    rows = torch.tensor([[2, -1, 4], [-1, -1, -1], [6, 4, -2 ** 31]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[1.0, math.nan, 3.0], [math.nan] * 3, [math.inf, 0.5, math.nan]], device="cuda")
    assert w8.combine_experts(Y, rows, weights)[:, 0].tolist() == [7.0, 0.0, 1.0]
    assert w8.combine_experts(Y[:0], rows, weights)[:, 0].tolist() == [0.0, 0.0, 0.0]


def test_combine_strides_and_alignments():
    g = gen(2)
    for dtype in DT.values():
        for D, pad, shift in ((64, 16, 0), (64, 3, 1), (66, 2, 2), (71, 5, 3), (128, 8, 4)):
            wide = lambda n: torch.randn(n, shift + D + pad, generator=g, device="cuda").to(dtype)[:, shift:shift + D]  # noqa: E731
            Y, add, out = wide(40), wide(9), wide(9)
            rows = torch.randint(0, 40, (9, 4), generator=g, device="cuda", dtype=torch.int32)
            weights = torch.rand(9, 4, generator=g, device="cuda")
            before = out._base.clone()
            got = check_combine(Y, rows, weights, add=add, out=out)
            assert got is out
            assert torch.equal(out._base[:, :shift], before[:, :shift])
            assert torch.equal(out._base[:, shift + D:], before[:, shift + D:])


@pytest.mark.parametrize("T,k,D", [(6000, 1, 1936), (9001, 1, 486), (20000, 2, 40), (7000, 3, 1000), (12001, 4, 73),
                                   (20011, 1, 8), (5003, 2, 257), (9000, 0, 136), (9000, 2, 1)])
@pytest.mark.parametrize("dtype,out", [("bf16", None), ("fp16", "fp32"), ("fp32", None)])
def test_combine_many_tokens_of_few_rows(T, k, D, dtype, out):
    g = gen(T + D)
    Y = torch.randn(997, D, generator=g, device="cuda").to(DT[dtype])
    rows = torch.randint(-1, 997, (T, k), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand(T, k, generator=g, device="cuda")
    add = torch.randn(T, D, generator=g, device="cuda").to(DT[out or dtype])
    check_combine(Y, rows, weights, out_dtype=out)
    check_combine(Y, rows, weights, add=add, out_dtype=out)


@pytest.mark.parametrize("M", [1, 2, 5])
@pytest.mark.parametrize("D", [1, 2, 63, 255, 256, 257, 769])
@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("dtype", list(DT))
def test_combine_sees_only_its_own_columns(M, D, shift, dtype):
    """What lies before, between and after the rows is NaN."""
    g = gen(M + D + shift)
    flat = torch.full((shift + M * (D + 3) + 5,), math.nan, device="cuda").to(DT[dtype])
    Y = torch.as_strided(flat, (M, D), (D + 3, 1), shift)
    Y.copy_(torch.randn(M, D, generator=g, device="cuda"))
    rows = torch.randint(0, M, (70, 5), generator=g, device="cuda", dtype=torch.int32)
    assert torch.isfinite(check_combine(Y, rows, torch.rand(70, 5, generator=g, device="cuda"))).all()


def test_combine_rows_past_2_31_elements():
    D = 4096
    M = (1 << 31) // D + 40
    Y = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    Y[M - 1], Y[M - 2] = 1.0, 2.0
    rows = torch.tensor([[M - 1, M - 2]], dtype=torch.int32, device="cuda")
    got = w8.combine_experts(Y, rows, torch.tensor([[1.0, 10.0]], device="cuda"))
    assert (got == 21.0).all()


# ---------------------------------------------------------------- adapters


def adapter_case(T, L, K, N, r, dtype, out, seed=0, none=0.2, sizes=1.0):
    g = gen(seed + T + K + N + r)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, max(L, 1), (T,), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.where(torch.rand(T, generator=g, device="cuda") < none, -1, ids) if L else torch.full_like(ids, -1)
    return dict(x=(sizes * randn(T, K)).to(DT[dtype]), A=(randn(L, r, K) / max(K, 1) ** 0.5).to(DT[dtype]),
                B=(randn(L, N, r) / max(r, 1) ** 0.5).to(DT[dtype]), ids=ids, base=randn(T, N).to(DT[out or dtype]),
                scales=torch.rand(L, generator=g, device="cuda") + 0.5)


def adapter_reference(x, A, B, ids, base, scales):
    """(out, bound on the error) in 64 bits, adapter by adapter."""
    want, bound = base.double(), torch.zeros(base.shape, device="cuda").double()
    K, r = x.shape[1], A.shape[1]
    # x A^T: every MMA adds 16 products to the sum, its roundings within 4 units of 2^-23 of the
    # sum of sizes, and the partial sums of warps and CTAs are joined by some 16 more; likewise
    # h B^T.  h in parts: bf16 leaves 2^-18 (two) or 2^-27 (three), fp16 2^-24.
    first, second = (K / 16 + 16) * 2.0 ** -21, (3 * r / 16 + 4) * 2.0 ** -21
    parts = 2.0 ** -22 if x.dtype is torch.float16 or base.dtype is torch.float32 else 2.0 ** -17
    for i in range(A.shape[0]):
        t = (ids == i).nonzero()[:, 0]
        if t.numel():
            a, b, s = A[i].double(), B[i].double(), 1.0 if scales is None else scales[i].double()
            h = x[t].double() @ a.t()
            want[t] += s * (h @ b.t())
            sizes = x[t].double().abs() @ a.abs().t()
            bound[t] += s * (first * (sizes @ b.abs().t()) + (second + parts) * (h.abs() @ b.abs().t()))
    bound += HALF_STEP[base.dtype] * (want.abs() + bound) + smallest(base.dtype)
    return want, bound


def check_adapters(c, **kw):
    order, offsets = w8.group_rows(c["ids"], c["A"].shape[0]) if c["A"].shape[0] else (
        torch.arange(c["ids"].numel(), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    want, bound = adapter_reference(**c)
    before = c["base"].clone()
    got = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], scales=c["scales"], **kw)
    assert torch.equal(c["base"], before)
    off = (got.double() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    assert torch.equal(got[c["ids"] < 0], before[c["ids"] < 0])
    # the same bits again, in place too
    again = c["base"].clone()
    assert w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, again, scales=c["scales"], out=again,
                             variant=kw.get("variant", 0)) is again
    assert torch.equal(again, got)
    ok()
    return got


@pytest.mark.parametrize("T,L,K,N,r", [
    (1, 1, 64, 64, 16), (1, 8, 4096, 4096, 16), (3, 2, 1, 1, 1), (5, 4, 7, 5, 3), (8, 1, 100, 33, 8), (16, 16, 520, 264, 64),
    (64, 32, 1024, 512, 64), (40, 3, 1000, 1537, 24), (130, 5, 264, 250, 100), (33, 2, 2048, 160, 256), (300, 7, 512, 520, 32),
    (700, 2, 136, 1040, 128), (9, 1024, 64, 32, 4), (2, 0, 64, 32, 8), (6, 3, 64, 32, 0), (6, 3, 0, 32, 8), (0, 2, 16, 16, 8),
    (513, 1, 320, 96, 16),
])
@pytest.mark.parametrize("dtype,out", [("bf16", None), ("fp16", None), ("bf16", "fp32"), ("fp16", "fp32")])
def test_adapters(T, L, K, N, r, dtype, out):
    c = adapter_case(T, L, K, N, r, dtype, out)
    check_adapters(c)
    c["scales"] = None
    c["ids"] = torch.sort(c["ids"], descending=True).values.clone()
    check_adapters(c)


SMALL, TILED = w8.W8A8_VARIANT_SMALLM, w8.W8A8_VARIANT_TILED


# The tiles of 128 rows.
@pytest.mark.parametrize("T,L,K,N,r", [
    (32, 1, 64, 8, 8), (128, 1, 128, 64, 16), (129, 1, 72, 72, 24), (255, 2, 4096, 256, 64), (1000, 3, 1000, 1032, 40),
    (640, 20, 256, 200, 56), (5000, 4, 512, 264, 48), (300, 2, 328, 4096, 128), (257, 1, 64, 136, 72), (400, 3, 2048, 64, 104),
    (3000, 16, 256, 520, 32), (64, 2, 8192, 8, 64),
])
@pytest.mark.parametrize("dtype,out", [("bf16", None), ("fp16", None), ("bf16", "fp32"), ("fp16", "fp32")])
def test_adapters_many_rows(T, L, K, N, r, dtype, out):
    c = adapter_case(T, L, K, N, r, dtype, out)
    check_adapters(c, variant=TILED)
    c["scales"] = None
    c["ids"] = torch.sort(c["ids"], descending=True).values.clone()
    check_adapters(c, variant=TILED)


def test_adapters_forms_chosen_by_themselves():
    """Either form at sizes that are its own, and TILED refused where it does not fit."""
    for T, L in ((100, 4), (6000, 4)):
        c = adapter_case(T, L, 256, 264, 16, "bf16", None)
        order, offsets = w8.group_rows(c["ids"], L)
        call = lambda **kw: w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], **kw)  # noqa: E731
        assert torch.equal(call(), call(variant=SMALL if T == 100 else TILED))
        check_adapters(c)
    with pytest.raises(w8.W8A8Error) as e:
        w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"][:, :259].contiguous()[:, :0], variant=TILED)
    assert e.value.status in (w8.W8A8_ERR_INVALID_ARG, w8.W8A8_ERR_UNSUPPORTED)


def test_adapters_many_rows_bad_order_and_offsets_stay_in_bounds():
    c = adapter_case(400, 3, 128, 64, 8, "bf16", None, none=0.0)
    order, offsets = w8.group_rows(c["ids"], 3)
    good = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], variant=TILED)
    bad = order.clone()
    bad[3], bad[200] = -5, 2 ** 30
    out = torch.full_like(c["base"], 7.0)
    w8.adapter_matmul(c["x"], c["A"], c["B"], bad, offsets, c["base"], out=out, variant=TILED)
    skipped = order[[3, 200]].long().tolist()
    rest = [i for i in range(400) if i not in skipped]
    assert (out[skipped] == 7.0).all() and torch.equal(out[rest], good[rest])
    for wrong in ([0, 999, -4, 400], [300, 200, 100, 0], [-1, 2 ** 31 - 1, -2 ** 31, 5]):
        w8.adapter_matmul(c["x"], c["A"], c["B"], order, torch.tensor(wrong, dtype=torch.int32, device="cuda"), c["base"],
                          variant=TILED)
    ok()


def test_adapters_many_rows_strides_not_finite_rows_and_large_fp16_sums():
    for dtype in ("bf16", "fp16"):
        c = adapter_case(500, 2, 200, 96, 16, dtype, "fp32", none=0.1)
        order, offsets = w8.group_rows(c["ids"], 2)
        clean = check_adapters(c, variant=TILED)
        x, base = torch.zeros(500, 264, device="cuda", dtype=c["x"].dtype), torch.zeros(500, 100, device="cuda")
        x[:, 8:208], base[:, :96] = c["x"], c["base"]
        assert torch.equal(check_adapters(dict(c, x=x[:, 8:208], base=base[:, :96]), variant=TILED), clean)
        t = (c["ids"] >= 0).nonzero()[:, 0][[5, 90]].tolist()
        c["x"][t[0], 17], c["x"][t[1], 3] = math.nan, math.inf
        got = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], scales=c["scales"], variant=TILED)
        assert got[t[0]].isnan().all() and not got[t[1]].isfinite().any()
        others = [i for i in range(500) if i not in t]
        assert torch.equal(got[others], clean[others])
    c = adapter_case(200, 2, 1024, 136, 40, "fp16", "fp32", sizes=200.0)
    c["A"] = (c["A"].float() * 256).half()
    check_adapters(c, variant=TILED)


def test_adapters_many_rows_captured_twice_and_replayed_at_once():
    graphs, cases, outs, kept = [], [], [], []
    for i in range(2):
        c = adapter_case(1500, 4, 512, 264, 32, "bf16", None, seed=i)
        order, offsets = w8.group_rows(c["ids"], 4)
        w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], scales=c["scales"], variant=TILED)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], scales=c["scales"], variant=TILED))
        graphs.append(graph), cases.append(c), kept.append((order, offsets))      # the graph reads them
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c in cases:
            c["x"].copy_(torch.randn_like(c["x"]))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            want, bound = adapter_reference(**c)
            assert ((out.double() - want).abs() <= bound).all()
    ok()


@pytest.mark.parametrize("rows_of", ["one", "none", "each"])
def test_adapters_all_rows_of_one_or_of_none(rows_of):
    for T in (1, 40, 200):
        c = adapter_case(T, 6, 256, 264, 16, "bf16", None)
        c["ids"] = {"one": torch.full_like(c["ids"], 4), "none": torch.full_like(c["ids"], -1),
                    "each": torch.arange(T, device="cuda", dtype=torch.int32) % 6}[rows_of]
        check_adapters(c)


def test_adapters_in_place_leave_rows_without_one_untouched():
    c = adapter_case(50, 3, 128, 72, 8, "bf16", None, none=0.6)
    order, offsets = w8.group_rows(c["ids"], 3)
    out = c["base"].clone()
    out[c["ids"] < 0] = math.nan
    bits = out.clone().view(torch.int16)
    w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, out, out=out)
    none = c["ids"] < 0
    assert torch.equal(out.view(torch.int16)[none], bits[none]) and out[~none].isfinite().all()


@pytest.mark.parametrize("size", [3e-4, 200.0])
def test_adapters_fp16_sums_beyond_fp16(size):
    """x A^T reaches 10^6 (fp16 ends at 65504), or lies where fp16 has few bits; base in fp32."""
    c = adapter_case(30, 3, 1024, 136, 40, "fp16", "fp32", sizes=size)
    c["A"] = (c["A"].float() * (256 if size > 1 else 1 / 16)).half()
    if size > 1:
        assert (c["x"].double() @ c["A"][0].double().t()).abs().max() > 65504
    check_adapters(c)


def test_adapters_a_row_that_is_not_finite_stays_alone():
    for dtype in ("bf16", "fp16"):
        c = adapter_case(24, 2, 200, 96, 16, dtype, "fp32", none=0.0)
        order, offsets = w8.group_rows(c["ids"], 2)
        clean = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"])
        c["x"][5, 17], c["x"][9, 3] = math.nan, math.inf
        got = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"])
        assert got[5].isnan().all() and not got[9].isfinite().any()
        others = [i for i in range(24) if i not in (5, 9)]
        assert torch.equal(got[others], clean[others])


def test_adapters_strides_and_alignments():
    g = gen(4)
    for dtype in ("bf16", "fp16"):
        for K, N, pad, shift in ((128, 64, 8, 0), (128, 64, 8, 8), (128, 64, 3, 1), (200, 71, 5, 2)):
            c = adapter_case(37, 3, K, N, 16, dtype, None)

            def wide(t):
                b = torch.randn(t.shape[0], shift + t.shape[1] + pad, generator=g, device="cuda").to(t.dtype)
                b[:, shift:shift + t.shape[1]] = t
                return b[:, shift:shift + t.shape[1]]

            dense = check_adapters(c)
            v = dict(c, x=wide(c["x"]), base=wide(c["base"]))
            out = wide(torch.zeros_like(c["base"]))
            before = out._base.clone()
            assert torch.equal(check_adapters(v, out=out), dense)
            assert torch.equal(out._base[:, :shift], before[:, :shift])
            assert torch.equal(out._base[:, shift + N:], before[:, shift + N:])
            # weights off 16-byte boundaries
            for name in ("A", "B"):
                flat = torch.empty(c[name].numel() + 1, dtype=c[name].dtype, device="cuda")[1:]
                v[name] = flat.copy_(c[name].reshape(-1)).view(c[name].shape)
            assert torch.equal(check_adapters(v), dense)


def test_adapters_bad_order_and_offsets_stay_in_bounds():
    """Entries that name no row are skipped; offsets out of order or range touch no other memory."""
    c = adapter_case(40, 3, 128, 64, 8, "bf16", None, none=0.0)
    order, offsets = w8.group_rows(c["ids"], 3)
    good = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"])
    bad = order.clone()
    bad[3], bad[20] = -5, 2 ** 30
    out = torch.full_like(c["base"], 7.0)
    w8.adapter_matmul(c["x"], c["A"], c["B"], bad, offsets, c["base"], out=out)
    skipped = order[[3, 20]].long().tolist()
    rest = [i for i in range(40) if i not in skipped]
    assert (out[skipped] == 7.0).all() and torch.equal(out[rest], good[rest])
    for wrong in ([0, 99, -4, 40], [30, 20, 10, 0], [-1, 2 ** 31 - 1, -2 ** 31, 5]):
        w8.adapter_matmul(c["x"], c["A"], c["B"], order, torch.tensor(wrong, dtype=torch.int32, device="cuda"), c["base"])
    ok()


def test_adapters_captured_and_replayed_over_new_rows():
    c = adapter_case(96, 5, 256, 264, 16, "bf16", None)
    order, offsets = w8.group_rows(c["ids"], 5)
    out = torch.empty_like(c["base"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, f = w8.group_rows(c["ids"], 5)
        w8.adapter_matmul(c["x"], c["A"], c["B"], o, f, c["base"], scales=c["scales"], out=out)
    for seed in range(4):
        n = adapter_case(96, 5, 256, 264, 16, "bf16", None, seed=seed)
        for name in ("x", "A", "B", "ids", "base", "scales"):
            c[name].copy_(n[name])
        graph.replay()
        want, bound = adapter_reference(**c)
        assert ((out.double() - want).abs() <= bound).all()
    ok()


@pytest.mark.parametrize("variant", [SMALL, TILED])
def test_adapters_rows_past_2_31_elements(variant):
    c = adapter_case(40, 3, 256, 264, 16, "bf16", None)
    order, offsets = w8.group_rows(c["ids"], 3)
    want = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"], variant=variant)
    ld = (1 << 26) + 8
    far = torch.zeros(40 * ld, dtype=torch.bfloat16, device="cuda")
    x, base, out = (torch.as_strided(far, (40, n), (ld, 1), at) for n, at in ((256, 0), (264, 1024), (264, 4096)))
    x.copy_(c["x"]), base.copy_(c["base"])
    w8.adapter_matmul(x, c["A"], c["B"], order, offsets, base, out=out, variant=variant)
    assert torch.equal(out, want)
    ok()


def test_route_rows_past_2_31_elements():
    g = gen(8)
    logits = torch.randn(40, 64, generator=g, device="cuda").half()
    far = torch.zeros(40 * ((1 << 26) + 3), dtype=torch.float16, device="cuda")
    strided = torch.as_strided(far, (40, 64), ((1 << 26) + 3, 1))
    strided.copy_(logits)
    for a, b in zip(w8.route_experts(logits, 4), w8.route_experts(strided, 4)):
        assert torch.equal(a, b)
    ok()


def test_threads_on_their_own_streams():
    errors = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                c = adapter_case(60 + seed, 4, 256, 264, 16, "bf16", None, seed=seed)
                g = gen(seed)
                logits = torch.randn(2000 + seed, 128, generator=g, device="cuda")
                first = None
                for _ in range(10):
                    r = w8.route_experts(logits, 6, "sigmoid")
                    order, offsets = w8.group_rows(c["ids"], 4)
                    y = w8.adapter_matmul(c["x"], c["A"], c["B"], order, offsets, c["base"])
                    z = w8.combine_experts(c["base"], (r[4][:50] % c["base"].shape[0]).contiguous(), r[1][:50].contiguous())
                    torch.cuda.current_stream().synchronize()
                    now = [*r, y, z]
                    first = first or now
                    assert all(torch.equal(a, b) for a, b in zip(now, first))
        except Exception as e:      # noqa: BLE001
            errors.append(repr(e))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in ts) and not errors, errors
    ok()
