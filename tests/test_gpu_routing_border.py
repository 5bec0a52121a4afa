"""GPU: the border between the last expert that is chosen and those that stay behind, where
biased scores are nearer than the bits that rank them first.

The router ranks by keys that lack their lowest bits and checks neighbours by whole scores.
Three experts whose keys agree may stand in any order; the best of them has to be found also where
the first two are surely apart and the third, behind both, is above them."""
import pytest
import torch

import block_scaled_fp8_w8a8_gb300 as w8
from test_gpu_routing import check_route, gen, ok

pytestmark = pytest.mark.gpu


# Sums of a score of 0.5 and a bias: the value in units `u` of its last place, the three
# experts' offsets in units, all in one run of as many units as a lane has slots (a key's lowest bits).
BUILT = [  # E, sum, u, (first, second, third)
    (1024, 0.5, 2.0 ** -24, (16, 0, 31)), (512, 0.5, 2.0 ** -24, (12, 0, 15)), (1024, 1.0, 2.0 ** -23, (16, 0, 31)),
    (512, 1.0, 2.0 ** -23, (9, 1, 14)), (256, 2.0, 2.0 ** -22, (5, 0, 7)), (256, 4.5, 2.0 ** -21, (6, 2, 7)),
    (512, 4.5, 2.0 ** -21, (9, 1, 10)), (1024, 8.0, 2.0 ** -20, (20, 3, 21)), (256, 8.0, 2.0 ** -20, (4, 0, 6)),
    (160, 8.0, 2.0 ** -20, (4, 0, 6)), (1000, 100.0, 2.0 ** -17, (20, 3, 21)), (129, 1000.0, 2.0 ** -14, (6, 0, 7)),
]


@pytest.mark.parametrize("E,value,u,offsets", BUILT)
@pytest.mark.parametrize("k", [1, 2, 5, 8, 31, 32])
def test_the_third_of_three_scores_with_one_key(E, value, u, offsets, k):
    """Logits of zero have the score 0.5, so the fp32 sums are exact and the order is that of
    the biases; k - 1 experts are far above the three."""
    per = (E + 31) // 32
    assert all(0 <= o < 2 ** (per - 1).bit_length() for o in offsets)
    for first in (0, 3 * per):
        bias = torch.full((E,), value - 50.5, device="cuda")
        for i, o in enumerate(offsets):
            bias[first + i * per] = value - 0.5 + o * u
        above = [e for e in range(E - 1, 0, -3) if e not in (first, first + per, first + 2 * per)][:k - 1]
        bias[above] = value + 1.0 + torch.arange(k - 1, device="cuda") / 64
        logits = torch.zeros(5, E, device="cuda")
        got = check_route(logits, k, scoring="sigmoid", bias=bias)
        assert (got[0][:, -1] == first + 2 * per).all()
        for groups in (2, 8):       # runs of whole lanes or not
            if E % groups == 0:
                check_route(logits, k, scoring="sigmoid", bias=bias, groups=groups, top_groups=groups, group_top=1)
                check_route(logits, k, scoring="sigmoid", bias=bias, groups=groups, top_groups=groups, group_top=2)


def test_the_third_of_three_sigmoids_near_one():
    x = torch.full((1, 1024), -10.0, device="cuda")
    x[0, 0], x[0, 40], x[0, 80] = 14.15, 13.303, 15.249
    assert check_route(x, 1, scoring="sigmoid", bias=torch.zeros(1024, device="cuda"))[0][0, 0] == 80
    assert check_route(x, 2, scoring="sigmoid", bias=torch.zeros(1024, device="cuda"))[0].tolist() == [[80, 0]]


@pytest.mark.parametrize("E,groups,top_groups,group_top", [(256, 1, 1, 2), (512, 1, 1, 2), (1024, 1, 1, 2), (250, 2, 1, 1),
                                                           (512, 8, 3, 2), (1000, 4, 2, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [0.0, 1.0, 2.0, 8.0, 300.0])
def test_many_rows_of_spread_logits_and_biases_of_one_level(E, groups, top_groups, group_top, scoring, level):
    """Against the sums in 64 bits, which are off by less than 4 units of 2^-53 of their size on
    either side: an expert that is chosen instead of another is no lower than that."""
    g = gen(E + int(level))
    T = 12000
    size = E // groups
    for spread, own in ((1.0, 0.0), (4.0, 0.0), (8.0, 0.05)):
        x = (spread * torch.randn(T, E, generator=g, device="cuda")).clamp(max=25.0)
        bias = level + own * torch.randn(E, generator=g, device="cuda")
        d = x.double()
        c = (d.sigmoid() if scoring == "sigmoid" else d.softmax(1)) + bias.double()
        unit = 8 * 2.0 ** -53 * (1 + c.abs().amax())
        value = c.view(T, groups, size).sort(dim=2, descending=True).values[:, :, :group_top].sum(2)
        for k in (1, 2, 8):
            ids, weights, order, offsets, rows = w8.route_experts(x, k, scoring, bias=bias, groups=groups,
                                                                  top_groups=top_groups, group_top=group_top)
            ids = ids.long()
            assert (ids >= 0).all() and (ids.sort(1).values.diff(dim=1) > 0).all()
            if groups > 1:      # no run that is left closed is above one that a choice lies in ...
                used = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, ids // size, True)
                assert (used.sum(1) <= top_groups).all()
                least = value.masked_fill(~used, torch.inf).amin(1)
                border = value.topk(top_groups, 1).values[:, -1]
                assert (least >= border - 2 * unit).all()
                # ... and where the border is told apart, the open runs are known
                after = value.topk(top_groups + 1, 1).values[:, -1]
                open_ = value >= border[:, None]
                rows_ = border - after > 4 * unit
                ranked = c.masked_fill(~open_.repeat_interleave(size, 1), -torch.inf)
            else:
                rows_, ranked = torch.ones(T, dtype=torch.bool, device="cuda"), c
            assert rows_.float().mean() > 0.5
            best = ranked.topk(k, 1).values
            mine = c.gather(1, ids)
            worst = torch.where(rows_[:, None], best - mine, 0.0)
            assert (worst <= unit).all(), (k, spread, (worst > unit).any(1).sum().item(), worst.max().item())
    ok()


@pytest.mark.parametrize("kw", [dict(groups=2 ** 32 + 1), dict(groups=2, top_groups=2 ** 32 + 2), dict(groups=2, group_top=2 ** 32 + 1)])
def test_numbers_of_groups_that_32_bits_do_not_hold_are_refused(kw):
    x = torch.randn(4, 8, device="cuda")
    out = w8.route_experts(x, 2)
    for given in (None, out):
        with pytest.raises(w8.W8A8Error) as e:
            w8.route_experts(x, 2, out=given, **kw)
        assert e.value.status == w8.W8A8_ERR_INVALID_ARG
    ok()
