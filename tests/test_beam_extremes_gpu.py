"""Beam search's choice where logits are far from 0 or from each other: mask
values of any size, offsets, infinities, ties.  Against the fp64 oracle, or
against the definition where the answer is plain."""
import numpy as np
import pytest
import torch

import gated_deltanet_scan_chunked_b200 as lib
from oracle import beam
from tests.test_beam_gpu import BF16, F32, LOG_SUM, check, rows

pytestmark = pytest.mark.gpu

# The bound on the log sum that `check` uses has 35 * 2^-24 for the exponents'
# arguments.  The rows here have at most 13,000 tokens, whose terms weigh nothing
# together below a difference of log 13,000 = 9.5.  Of the argument (x - m) log2 e
# + r the constant is off by 2^-25 (0.5 * 9.5), and its one rounding, where
# differing values count at all (from 2^27 on they lie 16 apart) of at most 8 +
# 9.5 * 1.44 < 32, by 2^-20 * log 2 = 11; equal values have r exactly.  The factor
# 2^-r is off by 2 * 2^-23 and a rounding, 5.  Where x - m is formed first, its
# rounding (9.5) and that of at most 13.7 (5.5) take the place of 11 and 5.
# 4.8 + max(11 + 5, 9.5 + 5.5) < 35.


def choice(x, s, M):
    """(scores, parents, tokens) of one group by the definition: the score, then the
    beam, then the logit (of finite scores), then the token."""
    x, s = x.double().cpu().numpy(), s.double().cpu().numpy()
    c = beam.table(x, s)
    k, v = np.indices(c.shape)
    by = np.where(np.isfinite(c), -x, 0.0)
    at = np.lexsort([a.reshape(-1) for a in (v, by, k, -c)])[:M]
    return c.reshape(-1)[at], at // x.shape[1], at % x.shape[1]


FILLS = [-1e4, -65504.0, -1e5, -1e7, -3e7, -6.7e7, -6.8e7, -1e9, -1e10, -1e12, -1e18, -1e20,
         -1e25, -1e31]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fill", FILLS)
def test_masks_of_any_low_value(fill, dtype):
    V = 5003
    x, s = rows(3, 7, 4, V, dtype, 3, 1)
    x[0, :, 7:] = fill                       # few tokens left, at the start
    x[1, :, :V - 5] = fill                   # at the end
    keep = torch.zeros(V, dtype=torch.bool, device="cuda")
    keep[::997] = True
    x[2][:, ~keep] = fill                    # scattered
    x[3, 1] = fill                           # a row that the mask leaves empty
    x[4] = fill                              # nothing but such rows
    x[5][:, torch.rand(V, generator=torch.Generator().manual_seed(1)) < 0.5] = fill
    x[6, :, ::2] = fill
    x[6, :, 1::4] = float("-inf")            # two masks
    check(x, s, 12)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fill", FILLS)
def test_one_beam_with_fewer_tokens_left_than_asked_for(fill, dtype):
    """Behind the tokens left come the masked ones, by index."""
    x, s = rows(4, 2, 1, 5003, dtype, 3, 1)
    x[:, :, 3:] = fill
    out = check(x, s, 9)
    assert out[2][:, 3:].tolist() == [[3, 4, 5, 6, 7, 8]] * 2


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset", [2e4, -3e4, 1e5, -1e6, 1e7, 6.5e7, -7e7, 1e9, 1e15, -1e24, 1e33])
def test_rows_far_from_zero(offset, dtype):
    x, s = rows(5, 3, 4, 5003, dtype, 3, 1)
    x += offset
    x[1, 2] -= offset                        # one row of the group near 0
    check(x, s, 12)


@pytest.mark.parametrize("step", [20, 40])
@pytest.mark.parametrize("m", [12345.678, -98765.4, 4321987.0, 6.1e7])
def test_sums_that_grow_in_steps(m, step):
    """A thread meets values about as far above its first ones as its sum's reference
    lies below, then a little more, so that it changes while both still count."""
    G, K, V = 150, 4, 13000
    x = torch.full((G, K, V), m, device="cuda")
    x[:, :, 4096] = x[0, 0, 0] + (step - 0.25)
    x[:, :, 8192] = x[0, 0, 0] + (step + 0.25)
    check(x, torch.zeros(G, K, device="cuda"), 8, groups=[0, 77, 149])


INF = float("inf")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 5003, 70001])
def test_infinite_logits_leave_the_others_nothing(V, dtype):
    """+inf logits share their row; its other tokens score -inf and come by index."""
    x, s = rows(6, 8, 3, V, dtype, 3, 1)
    hot = [V - 1, 5, V // 2]
    x[0, :, hot] = INF                       # all beams: 9 candidates that are finite
    x[1, 0, hot] = INF                       # one beam, the others as usual
    x[2, :, 0] = INF
    x[2, 1, 1::3] = float("nan")
    x[3, :, ::2] = INF                       # far more than are asked for
    x[4, 2, :] = INF
    x[5, 0, hot], x[5, 1:] = INF, -INF       # 3 finite candidates in all
    x[6, :, hot], s[6, :2] = INF, -INF       # dead beams beside it
    x[7, 0, 3], x[7, 1, 4], x[7, 2] = INF, torch.finfo(dtype).max, -INF
    x[7, 1, 5:] = torch.finfo(dtype).min
    for M in (2, 8, 20):
        out = check(x, s, M, groups=range(7))
        # Group 7's lowest candidates lie 2 max(type) below its highest, beyond fp32's
        # range: the score nearest to them is -inf.
        want, wp, wt = choice(x[7], s[7], M)
        with np.errstate(over="ignore"):
            want = want.astype(np.float32)
        got, out_of_range = out[0][7].cpu().numpy(), np.isinf(want)
        assert np.array_equal(np.isinf(got), out_of_range)
        got, want = got[~out_of_range], want[~out_of_range]
        assert (np.abs(got - want) <= LOG_SUM + 2.0 ** -24 * np.abs(want)).all()
        assert out[1][7].tolist() == wp.tolist() and out[2][7].tolist() == wt.tolist()
    assert torch.isfinite(out[0][0]).sum() == 9 and torch.isfinite(out[0][5]).sum() == 3
    assert out[1][5].tolist() == [0] * 20
    low = [v for v in range(20) if v not in hot][:17]
    assert out[2][5].tolist() == sorted(hot) + low


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_beam_with_an_infinite_logit(dtype):
    x, s = rows(7, 150, 1, 9000, dtype)
    x[:, 0, 7000] = INF
    sc, pa, to, fi = lib.gdn_beam_select(x, s, 4)
    assert torch.equal(sc[:, 0], s[:, 0]) and (sc[:, 1:] == -INF).all()
    assert to.tolist() == [[7000, 0, 1, 2]] * 150
    # a step later only one beam lives
    y = torch.randn(150, 4, 9000, device="cuda").to(dtype)
    assert (lib.gdn_beam_select(y, sc, 4)[1] == 0).all()


def test_the_largest_finite_logit_is_not_infinite():
    x = torch.zeros(1, 1, 5000, device="cuda")
    x[0, 0, 9], x[0, 0, 4] = INF, torch.finfo(F32).max
    sc, _, to, _ = lib.gdn_beam_select(x, torch.zeros(1, 1, device="cuda"), 3)
    assert to.tolist() == [[9, 0, 1]] and sc.tolist() == [[0.0, -INF, -INF]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top,score", [(1e20, 0.0), (3.0, 1e20), (1e17, -1e17)])
def test_a_beam_keeps_the_order_of_its_logits(top, score, dtype):
    """Where the top logit or the score swallows the others' differences in 64 bits,
    a beam's candidates still go by logit; of different beams, the lower first."""
    V, M = 5003, 12
    g = torch.Generator().manual_seed(2)
    x = torch.randn(2, 2, V, generator=g).clamp_(-2.9, 2.9).to(dtype).cuda()
    x[0, :, 4001] = top
    x[1, 0, 17] = top
    s = torch.full((2, 2), score, device="cuda")
    s[1, 1] = -INF                           # one beam; in group 0 two with equal scores
    sc, pa, to, _ = lib.gdn_beam_select(x, s, M)
    for n, k, M_k in ((1, 0, M), (0, 0, M if score == 1e20 else M - 1)):
        order = torch.sort(x[n, k].float(), descending=True, stable=True).indices
        mine = to[n][pa[n] == k].tolist()
        assert mine == order[:M_k].tolist() and len(mine) == M_k
    if score != 1e20:                        # the other beam's top comes before all the rest
        assert pa[0].tolist() == [0, 1] + [0] * (M - 2) and to[0, 1] == 4001


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [2 ** 31 - 1, 2 ** 31 - 9])
def test_the_longest_vocabulary(V, dtype):
    """K V just below 2^31.  The row's sum is V - 4 ones (exact: no partial sum but
    the last few is above 2^24, and those are multiples of its step) and 4 e^9."""
    x = torch.zeros(1, 1, V, dtype=dtype, device="cuda")
    at = [7, V // 2, V - 2, V - 1]
    x[0, 0, at] = 9.0
    sc, pa, to, _ = lib.gdn_beam_select(x, torch.zeros(1, 1, device="cuda"), 6)
    assert to.tolist() == [at + [0, 1]] and (pa == 0).all()
    want = torch.tensor([9.0] * 4 + [0.0] * 2, dtype=torch.float64) - np.log(V - 4 + 4 * np.exp(9))
    assert (sc[0].cpu().double() - want).abs().max() <= LOG_SUM + 2.0 ** -24 * 22
