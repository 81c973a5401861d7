"""Beam search's choice where logits are far from 0 or from each other: mask
values of any size, offsets, infinities, ties.  Against the fp64 oracle, or
against the definition where the answer is plain."""
import pytest
import torch

import gated_deltanet_scan_chunked_b200 as lib
from tests.test_beam_gpu import BF16, F32, check, rows

pytestmark = pytest.mark.gpu

# The bound on the log sum that `check` uses has 35 * 2^-24 for the exponents'
# arguments: 2.5 * 2^-24 of a difference of up to 14.  The rows here have at
# most 13,000 tokens, whose terms weigh nothing together below a difference of
# log 13,000 = 9.5, and take besides a factor 2^-r (2 * 2^-23 and a rounding,
# 5 * 2^-24) and a rounding of r + difference, up to 6 + 13.7 = 20 in units of
# 2 (20 * 0.7 * 2^-24 in the worst case, if all weight lay there; at most a
# difference of 4.5 + 9.5 counts): 2.5 * 9.5 + 5 + 4 < 35.

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


@pytest.mark.parametrize("m", [12345.678, -98765.4, 4321987.0, 6.1e7])
def test_sums_that_grow_in_steps(m):
    """A thread meets values 40 above its first ones, then a little more, so that
    its sum changes its reference while both still count."""
    G, K, V = 150, 4, 13000
    x = torch.full((G, K, V), m, device="cuda")
    x[:, :, 4096] = x[0, 0, 0] + 39.75
    x[:, :, 8192] = x[0, 0, 0] + 40.25
    check(x, torch.zeros(G, K, device="cuda"), 8, groups=[0, 77, 149])
