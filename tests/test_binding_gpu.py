"""Calls that the binding refuses on a GPU machine (most of the tensors have no rows)."""
import pytest
import torch

import gated_deltanet_scan_chunked_b200 as lib

pytestmark = pytest.mark.gpu
BIG = 2 ** 32  # what an int32 argument would be cut by


def test_sizes_past_32_bits_are_refused():
    x = torch.empty(0, BIG + 64, device="cuda", dtype=torch.bfloat16)
    h = torch.empty(0, BIG + 64, device="cuda")
    z, s = torch.zeros(1, 2, 50, device="cuda"), torch.zeros(1, 2, device="cuda")
    none = torch.empty(0, 2, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for call in (lambda: lib.gdn_glr_fwd(x, x, output_final_state=False),
                 lambda: lib.gdn_glr_bwd(x, x, x, want_d_initial_state=False),
                 lambda: lib.gdn_glr_step(x, x, h),
                 lambda: lib.gdn_beam_select(z, s, 2, end_token=BIG + 1),
                 lambda: lib.gdn_beam_select(z, s, BIG + 2),
                 lambda: lib.gdn_beam_select(torch.empty(0, 2, BIG + 8, device="cuda"), none, 2),
                 lambda: lib.gdn_state_reorder(torch.empty(0, 4, device="cuda"),
                                               torch.empty(0, BIG + 4, **i32)),
                 lambda: lib.gdn_state_reorder(torch.empty(0, 4, device="cuda"),
                                               torch.empty(BIG + 4, 0, **i32))):
        with pytest.raises(ValueError, match="32 bits"):
            call()
