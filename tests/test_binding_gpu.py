"""Calls that the binding refuses on a GPU machine (most of the tensors have no rows)."""
import pathlib
import subprocess
import sys

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


FAILED_LAUNCH = """
import ctypes, torch, gated_deltanet_scan_chunked_b200 as lib
from gated_deltanet_scan_chunked_b200 import gdn
cuda = ctypes.CDLL("libcuda.so.1")
x = torch.ones(8, 64, device="cuda"); la = torch.zeros_like(x); h = torch.zeros_like(x)
y, y2, h2 = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(x)
z, sc = torch.zeros(2, 4, 50, device="cuda"), torch.zeros(2, 4, device="cuda")
out = (torch.empty(2, 4, device="cuda"), torch.empty(2, 4, dtype=torch.int32, device="cuda"),
       torch.empty(2, 4, dtype=torch.int32, device="cuda"),
       torch.empty(2, 4, dtype=torch.uint8, device="cuda"))
p = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
lib.gdn_glr_step(x, la, h2, y=y2)
s = torch.cuda.Stream()
torch.cuda.synchronize()
bad = (lambda: lib.gdn_glr_step(x, la, h, y=y, stream=s),
       lambda: lib.gdn_glr_fwd(x, la, y=y, output_final_state=False, stream=s),
       lambda: lib.gdn_beam_select(z, sc, 4, out=out, stream=s),
       lambda: lib.gdn_state_reorder(h, p, stream=s))
good = (lambda: lib.gdn_glr_step(x, la, h, y=y), lambda: lib.gdn_state_reorder(h, p),
        lambda: lib.gdn_beam_select(z, sc, 4, out=out),
        lambda: lib.gdn_glr_fwd(x, la, y=y, output_final_state=False))
for call in bad:
    # a capture that the driver has given up: it refuses launches on the stream
    st, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    assert cuda.cuStreamBeginCapture_v2(st, 1) == 0
    assert cuda.cuStreamSynchronize(st) != 0
    try:
        call()
        raise SystemExit("a launch into a broken capture went through")
    except gdn.GdnError as e:
        assert e.status == gdn.GDN_ERR_CUDA
    assert cuda.cuStreamEndCapture(st, ctypes.byref(graph)) != 0
    for other in good:
        other()
    torch.cuda.synchronize()
assert (h == 4 * 1).all() and torch.equal(y, x.cumsum(0))
assert gdn.gdn_check_device_error() == gdn.GDN_OK
print("ok")
"""


def test_a_failed_launch_is_reported_once():
    """By the call that made it, and not by the next ones of its thread."""
    root = str(pathlib.Path(__file__).resolve().parent.parent)
    out = subprocess.run([sys.executable, "-c", FAILED_LAUNCH], cwd=root, capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stderr[-2000:]
