"""Rules of the Python binding, checked without a GPU."""
import inspect
import pathlib
import subprocess
import sys

import pytest
import torch

from gated_deltanet_scan_chunked_b200 import gdn


def test_every_call_that_takes_a_stream_runs_under_it():
    """Allocations of a call with a stream come from that stream's memory: the
    call is made again with the stream as torch's current one."""
    calls = [n for n in dir(gdn) if n.startswith("gdn_") and callable(getattr(gdn, n))
             and n != "gdn_check_device_error"]
    assert len(calls) >= 15
    for n in calls:
        f = getattr(gdn, n)
        names = list(inspect.signature(f).parameters)
        assert names[-1] == "stream", n
        text = inspect.getsource(f)
        body = text[text.index('"""', text.index('"""') + 3) + 3:]
        want = "if stream is not None: return _on_stream(stream, %s, %s)" % (
            n, ", ".join(names[:-1]))
        assert " ".join(body.split()).startswith(want), n
        assert body.count("stream, ") == 1, n


def test_tensors_of_arguments_and_results():
    a, b, c = (torch.zeros(1) for _ in range(3))
    got = list(gdn._tensors((a, None, [b, 3], dict(x=c, y="z"), 1.5)))
    assert [t is u for t, u in zip(got, (a, b, c))] == [True] * 3 and len(got) == 3


def test_imports_with_a_torch_that_has_no_cuda():
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import gated_deltanet_scan_chunked_b200 as lib
from gated_deltanet_scan_chunked_b200 import gdn
assert "gdn_glr_fwd" in gdn.header_functions()
x = torch.zeros(4, 8)
try:
    lib.gdn_glr_fwd(x, x)
except ValueError as e:
    print("refused:", e)
"""
    root = str(pathlib.Path(__file__).resolve().parent.parent)
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and out.stdout.startswith("refused:"), out.stderr[-2000:]


def test_numbers_past_32_bits_are_refused():
    for v in (0, -1, 2 ** 31 - 1, -2 ** 31):
        assert gdn._int32(v, "v") == v
    for v in (2 ** 31, -2 ** 31 - 1, 2 ** 32, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="v = "):
            gdn._int32(v, "v")
