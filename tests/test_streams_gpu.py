"""Calls given a stream: where their memory comes from, and when it may go to
others.  Everything is decided on the host, from addresses."""
import pytest
import torch

import gated_deltanet_scan_chunked_b200 as lib
from gated_deltanet_scan_chunked_b200 import gdn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
LATE = 200_000_000  # cycles that a stream is kept busy: about a tenth of a second


def randn(*shape, dtype=BF16):
    return torch.randn(*shape, device="cuda").to(dtype)


def delta(T=200, H=4, d=32):
    q, k, v = randn(T, H, d), randn(T, H, d), randn(T, H, d)
    return q, k, v, -torch.rand(T, H, device="cuda"), torch.rand(T, H, device="cuda")


def steps(N=8, H=4, d=32):
    return [t.reshape(N, 1, *t.shape[1:]) for t in delta(N, H, d)], randn(N, H, d, d,
                                                                         dtype=torch.float32)


def conv_w(H=4, d=32):
    return randn(3 * H * d, 4, dtype=torch.float32)


def residual(T=64, n_r=4, d=256, rank=64):
    codes = torch.zeros(T, n_r, d, dtype=torch.uint8, device="cuda")
    return (codes, torch.ones(T, n_r, device="cuda"), torch.zeros(n_r, d, device="cuda"),
            randn(rank, n_r * d), randn(n_r * d, rank), randn(n_r, n_r * d))


def cases():
    x, la = randn(1000, 512), -torch.rand(1000, 512, device="cuda").to(BF16)
    z, s = randn(8, 4, 5000), torch.zeros(8, 4, device="cuda")
    q5, (q6, S) = delta(), steps()
    dy, w, r = randn(200, 4, 32), conv_w(), residual()
    h = torch.zeros(1000, 512, device="cuda")  # (here: no call waits for the current stream)
    return {
        "glr_fwd": lambda **k: lib.gdn_glr_fwd(x, la, checkpoints=True, **k),
        "glr_bwd": lambda **k: lib.gdn_glr_bwd(x, la, x, **k),
        "glr_step": lambda **k: lib.gdn_glr_step(x, la, h, **k),
        "beam_select": lambda **k: lib.gdn_beam_select(z, s, 8, **k),
        "chunk_fwd": lambda **k: lib.gdn_chunk_fwd(*q5, **k),
        "chunk_bwd": lambda **k: lib.gdn_chunk_bwd(*q5, dy, **k),
        "decode_step": lambda **k: lib.gdn_decode_step(*(t[:, 0] for t in q6), S, **k),
        "decode_multi": lambda **k: lib.gdn_decode_multi(*q6, S, snapshots=True, **k),
        "conv_frontend": lambda **k: lib.gdn_conv_frontend(*q5[:3], w, **k),
        "chunk_fwd_conv": lambda **k: lib.gdn_chunk_fwd_conv(*q5[:3], w, *q5[3:], **k),
        "decode_conv": lambda **k: lib.gdn_decode_conv(*q6[:3], w, *q6[3:], S, None, snapshots=True,
                                                       **k),
        "gr_read": lambda **k: lib.gdn_gr_read(*r, **k),
    }


NAMES = ["glr_fwd", "glr_bwd", "glr_step", "beam_select", "chunk_fwd", "chunk_bwd", "decode_step",
         "decode_multi", "conv_frontend", "chunk_fwd_conv", "decode_conv", "gr_read"]


def outputs(r):
    return [t for t in gdn._tensors(r) if t.numel()]


@pytest.mark.parametrize("name", NAMES)
def test_results_never_lie_in_memory_just_freed_on_the_current_stream(name):
    call = cases()[name]
    want = call()                                   # (warm-up, and the sizes)
    sizes = [(t.shape, t.dtype) for t in outputs(want)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty(shape, dtype=dt, device="cuda") for shape, dt in sizes for _ in range(3)]
    spans = [(t.data_ptr(), t.data_ptr() + t.untyped_storage().nbytes()) for t in freed]
    del freed
    got = call(stream=s)
    for t in outputs(got):
        assert not any(lo < t.data_ptr() + t.nbytes and t.data_ptr() < hi for lo, hi in spans), name
    s.synchronize()
    for a, b in zip(outputs(got), outputs(want)):
        assert a.shape == b.shape and a.dtype == b.dtype


def test_a_workspace_comes_from_the_given_stream_too():
    """The current stream's cached blocks stay whole while a call on another stream
    makes its workspace."""
    x, la = randn(4096, 4096), -torch.rand(4096, 4096, device="cuda").to(BF16)
    n = lib.glr_bwd_workspace_size(4096, 4096)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty(n, dtype=torch.uint8, device="cuda")
    at = block.data_ptr()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):  # (the outputs' room, so that only the workspace has to be found)
        room = [torch.empty_like(x) for _ in range(2)]
        room.append(torch.empty(1, 4096, device="cuda"))
    torch.cuda.synchronize()
    del room, block
    before = torch.cuda.memory_reserved()
    lib.gdn_glr_bwd(x, la, x, stream=s)
    assert torch.cuda.memory_reserved() - before >= n
    assert torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr() == at
    torch.cuda.synchronize()


def test_arguments_are_kept_until_the_stream_has_read_them():
    s = torch.cuda.Stream()
    shape = (1000, 512)
    state = torch.zeros(shape, device="cuda")
    for _ in range(2):                              # (the second time without first-use costs)
        x, la = randn(*shape), -torch.rand(shape, device="cuda").to(BF16)
        want = lib.gdn_glr_step(x, la, state.clone())
        h = state.clone()
        held = {x.data_ptr(), la.data_ptr()}
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(LATE)
        y = lib.gdn_glr_step(x, la, h, stream=s)
        del x, la
        others = [torch.empty(shape, dtype=BF16, device="cuda") for _ in range(8)]
        busy = not s.query()
        assert busy and not held & {t.data_ptr() for t in others}
        for t in others:
            t.fill_(float("nan"))
        s.synchronize()
        assert torch.equal(y, want)
        del others


def test_results_are_kept_until_the_current_stream_has_read_them():
    s = torch.cuda.Stream()
    x, la = randn(1000, 512), -torch.rand(1000, 512, device="cuda").to(BF16)
    lib.gdn_glr_fwd(x, la, stream=s, output_final_state=False)
    torch.cuda.synchronize()
    y = lib.gdn_glr_fwd(x, la, stream=s, output_final_state=False)[0]
    s.synchronize()
    at, now = y.data_ptr(), torch.cuda.current_stream()
    torch.cuda._sleep(LATE)
    copy = y.clone()
    del y
    again = lib.gdn_glr_fwd(x, la, stream=s, output_final_state=False)[0]
    assert not now.query() and again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, again)


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_given_by_name(name):
    call = cases()[name]
    now = torch.cuda.current_stream()

    class Handle:
        cuda_stream = now.cuda_stream
    for s in (now, torch.cuda.default_stream(), Handle()):
        got = call(stream=s)
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == now
        if name in ("glr_fwd", "glr_bwd", "beam_select", "chunk_fwd"):
            want = call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outputs(got), outputs(want)))


def test_calls_on_a_given_stream_inside_a_capture():
    """A side stream that has joined the capture; replays follow new inputs."""
    x, la = randn(300, 64), -torch.rand(300, 64, device="cuda").to(BF16)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        y, h, _ = lib.gdn_glr_fwd(x, la, stream=s)
        d = lib.gdn_glr_bwd(x, la, y, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        twice = y * 2
    for _ in range(2):
        x.copy_(randn(300, 64))
        g.replay()
        want = lib.gdn_glr_fwd(x, la)[0]
        want_d = lib.gdn_glr_bwd(x, la, want)
        assert torch.equal(y, want) and torch.equal(twice, want * 2)
        assert all(torch.equal(d[k], want_d[k]) for k in d)
