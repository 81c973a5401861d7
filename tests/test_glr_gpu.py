"""Gated linear recurrence on the GPU against the fp64 oracle, elementwise
inside the oracle's derived fp32 bounds (plus half a step of the output's
type), and its contracts: packing, carrying, aliasing, streams, graphs."""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_deltanet_scan_chunked_b200 as lib
from gated_deltanet_scan_chunked_b200 import gdn
from oracle import glr

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROOT = str(pathlib.Path(__file__).resolve().parent.parent)
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
GATES = ["none", "beta", "complement"]


def make(seed, lens, C, gate, dtype, h0=True, slow=False):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens), len(lens)
    rate = torch.exp(torch.rand(C, generator=g) * (-7.0 if slow else -3.0))
    la = -torch.nn.functional.softplus(torch.randn(T, C, generator=g) * 2) * rate * 4
    p = dict(x=torch.randn(T, C, generator=g).to(dtype), log_alpha=la.to(dtype),
             dy=torch.randn(T, C, generator=g).to(dtype),
             beta=torch.rand(T, C, generator=g).to(dtype) if gate == "beta" else
             None if gate == "none" else gate,
             h0=torch.randn(n, C, generator=g) if h0 else None,
             dhT=torch.randn(n, C, generator=g),
             cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
    return p


def cuda(v):
    return v.cuda() if isinstance(v, torch.Tensor) else v


def f64(v):
    return v.double().cpu().numpy() if isinstance(v, torch.Tensor) else v


def inside(got, ref, bound, dtype, what):
    got = f64(got)
    tol = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / tol))


def forward(p, **kw):
    return lib.gdn_glr_fwd(cuda(p["x"]), cuda(p["log_alpha"]), cuda(p["beta"]),
                           initial_state=cuda(p["h0"]), cu_seqlens=cuda(p["cu"]), **kw)


def backward(p, **kw):
    return lib.gdn_glr_bwd(cuda(p["x"]), cuda(p["log_alpha"]), cuda(p["dy"]), cuda(p["beta"]),
                           initial_state=cuda(p["h0"]), d_final_state=cuda(p["dhT"]),
                           cu_seqlens=cuda(p["cu"]), **kw)


def check(p, dtype):
    args = (f64(p["x"]), f64(p["log_alpha"]))
    beta, h0, cu = f64(p["beta"]), f64(p["h0"]), p["cu"].tolist()
    ref = glr.forward(*args, beta, h0, cu)
    y, hT, ck = forward(p, checkpoints=True)
    inside(y, ref["y"], ref["y_bound"], dtype, "y")
    inside(hT, ref["final_state"], ref["final_bound"], F32, "final_state")
    ref_d, bound = glr.backward(*args, f64(p["dy"]), beta, h0, f64(p["dhT"]), cu)
    d = backward(p, checkpoints=ck)
    assert ("dbeta" in d) == isinstance(p["beta"], torch.Tensor)
    for name, got in d.items():
        inside(got, ref_d[name], bound[name], F32 if name == "d_initial_state" else dtype, name)
    again = backward(p)  # checkpoints computed again
    for name in d:
        assert torch.equal(d[name], again[name]), name
    assert gdn.gdn_check_device_error() == gdn.GDN_OK


SHAPES = [([1], 1), ([1], 2), ([2], 3), ([7], 33), ([8], 64), ([63], 65), ([64], 66), ([65], 2),
          ([511], 31), ([512], 128), ([513], 5), ([700], 130), ([1100], 64),
          ([1] * 70, 34), ([0, 3, 0, 0, 64, 1, 0], 7), ([64, 64, 0, 63, 2, 200, 0], 40),
          ([5, 0, 600, 9], 66), ([0], 3), ([0, 0], 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("lens,C", SHAPES)
def test_against_oracle(lens, C, gate, dtype):
    check(make(len(lens) * 100 + C, lens, C, gate, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,C", [([300], 8), ([40, 90, 7], 16), ([129], 24), ([2000, 61], 4),
                                    ([3000], 64), ([700, 900], 192)])
def test_narrow_against_oracle(lens, C, dtype):
    """Rows shorter than a CTA's channels; few channels, so the largest clusters."""
    check(make(40 + C, lens, C, "complement", dtype), dtype)


@pytest.mark.parametrize("lens", [[0] * 100 + [1] * 200 + [0] * 50 + [700] + [2] * 90,
                                  [3] * 500, [40, 0] * 30 + [1] * 300,
                                  [600] + [0] * 80 + [1] + [0] * 33 + [500]])
def test_many_sequences_against_oracle(lens):
    """More sequences between two runs than the walk counts at once."""
    check(make(len(lens), lens, 24, "beta", BF16), BF16)
    check(make(len(lens), lens, 9, "none", F32), F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,C", [([3000, 1, 1500], 70), ([4500], 33)])
def test_long_memory_against_oracle(lens, C, dtype):
    """Channels that remember thousands of tokens, over several cluster steps."""
    check(make(11, lens, C, "beta", dtype, slow=True), dtype)


@pytest.mark.parametrize("lens,C", [([140, 0, 90], 2560), ([140, 0, 90], 6145),
                                    ([1000, 300], 6144), ([700], 9216)])
def test_wide_against_oracle(lens, C):
    check(make(12, lens, C, "beta", BF16), BF16)


@pytest.mark.parametrize("C", [2048, 2049])
def test_offsets_past_32_bits(C):
    """More than 2^32 elements: the last sequence equals the same one alone."""
    T, n = (1 << 21) + 300, 200
    g = torch.Generator("cuda").manual_seed(C)
    tail = {k: torch.rand(n, C, generator=g, device="cuda").to(BF16) for k in ("x", "be", "dy")}
    tail["la"] = -torch.rand(n, C, generator=g, device="cuda").to(BF16)
    h0 = torch.randn(2, C, generator=g, device="cuda")
    big = {}
    for k, v in tail.items():
        big[k] = torch.full((T, C), -0.5 if k == "la" else 0.25, dtype=BF16, device="cuda")
        big[k][T - n:] = v
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    y, hT, ck = lib.gdn_glr_fwd(big["x"], big["la"], big["be"], initial_state=h0, cu_seqlens=cu,
                                checkpoints=True)
    d = lib.gdn_glr_bwd(big["x"], big["la"], big["dy"], big["be"], initial_state=h0,
                        cu_seqlens=cu, checkpoints=ck)
    ref = glr.forward(f64(tail["x"]), f64(tail["la"]), f64(tail["be"]), f64(h0[1:]))
    inside(y[T - n:], ref["y"], ref["y_bound"], BF16, "y")
    inside(hT[1:], ref["final_state"], ref["final_bound"], F32, "final_state")
    ref_d, bound = glr.backward(f64(tail["x"]), f64(tail["la"]), f64(tail["dy"]), f64(tail["be"]),
                                f64(h0[1:]))
    for k in ("dx", "dlog_alpha", "dbeta"):
        inside(d[k][T - n:], ref_d[k], bound[k], BF16, k)
    inside(d["d_initial_state"][1:], ref_d["d_initial_state"], bound["d_initial_state"], F32, "dh0")
    # the long sequence has settled: h = a h + b x with a = e^-1/2, b x = 1/16
    fixed = 0.0625 / (1 - np.exp(-0.5))
    assert (hT[0] - fixed).abs().max().item() < 1e-5 * fixed
    assert (y[T // 2].float() - fixed).abs().max().item() <= 2.0 ** -8 * fixed * 1.01


def test_no_initial_state_is_zeros():
    p = make(13, [30, 100], 20, "beta", F32, h0=False)
    check(p, F32)
    y, hT, _ = forward(p)
    q = dict(p, h0=torch.zeros(2, 20))
    y0, hT0, _ = forward(q)
    assert torch.equal(y, y0) and torch.equal(hT, hT0)


def test_single_sequence_without_cu_seqlens():
    p = make(14, [150], 24, "complement", F32)
    y, hT, ck = forward(p, checkpoints=True)
    q = dict(p, cu=None)
    y1, hT1, ck1 = forward(q, checkpoints=True)
    assert torch.equal(y, y1) and torch.equal(hT, hT1) and torch.equal(ck[1:], ck1[1:])
    d, d1 = backward(p), backward(q)
    assert all(torch.equal(d[k], d1[k]) for k in d)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_resets_inside_a_sequence(dtype):
    """log_alpha = -inf: a = 0, also at tile borders; dlog_alpha is 0 there."""
    p = make(15, [300, 40], 34, "beta", dtype)
    at = [0, 1, 63, 64, 65, 128, 200, 299, 300, 339]
    p["log_alpha"][at] = float("-inf")
    p["log_alpha"][250, ::2] = float("-inf")
    p["log_alpha"][251] = -200.0   # a = 0 in fp32 as well
    check(p, dtype)
    assert (backward(p)["dlog_alpha"][at] == 0).all()


def test_infinities_and_nan_stay_in_their_sequence():
    lens = [70, 130, 5, 61]
    clean = make(16, lens, 36, "beta", F32)
    y0, hT0, _ = forward(clean)
    d0 = backward(clean)
    p = dict(clean, x=clean["x"].clone(), dy=clean["dy"].clone(), h0=clean["h0"].clone())
    p["x"][3, 4], p["x"][69, 5] = float("inf"), float("nan")
    p["x"][201, 6] = float("nan")
    p["h0"][3, 7] = float("inf")
    p["dy"][204, 8], p["dy"][100, 9] = float("inf"), float("nan")
    y, hT, _ = forward(p)
    d = backward(p)
    same = [slice(70, 200)]           # forward: sequence 1 has clean inputs
    for s in same:
        assert torch.equal(y[s], y0[s])
    assert torch.equal(hT[1], hT0[1])
    clean_cols = [c for c in range(36) if c not in (4, 5, 6, 7, 8, 9)]
    assert torch.equal(y[:, clean_cols], y0[:, clean_cols])
    assert not torch.isfinite(y[3:70, 4]).any() and torch.isfinite(y[:3, 4]).all()
    for k in ("dx", "dlog_alpha", "dbeta"):
        assert torch.equal(d[k][:, clean_cols], d0[k][:, clean_cols]), k
        assert torch.equal(d[k][:70, 8], d0[k][:70, 8]) and torch.equal(d[k][:70, 9], d0[k][:70, 9])
        assert torch.equal(d[k][200:, 9], d0[k][200:, 9])
        assert torch.equal(d[k][70:200, [4, 5, 6, 7]], d0[k][70:200, [4, 5, 6, 7]]), k


@pytest.mark.parametrize("C", [32, 33])
@pytest.mark.parametrize("packed", [True, False])
def test_nan_is_not_forgotten_where_the_decays_underflow(C, packed):
    """exp(-20) is not 0, so a NaN stays to the end of its sequence (backward: to
    its beginning), although products of a few such decays are 0 in fp32."""
    lens = [100, 900, 200] if packed else [1200]
    p = make(19, lens, C, "none", F32)
    p["log_alpha"][:] = -20.0
    p["x"][150, 3] = p["dy"][950, 4] = float("nan")
    p["x"][170, 5] = float("inf")
    lo, hi = (100, 1000) if packed else (0, 1200)
    y, hT, _ = forward(p)
    d = backward(p)["dx"]
    for c, at in ((3, 150), (5, 170)):
        assert not torch.isfinite(y[at:hi, c]).any()
        assert torch.isfinite(y[:at, c]).all() and torch.isfinite(y[hi:, c]).all()
        assert not torch.isfinite(hT[1 if packed else 0, c])
    assert torch.isnan(y[150:hi, 3]).all()
    assert torch.isnan(d[lo:951, 4]).all()
    assert torch.isfinite(d[951:, 4]).all() and torch.isfinite(d[:lo, 4]).all()


def test_in_place_state_equals_separate():
    p = make(17, [100, 0, 1, 200], 50, "beta", BF16)
    y, hT, _ = forward(p)
    h = p["h0"].cuda()
    y2, h2, _ = lib.gdn_glr_fwd(p["x"].cuda(), p["log_alpha"].cuda(), p["beta"].cuda(),
                                initial_state=h, final_state=h, cu_seqlens=p["cu"].cuda())
    assert h2 is h and torch.equal(h, hT) and torch.equal(y, y2)


def test_split_and_carry():
    p = make(18, [333], 40, "beta", F32)
    ref = glr.forward(f64(p["x"]), f64(p["log_alpha"]), f64(p["beta"]), f64(p["h0"]))
    h = p["h0"].cuda()
    for lo, hi in ((0, 100), (100, 101), (101, 333)):
        a = [p[k][lo:hi].contiguous().cuda() for k in ("x", "log_alpha", "beta")]
        y, h, _ = lib.gdn_glr_fwd(*a, initial_state=h)
        inside(y, ref["y"][lo:hi], ref["y_bound"][lo:hi], F32, "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("N,C", [(1, 1), (1, 8), (3, 5), (2, 2561), (300, 129)])
def test_step_against_oracle(N, C, gate, dtype):
    p = make(19, [1] * N, C, gate, dtype)
    ref = glr.forward(f64(p["x"]), f64(p["log_alpha"]), f64(p["beta"]), f64(p["h0"]),
                      list(range(N + 1)))
    h = p["h0"].cuda()
    y = lib.gdn_glr_step(cuda(p["x"]), cuda(p["log_alpha"]), h, cuda(p["beta"]))
    inside(y, ref["y"], ref["y_bound"], dtype, "y")
    inside(h, ref["final_state"], ref["final_bound"], F32, "state")


def test_decode_continues_a_prefill():
    lens, C, steps = [90, 3, 0], 24, 5
    p = make(20, [n + steps for n in lens], C, "beta", BF16)
    starts = np.concatenate([[0], np.cumsum([n + steps for n in lens])])
    pre = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)])
    q = dict(p, cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32),
             **{k: p[k][pre].contiguous() for k in ("x", "log_alpha", "beta")})
    ref = glr.forward(f64(p["x"]), f64(p["log_alpha"]), f64(p["beta"]), f64(p["h0"]), starts)
    _, h, _ = forward(q)
    for i in range(steps):
        at = [int(s + n + i) for s, n in zip(starts, lens)]
        y = lib.gdn_glr_step(*(cuda(p[k][at]) for k in ("x", "log_alpha")), h,
                             cuda(p["beta"][at]))
        inside(y, ref["y"][at], ref["y_bound"][at], BF16, "token %d" % i)


@pytest.mark.parametrize("gate", GATES)
def test_gradient_against_differences_of_the_forward(gate):
    """Directional differences of the fp32 forward.  The loss is linear in x,
    h_0 and beta, so those differences are off by rounding only; in
    log_alpha the two-step combination (4 D(h) - D(2h)) / 3 is off by h^4 of
    the fifth derivative.  Rounding: each y is within its bound E, so the
    loss within sum |dy| E on either side of a difference of 2 h."""
    lens, C = [40, 0, 75], 12
    p = make(21, lens, C, gate, F32)
    p["log_alpha"] = -torch.rand(p["x"].shape, generator=torch.Generator().manual_seed(1)) * 0.5
    d = backward(p)
    ref = glr.forward(f64(p["x"]), f64(p["log_alpha"]), f64(p["beta"]), f64(p["h0"]),
                      p["cu"].tolist())
    dy, dhT = f64(p["dy"]), f64(p["dhT"])
    noise = 4 * ((np.abs(dy) * ref["y_bound"]).sum()
                 + (np.abs(dhT) * ref["final_bound"]).sum())

    def loss(q):
        y, hT, _ = forward(q)
        return float((f64(y) * dy).sum() + (f64(hT) * dhT).sum())

    g = torch.Generator().manual_seed(2)
    names = dict(x="dx", log_alpha="dlog_alpha", h0="d_initial_state")
    if gate == "beta":
        names["beta"] = "dbeta"
    for name, dname in names.items():
        v = torch.randn(p[name].shape, generator=g)

        def diff(h):
            q = [dict(p, **{name: p[name] + s * h * v}) for s in (1, -1)]
            # the step that was taken, after rounding of the input
            taken = (q[0][name].double() - q[1][name].double()) / (2 * h)
            want = float((f64(taken) * f64(d[dname])).sum())
            return (loss(q[0]) - loss(q[1])) / (2 * h), want

        h = 2.0 ** -5
        (d1, want), (d2, want2) = diff(h), diff(2 * h)
        if name == "log_alpha":
            d1, h4 = (4 * d1 - d2) / 3, h ** 4
            # the fifth derivative along v of sums of products of up to ~10
            # effective decays, from the same quotient at double the step
            d4 = (4 * d2 - diff(4 * h)[0]) / 3
            assert abs(d1 - want) <= abs(d4 - d1) / 4 + 3 * noise / h + h4, (d1, d4, want)
        else:
            assert abs(d1 - want) <= noise / h + 1e-6 * abs(want), (name, d1, want, noise / h)


def test_results_do_not_depend_on_timing_or_stream():
    p = make(22, [900, 4, 1200], 200, "beta", BF16)
    y, hT, ck = forward(p, checkpoints=True)
    d = backward(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y2, hT2, ck2 = forward(p, checkpoints=True, stream=s)
        d2 = backward(p, stream=s)
        s.synchronize()
        assert torch.equal(y, y2) and torch.equal(hT, hT2) and torch.equal(ck, ck2)
        assert all(torch.equal(d[k], d2[k]) for k in d)


def test_calls_at_the_same_time():
    """Different batches on streams that overlap: nothing is shared between calls."""
    ps = [{k: cuda(v) for k, v in make(50 + i, [900 + 37 * i, 5], 640 + 8 * i, "beta", BF16).items()}
          for i in range(4)]
    want = [(forward(p, checkpoints=True), backward(p)) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[] for _ in ps]
    for _ in range(5):
        for i, (p, s) in enumerate(zip(ps, streams)):
            got[i].append((forward(p, checkpoints=True, stream=s), backward(p, stream=s)))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for f, d in g:
            assert all(torch.equal(a, b) for a, b in zip(f, w[0]))
            assert all(torch.equal(d[k], w[1][k]) for k in d)


FIRST = """
import torch, gated_deltanet_scan_chunked_b200 as lib
x = torch.ones(200, 64, device="cuda", dtype=torch.bfloat16)
la = torch.full_like(x, float("-inf"))
z = torch.zeros(1, 2, 50, device="cuda"); z[0, 1, 7] = 9
s = torch.zeros(1, 2, device="cuda"); S = torch.arange(8.0, device="cuda").reshape(2, 4)
h = torch.zeros(200, 64, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, hT, ck = lib.gdn_glr_fwd(x, la, checkpoints=True)
    d = lib.gdn_glr_bwd(x, la, x, checkpoints=ck)
    ys = lib.gdn_glr_step(x, la, h)
    sc, pa, to, fi = lib.gdn_beam_select(z, s, 2)
    lib.gdn_state_reorder(S, pa)
g.replay(); torch.cuda.synchronize()
assert (y == 1).all() and (hT == 1).all() and (d["dx"] == 1).all() and (ys == 1).all()
assert (h == 1).all() and pa.tolist()[0][0] == 1 and to.tolist()[0][0] == 7
assert S[0].tolist() == [4.0, 5.0, 6.0, 7.0], S
print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture():
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stderr[-2000:]


def test_captured_and_replayed():
    """Forward, backward and step in one graph; replays follow new inputs, and a
    second graph of the same calls lives beside it."""
    ps = [{k: cuda(v) for k, v in make(s, [70, 300], 48, "beta", BF16).items()} for s in (23, 24)]
    want = []
    for p in ps:
        y, hT, ck = forward(p, checkpoints=True)
        h = p["h0"].clone()
        ys = lib.gdn_glr_step(p["x"][:2], p["log_alpha"][:2], h, p["beta"][:2])
        want.append((y, hT, backward(p, checkpoints=ck), ys, h))
    cur = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in ps[0].items()}
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        h = torch.empty_like(cur["h0"])
        with torch.cuda.graph(g):
            h.copy_(cur["h0"])
            y, hT, ck = forward(cur, checkpoints=True)
            d = backward(cur, checkpoints=ck)
            d_again = backward(cur)
            ys = lib.gdn_glr_step(cur["x"][:2], cur["log_alpha"][:2], h, cur["beta"][:2])
        graphs.append((g, y, hT, d, d_again, ys, h))
    for p, w in ((ps[1], want[1]), (ps[0], want[0])):
        for k in cur:
            if isinstance(cur[k], torch.Tensor):
                cur[k].copy_(p[k])
        for g, y, hT, d, d_again, ys, h in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, y, hT, d, d_again, ys, h in graphs:
            assert torch.equal(y, w[0]) and torch.equal(hT, w[1])
            assert all(torch.equal(d[k], w[2][k]) for k in d)
            assert all(torch.equal(d_again[k], w[2][k]) for k in d)
            assert torch.equal(ys, w[3]) and torch.equal(h, w[4])


@pytest.mark.parametrize("cu", [[0, 9, 4, 20], [1, 5, 9, 20], [0, 5, 9, 19], [0, 5, 30, 20],
                                [0, -3, 9, 20]])
def test_malformed_sequence_offsets_are_reported(cu):
    p = make(25, [5, 4, 11], 10, "beta", F32)
    guard = torch.full((20 + 64, 10), 7.0, device="cuda")
    p["cu"] = torch.tensor(cu, dtype=torch.int32)
    lib.gdn_glr_fwd(cuda(p["x"]), cuda(p["log_alpha"]), cuda(p["beta"]), cu_seqlens=p["cu"].cuda(),
                    initial_state=p["h0"].cuda(), y=guard[:20])
    assert gdn.gdn_check_device_error() == gdn.GDN_ERR_INVALID_ARG
    assert (guard[20:] == 7.0).all()
    backward(p)
    assert gdn.gdn_check_device_error() == gdn.GDN_ERR_INVALID_ARG
    assert gdn.gdn_check_device_error() == gdn.GDN_OK


@pytest.mark.parametrize("seed", range(6))
def test_malformed_offsets_of_many_sequences_write_nothing_outside(seed):
    """Offsets out of order and far out of range among 300, at widths with and without
    aligned rows: reported, and nothing but the outputs is written."""
    rng = np.random.default_rng(seed)
    T, C, n = 1500, (40, 33)[seed % 2], 300
    p = make(27, [T], C, "beta", F32)
    cu = np.concatenate([[0], np.sort(rng.integers(0, T, n - 1)), [T]])
    cu[rng.integers(1, n, 5)] = [-2 ** 31, 2 ** 31 - 1, T + 1, -1, 0]
    p["cu"] = torch.tensor(cu, dtype=torch.int32)
    p["h0"] = torch.randn(n, C)
    p["dhT"] = torch.randn(n, C)
    y = torch.full((T + 64, C), 7.0, device="cuda")
    h = torch.full((n + 64, C), 7.0, device="cuda")
    lib.gdn_glr_fwd(cuda(p["x"]), cuda(p["log_alpha"]), cuda(p["beta"]), cu_seqlens=p["cu"].cuda(),
                    initial_state=p["h0"].cuda(), y=y[:T], final_state=h[:n])
    assert gdn.gdn_check_device_error() == gdn.GDN_ERR_INVALID_ARG
    assert (y[T:] == 7.0).all() and (h[n:] == 7.0).all()
    backward(p)
    assert gdn.gdn_check_device_error() == gdn.GDN_ERR_INVALID_ARG


def test_binding_refuses_mismatches():
    p = {k: cuda(v) for k, v in make(26, [9], 6, "beta", F32).items()}
    x, la, be = p["x"], p["log_alpha"], p["beta"]
    for bad in (lambda: lib.gdn_glr_fwd(x, la[:8], be), lambda: lib.gdn_glr_fwd(x, la.bfloat16()),
                lambda: lib.gdn_glr_fwd(x.t(), la.t()), lambda: lib.gdn_glr_fwd(x, la, "other"),
                lambda: lib.gdn_glr_fwd(x, la.cpu()), lambda: lib.gdn_glr_fwd(x.half(), la.half()),
                lambda: lib.gdn_glr_fwd(x, la, initial_state=p["h0"][:, :5].contiguous()),
                lambda: lib.gdn_glr_fwd(x, la, checkpoints=torch.empty(2, 6, device="cuda")),
                lambda: lib.gdn_glr_fwd(x[0], la[0]),
                lambda: lib.gdn_glr_step(x, la, p["h0"]),
                lambda: lib.gdn_glr_bwd(x, la, p["dy"][:4]),
                lambda: lib.gdn_glr_fwd(x, la, y=x),          # output on an input
                lambda: lib.gdn_glr_step(x, la, x)):
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            bad()
