"""Beam search's choice and the reordering of states on the GPU, against plain
fp64 numpy, and with decode steps as a search uses them."""
import numpy as np
import pytest
import torch

import gated_deltanet_scan_chunked_b200 as lib
from gated_deltanet_scan_chunked_b200 import gdn
import oracle
from oracle import beam, glr

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")

# What the kernel's log sum can be off.  An exponent's argument: the
# difference and its product with log2(e), a constant rounded too, 2.5 * 2^-24
# relative, of at most ~14 (differences far below the maximum weigh nothing)
# -> 2^-18.8 of the exponent; 2^x itself 2^-22; a thread's sum of up to 300
# partial sums of 8 in order -> 308 * 2^-24, the tree behind it 13 * 2^-24.
LOG_SUM = 2.0 ** -18.8 + 2.0 ** -22 + 330 * 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def check_group(got, logits, scores, M, finished=None, end_token=-1):
    """got: (scores, parents, tokens, finished) of one group.  Equal to the
    oracle's choice; where candidates of different beams lie closer than the
    log sums can tell, any order of them is right."""
    sc, pa, to, fi = got
    V = logits.shape[1]
    c = beam.table(logits, scores, finished, end_token).reshape(-1)
    want, wp, wt, wf = beam.select(logits, scores, M, finished, end_token)
    flat = pa.astype(np.int64) * V + to
    assert len(set(flat.tolist())) == M and (pa >= 0).all() and (to >= 0).all() and (to < V).all()
    mine = c[flat]
    with np.errstate(invalid="ignore"):
        close = (mine == want) | (np.abs(mine - want) <= 2 * LOG_SUM)
        near = (sc == mine) | (np.abs(sc - mine) <= LOG_SUM + 2.0 ** -24 * np.abs(mine))
    assert close.all(), (mine, want)
    assert near.all(), (sc, mine)
    swapped = flat != wp * V + wt
    for r in np.nonzero(swapped)[0]:  # another candidate than the oracle's: a near tie
        assert mine[r] != want[r] or pa[r] != wp[r], (r, flat[r], wp[r] * V + wt[r])
        assert np.isfinite(mine[r])
        others = np.nonzero(np.abs(c - mine[r]) <= 2 * LOG_SUM)[0]
        assert len(set((others // V).tolist())) > 1, "a wrong choice, not a near tie"
    assert swapped.mean() <= 0.1
    done = np.zeros(len(scores), bool) if finished is None else np.asarray(finished, bool)
    assert np.array_equal(fi.astype(bool), done[pa] | (to == end_token))


def check(logits, scores, M, finished=None, end_token=-1, groups=None, **kw):
    out = lib.gdn_beam_select(logits, scores, M, finished=finished, end_token=end_token, **kw)
    torch.cuda.synchronize()
    G = logits.shape[0]
    assert [tuple(t.shape) for t in out] == [(G, M)] * 4
    host = [t.cpu().numpy() for t in out]
    for g in range(G) if groups is None else groups:
        check_group([h[g] for h in host], f64(logits[g].float()), f64(scores[g]), M,
                    None if finished is None else f64(finished[g]), end_token)
    return out


def rows(seed, G, K, V, dtype, pad=0, offset=0, scale=2.5):
    """Logits [G, K, V] inside a larger buffer whose other elements are NaN:
    rows V + pad apart, the first at `offset`."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((offset + G * K * (V + pad) + 64,), float("nan"), dtype=dtype, device="cuda")
    x = buf[offset:].as_strided((G, K, V), (K * (V + pad), V + pad, 1))
    x.copy_(torch.randn(G, K, V, generator=g).mul_(scale))
    s = -torch.rand(G, K, generator=g).mul_(8).cuda()
    return x, s


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,K,V,M,pad,offset", [
    (1, 1, 1, 1, 0, 0), (3, 1, 2, 2, 0, 0), (2, 3, 3, 9, 0, 1), (5, 2, 7, 4, 2, 0),
    (2, 4, 8, 8, 0, 0), (2, 4, 9, 8, 0, 3), (4, 3, 255, 6, 1, 0), (1, 4, 2047, 8, 0, 0),
    (2, 4, 2048, 4, 0, 0), (2, 4, 2049, 4, 0, 5), (1, 32, 1025, 64, 0, 0),
    (3, 5, 5000, 10, 3, 2), (1, 1, 70001, 64, 0, 0), (1, 16, 33000, 32, 1, 7),
    (150, 4, 1500, 8, 0, 0), (700, 2, 300, 4, 5, 1)])
def test_select_against_oracle(G, K, V, M, pad, offset, dtype):
    x, s = rows(G * 1000 + V, G, K, V, dtype, pad, offset)
    check(x, s, M, groups=range(0, G, max(1, G // 20)))
    g = torch.Generator().manual_seed(V)
    fin = (torch.rand(G, K, generator=g) < 0.4).to(torch.uint8).cuda()
    check(x, s, M, finished=fin, end_token=V // 2, groups=range(0, G, max(1, G // 20)))
    check(x, s, M, end_token=0, groups=range(0, G, max(1, G // 20)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,K,V,M", [(3000, 4, 700, 8), (65535, 1, 40, 3), (1, 32, 9000, 64),
                                     (5, 12, 70001, 24), (2, 31, 20011, 1), (40, 3, 33333, 6)])
def test_select_over_groups_and_beams(G, K, V, M, dtype):
    x, s = rows(V, G, K, V, dtype)
    check(x, s, M, groups=sorted({0, 1 % G, G // 3, G // 2, G - 1}))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_with_few_tokens_allowed(dtype):
    """Masks that leave a few tokens of a large vocabulary, at its start, its end
    and scattered: fewer finite values than threads, M, or one."""
    V = 70001
    x, s = rows(61, 6, 4, V, dtype, 3, 1)
    keep = [[0], [V - 1], [5, V - 2], list(range(100, 106)), list(range(0, V, 9973)),
            list(range(V - 300, V))]
    for g, k in enumerate(keep):
        m = torch.ones(V, dtype=torch.bool, device="cuda")
        m[k] = False
        x[g][:, m] = -INF
    check(x, s, 12)


def test_select_past_32_bit_offsets():
    """Rows that begin more than 2^32 elements into the logits."""
    ld = (1 << 31) + 1003
    buf = torch.empty(3 * ld + 4096, dtype=BF16, device="cuda")
    x = buf.as_strided((1, 4, 4001), (4 * ld, ld, 1))
    x.copy_(torch.randn(1, 4, 4001, generator=torch.Generator().manual_seed(1)))
    check(x, torch.tensor([[-1.0, -2.0, -0.5, -0.25]], device="cuda"), 8)


def test_select_long_vocabulary():
    x, s = rows(3, 1, 2, 1 << 20, BF16, 0, 0)
    check(x, s, 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_ties_go_to_the_lowest_index(dtype):
    V, K, M = 4099, 3, 24
    x = torch.zeros(2, K, V, dtype=dtype, device="cuda")
    x[1, :, 17:4000:13] = 1.0          # many equal maxima in every row
    x[0, 1, ::2] = -0.0                # -0 equals 0
    s = torch.zeros(2, K, device="cuda")
    sc, pa, to, _ = lib.gdn_beam_select(x, s, M)
    # equal rows, wherever they begin in memory: beam by beam at the same index
    assert pa[0].tolist() == [0] * M and to[0].tolist() == list(range(M))
    ones = list(range(17, 4000, 13))
    assert pa[1].tolist() == [0] * M and to[1].tolist() == ones[:M]
    s[1] = torch.tensor([-1.0, 0.0, 0.0])
    _, pa, to, _ = lib.gdn_beam_select(x, s, M)
    assert pa[1].tolist() == [1] * M and to[1].tolist() == ones[:M]
    # few equal maxima: beam 0's, then beam 1's, then beam 2's
    x[1] = 0
    x[1, :, [5, 4098]] = 9.0
    s[1] = 0
    _, pa, to, _ = lib.gdn_beam_select(x, s, 6)
    assert pa[1].tolist() == [0, 0, 1, 1, 2, 2] and to[1].tolist() == [5, 4098] * 3


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [4099, 32000])
def test_equal_rows_have_equal_sums_wherever_they_begin(V, dtype):
    g = torch.Generator().manual_seed(V)
    row = torch.randn(V, generator=g).to(dtype).cuda()
    x = row.expand(1, 8, V).contiguous()   # an odd V: every row begins elsewhere
    sc, pa, to, _ = lib.gdn_beam_select(x, torch.zeros(1, 8, device="cuda"), 32)
    order = torch.sort(row.float(), descending=True, stable=True).indices[:32].tolist()
    vals = row.float()[order].tolist()
    want, i = [], 0
    while len(want) < 32:                  # equal values by beam, then index
        n = sum(v == vals[i] for v in vals[i:])
        want += [(k, t) for k in range(8) for t in order[i:i + n]]
        i += n
    assert list(zip(pa[0].tolist(), to[0].tolist())) == want[:32]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_masks_and_values_that_are_no_numbers(dtype):
    V, K, M = 3001, 4, 12
    low = torch.finfo(dtype).min
    x, s = rows(5, 9, K, V, dtype, 3, 1)
    x[0, :, 100:] = -INF                    # a mask that leaves 100 tokens
    x[1, :, 3:] = -INF                      # 3 tokens a beam: exactly M
    x[2, :, 2:] = -INF                      # fewer than M
    x[3, 1] = -INF                          # an empty row
    x[4] = -INF                             # nothing at all
    x[5, :, 5:] = low                       # masked with the lowest value
    x[6, 2] = low                           # a row of it
    x[7, 0, 7], x[7, 1, 9] = float("nan"), INF
    x[7, 1, 2999] = INF
    x[8, 0] = float("nan")
    x[8, 3, 1500:] = float("nan")
    check(x, s, M)


def test_select_first_step_and_dead_beams():
    x, s = rows(6, 5, 4, 2500, BF16)
    s[0] = torch.tensor([0.0, -INF, -INF, -INF])    # the first step of a search
    s[1] = torch.tensor([-INF, -2.0, float("nan"), INF])
    s[2] = -INF
    fin = torch.zeros(5, 4, dtype=torch.uint8, device="cuda")
    fin[1, 1] = fin[3] = 1                          # one candidate; four
    fin[4, 0] = fin[2, 3] = 1
    out = check(x, s, 8, finished=fin, end_token=2499)
    assert out[1][0].tolist() == [0] * 8
    assert out[2][1].tolist() == [2499] + list(range(7)) and out[1][1].tolist() == [1] + [0] * 7
    assert out[2][3, :4].tolist() == [2499] * 4
    assert sorted(out[1][3, :4].tolist()) == [0, 1, 2, 3]
    check(x, s, 64, finished=fin.bool(), end_token=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 64])
def test_select_when_a_few_threads_hold_the_largest_values(M, dtype):
    """The largest elements recur at the distance at which a CTA's thread meets
    them again: more candidates than the kernel holds at once."""
    G, K, V = 150, 4, 131072
    step = 256 * (8 if dtype == BF16 else 4)
    x = torch.randn(G, K, V, generator=torch.Generator("cuda").manual_seed(7),
                    device="cuda").to(dtype)
    at = torch.arange(V, device="cuda")
    big = (at % step) < 128
    g = torch.Generator("cuda").manual_seed(8)
    for k in range(K):
        x[3, k, big] = 10 + torch.rand(int(big.sum()), generator=g, device="cuda").to(dtype)
    x[149, 2, big] = 9.0
    s = torch.zeros(G, K, device="cuda")
    check(x, s, M, groups=[0, 3, 149])


def test_select_in_place():
    G, K, V = 3, 6, 3000
    x, s = rows(9, G, K, V, F32)
    fin = torch.zeros(G, K, dtype=torch.uint8, device="cuda")
    fin[1, 2] = 1
    want = lib.gdn_beam_select(x, s, K, finished=fin, end_token=1)
    pa, to = (torch.empty(G, K, dtype=torch.int32, device="cuda") for _ in range(2))
    out = lib.gdn_beam_select(x, s, K, finished=fin, end_token=1, out=(s, pa, to, fin))
    assert out[0] is s and all(torch.equal(a, b) for a, b in zip(out, want))


def test_select_is_the_same_each_time_and_on_other_streams():
    x, s = rows(10, 4, 8, 50001, BF16, 3, 1)
    want = lib.gdn_beam_select(x, s, 16)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [lib.gdn_beam_select(x, s, 16, stream=st) for st in streams for _ in range(4)]
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_binding_refuses_mismatches():
    x, s = rows(11, 2, 3, 100, BF16)
    ok = dict(finished=torch.zeros(2, 3, dtype=torch.uint8, device="cuda"), end_token=4)
    bad = [lambda: lib.gdn_beam_select(x.transpose(1, 2), s, 2),
           lambda: lib.gdn_beam_select(x[..., ::2], s, 2), lambda: lib.gdn_beam_select(x[0], s, 2),
           lambda: lib.gdn_beam_select(x.half(), s, 2), lambda: lib.gdn_beam_select(x, s[:1], 2),
           lambda: lib.gdn_beam_select(x, s.double(), 2), lambda: lib.gdn_beam_select(x, s, 0),
           lambda: lib.gdn_beam_select(x, s, 65), lambda: lib.gdn_beam_select(x.cpu(), s, 2),
           lambda: lib.gdn_beam_select(x, s, 2, end_token=100),
           lambda: lib.gdn_beam_select(x, s, 2, finished=ok["finished"]),   # no end token
           lambda: lib.gdn_beam_select(x, s, 2, finished=s, end_token=1),
           lambda: lib.gdn_beam_select(x, s, 2, out=(s, s, s, s)),
           lambda: lib.gdn_state_reorder(torch.zeros(5, 2, device="cuda"),
                                         torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           lambda: lib.gdn_state_reorder(torch.zeros(6, 2),
                                         torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           lambda: lib.gdn_state_reorder(torch.zeros(2, 6, device="cuda").t(),
                                         torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           lambda: lib.gdn_state_reorder([], torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           lambda: lib.gdn_state_reorder(torch.zeros(6, 2, device="cuda"),
                                         torch.zeros(2, 3, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            call()
            print("case", i)


# --- reordering ---------------------------------------------------------------


def maps(G, K, seed):
    r = np.random.default_rng(seed)
    yield np.tile(np.arange(K), (G, 1))                  # nothing moves
    yield np.zeros((G, K), int)                          # all from one
    yield np.tile((np.arange(K) + 1) % K, (G, 1))        # a cycle
    yield np.tile(np.arange(K)[::-1], (G, 1))
    for _ in range(3):
        yield r.integers(0, K, (G, K))


@pytest.mark.parametrize("G,K", [(1, 1), (2, 2), (3, 4), (2, 5), (1, 8), (2, 13), (1, 16), (2, 32)])
def test_reorder_against_oracle(G, K):
    g = torch.Generator().manual_seed(G * K)
    kinds = [((3, 16, 16), F32), ((7,), F32), ((4,), BF16), ((3,), BF16), ((5,), torch.uint8),
             ((1,), torch.uint8), ((260, 4), F32), ((9,), torch.int64), ((0,), F32),
             ((), torch.int32)]
    for p in maps(G, K, K):
        states = [torch.randint(0, 200, (G * K,) + shape, generator=g).to(dt).cuda()
                  for shape, dt in kinds]
        want = [beam.reorder(s.float().cpu().numpy(), p) for s in states]
        parents = torch.tensor(p, dtype=torch.int32, device="cuda")
        assert lib.gdn_state_reorder(states, parents) is states
        for s, w in zip(states, want):
            assert np.array_equal(s.float().cpu().numpy(), w)
    assert gdn.gdn_check_device_error() == gdn.GDN_OK


def test_reorder_leaves_its_surroundings():
    buf = torch.arange(40 * 7, dtype=F32, device="cuda").reshape(40, 7)
    before = buf.clone()
    lib.gdn_state_reorder(buf[9:21], torch.tensor([[1, 0, 2, 2]] * 3, dtype=torch.int32,
                                                  device="cuda"))
    assert torch.equal(buf[:9], before[:9]) and torch.equal(buf[21:], before[21:])
    assert np.array_equal(buf[9:21].cpu().numpy(),
                          beam.reorder(before[9:21].cpu().numpy(), np.array([[1, 0, 2, 2]] * 3)))


def test_reorder_reports_parents_out_of_range():
    s = torch.arange(24, dtype=F32, device="cuda").reshape(8, 3)
    p = torch.tensor([[1, 4, -1, 0], [3, 2, 1, 1 << 30]], dtype=torch.int32, device="cuda")
    want = beam.reorder(s.cpu().numpy(), p.cpu().numpy())
    lib.gdn_state_reorder(s, p)
    assert gdn.gdn_check_device_error() == gdn.GDN_ERR_INVALID_ARG
    assert gdn.gdn_check_device_error() == gdn.GDN_OK
    assert np.array_equal(s.cpu().numpy(), want)


def test_reorder_states_past_four_gigabytes():
    n = 12_000_003 * 4                    # bytes of a row; 96 rows
    s = torch.empty(96, n // 4, device="cuda")
    s[:, 0] = torch.arange(96, device="cuda")
    s[:, -1] = torch.arange(96, device="cuda") + 1000
    s[:, n // 8] = torch.arange(96, device="cuda") + 2000
    p = torch.tensor(np.random.default_rng(1).integers(0, 16, (6, 16)), dtype=torch.int32)
    at = (p.long() + 16 * torch.arange(6)[:, None]).flatten().float()
    lib.gdn_state_reorder(s, p.cuda())
    assert torch.equal(s[:, 0].cpu(), at) and torch.equal(s[:, -1].cpu(), at + 1000)
    assert torch.equal(s[:, n // 8].cpu(), at + 2000)


# --- a search -----------------------------------------------------------------

HQK, HV, D, C, V, G, K, STEPS = 1, 2, 32, 40, 601, 2, 4, 6


class Model:
    """One delta-rule mixer and one recurrence over embedding tables, a readout
    of both, random weights."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q, self.k, self.v = r(V, HQK, D), r(V, HQK, D), r(V, HV, D)
        self.la, self.be = -torch.rand(V, HV, generator=g), torch.rand(V, HV, generator=g)
        self.x, self.lc, self.bc = r(V, C), -torch.rand(V, C, generator=g), torch.rand(
            V, C, generator=g)
        self.w = r(HV * D + C, V) * 0.3
        self.S0, self.h0 = r(G, HV, D, D) * 0.1, r(G, C)

    def cuda(self):
        for k, v in vars(self).items():
            setattr(self, k, v.cuda())
        return self


def search_step(m, b):
    """One step of the search, all on the device: b holds its buffers."""
    t = b["token"].flatten().long()
    y = lib.gdn_decode_step(m.q[t], m.k[t], m.v[t], m.la[t], m.be[t], b["S"])
    z = lib.gdn_glr_step(m.x[t], m.lc[t], b["h"], m.bc[t])
    logits = torch.cat([y.flatten(1), z], 1) @ m.w
    lib.gdn_beam_select(logits.view(G, K, V), b["scores"], K, finished=b["finished"], end_token=0,
                        out=(b["scores"], b["parents"], b["token"], b["finished"]))
    lib.gdn_state_reorder([b["S"], b["h"], b["history"]], b["parents"])
    b["history"].scatter_(1, b["at"].expand(G * K, 1), b["token"].reshape(-1, 1))
    b["at"] += 1


def buffers(m):
    i32 = dict(dtype=torch.int32, device="cuda")
    scores = torch.full((G, K), -INF, device="cuda")
    scores[:, 0] = 0
    return dict(S=m.S0.repeat_interleave(K, 0).contiguous(),
                h=m.h0.repeat_interleave(K, 0).contiguous(), scores=scores,
                finished=torch.zeros(G, K, dtype=torch.uint8, device="cuda"),
                token=torch.tensor([[5] * K, [9] * K], **i32), parents=torch.zeros(G, K, **i32),
                history=torch.full((G * K, STEPS), -1, **i32),
                at=torch.zeros(1, dtype=torch.int64, device="cuda"))


def test_a_search_keeps_states_histories_and_scores_together():
    """Every surviving beam's states and score equal those of its own history
    run alone through the oracles."""
    m = Model(1).cuda()
    b = buffers(m)
    for _ in range(STEPS):
        search_step(m, b)
    assert gdn.gdn_check_device_error() == gdn.GDN_OK
    hist = b["history"].cpu().numpy()
    assert len({tuple(h) for h in hist[:K]}) == K          # four different continuations
    assert (np.diff(b["scores"].cpu().numpy(), axis=1) <= 0).all()
    for i in range(G * K):
        tok = np.concatenate([[5 if i < K else 9], hist[i][:-1]]).astype(int)
        f = lambda t: f64(t[torch.tensor(tok, device="cuda")])  # noqa: E731
        heads = lambda a: np.repeat(a, HV // HQK, 1)  # noqa: E731
        y, S = oracle.recurrence(heads(f(m.q)), heads(f(m.k)), f(m.v), f(m.la), f(m.be),
                                 initial_state=f64(m.S0[i // K])[None])
        r = glr.forward(f(m.x), f(m.lc), f(m.bc), f64(m.h0[i // K])[None])
        ref = np.asarray(S)[0]
        rel = np.linalg.norm(f64(b["S"][i]) - ref) / np.linalg.norm(ref)
        assert rel < 1e-4, (i, rel)                        # the library's fp32 bar
        assert (np.abs(f64(b["h"][i]) - r["final_state"][0]) <= r["final_bound"][0]).all(), i
        logits = np.concatenate([np.asarray(y).reshape(len(tok), -1), r["y"]], 1) @ f64(m.w)
        score, ended = 0.0, False
        for z, t in zip(logits, hist[i]):
            if not ended:
                score += z[t] - z.max() - np.log(np.exp(z - z.max()).sum())
            else:
                assert t == 0
            ended = ended or t == 0
        # fp32 (TF32-free) products of 104 terms, at the library's 1e-4 bar on y
        assert abs(score - float(b["scores"].flatten()[i])) < STEPS * 1e-3
        assert bool(b["finished"].flatten()[i]) == ended


def test_a_captured_search_equals_the_eager_one():
    m = Model(2).cuda()
    want, b = buffers(m), buffers(m)
    for _ in range(STEPS):
        search_step(m, want)
    fresh = {k: v.clone() for k, v in b.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        search_step(m, b)                                  # warm-up: library handles
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        search_step(m, b)
    for _ in range(2):                                     # the search, twice over
        for k, v in b.items():
            v.copy_(fresh[k])
        for _ in range(STEPS):
            g.replay()
        torch.cuda.synchronize()
        for k in ("S", "h", "scores", "finished", "token", "parents", "history"):
            assert torch.equal(b[k], want[k]), k
