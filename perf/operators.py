"""Workloads of the recurrence and beam-search operators, and their plain forms.

Operators (see include/gdn.h for the calls):

- fwd:     the gated linear recurrence h_t = a_t h_{t-1} + b_t x_t over packed
           sequences, per channel, with a = exp(log_alpha) and b = 1, a given
           gate, or 1 - a (prefill).
- train:   that forward and its backward, as one training step makes them.
- step:    one token per sequence, the state updated in place (decode).
- select:  beam search's choice of the best continuations over beams and
           vocabulary.
- reorder: the recurrent states of the surviving beams moved in place.

`run` computes the plain form in elementary torch operations where `own` is
false and calls the library where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a short prompt of one request: latency counts
        dict(name="fwd_prompt_128", op="fwd", T=128, C=2560, n_seq=1, gate="beta", dtype="bf16"),
        # one 4k-token prefill, 48 heads x 128 channels
        dict(name="fwd_prefill_4k", op="fwd", T=4096, C=6144, n_seq=1, gate="beta", dtype="bf16"),
        # a long document at the model width, 1 - a as the input gate
        dict(name="fwd_long_128k", op="fwd", T=131072, C=2560, n_seq=1, gate="complement",
             dtype="bf16"),
        # a ragged packed batch of prompts in fp32 with an odd width
        dict(name="fwd_packed_odd", op="fwd", T=20011, C=1333, n_seq=24, gate="none",
             dtype="fp32"),
        # a training step on one 4k sequence
        dict(name="train_4k", op="train", T=4096, C=2560, n_seq=1, gate="beta", dtype="bf16"),
        # a training step on a packed batch, 48 heads x 128 channels
        dict(name="train_packed_32k", op="train", T=32768, C=6144, n_seq=24, gate="beta",
             dtype="bf16"),
        # decode of a few sequences, and of the large decode batch
        dict(name="step_3", op="step", N=3, C=2561, gate="beta", dtype="bf16"),
        dict(name="step_256", op="step", N=256, C=6144, gate="beta", dtype="bf16"),
        # one request with four beams; a batch of requests over a large vocabulary whose rows
        # are padded in memory
        dict(name="select_1x4", op="select", G=1, K=4, V=32000, pad=0, M=8, dtype="bf16"),
        dict(name="select_32x8", op="select", G=32, K=8, V=130001, pad=47, M=16, dtype="bf16"),
        # the states of two requests' beams (d = 128, 48 heads); of the large decode batch
        dict(name="reorder_2x4", op="reorder", G=2, K=4, H=48, d=128, C=2560, pattern="halve"),
        dict(name="reorder_32x8", op="reorder", G=32, K=8, H=48, d=128, C=6144,
             pattern="halve"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "train", "step", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("fwd", "train"):
        C = _log_int(rng, 64, 8192)
        T = _log_int(rng, 1, min(131072, (1 << 26) // C))
        return dict(op=op, T=T, C=C, n_seq=rng.randint(1, max(1, min(64, T))),
                    gate=rng.choice(["none", "beta", "complement"]), dtype=dtype)
    if op == "step":
        return dict(op=op, N=_log_int(rng, 1, 1024), C=_log_int(rng, 64, 8192),
                    gate=rng.choice(["none", "beta", "complement"]), dtype=dtype)
    K = rng.randint(1, 16)
    if op == "select":
        V = _log_int(rng, 1000, 260000)
        return dict(op=op, G=_log_int(rng, 1, max(1, min(256, (1 << 25) // (K * V)))), K=K, V=V,
                    pad=rng.choice([0, 0, rng.randint(1, 127)]), M=rng.choice([K, 2 * K]),
                    dtype=dtype)
    d = rng.choice([64, 128])
    return dict(op=op, G=_log_int(rng, 1, max(1, 256 // K)), K=K, H=rng.randint(1, 48), d=d,
                C=_log_int(rng, 64, 8192), pattern=rng.choice(["halve", "shift"]))


# --- inputs ------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _gates(shape, C, g, dtype):
    """log_alpha: -softplus(N(0, 1)) times a channel's rate, log-uniform in [1e-3, 1], so that
    channels remember between about one token and a thousand."""
    rate = torch.exp(torch.rand(C, generator=g, device="cuda") * math.log(1e-3))
    z = torch.randn(shape, generator=g, device="cuda")
    return (-torch.nn.functional.softplus(z) * rate).to(dtype)


def _cu_seqlens(T, n_seq, g):
    cuts = torch.randint(0, T + 1, (n_seq - 1,), generator=g, device="cuda").sort().values
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _parents(case, g):
    """Parents of every group: "halve": half the beams survive, two children each; "shift":
    every beam moves.  The beams of each group are numbered in an order of its own."""
    G, K = case["G"], case["K"]
    j = torch.arange(K, device="cuda")
    p = j // 2 if case["pattern"] == "halve" else (j + 1) % K
    order = torch.rand(G, K, generator=g, device="cuda").argsort(1)
    out = torch.empty(G, K, dtype=torch.int64, device="cuda")
    out.scatter_(1, order, order[:, p])
    return out.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if op in ("fwd", "train", "step"):
        dt = DTYPES[case["dtype"]]
        C = case["C"]
        n = case["N"] if op == "step" else case["T"]
        s["x"] = randn(n, C).to(dt)
        s["log_alpha"] = _gates((n, C), C, g, dt)
        s["beta"] = torch.sigmoid(randn(n, C)).to(dt) if case["gate"] == "beta" else None
        rows = n if op == "step" else case["n_seq"]
        s["h0"] = randn(rows, C)
        if op != "step":
            s["cu"] = _cu_seqlens(case["T"], case["n_seq"], g) if case["n_seq"] > 1 else None
        if op == "train":
            s["dy"] = randn(n, C).to(dt)
            s["dhT"] = randn(rows, C)
    elif op == "select":
        G, K, V, ld = case["G"], case["K"], case["V"], case["V"] + case["pad"]
        # the rows of a language model's logits: some 2.5 wide, a few tokens far above
        z = randn(G * K * ld).mul_(2.5).to(DTYPES[case["dtype"]])
        s["logits"] = z.as_strided((G, K, V), (K * ld, ld, 1))
        s["scores"] = -10.0 * torch.rand(G, K, generator=g, device="cuda")
        s["finished"] = (torch.rand(G, K, generator=g, device="cuda") < 0.15).to(torch.uint8)
        s["end_token"] = 2
    else:
        n = case["G"] * case["K"]
        H, d = case["H"], case["d"]
        s["S"] = randn(n, H, d, d)
        s["conv"] = randn(n, H, 3, 3 * d)
        s["h"] = randn(n, case["C"])
        s["parents"] = _parents(case, g)
    return s


# --- one pass ----------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    if op == "fwd":
        return _plain_forward(s)[:2]
    if op == "train":
        return _plain_train(s)
    if op == "step":
        return _plain_step(s)
    if op == "select":
        return _plain_select(s)
    return _plain_reorder(s)


def _own(op, s):
    import gated_deltanet_scan_chunked_b200 as lib

    if op in ("fwd", "train", "step"):
        beta = "complement" if s["case"]["gate"] == "complement" else s["beta"]
    if op == "fwd":
        y, h, _ = lib.gdn_glr_fwd(s["x"], s["log_alpha"], beta, initial_state=s["h0"],
                                  cu_seqlens=s["cu"])
        return y, h
    if op == "train":
        y, h, ckpt = lib.gdn_glr_fwd(s["x"], s["log_alpha"], beta, initial_state=s["h0"],
                                     cu_seqlens=s["cu"], checkpoints=True)
        d = lib.gdn_glr_bwd(s["x"], s["log_alpha"], s["dy"], beta, initial_state=s["h0"],
                            d_final_state=s["dhT"], cu_seqlens=s["cu"], checkpoints=ckpt)
        return y, h, d["dx"], d["dlog_alpha"], d.get("dbeta"), d["d_initial_state"]
    if op == "step":
        y = lib.gdn_glr_step(s["x"], s["log_alpha"], s["h0"], beta)
        return y, s["h0"]
    if op == "select":
        return lib.gdn_beam_select(s["logits"], s["scores"], s["case"]["M"],
                                   finished=s["finished"], end_token=s["end_token"])
    lib.gdn_state_reorder([s["S"], s["conv"], s["h"]], s["parents"])
    return s["S"], s["conv"], s["h"]


# --- plain forms (32 bits, rounded once at the end) ---------------------------


def _decay_and_gate(s):
    la = s["log_alpha"].float()
    # exp in 64 bits: an error of a in one direction adds up over a thousand tokens
    a = torch.exp(la.double()).float()
    gate = s["case"]["gate"]
    b = s["beta"].float() if gate == "beta" else -torch.expm1(la) if gate == "complement" else None
    return a, b


def _packing(s):
    """Of every token: its sequence, whether it is the first, the last (as columns); of every
    sequence: its first and last token and whether it has any."""
    T = s["x"].shape[0]
    cu = torch.tensor([0, T], device="cuda") if s["cu"] is None else s["cu"].long()
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    is_first, is_last = (t == cu[seq])[:, None], (t == cu[seq + 1] - 1)[:, None]
    first, last = cu[:-1].clamp(max=T - 1), (cu[1:] - 1).clamp(min=0)
    return seq, is_first, is_last, first, last, (cu[1:] > cu[:-1])[:, None]


def _scan(a, b):
    """All h_t = a_t h_{t-1} + b_t along dimension 0 (h_{-1} = 0), by doubling."""
    d, n = 1, a.shape[0]
    while d < n:
        b = torch.cat([b[:d], torch.addcmul(b[d:], a[d:], b[:-d])])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_forward(s):
    a, b = _decay_and_gate(s)
    seq, is_first, is_last, first, last, some = where = _packing(s)
    x = s["x"].float()
    u = x if b is None else b * x
    u = torch.where(is_first, torch.addcmul(u, a, s["h0"][seq]), u)
    h = _scan(a * ~is_first, u)
    return h.to(s["x"].dtype), torch.where(some, h[last], s["h0"]), (h, a, b, x, where)


def _plain_train(s):
    y, hT, (h, a, b, x, (seq, is_first, is_last, first, last, some)) = _plain_forward(s)
    dt, gate = s["x"].dtype, s["case"]["gate"]
    dy = s["dy"].float() + torch.where(is_last, s["dhT"][seq], 0.0)
    # e_t = a_t (dy_t + e_{t+1}), cut behind each sequence's last token
    e = _scan((a * ~is_last).flip(0), (a * dy).flip(0)).flip(0)
    dh = dy + torch.cat([e[1:], e[:1]]) * ~is_last
    before = torch.where(is_first, s["h0"][seq], torch.cat([h[:1], h[:-1]]))
    dx = (dh if b is None else b * dh).to(dt)
    dla = (a * (before - x if gate == "complement" else before) * dh).to(dt)
    dbeta = (x * dh).to(dt) if gate == "beta" else None
    return y, hT, dx, dla, dbeta, torch.where(some, e[first], s["dhT"])


def _plain_step(s):
    a, b = _decay_and_gate(s)
    x = s["x"].float()
    h = a * s["h0"] + (x if b is None else b * x)
    s["h0"].copy_(h)
    return h.to(s["x"].dtype), s["h0"]


def _plain_select(s):
    # 64 bits: which candidate is chosen goes by differences near 32-bit rounding
    z = s["logits"].double()
    top = z.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(-1, keepdim=True))
    logp = z - lse
    done = s["finished"].bool()
    only_end = torch.full_like(logp[:1, :1], -math.inf)
    only_end[..., s["end_token"]] = 0
    logp = torch.where(done[..., None], only_end, logp)
    total = (s["scores"].double()[..., None] + logp).flatten(1)
    order = torch.sort(total, dim=1, descending=True, stable=True)
    M, V = s["case"]["M"], s["case"]["V"]
    at = order.indices[:, :M]
    parents, tokens = at // V, at % V
    ended = (done.gather(1, parents) | (tokens == s["end_token"])).to(torch.uint8)
    return (order.values[:, :M].float(), parents.to(torch.int32), tokens.to(torch.int32), ended)


def _plain_reorder(s):
    K = s["case"]["K"]
    G = s["case"]["G"]
    at = (s["parents"].long() + torch.arange(G, device="cuda")[:, None] * K).flatten()
    for name in ("S", "conv", "h"):
        s[name].copy_(s[name][at])
    return s["S"], s["conv"], s["h"]


# --- what a pass cannot do without -------------------------------------------


def work(case):
    op = case["op"]
    if op in ("fwd", "train", "step"):
        es = 2 if case["dtype"] == "bf16" else 4
        ins = 3 if case["gate"] == "beta" else 2
        n = (case["N"] if op == "step" else case["T"]) * case["C"]
        states = 8 * case["C"] * (case["N"] if op == "step" else case["n_seq"])
        if op == "train":
            # forward, then inputs and dy read, a gradient of each input written
            return dict(bytes=n * es * (ins + 1 + ins + 1 + ins) + 2 * states, flops=14 * n)
        return dict(bytes=n * es * (ins + 1) + states, flops=4 * n)
    if op == "select":
        n = case["G"] * case["K"] * case["V"]
        return dict(bytes=n * (2 if case["dtype"] == "bf16" else 4)
                    + case["G"] * (5 * case["K"] + 13 * case["M"]), flops=4 * n)
    K = case["K"]
    row = 4 * (case["H"] * case["d"] * (case["d"] + 9) + case["C"])
    if case["pattern"] == "halve":  # beam 0 stays; the others are written, (K + 1) // 2 read
        moved, read = K - 1, (K + 1) // 2 if K > 1 else 0
    else:
        moved = read = K if K > 1 else 0
    return dict(bytes=case["G"] * ((moved + read) * row + 4 * K), flops=0)


# --- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return _exact_select(s)
    if op == "reorder":
        return _exact_reorder(s)
    la = s["log_alpha"].to(torch.float64)
    alpha = la.exp()
    x = s["x"].to(torch.float64)
    if case["gate"] == "beta":
        w = s["beta"].to(torch.float64)
    elif case["gate"] == "complement":
        w = -la.expm1()
    else:
        w = torch.ones_like(x)
    h0 = s["h0"].to(torch.float64)
    if op == "step":
        h = alpha * h0 + w * x
        return h, h
    T = case["T"]
    cu = [0, T] if s["cu"] is None else s["cu"].tolist()
    h = torch.empty_like(x)
    hT = h0.clone()
    wx = w * x
    for n in range(len(cu) - 1):  # token by token, sequence by sequence
        prev = h0[n]
        for t in range(cu[n], cu[n + 1]):
            prev = torch.addcmul(wx[t], alpha[t], prev, out=h[t])
        hT[n] = prev
    if op == "fwd":
        return h, hT
    del wx
    dh = s["dy"].to(torch.float64)
    dh0 = s["dhT"].to(torch.float64)
    dalpha = torch.empty_like(x)
    for n in range(len(cu) - 1):
        lo, hi = cu[n], cu[n + 1]
        if lo == hi:
            continue
        dh[hi - 1] += dh0[n]
        for t in range(hi - 2, lo - 1, -1):
            dh[t].addcmul_(alpha[t + 1], dh[t + 1])
        torch.mul(dh[lo], h0[n], out=dalpha[lo])
        torch.mul(dh[lo + 1:hi], h[lo:hi - 1], out=dalpha[lo + 1:hi])
        dh0[n] = alpha[lo] * dh[lo]
    if case["gate"] == "complement":
        dalpha -= x * dh
    dbeta = x * dh if case["gate"] == "beta" else None
    return h, hT, w * dh, alpha * dalpha, dbeta, dh0


def _exact_select(s):
    G, K, V, M = (s["case"][k] for k in ("G", "K", "V", "M"))
    end = s["end_token"]
    vals, rows, toks, ends = [], [], [], []
    for i in range(G):
        table = torch.empty(K, V, dtype=torch.float64, device="cuda")
        for k in range(K):
            if s["finished"][i, k]:
                table[k].fill_(-math.inf)
                table[k, end] = 0
            else:
                z = s["logits"][i, k].to(torch.float64)
                table[k] = z - torch.logsumexp(z, 0)
            table[k] += s["scores"][i, k].to(torch.float64)
        flat = table.reshape(-1)
        for _ in range(M):
            best = flat[~flat.isnan()].max()
            at = int(torch.nonzero(flat == best)[0])
            vals.append(float(best))
            rows.append(at // V)
            toks.append(at % V)
            ends.append(bool(s["finished"][i, at // V]) or at % V == end)
            flat[at] = math.nan  # taken
    back = lambda v, t: torch.tensor(v, dtype=t, device="cuda").reshape(G, M)  # noqa: E731
    return (back(vals, torch.float64), back(rows, torch.int32), back(toks, torch.int32),
            back(ends, torch.uint8))


def _exact_reorder(s):
    K = s["case"]["K"]
    p = s["parents"].tolist()
    out = []
    for name in ("S", "conv", "h"):
        old = s[name]
        rows = [old[g * K + p[g][j]] for g in range(len(p)) for j in range(K)]
        out.append(torch.stack(rows).to(torch.float64) if old.numel() < 1 << 28
                   else torch.stack(rows))
    return tuple(out)
