"""Gated linear recurrence in fp64 numpy, token by token, with elementwise
bounds on what fp32 arithmetic can be off.

    h_t = a_t h_{t-1} + b_t x_t,  a = exp(log_alpha),  b = 1 | beta | 1 - a

Independent of the CUDA path.  Used by the tests only.
"""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def gates(log_alpha, beta):
    """(a, b) from log_alpha and beta (None, "complement" or an array)."""
    la = _f64(log_alpha)
    a = np.exp(la)
    if beta is None:
        return a, np.ones_like(a)
    if isinstance(beta, str):
        assert beta == "complement"
        return a, -np.expm1(la)
    return a, _f64(beta)


def forward(x, log_alpha, beta=None, h0=None, cu=None):
    """y [T, C], final state [n, C], the state before every token [T, C], and
    bounds on the error of y and of the final state in fp32.

    The bound follows the recurrence.  Let H be the recurrence on absolute
    values.  In units of U, a token's a is off by at most 4 + 2 |l| relative
    (near 0 the series and one rounding; further out 2^x to 2^-22, its
    argument l log2(e) rounded), at most doubled where a enters through the
    product of a run as well as through the token itself, with one rounding
    of that product; b x by 20 (1 - a at |l| >= 1/4 is a difference that
    loses at most 1/(1 - 0.78) of a's 4 U), and the sum by 2.  Hence
        E_t = a E_{t-1} + U ((10 + 4 |l|) a H_{t-1} + 20 |b x| + 2 H_t).
    (|l| is capped at 104, behind which a is 0 in fp32.)
    """
    x, la = _f64(x), _f64(log_alpha)
    a, b = gates(log_alpha, beta)
    T, C = x.shape
    cu = [0, T] if cu is None else [int(v) for v in cu]
    n = len(cu) - 1
    h0 = np.zeros((n, C)) if h0 is None else _f64(h0)
    kap = 10.0 + 4.0 * np.minimum(np.abs(la), 104.0)
    y, before, ey = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    hT, eT = h0.copy(), np.zeros_like(h0)
    for s in range(n):
        h, H, E = h0[s].copy(), np.abs(h0[s]), np.zeros(C)
        for t in range(cu[s], cu[s + 1]):
            before[t] = h
            bx = b[t] * x[t]
            h = np.where(a[t] == 0, 0.0, a[t] * h) + bx
            Hn = np.where(a[t] == 0, 0.0, a[t] * H) + np.abs(bx)
            E = a[t] * E + U * (kap[t] * a[t] * H + 20 * np.abs(bx) + 2 * Hn)
            H = Hn
            y[t], ey[t] = h, E
        hT[s], eT[s] = h, E
    return dict(y=y, final_state=hT, before=before, y_bound=ey, final_bound=eT)


def backward(x, log_alpha, dy, beta=None, h0=None, dhT=None, cu=None):
    """Gradients and their fp32 bounds: e_t = a_t dh_t, dh_t = dy_t + e_{t+1},
    dx = b dh, dbeta = x dh, dlog_alpha = h_{t-1} e (b = 1 - a: (h_{t-1} - x)
    e), dh_0 = the first token's e.  The bound on e is the forward's, run
    backwards; products add the bounds of their factors and a rounding."""
    f = forward(x, log_alpha, beta, h0, cu)
    x, la, dy = _f64(x), _f64(log_alpha), _f64(dy)
    a, b = gates(log_alpha, beta)
    T, C = x.shape
    cu = [0, T] if cu is None else [int(v) for v in cu]
    n = len(cu) - 1
    dhT = np.zeros((n, C)) if dhT is None else _f64(dhT)
    kap = 10.0 + 4.0 * np.minimum(np.abs(la), 104.0)
    comp = isinstance(beta, str)
    # the bound on h before a token: the forward's of the token before (0 for h_0)
    eb = np.zeros_like(x)
    out = {k: np.zeros_like(x) for k in ("dx", "dlog_alpha", "dbeta")}
    bound = {k: np.zeros_like(x) for k in out}
    dh0, e0 = dhT.copy(), np.zeros_like(dhT)
    for s in range(n):
        lo, hi = cu[s], cu[s + 1]
        if lo == hi:
            continue
        eb[lo + 1:hi] = f["y_bound"][lo:hi - 1]
        e, R, E = dhT[s].copy(), np.abs(dhT[s]), np.zeros(C)
        for t in range(hi - 1, lo - 1, -1):
            dh = dy[t] + e
            adh = np.abs(dy[t]) + R
            edh = E + 2 * U * adh
            e = a[t] * dh
            R = a[t] * adh
            E = a[t] * edh + U * kap[t] * R
            hb = f["before"][t] - (x[t] if comp else 0.0)
            ahb = np.abs(f["before"][t]) + (np.abs(x[t]) if comp else 0.0)
            out["dx"][t] = b[t] * dh
            bound["dx"][t] = np.abs(b[t]) * (edh + 20 * U * np.abs(dh))
            out["dbeta"][t] = x[t] * dh
            bound["dbeta"][t] = np.abs(x[t]) * (edh + 2 * U * np.abs(dh))
            out["dlog_alpha"][t] = np.where(a[t] == 0, 0.0, hb * e)
            bound["dlog_alpha"][t] = (ahb + eb[t]) * (E + 2 * U * np.abs(e)) \
                + eb[t] * np.abs(e)
        dh0[s], e0[s] = e, E
    out["d_initial_state"], bound["d_initial_state"] = dh0, e0
    return out, bound
