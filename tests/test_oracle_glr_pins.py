"""Pins of the gated linear recurrence's oracle (CPU): closed forms, central
differences of every input, torch autograd in fp64, packing."""
import numpy as np
import pytest
import torch

from oracle import glr


def _case(seed, T, C, n, gate):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.sort(r.integers(0, T + 1, n - 1)), [T]])
    p = dict(x=r.normal(size=(T, C)), log_alpha=-r.exponential(size=(T, C)) * 0.3,
             h0=r.normal(size=(n, C)))
    beta = r.uniform(size=(T, C)) if gate == "beta" else gate
    if gate == "beta":
        p["beta"] = beta
    return p, beta, cu, r.normal(size=(T, C)), r.normal(size=(n, C))


def test_closed_forms():
    x = np.arange(1.0, 6.0)[:, None]
    f = glr.forward(x, np.zeros((5, 1)))
    assert np.array_equal(f["y"][:, 0], [1, 3, 6, 10, 15])          # a = 1: a cumulative sum
    f = glr.forward(x, np.full((5, 1), -np.inf))
    assert np.array_equal(f["y"], x)                                 # a = 0: nothing is kept
    f = glr.forward(np.zeros((4, 1)), np.full((4, 1), np.log(0.5)), h0=[[16.0]])
    assert np.allclose(f["y"][:, 0], [8, 4, 2, 1], rtol=1e-15)       # decay of h_0
    f = glr.forward(np.full((60, 1), 3.0), np.full((60, 1), np.log(0.5)), "complement")
    assert abs(f["final_state"][0, 0] - 3.0) < 1e-15                 # a moving average


@pytest.mark.parametrize("gate", [None, "beta", "complement"])
def test_gradients_match_differences(gate):
    p, beta, cu, dy, dhT = _case(3, 11, 2, 4, gate)

    def loss(q):
        f = glr.forward(q["x"], q["log_alpha"], q.get("beta", beta), q["h0"], cu)
        return (f["y"] * dy).sum() + (f["final_state"] * dhT).sum()

    out, _ = glr.backward(p["x"], p["log_alpha"], dy, beta, p["h0"], dhT, cu)
    grads = dict(x=out["dx"], log_alpha=out["dlog_alpha"], beta=out["dbeta"],
                 h0=out["d_initial_state"])
    h = 1e-5
    for name, v in p.items():
        for i in np.ndindex(v.shape):
            ls = []
            for d in (h, -h):
                q = dict(p, **{name: v.copy()})
                q[name][i] += d
                ls.append(loss(q))
            # central differences: h^2 of the third derivative, and rounding / h
            assert abs((ls[0] - ls[1]) / (2 * h) - grads[name][i]) < 1e-8, (name, i)


@pytest.mark.parametrize("gate", [None, "beta", "complement"])
def test_gradients_match_autograd(gate):
    p, beta, cu, dy, dhT = _case(5, 40, 3, 6, gate)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in p.items()}
    a = t["log_alpha"].exp()
    b = t["beta"] if gate == "beta" else (1 - a if gate else torch.ones_like(a))
    loss = 0.0
    for s in range(len(cu) - 1):
        h = t["h0"][s]
        for i in range(cu[s], cu[s + 1]):
            h = a[i] * h + b[i] * t["x"][i]
            loss = loss + (h * torch.tensor(dy[i])).sum()
        loss = loss + (h * torch.tensor(dhT[s])).sum()
    loss.backward()
    out, _ = glr.backward(p["x"], p["log_alpha"], dy, beta, p["h0"], dhT, cu)
    grads = dict(x=out["dx"], log_alpha=out["dlog_alpha"], beta=out["dbeta"],
                 h0=out["d_initial_state"])
    for k in p:
        assert np.allclose(t[k].grad.numpy(), grads[k], rtol=1e-12, atol=1e-12), k


def test_packing_equals_separate_sequences():
    p, beta, cu, _, _ = _case(7, 30, 2, 5, "beta")
    f = glr.forward(p["x"], p["log_alpha"], beta, p["h0"], cu)
    for s in range(len(cu) - 1):
        lo, hi = cu[s], cu[s + 1]
        g = glr.forward(p["x"][lo:hi], p["log_alpha"][lo:hi], beta[lo:hi], p["h0"][s:s + 1])
        assert np.array_equal(f["y"][lo:hi], g["y"])
        assert np.array_equal(f["final_state"][s], g["final_state"][0])


def test_fp32_recurrence_stays_inside_the_bound():
    """A plain fp32 evaluation, and one composed from runs of 8 tokens."""
    p, _, _, _, _ = _case(9, 400, 16, 1, None)
    x, la = p["x"].astype(np.float32), (p["log_alpha"] * 0.01).astype(np.float32)
    f = glr.forward(x, la)
    a = np.exp(la.astype(np.float64)).astype(np.float32)
    h = np.zeros(16, np.float32)
    carry = np.zeros(16, np.float32)
    for t0 in range(0, 400, 8):
        A, g = np.ones(16, np.float32), np.zeros(16, np.float32)
        for t in range(t0, t0 + 8):
            h = a[t] * h + x[t]
            A, g = A * a[t], a[t] * g + x[t]
            assert (np.abs(h - f["y"][t]) <= f["y_bound"][t]).all()
        carry = A * carry + g
        assert (np.abs(carry - f["y"][t0 + 7]) <= f["y_bound"][t0 + 7]).all()
