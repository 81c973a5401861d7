"""Beam search's choice and the reordering of states, in plain numpy (fp64).
Independent of the CUDA path.  Used by the tests only."""
import numpy as np


def table(logits, scores, finished=None, end_token=-1):
    """c[k, v] = scores[k] + ((x - top) - log sum exp(x - top)) of one group:
    logits [K, V].  NaN logits count as -inf, +inf ones share their row; a
    finished beam has its end token alone, at its score; beams with a score
    that is not finite, and rows of -inf, are -inf throughout."""
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    c = np.full(x.shape, -np.inf)
    for k in range(x.shape[0]):
        s = float(scores[k])
        if not np.isfinite(s):
            continue
        if finished is not None and finished[k]:
            c[k, end_token] = s
            continue
        top = x[k].max()
        if top == -np.inf:
            continue
        if top == np.inf:
            c[k] = np.where(x[k] == np.inf, s - np.log((x[k] == np.inf).sum()), -np.inf)
            continue
        d = x[k] - top
        c[k] = s + (d - np.log(np.exp(d).sum()))
    return c


def select(logits, scores, M, finished=None, end_token=-1):
    """(scores, parents, tokens, finished) of one group, best first; ties to
    the lowest k V + v."""
    c = table(logits, scores, finished, end_token).reshape(-1)
    V = np.shape(logits)[1]
    at = np.argsort(-c, kind="stable")[:M]
    done = np.zeros(len(scores), bool) if finished is None else np.asarray(finished, bool)
    parents, tokens = at // V, at % V
    return c[at], parents, tokens, done[parents] | (tokens == end_token)


def reorder(state, parents):
    """Rows of state [G * K, ...] after the move; out-of-range parents stay."""
    G, K = parents.shape
    out = state.copy()
    for g in range(G):
        for j in range(K):
            p = int(parents[g, j])
            if 0 <= p < K:
                out[g * K + j] = state[g * K + p]
    return out
