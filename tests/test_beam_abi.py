"""Host-side refusals of the beam-search entry points, and pins of their
numpy oracle (CPU)."""
import ctypes

import numpy as np
import pytest

from gated_deltanet_scan_chunked_b200 import build as gbuild
from gated_deltanet_scan_chunked_b200 import gdn
from oracle import beam

FAKE = 0x1000
MB = 1 << 20
BAD, UNSUP, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def at(i):
    return FAKE + i * 256 * MB


def _select(lib, **kw):
    a = dict(x=at(1), ld=1000, s=at(2), f=at(3), end=7, G=2, K=4, V=1000, M=8, dt=0, os=at(4),
             op=at(5), ot=at(6), of=at(7))
    a.update(kw)
    return lib.gdn_beam_select(a["x"], a["ld"], a["s"], a["f"], a["end"], a["G"], a["K"], a["V"],
                               a["M"], a["dt"], a["os"], a["op"], a["ot"], a["of"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(s=None), BAD), (dict(os=None), BAD), (dict(op=None), BAD),
    (dict(ot=None), BAD), (dict(x=at(1) + 1), BAD), (dict(dt=1, x=at(1) + 2), BAD),
    (dict(s=at(2) + 2), BAD), (dict(ot=at(6) + 1), BAD),
    (dict(ld=999), BAD), (dict(ld=1 << 62), BAD), (dict(end=1000), BAD), (dict(end=-2), BAD),
    (dict(end=-1), BAD),                                   # finished beams without an end token
    (dict(G=-1), BAD), (dict(K=0), BAD), (dict(V=0), BAD), (dict(M=0), BAD),
    (dict(V=1, ld=1, end=0, M=5), BAD),                    # fewer candidates than asked for
    (dict(K=33), UNSUP), (dict(M=65), UNSUP), (dict(dt=2), UNSUP),
    (dict(K=32, V=1 << 26, ld=1 << 26), UNSUP),            # K V = 2^31
    (dict(G=65536), UNSUP),
    (dict(os=at(2)), BAD),                                 # in place needs M = K
    (dict(of=at(3)), BAD), (dict(op=at(4)), BAD), (dict(os=at(1) + 64), BAD),
    (dict(M=4, os=at(2) + 4), BAD),                        # a partial overlap
    (dict(M=4, op=at(2)), BAD),
    (dict(G=0, x=None, s=None, os=None), OK),
])
def test_select_rejects(lib, kw, code):
    assert _select(lib, **kw) == code


def _reorder(lib, ptrs=(at(1),), sizes=(64,), parents=at(9), G=2, K=4, n=None):
    n = len(ptrs) if n is None else n
    p = (ctypes.c_void_p * max(n, 1))(*ptrs)
    s = (ctypes.c_size_t * max(n, 1))(*sizes)
    return lib.gdn_state_reorder(p, s, n, parents, G, K, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ptrs=(None,)), BAD), (dict(parents=None), BAD), (dict(parents=at(9) + 2), BAD),
    (dict(G=-1), BAD), (dict(K=0), BAD), (dict(K=33), UNSUP), (dict(n=0), BAD),
    (dict(ptrs=(at(1),) * 17, sizes=(64,) * 17), UNSUP),
    (dict(ptrs=(at(1), at(1) + 504), sizes=(64, 64)), BAD),   # overlapping states
    (dict(ptrs=(at(9) - 500,)), BAD),                          # a state over the parents
    (dict(sizes=(1 << 60,)), BAD),
    (dict(G=0, ptrs=(None,), parents=None), OK),
    (dict(ptrs=(None,), sizes=(0,)), OK),                      # rows without bytes
])
def test_reorder_rejects(lib, kw, code):
    assert _reorder(lib, **kw) == code


def test_reorder_rejects_null_arrays(lib):
    assert lib.gdn_state_reorder(None, None, 1, at(9), 2, 4, None) == BAD


def test_binding_refuses_cpu_tensors(lib):
    import torch
    with pytest.raises(ValueError):
        gdn.gdn_beam_select(torch.zeros(1, 2, 5), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        gdn.gdn_state_reorder(torch.zeros(2, 5), torch.zeros(1, 2, dtype=torch.int32))


# --- pins of the oracle -----------------------------------------------------


def test_oracle_by_hand():
    # two beams over three tokens, probabilities 1/2 1/4 1/4 and 1/8 1/8 3/4
    x = np.log([[2.0, 1.0, 1.0], [1.0, 1.0, 6.0]])
    s = np.log([0.5, 0.5])
    c, p, t, f = beam.select(x, s, 6, end_token=2)
    assert np.allclose(np.exp(c), [0.375, 0.25, 0.125, 0.125, 0.0625, 0.0625])
    assert p.tolist() == [1, 0, 0, 0, 1, 1] and t.tolist() == [2, 0, 1, 2, 0, 1]
    assert f.tolist() == [True, False, False, True, False, False]


def test_oracle_probabilities_sum_to_the_scores():
    r = np.random.default_rng(0)
    x, s = r.normal(size=(3, 50)) * 4, r.normal(size=3)
    c = beam.table(x, s)
    assert np.allclose(np.exp(c).sum(1), np.exp(s))
    # a shift of a row's logits changes nothing
    assert np.allclose(beam.table(x + [[100.0], [-7.0], [0.5]], s), c)


def test_oracle_finished_dead_and_empty():
    x = np.array([[1.0, 2.0], [3.0, 1.0], [-np.inf, -np.inf]])
    c, p, t, f = beam.select(x, [-1.0, -np.inf, 0.0], 4, finished=[1, 0, 0], end_token=1)
    assert c[0] == -1.0 and (c[1:] == -np.inf).all()
    assert list(zip(p, t)) == [(0, 1), (0, 0), (1, 0), (1, 1)]


def test_oracle_reorder():
    s = np.arange(12).reshape(6, 2)
    out = beam.reorder(s, np.array([[2, 2, 0], [1, 0, 5]]))
    assert out[:, 0].tolist() == [4, 4, 0, 8, 6, 10]
