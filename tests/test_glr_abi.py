"""Host-side refusals of the gated linear recurrence's entry points (CPU)."""
import pytest

from gated_deltanet_scan_chunked_b200 import build as gbuild
from gated_deltanet_scan_chunked_b200 import gdn

FAKE = 0x1000  # 16-byte aligned, never dereferenced
MB = 1 << 20
BAD, UNSUP = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def at(i):
    return FAKE + i * 64 * MB


def _fwd(lib, **kw):
    a = dict(x=at(1), la=at(2), be=at(3), gate=1, h0=at(4), cu=at(5), n=2, T=64, C=100, dt=0,
             y=at(6), hT=at(7), ck=None)
    a.update(kw)
    return lib.gdn_glr_fwd(a["x"], a["la"], a["be"], a["gate"], a["h0"], a["cu"], a["n"], a["T"],
                           a["C"], a["dt"], a["y"], a["hT"], a["ck"], None)


PACKED = [
    (dict(x=None), BAD), (dict(la=None), BAD), (dict(be=None), BAD),
    (dict(gate=0), BAD),                       # a beta that the gate does not use
    (dict(gate=2), BAD), (dict(gate=3, be=None), BAD), (dict(gate=-1, be=None), BAD),
    (dict(n=0), BAD), (dict(cu=None), BAD),    # two sequences need offsets
    (dict(cu=at(5) + 2), BAD), (dict(T=-1), BAD), (dict(T=1 << 31), BAD),
    (dict(C=0), BAD), (dict(C=-5), BAD), (dict(C=65535 * 32 + 1), UNSUP),
    (dict(dt=2), UNSUP), (dict(dt=-1), UNSUP),
    (dict(x=at(1) + 8), BAD), (dict(h0=at(4) + 4), BAD),
    (dict(n=(1 << 30) + 1), UNSUP),
]


@pytest.mark.parametrize("kw,code", PACKED + [
    (dict(y=None), BAD), (dict(y=at(1)), BAD),            # y on x
    (dict(y=at(2) + 16), BAD), (dict(hT=at(4) + 16), BAD),  # a partial overlap of the state
    (dict(ck=at(6) + 64), BAD),                           # checkpoints inside y
    (dict(hT=at(7) + 2), BAD),
    (dict(y=at(5)), BAD), (dict(hT=at(5) - 16), BAD), (dict(ck=at(5)), BAD),  # on the offsets
])
def test_forward_rejects(lib, kw, code):
    assert _fwd(lib, **kw) == code


def _bwd(lib, **kw):
    a = dict(x=at(1), la=at(2), be=at(3), gate=1, h0=at(4), cu=at(5), n=2, T=64, C=100, dt=0,
             dy=at(6), dhT=at(7), ck=at(8), dx=at(9), dla=at(10), dbe=at(11), dh0=at(12), ws=None,
             wsb=0)
    a.update(kw)
    return lib.gdn_glr_bwd(a["x"], a["la"], a["be"], a["gate"], a["h0"], a["cu"], a["n"], a["T"],
                           a["C"], a["dt"], a["dy"], a["dhT"], a["ck"], a["dx"], a["dla"],
                           a["dbe"], a["dh0"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", PACKED + [
    (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dla=None), BAD), (dict(dbe=None), BAD),
    (dict(gate=0, be=None), BAD),                         # dbeta without a beta
    (dict(ck=None), BAD),                                 # neither checkpoints nor workspace
    (dict(ck=None, ws=at(13), wsb=64), BAD),              # too small
    (dict(ck=None, ws=at(13) + 16, wsb=MB), BAD),         # not 256-byte aligned
    (dict(ck=None, ws=at(9), wsb=MB), BAD),               # the workspace on an output
    (dict(dx=at(6)), BAD), (dict(dx=at(10)), BAD), (dict(dh0=at(7)), BAD),
    (dict(dx=at(5)), BAD), (dict(dbe=at(5)), BAD), (dict(dh0=at(5)), BAD),  # on the offsets
])
def test_backward_rejects(lib, kw, code):
    assert _bwd(lib, **kw) == code


def _step(lib, **kw):
    a = dict(x=at(1), la=at(2), be=at(3), gate=1, h=at(4), N=3, C=100, dt=0, y=at(5))
    a.update(kw)
    return lib.gdn_glr_step(a["x"], a["la"], a["be"], a["gate"], a["h"], a["N"], a["C"], a["dt"],
                            a["y"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(la=None), BAD), (dict(be=None), BAD), (dict(h=None), BAD),
    (dict(y=None), BAD), (dict(N=-1), BAD), (dict(C=0), BAD), (dict(gate=0), BAD),
    (dict(dt=5), UNSUP), (dict(h=at(4) + 8), BAD), (dict(y=at(4) + 16), BAD),
    (dict(N=0, x=None, la=None, be=None, h=None, y=None), gdn.GDN_OK),
])
def test_step_rejects(lib, kw, code):
    assert _step(lib, **kw) == code


def test_workspace_and_checkpoint_sizes(lib):
    assert gdn.glr_bwd_workspace_size(0, 10) == 0
    assert gdn.glr_bwd_workspace_size(1, 10) == 256
    assert gdn.glr_bwd_workspace_size(4096, 2560) == 128 * 2560 * 4
    assert gdn.glr_bwd_workspace_size(-1, 10) == 0
    assert gdn.glr_bwd_workspace_size(10, 0) == 0
    assert gdn.glr_checkpoint_shape(32, 5) == (1, 5)
    assert gdn.glr_checkpoint_shape(33, 5) == (2, 5)


def test_binding_refuses_cpu_tensors(lib):
    import torch
    x = torch.zeros(4, 6)
    for call in (lambda: gdn.gdn_glr_fwd(x, x), lambda: gdn.gdn_glr_bwd(x, x, x),
                 lambda: gdn.gdn_glr_step(x, x, x)):
        with pytest.raises(ValueError):
            call()
