"""Host-side checks of the layer-step entry points: each bad argument is
refused with its code before anything reaches CUDA."""
import ctypes

import pytest

from long_context_sequence_sca_b200 import build as B
from long_context_sequence_sca_b200 import lib as L

FAKE = 0x100000  # 16-byte aligned, never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def so():
    B.build()
    return L.load()


def _with(ptrs, changes):
    ptrs = list(ptrs)
    for i, v in changes.items():
        ptrs[i] = v
    return ptrs


def _scan(at={}, B=1, Lt=100, D=64, dtype=1, ws=FAKE, n=BIG):
    return L.gecko_gated_scan_forward(*_with([FAKE, FAKE, FAKE, 0, 0, 0, 0], at), B, Lt, D, dtype, ws, n, None)


def _scan_bwd(at={}, B=1, Lt=100, D=64, dtype=1, ws=FAKE, n=BIG):
    return L.gecko_gated_scan_backward(*_with([FAKE, FAKE, FAKE, 0, FAKE, 0, FAKE, FAKE, 0], at), B, Lt, D, dtype,
                                       ws, n, None)


SIZES = [(dict(B=0), 1), (dict(Lt=0), 1), (dict(D=-8), 1), (dict(dtype=2), 1), (dict(D=60), 2), (dict(B=65536), 2),
         (dict(Lt=65535 * 256 + 1), 2), (dict(D=1 << 25), 2), (dict(B=65535, Lt=65535 * 256, D=1 << 24), 2)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(at={0: 0}), 1), (dict(at={2: 0}), 1), (dict(at={1: FAKE + 8}), 3), (dict(at={4: FAKE + 4}), 3),
    (dict(at={6: FAKE + 8}), 3), (dict(n=-1), 1)])
def test_scan_rejects(so, kw, code):
    assert _scan(**kw) == code and L.gecko_last_error()


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(at={4: 0}), 1), (dict(at={7: 0}), 1), (dict(at={5: FAKE + 4}), 3), (dict(at={8: FAKE + 2}), 3),
    (dict(n=0), 1), (dict(ws=0), 1), (dict(ws=FAKE + 8), 3)])
def test_scan_backward_rejects(so, kw, code):
    kw = dict(kw)
    if kw.get("n") == 0 or "ws" in kw:
        kw["Lt"] = 5000     # long enough to need working memory
    assert _scan_bwd(**kw) == code and L.gecko_last_error()


def _qk(at={}, B=1, T=10, H=2, d=64, eps=1e-6, pos0=0, rot=64, base=10000.0, dtype=1):
    return L.gecko_qk_forward(*_with([FAKE] * 3 + [0] + [FAKE] * 4, at), B, T, H, d, eps, pos0, rot, base, 0, dtype,
                              None)


def _qk_bwd(at={}, B=1, T=10, H=2, d=64, eps=1e-6, pos0=0, rot=64, base=10000.0, dtype=1, ws=FAKE, n=BIG):
    return L.gecko_qk_backward(*_with([FAKE] * 2 + [0] + [FAKE] * 7, at), B, T, H, d, eps, pos0, rot, base, 0, dtype,
                               ws, n, None)


QK = [(dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(dtype=9), 1), (dict(eps=0.0), 1), (dict(eps=1e-20), 1),
      (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(rot=-16), 1), (dict(base=0.5), 1),
      (dict(base=float("inf")), 1), (dict(d=96), 2), (dict(rot=24), 2), (dict(rot=80), 2), (dict(H=65536), 2),
      (dict(B=1 << 31), 2), (dict(B=1 << 18, T=1 << 18), 2)]


@pytest.mark.parametrize("kw,code", QK + [(dict(at={0: 0}), 1), (dict(at={7: 0}), 1), (dict(at={3: FAKE + 4}), 3),
                                          (dict(at={5: FAKE + 4}), 3)])
def test_qk_rejects(so, kw, code):
    assert _qk(**kw) == code and L.gecko_last_error()


@pytest.mark.parametrize("kw,code", QK + [(dict(at={9: 0}), 1), (dict(at={6: FAKE + 8}), 3), (dict(n=16), 1),
                                          (dict(ws=0), 1), (dict(ws=FAKE + 4), 3)])
def test_qk_backward_rejects(so, kw, code):
    assert _qk_bwd(**kw) == code and L.gecko_last_error()


def _lin(at={}, B=1, T=10, N=64, K=72, H=0, act=0, dtype=1, ws=FAKE, n=BIG):
    return L.gecko_linear_forward(*_with([FAKE, FAKE, 0, 0, FAKE, 0], at), B, T, N, K, H, act, dtype, ws, n, None)


def _lin_bwd(at={}, B=1, T=10, N=64, K=72, H=0, act=0, dtype=1, ws=FAKE, n=BIG):
    return L.gecko_linear_backward(*_with([FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE], at), B, T, N, K, H, act, dtype, ws,
                                   n, None)


LIN = [(dict(B=0), 1), (dict(T=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(H=-1), 1), (dict(act=3), 1),
       (dict(act=-1), 1), (dict(dtype=2), 1), (dict(N=60), 2), (dict(K=20), 2), (dict(H=3), 2), (dict(N=72, H=2), 2),
       (dict(B=1 << 16, T=1 << 15), 2), (dict(N=(1 << 20) + 8), 2), (dict(K=(1 << 20) + 8), 2), (dict(B=1 << 62, T=4), 2)]


@pytest.mark.parametrize("kw,code", LIN + [(dict(at={0: 0}), 1), (dict(at={4: 0}), 1), (dict(at={2: FAKE + 4}), 3),
                                           (dict(at={5: FAKE + 8}), 3)])
def test_linear_rejects(so, kw, code):
    assert _lin(**kw) == code and L.gecko_last_error()


@pytest.mark.parametrize("kw,code", LIN + [(dict(at={2: 0}), 1), (dict(at={4: 0, 5: 0, 6: 0}), 1),
                                           (dict(at={6: FAKE + 4}), 3), (dict(act=1), 1), (dict(n=1), 1),
                                           (dict(ws=0), 1), (dict(ws=FAKE + 8), 3)])
def test_linear_backward_rejects(so, kw, code):
    assert _lin_bwd(**kw) == code and L.gecko_last_error()


def test_workspace_queries(so):
    n = ctypes.c_int64(-1)
    out = ctypes.byref(n)
    assert L.gecko_linear_workspace(2, 100, 64, 72, 0, 1, 1, 1, out) == 0 and n.value >= 2 * 200 * 64
    assert L.gecko_qk_workspace(2, 100, 3, 64, 1, out) == 0 and n.value >= 4 * 8 * 3 * 64
    assert L.gecko_gated_scan_workspace(2, 5000, 64, 1, 1, out) == 0 and n.value > 0
    assert L.gecko_linear_workspace(2, 100, 63, 72, 0, 1, 1, 1, out) == 2
    assert L.gecko_qk_workspace(0, 100, 3, 64, 1, out) == 1
    assert L.gecko_gated_scan_workspace(2, 5000, 63, 1, 1, out) == 2
    assert L.gecko_qk_workspace(2, 100, 3, 64, 1, None) == 1


def test_scan_length_limit(so):
    """65535 chunks of 128 tokens, and not one token more."""
    n = ctypes.c_int64(-1)
    most = 65535 * L.SCAN_CHUNK
    assert L.gecko_gated_scan_workspace(1, most, 64, 1, 1, ctypes.byref(n)) == 0 and n.value > 0
    assert L.gecko_gated_scan_workspace(1, most + 1, 64, 1, 1, ctypes.byref(n)) == 2
    assert _scan(Lt=most + 1) == 2 and _scan_bwd(Lt=most + 1) == 2 and L.gecko_last_error()
