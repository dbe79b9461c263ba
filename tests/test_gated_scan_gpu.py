"""GPU parity of the gated recurrence and its gradients against the fp64
oracle, element by element.

Bounds.  The gate a = exp(log_a) is off by at most GATE relative: 2 units in
the last place of the exponential (2^-22), and |log_a| 2^-23 from scaling the
argument by log2 e.  So with H the same recurrence over |x| and |state|, the
state's error E obeys E_t <= a_t E_{t-1} + GATE a_t H_{t-1} + 2^-24 H_t to first
order, in whatever order the affine maps are composed (composing rounds each
product and sum once more: the factor 4).  The reverse recurrence is the same
one.  An output adds one rounding to its type."""
import numpy as np
import pytest
import torch

from layer_steps import DT, F32, UNIT, host, library, within
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return library()


def _inputs(B, T, D, dtype, seed, resets="some", state=True):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)
    log_a = -torch.exp(1.5 * n(B, T, D) - 3.0)
    x = n(B, T, D) * torch.sqrt(-torch.expm1(2 * log_a))
    reset = None
    if resets == "some":
        reset = (torch.rand(B, T, generator=r) < 0.02).to(torch.uint8)
    elif resets == "all":
        reset = torch.full((B, T), 255, dtype=torch.uint8)
    inp = dict(x=x.to(DT[dtype]), log_a=log_a.to(DT[dtype]), reset=reset, state=n(B, D) if state else None,
               dy=n(B, T, D).to(DT[dtype]), dstate=n(B, D) if state else None)
    return {k: v.cuda() if v is not None else None for k, v in inp.items()}


def _gate(log_a):
    g = np.where(np.isfinite(log_a), np.abs(log_a), 0.0)
    return 2.0 ** -22 + g * 2.0 ** -23


def _forward_bound(x, log_a, state, reset):
    a = O.decay(log_a, reset)
    gate = _gate(log_a)
    B, T, D = x.shape
    H = np.zeros((B, D)) if state is None else np.abs(state)
    E = np.zeros((B, D))
    out = np.empty_like(x)
    for t in range(T):
        E = a[:, t] * E + gate[:, t] * a[:, t] * H
        H = a[:, t] * H + np.abs(x[:, t])
        E = E + F32 * H
        out[:, t] = 4 * E
    return out


def check(L, inp, dtype):
    u = UNIT[dtype]
    hx, hg, hs, hr = (host(inp[k]) for k in ("x", "log_a", "state", "reset"))
    y, last, chunks = L.gated_scan_forward(inp["x"], inp["log_a"], reset=inp["reset"], state_in=inp["state"],
                                           return_state=True, keep_chunks=True)
    want, wlast = O.gated_scan(hx, hg, hs, hr)
    E = _forward_bound(hx, hg, hs, hr)
    within(y, want, E + u * (np.abs(want) + E), "y")
    within(last, wlast, E[:, -1], "state")
    at = np.arange(0, hx.shape[1], L.SCAN_CHUNK)
    enter = np.concatenate([(np.zeros_like(want[:, :1]) if hs is None else hs[:, None]), want], 1)[:, at]
    bound = np.concatenate([np.zeros_like(E[:, :1]), E], 1)[:, at]
    within(chunks, enter, bound, "chunk states")

    dx, dg, ds = L.gated_scan_backward(inp["x"], inp["log_a"], inp["dy"], chunks, reset=inp["reset"],
                                       dstate_out=inp["dstate"])
    hd, hds = host(inp["dy"]), host(inp["dstate"])
    wx, wg, ws = O.gated_scan_grad(hx, hg, hd, hs, hr, hds)
    # the reverse recurrence runs over the gates moved by one token
    a, gate = O.decay(hg, hr), _gate(hg)
    B, T, D = hx.shape
    R, Er = (np.zeros((B, D)) if hds is None else np.abs(hds)), np.zeros((B, D))
    Ex, Rx = np.empty_like(hx), np.empty_like(hx)
    for t in range(T - 1, -1, -1):
        R = R + np.abs(hd[:, t])
        Er = Er + F32 * R
        Ex[:, t], Rx[:, t] = 4 * Er, R
        Er = a[:, t] * Er + (gate[:, t] + F32) * a[:, t] * R
        R = a[:, t] * R
    within(dx, wx, Ex + u * (np.abs(wx) + Ex), "dx")
    within(ds, ws, 4 * Er + F32 * R, "dstate_in")
    before = np.concatenate([np.zeros_like(want[:, :1]) if hs is None else hs[:, None], want[:, :-1]], 1)
    Eb = np.concatenate([np.zeros_like(E[:, :1]), E[:, :-1]], 1)
    Eg = a * (Ex * (np.abs(before) + Eb) + np.abs(wx) * Eb + (gate + 3 * F32) * np.abs(wx * before))
    within(dg, wg, Eg + u * (np.abs(wg) + Eg), "dlog_a")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (3, 1, 264), (5, 2, 72), (2, 17, 16), (2, 255, 24), (2, 256, 8),
                                   (1, 257, 72), (2, 1000, 136), (1, 5000, 40), (4, 700, 520), (1, 33, 4096)])
def test_matches_oracle(L, B, T, D, dtype):
    check(L, _inputs(B, T, D, dtype, seed=B * 1000003 + T * 101 + D), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("resets,state", [(None, False), ("all", True), (None, True), ("some", False)])
def test_resets_and_states(L, resets, state, dtype):
    check(L, _inputs(2, 600, 40, dtype, seed=7, resets=resets, state=state), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_closed_and_open_gates(L, dtype):
    """log_a of -inf, of the type's lowest value, and of 0 (a plain sum)."""
    inp = _inputs(2, 600, 24, dtype, seed=8)
    g = inp["log_a"]
    g[:, 5::61] = -torch.inf
    g[:, 11::67] = torch.finfo(g.dtype).min
    g[:, 100:160, :8] = 0.0
    check(L, inp, dtype)
    g[:] = -torch.inf
    check(L, inp, dtype)


def test_closed_gate_drops_what_is_not_finite(L):
    """What lies before a document start does not reach it, even if it is NaN or infinite."""
    inp = _inputs(1, 700, 16, "f32", seed=9, resets=None)
    inp["reset"] = torch.zeros(1, 700, dtype=torch.uint8, device="cuda")
    inp["reset"][0, 300] = 1
    clean = L.gated_scan_forward(inp["x"], inp["log_a"], reset=inp["reset"], state_in=inp["state"])
    x = inp["x"].clone()
    x[0, 299, :8], x[0, 10, 8:] = torch.nan, torch.inf
    y = L.gated_scan_forward(x, inp["log_a"], reset=inp["reset"], state_in=inp["state"])
    assert torch.equal(y[:, 300:], clean[:, 300:])
    assert torch.isnan(y[0, 299, :8]).all() and torch.isinf(y[0, 299, 8:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_and_single_tokens_chain(L, dtype):
    """Segments down to one token, chained by their states, give the whole sequence."""
    inp = _inputs(2, 530, 48, dtype, seed=10)
    hx, hg, hs, hr = (host(inp[k]) for k in ("x", "log_a", "state", "reset"))
    want, wlast = O.gated_scan(hx, hg, hs, hr)
    E = _forward_bound(hx, hg, hs, hr)
    s, ys = inp["state"], []
    for t0, t1 in ((0, 1), (1, 2), (2, 260), (260, 261), (261, 530)):
        cut = lambda k: inp[k][:, t0:t1].contiguous()
        y, s = L.gated_scan_forward(cut("x"), cut("log_a"), reset=cut("reset"), state_in=s, return_state=True)
        ys.append(y)
    y = torch.cat(ys, 1)
    within(y, want, E + UNIT[dtype] * (np.abs(want) + E), "y")
    within(s, wlast, E[:, -1], "state")


@pytest.mark.parametrize("T", [1, 40, 900])
def test_in_place(L, T):
    inp = _inputs(2, T, 72, "bf16", seed=11)
    want = L.gated_scan_forward(inp["x"], inp["log_a"], reset=inp["reset"], state_in=inp["state"])
    x = inp["x"].clone()
    got = L.gated_scan_forward(x, inp["log_a"], reset=inp["reset"], state_in=inp["state"], y=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


def test_aliases_of_the_c_call(L):
    """state_out over state_in, dx over dy and dstate_in over dstate_out."""
    import ctypes
    inp = _inputs(2, 600, 40, "f32", seed=12)
    B, T, D = inp["x"].shape
    y, last, chunks = L.gated_scan_forward(inp["x"], inp["log_a"], reset=inp["reset"], state_in=inp["state"],
                                           return_state=True, keep_chunks=True)
    dx, dg, ds = L.gated_scan_backward(inp["x"], inp["log_a"], inp["dy"], chunks, reset=inp["reset"],
                                       dstate_out=inp["dstate"])
    n = ctypes.c_int64()
    assert L.gecko_gated_scan_workspace(B, T, D, 0, 1, ctypes.byref(n)) == 0
    ws = torch.empty(max(n.value, 1 << 20), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    s, y2 = inp["state"].clone(), torch.empty_like(y)
    assert L.gecko_gated_scan_forward(inp["x"].data_ptr(), inp["log_a"].data_ptr(), y2.data_ptr(),
                                      inp["reset"].data_ptr(), s.data_ptr(), s.data_ptr(), 0, B, T, D, 0,
                                      ws.data_ptr(), ws.numel(), st) == 0
    assert torch.equal(y2, y) and torch.equal(s, last)
    d, e, dg2 = inp["dy"].clone(), inp["dstate"].clone(), torch.empty_like(dg)
    assert L.gecko_gated_scan_backward(inp["x"].data_ptr(), inp["log_a"].data_ptr(), d.data_ptr(),
                                       inp["reset"].data_ptr(), chunks.data_ptr(), e.data_ptr(), d.data_ptr(),
                                       dg2.data_ptr(), e.data_ptr(), B, T, D, 0, ws.data_ptr(), ws.numel(), st) == 0
    assert torch.equal(d, dx) and torch.equal(dg2, dg) and torch.equal(e, ds)


def test_autograd(L):
    """GatedScanFunction against torch's own differentiation of the recurrence in fp64."""
    inp = _inputs(2, 40, 16, "f32", seed=13, resets="some")
    leaves = [inp[k].clone().requires_grad_() for k in ("x", "log_a", "state")]
    y, s = L.GatedScanFunction.apply(leaves[0], leaves[1], leaves[2], inp["reset"])
    (y * inp["dy"]).sum().add((s * inp["dstate"]).sum()).backward()
    ref = [l.detach().double().requires_grad_() for l in leaves]
    a = torch.exp(ref[1]) * (inp["reset"] == 0)[..., None]
    h, ys = ref[2], []
    for t in range(40):
        h = a[:, t] * h + ref[0][:, t]
        ys.append(h)
    (torch.stack(ys, 1) * inp["dy"].double()).sum().add((h * inp["dstate"].double()).sum()).backward()
    for got, want in zip(leaves, ref):
        # at most 40 steps, each off by a few units of 2^-22 of terms up to about 30
        torch.testing.assert_close(got.grad.double(), want.grad, rtol=1e-4, atol=1e-4)
