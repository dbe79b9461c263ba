"""The gated recurrence on values that are not finite: a NaN or an infinity
stays in the state for as long as the gates are open, however little of it
their product would leave of a finite value, and no longer.

What is finite in the fp64 oracle is finite here, within the element-wise
bounds that the other tests of the recurrence derive (and a few of fp32's
subnormal steps: a product of values below 10 is rounded to those at most three
times); what is not is the same NaN or infinity."""
import numpy as np
import pytest
import torch

from layer_steps import DT, F32, UNIT, host, library, within
from oracle import layer_oracle as O
from test_gated_scan_gpu import _forward_bound, _gate, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return library()


def same(got, want, bound, what):
    """Equal where the oracle is not finite, within the bound where it is."""
    got = host(got)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), what
    keep = lambda t: np.where(odd, 0.0, t)
    within(keep(got), keep(want), keep(np.where(np.isfinite(bound), bound, 0.0)) + 2.0 ** -144, what)


def check(L, inp, dtype):
    """Forward and backward, patterns and values."""
    u = UNIT[dtype]
    hx, hg, hs, hr, hd, hds = (host(inp[k]) for k in ("x", "log_a", "state", "reset", "dy", "dstate"))
    finite = lambda t: None if t is None else np.where(np.isfinite(t), t, 0.0)
    with np.errstate(all="ignore"):
        want, wlast = O.gated_scan(hx, hg, hs, hr)
        wx, wg, ws = O.gated_scan_grad(hx, hg, hd, hs, hr, hds)
    E = _forward_bound(finite(hx), np.where(np.isnan(hg), 0.0, hg), finite(hs), hr)
    y, last, chunks = L.gated_scan_forward(inp["x"], inp["log_a"], reset=inp["reset"], state_in=inp["state"],
                                           return_state=True, keep_chunks=True)
    same(y, want, E + u * (np.abs(want) + E), "y")
    same(last, wlast, E[:, -1], "state")
    at = np.arange(0, hx.shape[1], L.SCAN_CHUNK)
    same(chunks, np.concatenate([hs[:, None], want], 1)[:, at],
         np.concatenate([np.zeros_like(E[:, :1]), E], 1)[:, at], "chunk states")
    dx, dg, ds = L.gated_scan_backward(inp["x"], inp["log_a"], inp["dy"], chunks, reset=inp["reset"],
                                       dstate_out=inp["dstate"])
    # (the bounds of the gradients: as in the other tests, over the finite values)
    fg, fd, fds = np.where(np.isnan(hg), 0.0, hg), finite(hd), finite(hds)
    a, gate = O.decay(fg, hr), _gate(fg)
    R, Er = np.abs(fds), np.zeros_like(fds)
    Ex = np.empty_like(hx)
    for t in range(hx.shape[1] - 1, -1, -1):
        R = R + np.abs(fd[:, t])
        Er = Er + F32 * R
        Ex[:, t] = 4 * Er
        Er = a[:, t] * Er + (gate[:, t] + F32) * a[:, t] * R
        R = a[:, t] * R
    same(dx, wx, Ex + u * (np.abs(wx) + Ex), "dx")
    same(ds, ws, 4 * Er + F32 * R, "dstate_in")
    before = np.concatenate([hs[:, None], want[:, :-1]], 1)
    Eb = np.concatenate([np.zeros_like(E[:, :1]), E[:, :-1]], 1)
    with np.errstate(all="ignore"):
        Eg = a * (Ex * (np.abs(before) + Eb) + np.abs(wx) * Eb + (gate + 3 * F32) * np.abs(wx * before))
        bound = Eg + u * (np.abs(wg) + Eg)
    same(dg, wg, bound, "dlog_a")


def _decaying(T, D, dtype, log_a, seed):
    """Gates all alike: their product over a span of 32 tokens is as small as can be (-4), over a chunk (-1), or not
    even that (-0.01)."""
    inp = _inputs(2, T, D, dtype, seed, resets=None)
    inp["log_a"].fill_(log_a)
    return inp


FAST = [-0.01, -1.0, -4.0, -30.0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(40, 24), (1000, 24), (5000, 8), (1000, 4096)])
@pytest.mark.parametrize("log_a", FAST)
def test_open_gates_keep_what_is_not_finite(L, log_a, T, D, dtype):
    if D == 4096 and (log_a != -4.0 or dtype == "f32"):
        pytest.skip("the wide tensor once")
    inp = _decaying(T, D, dtype, log_a, seed=31)
    x, dy = inp["x"], inp["dy"]
    x[0, 3, 0], x[0, 5, 1], x[1, T // 2, 2] = torch.nan, torch.inf, -torch.inf
    dy[0, T - 4, 3], dy[0, T - 9, 4], dy[1, T // 3, 5] = torch.nan, torch.inf, -torch.inf
    check(L, inp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_at_the_ends(L, dtype):
    """state_in and dstate_out that are not finite, and a value with gates that underflow only in fp32's subnormals."""
    inp = _decaying(700, 16, dtype, -2.0, seed=32)
    inp["state"][0, :3] = torch.tensor([torch.nan, torch.inf, -torch.inf])
    inp["dstate"][1, 4:7] = torch.tensor([torch.nan, torch.inf, -torch.inf])
    if dtype == "f32":   # (a gate this low is shut in bf16, whose exponential has no subnormals)
        inp["log_a"][:, 300:302] = -95.0
    check(L, inp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("log_a", FAST)
@pytest.mark.parametrize("at", [64, 100, 128, 300, 2049, 2300])
def test_shut_gate_ends_it(L, at, log_a, dtype):
    """A document start, or a gate of -inf, ends what is not finite: values, states, and a gate that is NaN itself."""
    inp = _decaying(2600, 16, dtype, log_a, seed=33)
    inp["reset"] = torch.zeros(2, 2600, dtype=torch.uint8, device="cuda")
    inp["reset"][0, at] = 1
    inp["log_a"][1, at] = -torch.inf
    x, g, dy = inp["x"], inp["log_a"], inp["dy"]
    x[:, at - 1, 0], x[:, 10, 1] = torch.nan, torch.inf
    g[:, 7, 2], g[:, at - 3, 3], g[:, at - 40, 4] = torch.nan, torch.nan, torch.nan
    dy[:, at, 5], dy[:, 2599, 6] = torch.nan, torch.inf
    inp["state"][:, 7] = torch.nan
    inp["dstate"][:, 8] = torch.nan
    g[:, at + 5, 9] = torch.nan
    check(L, inp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_gradient_does_not_hide_it(L, dtype):
    """dlog_a = dh a h is NaN where h is and the gate is open, also for dh = 0 and beside a shut gate."""
    inp = _decaying(200, 16, dtype, -0.5, seed=34)
    inp["reset"] = torch.zeros(2, 200, dtype=torch.uint8, device="cuda")
    inp["reset"][0, 75] = 1
    inp["x"][:, 64, :8] = torch.nan
    inp["dy"].zero_()
    inp["dstate"].zero_()
    check(L, inp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_keep_it_too(L, dtype):
    """A sequence in segments, down to one token, has the same NaN and infinities as the whole."""
    inp = _decaying(1000, 16, dtype, -1.0, seed=35)
    inp["x"][0, 3, 0], inp["x"][1, 400, 1] = torch.nan, torch.inf
    whole = L.gated_scan_forward(inp["x"], inp["log_a"], state_in=inp["state"])
    s, ys = inp["state"], []
    for t0, t1 in ((0, 1), (1, 260), (260, 300), (300, 301), (301, 1000)):
        cut = lambda k: inp[k][:, t0:t1].contiguous()
        y, s = L.gated_scan_forward(cut("x"), cut("log_a"), state_in=s, return_state=True)
        ys.append(y)
    y = torch.cat(ys, 1)
    odd = ~torch.isfinite(whole)
    assert torch.equal(odd, ~torch.isfinite(y)) and torch.equal(torch.isnan(whole), torch.isnan(y))
    assert torch.isnan(y[0, 3:, 0]).all() and torch.isinf(y[1, 400:, 1]).all()
