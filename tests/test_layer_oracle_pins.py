"""Pins of the layer-step oracle: every gradient against central differences
of the forward, and the forwards against independent forms (closed sums,
complex rotation, torch's own layers in fp64)."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as O

RNG = np.random.default_rng


def _difference(f, x, cotangents, step=1e-6):
    """d sum(f(x) * cotangents) / dx by central differences."""
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        old = flat[i]
        vals = []
        for s in (step, -step):
            flat[i] = old + s
            vals.append(sum((np.asarray(o) * c).sum() for o, c in zip(f(), cotangents)))
        flat[i] = old
        out[i] = (vals[0] - vals[1]) / (2 * step)
    return g


def test_scan_is_the_sum_over_history():
    r = RNG(0)
    x, g = r.normal(size=(2, 9, 3)), -r.random((2, 9, 3))
    s0 = r.normal(size=(2, 3))
    h, last = O.gated_scan(x, g, s0)
    for t in range(9):
        want = np.exp(g[:, :t + 1].sum(1)) * s0
        for u in range(t + 1):
            want = want + np.exp(g[:, u + 1:t + 1].sum(1)) * x[:, u]
        np.testing.assert_allclose(h[:, t], want, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(last, h[:, -1])


def test_scan_reset_equals_two_sequences():
    r = RNG(1)
    x, g = r.normal(size=(1, 8, 4)), -r.random((1, 8, 4))
    reset = np.zeros((1, 8), np.uint8)
    reset[0, 5] = 1
    h, _ = O.gated_scan(x, g, reset=reset)
    np.testing.assert_array_equal(h[:, 5:], O.gated_scan(x[:, 5:], g[:, 5:])[0])
    gi = g.copy()
    gi[0, 5] = -np.inf
    np.testing.assert_array_equal(h, O.gated_scan(x, gi)[0])


def test_scan_gradients_match_differences():
    r = RNG(2)
    x, g, s0 = r.normal(size=(2, 6, 2)), -r.random((2, 6, 2)), r.normal(size=(2, 2))
    reset = (r.random((2, 6)) < 0.3).astype(np.uint8)
    dy, ds = r.normal(size=x.shape), r.normal(size=s0.shape)
    f = lambda: O.gated_scan(x, g, s0, reset)
    got = O.gated_scan_grad(x, g, dy, s0, reset, ds)
    for v, want in zip((x, g, s0), got):
        np.testing.assert_allclose(_difference(f, v, (dy, ds)), want, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (32, True), (64, False)])
def test_qk_forward_and_gradients(rot, inter):
    r = RNG(3)
    H, d, eps = 2, 64, 1e-6
    z, sc, sh = r.normal(size=(1, 2, H * d)), 1 + 0.1 * r.normal(size=(4, H, d)), 0.1 * r.normal(size=(4, H, d))
    pos = np.array([[3, 1000]])
    kw = dict(rot_dim=rot, interleaved=inter, pos=pos)
    out = O.qk(z, sc, sh, eps, **kw)
    unit = z.reshape(1, 2, H, d) / np.linalg.norm(z.reshape(1, 2, H, d), axis=-1, keepdims=True)
    plain = (unit * sc[0] + sh[0]).transpose(0, 2, 1, 3)
    if rot:
        if inter:
            c = plain[..., 0:rot:2] + 1j * plain[..., 1:rot:2]
        else:
            c = plain[..., :rot // 2] + 1j * plain[..., rot // 2:rot]
        c = c * np.exp(1j * O.turns(pos, rot, 10000.0))[:, None]
        got = (out[0][..., 0:rot:2], out[0][..., 1:rot:2]) if inter else (out[0][..., :rot // 2],
                                                                          out[0][..., rot // 2:rot])
        np.testing.assert_allclose(got[0], c.real, atol=1e-12)
        np.testing.assert_allclose(got[1], c.imag, atol=1e-12)
    np.testing.assert_allclose(out[0][..., rot:], plain[..., rot:], atol=1e-13)
    np.testing.assert_allclose(out[2], (unit * sc[2] + sh[2]).transpose(0, 2, 1, 3), atol=1e-13)
    grads = [r.normal(size=o.shape) for o in out]
    dz, dsc, dsh = O.qk_grad(z, sc, grads, eps, **kw)
    f = lambda: O.qk(z, sc, sh, eps, **kw)
    for v, want in ((z, dz), (sc, dsc), (sh, dsh)):
        np.testing.assert_allclose(_difference(f, v, grads), want, rtol=1e-6, atol=1e-7)


def test_qk_rows_below_eps():
    """Below eps the norm is the constant eps: a linear map and its gradient."""
    r = RNG(4)
    z = 1e-3 * r.normal(size=(1, 1, 64))
    z[..., 32:] = 0.0
    sc, sh = np.ones((4, 1, 64)), np.zeros((4, 1, 64))
    np.testing.assert_allclose(O.qk(z, sc, sh, 1.0)[2].reshape(-1), z.reshape(-1))
    g = [r.normal(size=(1, 1, 1, 64)) for _ in range(4)]
    dz = O.qk_grad(z, sc, g, 1.0)[0]
    np.testing.assert_allclose(dz.reshape(-1), sum(g).reshape(-1))


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("H", [0, 2])
def test_linear_matches_torch_and_differences(name, H):
    r = RNG(5)
    x, w, b = r.normal(size=(2, 3, 4)), r.normal(size=(6, 4)), r.normal(size=6)
    y, u = O.linear(x, w, b, None, name, H)
    ref = torch.nn.functional.linear(*(torch.from_numpy(v) for v in (x, w, b)))
    fn = {"none": lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[name]
    want = fn(ref)
    if H:
        want = want.view(2, 3, H, -1).transpose(1, 2)
    np.testing.assert_allclose(y, want.numpy(), atol=1e-12)
    res = r.normal(size=y.shape)
    np.testing.assert_allclose(O.linear(x, w, b, res, name, H)[0], y + res, atol=1e-12)
    dy = r.normal(size=y.shape)
    dx, dw, db, _ = O.linear_grad(x, w, dy, b, name, H)
    f = lambda: O.linear(x, w, b, None, name, H)[:1]
    for v, want in ((x, dx), (w, dw), (b, db)):
        np.testing.assert_allclose(_difference(f, v, (dy,)), want, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("mutant", ["gate_late", "no_norm_term", "turn_forward", "slope_of_y"])
def test_planted_mistakes_fail_the_differences(mutant):
    """A wrong gradient is told apart from the differences of the forward."""
    r = RNG(6)
    if mutant == "gate_late":      # the gate of token t on dh_t instead of a_{t+1}
        x, g = r.normal(size=(1, 5, 2)), -r.random((1, 5, 2))
        dy = r.normal(size=x.shape)
        bad = O.gated_scan_grad(x, np.roll(g, 1, 1), dy)[0]
        want = _difference(lambda: O.gated_scan(x, g)[:1], x, (dy,))
    elif mutant in ("no_norm_term", "turn_forward"):
        z = r.normal(size=(1, 2, 64))
        sc, sh, pos = np.ones((4, 1, 64)), np.zeros((4, 1, 64)), np.array([[1, 2]])
        grads = [r.normal(size=(1, 1, 2, 64)) for _ in range(4)]
        want = _difference(lambda: O.qk(z, sc, sh, 1e-6, 64, pos=pos), z, grads)
        if mutant == "no_norm_term":
            bad = O.qk_grad(z, sc, grads, 1e3, 64, pos=pos)[0] * 1e3 / np.linalg.norm(z, axis=-1, keepdims=True)
        else:
            bad = O.qk_grad(z, sc, grads, 1e-6, 64, pos=-pos)[0]
    else:
        x, w, dy = r.normal(size=(1, 3, 4)), r.normal(size=(5, 4)), r.normal(size=(1, 3, 5))
        bad = (dy * O.act_slope(O.linear(x, w, name="silu")[0], "silu")) @ w
        want = _difference(lambda: O.linear(x, w, name="silu")[:1], x, (dy,))
    assert np.abs(bad - want).max() > 1e-2
