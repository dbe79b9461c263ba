"""GPU parity of the query/key step and its gradients against the fp64
oracle, element by element.

Bounds.  The norm sums d squares (d + 2 roundings), a root, a reciprocal and a
product: z' is off by at most (d / 2 + 4) units relative.  Each affine adds two
roundings of at most |scale z'| + |shift|.  An angle is reduced in fp64 to
within 2^-25 of half a revolution's argument, so cos and sin are off by at most
2^-22 (the argument's rounding times pi, and 2 units of the function); a turn
then mixes two values with three roundings.  An output adds one rounding to its
type; the parameter gradients sum B T terms in fp32."""
import numpy as np
import pytest
import torch

from layer_steps import DT, F32, UNIT, host, library, within
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return library()


def _inputs(B, T, H, d, dtype, seed, far=False):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)
    pos = None
    if far:
        pos = torch.randint(0, 1 << 31, (B, 1), generator=r) + torch.arange(T)
    inp = dict(z=n(B, T, H * d).to(DT[dtype]), scale=1 + 0.1 * n(4, H, d), shift=0.1 * n(4, H, d), pos=pos)
    inp = {k: v.cuda() if v is not None else None for k, v in inp.items()}
    inp["grads"] = [n(B, H, T, d).to(DT[dtype]).cuda() for _ in range(4)]
    return inp


def _partner(p, rot, inter):
    """|other member of the pair| for each rotated feature, 0 elsewhere."""
    out = np.zeros_like(p)
    if rot:
        ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
        ib = ia + (1 if inter else rot // 2)
        out[..., ia], out[..., ib] = np.abs(p[..., ib]), np.abs(p[..., ia])
    return out


def check(L, inp, dtype, rot=0, inter=False, eps=1e-6, pos0=0, base=10000.0):
    u = UNIT[dtype]
    B, T, W = inp["z"].shape
    H, d = inp["scale"].shape[1:]
    pos = host(inp["pos"]) if inp["pos"] is not None else np.broadcast_to(np.arange(T) + pos0, (B, T))
    kw = dict(rot_dim=rot, interleaved=inter)
    out = L.qk_forward(inp["z"], inp["scale"], inp["shift"], eps=eps, pos=inp["pos"], pos0=pos0, rot_base=base, **kw)
    hz, hs, hf = host(inp["z"]), host(inp["scale"]), host(inp["shift"])
    want = O.qk(hz, hs, hf, eps, pos=pos, base=base, **kw)
    flat = O.qk(hz, hs, hf, eps)   # before the turn
    E_unit = (d / 2 + 4) * F32
    for i, name in enumerate(("q", "k", "qm", "km")):
        size = np.abs(flat[i]) + 2 * np.abs(hf[i])[None, :, None]
        E = (E_unit + 2 * F32) * size
        if i < 2 and rot:
            E = E + _partner(E, rot, inter) + (2.0 ** -22 + 3 * F32) * (np.abs(flat[i]) +
                                                                        _partner(flat[i], rot, inter))
        within(out[i], want[i], E + u * (np.abs(want[i]) + E), name)

    dz, dsc, dsh = L.qk_backward(inp["z"], inp["scale"], *inp["grads"], eps=eps, pos=inp["pos"], pos0=pos0,
                                 rot_base=base, **kw)
    hg = [host(g) for g in inp["grads"]]
    wz, wsc, wsh = O.qk_grad(hz, hs, hg, eps, pos=pos, base=base, **kw)
    zh = hz.reshape(B, T, H, d)
    norm = np.sqrt((zh * zh).sum(-1, keepdims=True))
    n = np.maximum(norm, eps)
    unit = np.abs(zh / n)
    back = [g.transpose(0, 2, 1, 3) for g in hg]
    size, E = [], []
    for i in range(4):
        pr = _partner(back[i], rot, inter) if i < 2 else np.zeros_like(back[i])
        turned = i < 2 and rot
        size.append(np.abs(back[i]) + pr)
        E.append((2.0 ** -22 + 3 * F32) * size[i] if turned else np.zeros_like(pr))
    up = sum(np.abs(hs[i]) * size[i] for i in range(4))
    E_up = sum(np.abs(hs[i]) * E[i] for i in range(4)) + 4 * F32 * up
    along = (unit * up).sum(-1, keepdims=True)
    E_along = (unit * E_up).sum(-1, keepdims=True) + (E_unit + d * F32) * along
    Ez = (E_up + unit * E_along + (2 * E_unit + 4 * F32) * (up + unit * along)) / n
    Ez = Ez.reshape(B, T, W)
    within(dz, wz, Ez + u * (np.abs(wz) + Ez), "dz")
    N = B * T
    Esc = np.stack([(E[i] * unit + (E_unit + 2 * F32) * size[i] * unit).sum((0, 1)) for i in range(4)])
    Esc += N * F32 * np.stack([(size[i] * unit).sum((0, 1)) for i in range(4)])
    within(dsc, wsc, Esc, "dscale")
    Esh = np.stack([E[i].sum((0, 1)) + (N + 1) * F32 * size[i].sum((0, 1)) for i in range(4)])
    within(dsh, wsh, Esh, "dshift")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,d,rot,inter", [
    (1, 1, 1, 64, 64, False), (16, 1, 32, 128, 128, False), (2, 37, 5, 64, 32, True), (1, 130, 3, 128, 0, False),
    (3, 200, 32, 64, 48, False), (1, 70, 33, 128, 128, True), (2, 333, 1, 128, 16, False), (7, 5, 17, 64, 16, True),
    (1, 1000, 2, 64, 64, True), (2, 600, 16, 128, 112, False)])
def test_matches_oracle(L, B, T, H, d, rot, inter, dtype):
    check(L, _inputs(B, T, H, d, dtype, seed=T * 1009 + H * 7 + d), dtype, rot, inter)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_far_and_given_positions(L, inter, dtype):
    check(L, _inputs(3, 41, 4, 128, dtype, seed=3, far=True), dtype, 128, inter)
    check(L, _inputs(2, 65, 4, 64, dtype, seed=4), dtype, 64, inter, pos0=4194303)
    check(L, _inputs(1, 9, 2, 64, dtype, seed=5), dtype, 32, inter, pos0=-7, base=500000.0)


def test_one_token_of_a_row_of_positions(L):
    """A generated token's position as a slice of its sequence's: 8-byte aligned."""
    inp = _inputs(1, 1, 4, 64, "bf16", seed=8)
    row = torch.arange(100, 110, device="cuda")[None]
    for t in (4, 5):
        inp["pos"] = row[:, t:t + 1]
        check(L, inp, "bf16", 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_and_tiny_rows(L, dtype):
    """A row of zeros gives z' = 0, rows shorter than eps a linear map."""
    inp = _inputs(2, 20, 4, 64, dtype, seed=6)
    z = inp["z"].view(2, 20, 4, 64)
    z[0, 3] = 0
    z[1, 5, 2] = 0
    z[:, 7:9] *= 2.0 ** -12
    z[0, 11, 1, 1:] = 0
    check(L, inp, dtype, 64, False, eps=2.0 ** -5)
    inp["z"].zero_()
    check(L, inp, dtype, 16, True)


def test_rows_do_not_mix(L):
    """A row that is not finite leaves every other row as it was."""
    inp = _inputs(1, 50, 5, 64, "bf16", seed=7)
    kw = dict(rot_dim=64)
    clean = L.qk_forward(inp["z"], inp["scale"], inp["shift"], **kw)
    z = inp["z"].clone()
    z.view(1, 50, 5, 64)[0, 17, 3, 5] = torch.nan
    z.view(1, 50, 5, 64)[0, 18, 1, 6] = torch.inf
    keep = torch.ones(5, 50, dtype=torch.bool, device="cuda")
    keep[3, 17] = keep[1, 18] = False
    for a, b in zip(L.qk_forward(z, inp["scale"], inp["shift"], **kw), clean):
        assert torch.equal(a[0][keep], b[0][keep])
        assert torch.isnan(a[0, 3, 17]).all() and torch.isnan(a[0, 1, 18]).any()


def test_gradients_repeat_bit_for_bit(L):
    inp = _inputs(2, 3000, 9, 64, "bf16", seed=8)
    first = L.qk_backward(inp["z"], inp["scale"], *inp["grads"], rot_dim=64)
    for _ in range(3):
        for a, b in zip(L.qk_backward(inp["z"], inp["scale"], *inp["grads"], rot_dim=64), first):
            assert torch.equal(a, b)


def test_autograd_matches_differences(L):
    """QkFunction's gradient along random directions against central differences of the fp32 forward."""
    inp = _inputs(1, 12, 2, 64, "f32", seed=9)
    leaves = [inp[k].clone().requires_grad_() for k in ("z", "scale", "shift")]
    opts = dict(rot_dim=32, interleaved=True, pos0=100)
    f = lambda *a: sum((o.double() * g.double()).sum() for o, g in
                       zip(L.QkFunction.apply(*a, None, opts), inp["grads"]))
    f(*leaves).backward()
    gen = torch.Generator().manual_seed(1)
    for i, leaf in enumerate(leaves):
        v = torch.randn(leaf.shape, generator=gen).cuda()
        h = 2.0 ** -7
        args = lambda s: [l.detach() + (s * h * v if j == i else 0) for j, l in enumerate(leaves)]
        diff = (f(*args(1)) - f(*args(-1))) / (2 * h)
        slope = (leaf.grad.double() * v.double()).sum()
        # 1536 outputs of about 1, each rounded to 2^-24: noise 2^-24 sqrt(6144) / 2^-7 < 1e-3; the second-order
        # term of the unit norm (|z| about 8, |v| about 8) is about h^2 of the slope's terms, below 1e-2
        assert abs(diff - slope) <= 2e-2 * max(1.0, abs(slope)), (i, diff, slope)


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_norm_is_rounded(L, d):
    """A row of one value v of 12 bits: v^2 and its root are exact, so z' = v fl(1 / v), of which the reciprocal's
    rounding leaves 1 or the number below it (above 1 the next is 2^-23 away, and 1 + 2^-24 rounds to 1)."""
    v = torch.arange(2048, 4096, device="cuda").float() * 2.0 ** -9
    z = torch.zeros(1, 2048, d, device="cuda")
    z[0, :, 5] = torch.where(torch.arange(2048, device="cuda") % 2 == 0, v, -v)
    scale, shift = torch.ones(4, 1, d, device="cuda"), torch.zeros(4, 1, d, device="cuda")
    for out in L.qk_forward(z, scale, shift):
        assert ((out[0, 0, :, 5].double().abs() - 1).abs() <= F32).all()
