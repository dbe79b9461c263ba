"""GPU parity of the projection and its gradients against the fp64 oracle,
element by element.

Bounds.  A product of length K accumulated in fp32, in any order, is off by at
most (K + 2) 2^-24 sum |x w|; the bias adds one rounding.  An activation's slope
is at most 1.13 and its own arithmetic is off by at most ACT relative to |u|
(SiLU: the exponential to 2^-21 + |u| 2^-23, of which u s(u) keeps at most the
share 1 - s; GELU: erfc to 2^-20).  y adds the residual and one rounding to the
type.  The gradient of u reads u in fp32 (f'' is at most 0.8 in size) and is
itself rounded to the type as the operand of dx and dw."""
import numpy as np
import pytest
import torch

from layer_steps import DT, F32, UNIT, host, library, within
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
ACT = 2.0 ** -18


@pytest.fixture(scope="module")
def L():
    return library()


def _inputs(B, T, N, K, H, dtype, seed, bias=True, residual=True):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)
    out = (B, H, T, N // H) if H else (B, T, N)
    inp = dict(x=n(B, T, K).to(DT[dtype]), w=(n(N, K) * K ** -0.5).to(DT[dtype]), bias=n(N) if bias else None,
               residual=n(*out).to(DT[dtype]) if residual else None, dy=n(*out).to(DT[dtype]))
    return {k: v.cuda() if v is not None else None for k, v in inp.items()}


def check(L, inp, dtype, act, H):
    u = UNIT[dtype]
    hx, hw, hb, hr, hd = (host(inp[k]) for k in ("x", "w", "bias", "residual", "dy"))
    B, T, K = hx.shape
    N = hw.shape[0]
    y, pre = L.linear_forward(inp["x"], inp["w"], bias=inp["bias"], residual=inp["residual"], act=act, heads=H,
                              keep_pre=True)
    wy, wu = O.linear(hx, hw, hb, hr, act, H)
    sums = np.abs(hx) @ np.abs(hw).T + (0 if hb is None else np.abs(hb))
    Eu = O.split_heads((K + 3) * F32 * sums, H)
    within(pre, wu, Eu, "pre")
    own = ACT * np.abs(wu) if act != "none" else 0.0
    Ey = (1.13 if act != "none" else 1.0) * Eu + own + 2 * F32 * (np.abs(wy) + (0 if hr is None else np.abs(hr)))
    within(y, wy, Ey + u * (np.abs(wy) + Ey), "y")
    only = L.linear_forward(inp["x"], inp["w"], bias=inp["bias"], residual=inp["residual"], act=act, heads=H)
    within(only, wy, Ey + u * (np.abs(wy) + Ey), "y without pre")

    dx, dw, db = L.linear_backward(inp["x"], inp["w"], inp["dy"], pre=pre if act != "none" else None, act=act,
                                   heads=H)
    wx, ww, wb, du = O.linear_grad(hx, hw, hd, hb, act, H)
    g, Em = (np.abs(O.merge_heads(v, H)) for v in (hd, Eu))
    Edu = np.zeros_like(du) if act == "none" else g * (0.8 * Em + ACT) + 2 * F32 * np.abs(du)
    Eb = Edu.sum((0, 1)) + (B * T + 2) * F32 * (np.abs(du) + Edu).sum((0, 1))
    within(db, wb, Eb, "db")
    Er = Edu + (u * (np.abs(du) + Edu) if act != "none" else 0.0)   # rounded as an operand
    ax = (np.abs(du) + Er) @ np.abs(hw)
    Ex = Er @ np.abs(hw) + (N + 2) * F32 * ax
    within(dx, wx, Ex + u * (np.abs(wx) + Ex), "dx")
    Ew = np.einsum("btn,btk->nk", Er, np.abs(hx))
    Ew = Ew + (B * T + 2) * F32 * np.einsum("btn,btk->nk", np.abs(du) + Er, np.abs(hx))
    within(dw, ww, Ew + u * (np.abs(ww) + Ew), "dw")


SIZES = [(1, 1, 8, 8, 0), (1, 3, 24, 16, 0), (2, 65, 136, 72, 0), (5, 1, 64, 200, 8), (3, 129, 264, 520, 3),
         (1, 300, 1000, 1288, 0), (8, 1, 512, 1024, 4), (33, 1, 256, 264, 2), (2, 64, 128, 64, 1), (1, 500, 512, 256, 4),
         (3, 257, 640, 136, 5), (1, 2000, 264, 72, 0), (1, 17, 2048, 136, 16), (1, 130, 72, 5000, 0), (1, 5003, 16, 24, 2),
         (1, 100, 136, 5000, 0), (1, 128, 520, 128, 0), (2, 3, 2056, 200, 0), (1, 9, 24, 10000, 0),
         (1, 300, 1032, 2560, 0), (3, 171, 512, 1544, 4), (1, 1100, 264, 520, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,N,K,H", SIZES)
def test_matches_oracle(L, B, T, N, K, H, dtype):
    act = ("none", "silu", "gelu")[(T + N) % 3]
    check(L, _inputs(B, T, N, K, H, dtype, seed=T * 31 + N * 7 + K), dtype, act, H)


@pytest.mark.parametrize("B,T,N,K,H,act", [(5, 500, 2048, 2056, 16, "silu"), (1, 2700, 2184, 2048, 0, "none")])
def test_many_tiles(L, B, T, N, K, H, act):
    """Enough output tiles, in every product, for the large tiles shared by two CTAs; several per CTA."""
    check(L, _inputs(B, T, N, K, H, "bf16", seed=3), "bf16", act, H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bias,residual,H", [(True, False, 0), (False, True, 4), (False, False, 0), (True, True, 2)])
def test_epilogues(L, bias, residual, H, act, dtype):
    check(L, _inputs(2, 150, 320, 264, H, dtype, seed=2, bias=bias, residual=residual), dtype, act, H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,act", [(0, "none"), (4, "silu")])
def test_cuda_core_products(L, monkeypatch, H, act, dtype):
    """GECKO_KERNELS=simt: the second implementation, within the same bounds."""
    monkeypatch.setenv("GECKO_KERNELS", "simt")
    check(L, _inputs(2, 70, 96, 136, H, dtype, seed=12), dtype, act, H)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_large_arguments(L, act):
    """f far from 0: SiLU and GELU tend to u and to 0, their slopes to 1 and 0."""
    x = torch.tensor([[-200.0, -90.0, -30.0, -10.0, 0.0, 10.0, 90.0, 200.0]], device="cuda").T.contiguous()
    x = torch.cat([x, torch.zeros(8, 7, device="cuda")], 1)
    w = torch.zeros(8, 8, device="cuda")
    w[:, 0] = 1.0
    y, pre = L.linear_forward(x, w, act=act, keep_pre=True)
    want = O.act(host(pre), act)
    within(y, want, 2.0 ** -18 * np.abs(host(pre)) * (np.abs(want) > 1e-30) + 1e-30, "y")
    dx, _, _ = L.linear_backward(x, w, torch.ones_like(y), pre=pre, act=act)
    slope = O.act_slope(host(pre), act)
    within(dx[:, :1], slope.sum(1, keepdims=True), 8 * 2.0 ** -17, "dx")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_of_the_gradient(L, dtype):
    """Any of dx, dw, db alone is what the whole call gives."""
    inp = _inputs(2, 90, 136, 72, 0, dtype, seed=4)
    _, pre = L.linear_forward(inp["x"], inp["w"], bias=inp["bias"], act="silu", keep_pre=True)
    for act, p in (("silu", pre), ("none", None)):
        whole = L.linear_backward(inp["x"], inp["w"], inp["dy"], pre=p, act=act)
        for i in range(3):
            need = [j == i for j in range(3)]
            got = L.linear_backward(inp["x"], inp["w"], inp["dy"], pre=p, act=act, need=need)
            assert torch.equal(got[i], whole[i]) and all((got[j] is None) != need[j] for j in range(3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_do_not_mix(L, dtype):
    """NaN or infinity in one token's row reaches that row only."""
    inp = _inputs(1, 140, 136, 72, 0, dtype, seed=5, residual=False)
    clean = L.linear_forward(inp["x"], inp["w"], bias=inp["bias"])
    x = inp["x"].clone()
    x[0, 77, 3], x[0, 139, 0] = torch.nan, torch.inf
    y = L.linear_forward(x, inp["w"], bias=inp["bias"])
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[[77, 139]] = False
    assert torch.equal(y[0][keep], clean[0][keep]) and torch.isnan(y[0, 77]).all()


@pytest.mark.parametrize("T,N,K", [(300, 512, 520), (4, 1024, 1032), (3000, 128, 64)])
def test_repeats_bit_for_bit(L, T, N, K):
    inp = _inputs(1, T, N, K, 0, "bf16", seed=6)
    f = lambda: (L.linear_forward(inp["x"], inp["w"], bias=inp["bias"]),
                 *L.linear_backward(inp["x"], inp["w"], inp["dy"]))
    first = f()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(f(), first))


def test_two_dimensional_input(L):
    inp = _inputs(1, 37, 64, 72, 0, "bf16", seed=7)
    y = L.linear_forward(inp["x"], inp["w"], bias=inp["bias"], residual=inp["residual"], act="silu")
    y2 = L.linear_forward(inp["x"][0], inp["w"], bias=inp["bias"], residual=inp["residual"][0], act="silu")
    assert y2.shape == (37, 64) and torch.equal(y2, y[0])


@pytest.mark.parametrize("T,N,K", [(17, 136, 8), (100, 72, 4096), (700, 264, 72), (1024, 1024, 1024), (120, 1024, 2056),
                                   (640, 1000, 4096), (2100, 1032, 520), (4096, 64, 200)])
def test_fp32_products_are_as_good_as_fp32(L, T, N, K):
    """In the norm.  A step of 16 products cuts about 2^-25.5 of the sum, always to
    zero, and at most 64 steps follow one another before the sums are rounded:
    2^-19.5 together, far above what the roundings add (their signs differ).
    Without the third planes the products would be off by 2^-18 and more."""
    inp = _inputs(1, T, N, K, 0, "f32", seed=T + N + K, bias=False, residual=False)
    hx, hw, hd = (host(inp[k])[0] if k != "w" else host(inp[k]) for k in ("x", "w", "dy"))
    y = L.linear_forward(inp["x"], inp["w"])
    dx, dw, _ = L.linear_backward(inp["x"], inp["w"], inp["dy"])
    for got, want in ((y, hx @ hw.T), (dx, hd @ hw), (dw, hd.T @ hx)):
        err = np.linalg.norm(host(got).reshape(want.shape) - want) / np.linalg.norm(want)
        assert err <= 2.0 ** -19, err


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K,H", [(100, 72, 4096, 0), (640, 1000, 4096, 0), (120, 1024, 2056, 8), (260, 4096, 520, 0)])
def test_shared_depth(L, T, N, K, H, dtype):
    """Clusters of two and four CTAs, parts of one run and of several, ragged rows and columns."""
    check(L, _inputs(1, T, N, K, H, dtype, seed=T + K), dtype, "gelu", H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(20000, 64, 264), (30011, 128, 72)])
def test_many_tokens_few_features(L, T, N, K, dtype):
    """dw and dx of much depth or many rows and hardly any columns."""
    check(L, _inputs(1, T, N, K, 0, dtype, seed=T, residual=False), dtype, "silu", 0)
