"""Products whose depth is cut into parts, blocks and stages: nothing of it is
lost, and rows and columns do not mix.

A bf16 result is off by one rounding, 2^-8 of it at most (and what the tensor
core cuts of its sums, 2^-13.5 at the depths here), so that is what its 2-norm may be
off by; one lost block of 64 terms of 30011 would be 4.6e-2.  With operands that
are not zero in a few blocks only, a row (or column) of the result has the norm of just
those, and a lost one is most of it."""
import numpy as np
import pytest
import torch

from layer_steps import DT, host, library

pytestmark = pytest.mark.gpu

# M, N, K of y = x w^T; each is the depth of one of the three products
SIZES = [(30011, 128, 72), (20000, 64, 264), (9, 24, 10000), (100, 136, 5000), (640, 1000, 4096), (300, 1032, 2560),
         (1100, 264, 520), (2500, 2048, 2056), (1024, 1024, 1024), (3, 4096, 1032), (129, 4104, 200), (77, 16400, 264),
         (128, 72, 8200), (5000, 24, 16), (1, 512, 4104), (50000, 128, 136), (100, 264, 100000), (128, 4096, 33000),
         (16, 40, 131072), (250, 33000, 512), (300, 264, 24008)]


@pytest.fixture(scope="module")
def L():
    return library()


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _in_few_blocks(t, dim):
    """Of every row (column) of t, one block of 64 in (blocks, or as many as there are rows) along its depth `dim`."""
    depth, rows = torch.arange(t.shape[dim], device="cuda") // 64, torch.arange(t.shape[1 - dim], device="cuda")
    n = min(int(depth[-1]) + 1, t.shape[1 - dim])
    on = depth[:, None] % n == rows[None] % n
    return t * (on if dim == 0 else on.T)


def _check(got, want, what, by=None):
    got, want = got.double(), want.double()
    off = (got - want).norm(dim=by) if by is not None else (got - want).norm()
    size = want.norm(dim=by) if by is not None else want.norm()
    worst = (off / size.clamp_min(1e-30)).max().item()
    assert worst <= 2.0 ** -8 + 2.0 ** -13, (what, worst)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_depth(L, M, N, K, dtype):
    dt = DT[dtype]
    x, w, dy = (_normal(i, *s).to(dt) for i, s in enumerate([(M, K), (N, K), (M, N)]))
    xd, wd, dyd = x.double(), w.double(), dy.double()
    y = xd @ wd.T
    _check(L.linear_forward(x, w), y, "y")
    got, pre = L.linear_forward(x, w, keep_pre=True)
    _check(got, y, "y with pre")
    _check(pre, y, "pre")
    dx, dw, db = L.linear_backward(x, w, dy)
    _check(dx, dyd @ wd, "dx")
    _check(dw, dyd.T @ xd, "dw")
    _check(db, dyd.sum(0), "db")
    few = _in_few_blocks(x, 1)
    y = few.double() @ wd.T
    _check(L.linear_forward(few, w), y, "y in few blocks", 1)
    _check(L.linear_forward(few, w, keep_pre=True)[1], y, "pre in few blocks", 1)
    few = _in_few_blocks(dy, 1)
    _check(L.linear_backward(x, w, few, need=(True, False, False))[0], few.double() @ wd, "dx in few blocks", 1)
    few = _in_few_blocks(dy, 0)
    _check(L.linear_backward(x, w, few, need=(False, True, False))[1], few.double().T @ xd, "dw in few blocks", 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 9, 16, 17, 77, 140, 3000])
def test_rows_and_columns_do_not_mix(L, T, dtype):
    """NaN or infinity in a token's row, or in a row of w, is in that row or column of every result that reads it, as
    something that is not finite, and nowhere else."""
    N, K = 136, 328
    x, w, dy = (_normal(i, *s).to(DT[dtype]) for i, s in enumerate([(T, K), (N, K), (T, N)]))
    bad = [T // 2, T - 1]
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[bad] = False
    xb = x.clone()
    xb[bad[0], 3] = torch.nan
    xb[bad[1], 0] = torch.inf
    for keep_pre in (False, True):
        f = lambda *a: (lambda o: list(o) if keep_pre else [o])(L.linear_forward(*a, keep_pre=keep_pre))
        for a, b in zip(f(xb, w), f(x, w)):
            assert torch.equal(a[good], b[good]) and not torch.isfinite(a[bad]).any()
        wb = w.clone()
        wb[5, 7], wb[N - 1, K - 1] = torch.inf, torch.nan
        cols = torch.ones(N, dtype=torch.bool, device="cuda")
        cols[[5, N - 1]] = False
        for a, b in zip(f(x, wb), f(x, w)):
            assert torch.equal(a[:, cols], b[:, cols]) and not torch.isfinite(a[:, ~cols]).any()
    db = dy.clone()
    db[bad[0], 3], db[bad[1], 0] = torch.nan, torch.inf
    a, b = L.linear_backward(x, w, db), L.linear_backward(x, w, dy)
    assert torch.equal(a[0][good], b[0][good]) and not torch.isfinite(a[0][bad]).any()
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[[0, 3]] = False
    for i in (1, 2):
        assert torch.equal(a[i][cols], b[i][cols]) and not torch.isfinite(a[i][~cols]).any()
