"""The projection's activations far from zero, where f and f' are small and
only a relative error says anything: u comes exactly, as the bias of a product
with zeros.

Bounds, in units of 2^-24 of the value unless said otherwise."""
import numpy as np
import pytest
import torch

from layer_steps import DT, F32, UNIT, host, library, within
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
N = 4096


@pytest.fixture(scope="module")
def L():
    return library()


def outputs(L, u, act, dtype, B=1, T=1):
    """f(u) in the type, and f'(u) in fp32 (db of a single token with dy = 1)."""
    u = torch.from_numpy(u.astype(np.float32)).cuda()
    x, w = torch.zeros(B, T, 8, dtype=DT[dtype], device="cuda"), torch.zeros(N, 8, dtype=DT[dtype], device="cuda")
    y, pre = L.linear_forward(x, w, bias=u, act=act, keep_pre=True)
    assert torch.equal(pre, u.expand(B, T, N))
    _, _, db = L.linear_backward(x[:1, :1].contiguous(), w, torch.ones(1, 1, N, dtype=DT[dtype], device="cuda"),
                                 pre=pre[:1, :1].contiguous(), act=act)
    return u.double().cpu().numpy(), host(y), host(db)


@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gelu(L, dtype, T):
    """Phi(-|u|) to 2^-20 relative, and what the exponential makes of its argument u^2 / 2 log2 e: two roundings and
    that of log2 e itself, below 2^-26, together u^2 / 2 (2 + 1 / 2) 2^-24.  (A slope is Phi + u phi, two terms of which
    the second is rounded like the first.)  What is rounded to bf16 has a Phi to 2^-16.  Down to where Phi leaves the normal
    range."""
    u, y, db = outputs(L, np.linspace(-12.5, 12.5, N), "gelu", dtype, T=T)
    rel = 2.0 ** -20 + 1.25 * u * u * F32
    want = O.act(u, "gelu")
    own = 2.0 ** -16 if dtype == "bf16" else 0.0
    within(y, np.broadcast_to(want, y.shape), np.abs(want) * (rel + own + UNIT[dtype]), "y")
    phi = np.exp(-0.5 * u * u) / np.sqrt(2 * np.pi)
    size = np.abs(want) / np.maximum(np.abs(u), 1e-30) + np.abs(u) * phi
    within(db, O.act_slope(u, "gelu"), size * (rel + 2 * F32), "slope")


@pytest.mark.parametrize("T", [1, 200])
def test_silu_fp32(L, T):
    """s(u) from an exponential to 2 units, a sum and a quotient: 5 units with the product.  The slope s (1 + u (1 - s))
    has three roundings more."""
    u, y, db = outputs(L, np.linspace(-80.0, 80.0, N), "silu", "f32", T=T)
    want = O.act(u, "silu")
    within(y, np.broadcast_to(want, y.shape), 6 * F32 * np.abs(want), "y")
    e = np.exp(-np.abs(u))
    s, r = np.where(u < 0, e, 1.0) / (1 + e), np.where(u < 0, 1.0, e) / (1 + e)
    within(db, O.act_slope(u, "silu"), 12 * F32 * s * (1 + np.abs(u) * r), "slope")
