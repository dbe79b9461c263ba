"""bf16 products of much depth: the tensor core's cut sums do not draw them to zero.

A sum of positive terms loses about 2^-23.5 of itself every 16 terms (measured;
2^-25.5 where their signs are random): 6e-3 after a million, always in the same
direction.  One rounding to bf16
errs by 2^-8 / sqrt 3 at most in the mean square, in either direction, so that the mean
of n relative errors is within 6 2^-8 / sqrt(3 n) but for one draw in 5e8."""
import pytest
import torch

from layer_steps import library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return library()


def _positive(rows, cols, seed):
    """Uniform in [0, 1), the columns scaled by a factor in [1, 2) each, so that results are spread over binades."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.rand(rows, cols, generator=g, device="cuda")
    return t.mul_(1 + torch.rand(cols, generator=g, device="cuda")).bfloat16()


def _unbiased(got, want, cut):
    rel = (got.double() - want) / want
    assert rel.abs().max() <= 2.0 ** -8 + cut
    assert rel.mean().abs() <= 6 * 2.0 ** -8 / (3 * rel.numel()) ** 0.5 + cut


# What may be lost where the accumulator is emptied: 2^13 of the depth at most in one sum, 512 steps (2^-14.5),
# and fp32 additions of the parts.
CUT = 2.0 ** -14


@pytest.mark.parametrize("M,N,K", [(1 << 21, 512, 264), (1_000_003, 2048, 1032), (400_000, 128, 136),
                                   (300_001, 1200, 96)])
def test_weight_gradient(L, M, N, K):
    """dw over 300 thousand to two million tokens: with its depth in parts, and with whole tiles."""
    x, dy = _positive(M, K, 1), _positive(M, N, 2)
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    _, dw, _ = L.linear_backward(x, w, dy, need=(False, True, False))
    cols = torch.arange(0, N, N // 16, device="cuda")
    want = torch.zeros(cols.numel(), K, dtype=torch.float64, device="cuda")
    for a in range(0, M, 100_000):
        want += dy[a:a + 100_000][:, cols].double().T @ x[a:a + 100_000].double()
    _unbiased(dw[cols], want, CUT)


@pytest.mark.parametrize("M,keep_pre,D", [(1, False, 1 << 20), (100, False, 1 << 20), (100, True, 1 << 20),
                                          (600, False, 1 << 20), (1, False, 131072), (128, False, 100_000),
                                          (600, False, 131072), (300, False, 33_000)])
def test_forward_and_input_gradient(L, M, keep_pre, D):
    """y of as many features, dx of as many."""
    n = 264
    x, w = _positive(D, M, 3).T.contiguous(), _positive(D, n, 4).T.contiguous()
    out = L.linear_forward(x, w, keep_pre=keep_pre)
    y = out[0] if keep_pre else out
    want = torch.zeros(M, n, dtype=torch.float64, device="cuda")
    for a in range(0, D, 65536):
        want += x[:, a:a + 65536].double() @ w[:, a:a + 65536].double().T
    _unbiased(y, want, CUT)
    if keep_pre:
        return
    dx, _, _ = L.linear_backward(torch.zeros(M, n, dtype=x.dtype, device="cuda"), w.T.contiguous(), x,
                                 need=(True, False, False))
    _unbiased(dx, want, CUT)


def test_captured_and_at_once(L):
    """Deep products (in runs of the large tiles, of the cluster tiles, in parts) captured and replayed on new inputs,
    and on two streams at once, are what a call alone gives, bit for bit."""
    sizes = [(40_000, 2048, 1536), (50_000, 128, 136), (20_000, 1024, 1024), (90_000, 256, 264)]
    x, dy = ([_positive(M, n, i) for i, (M, *nk) in enumerate(sizes) for n in (nk[j],)] for j in (1, 0))
    w = [torch.zeros(N, K, dtype=torch.bfloat16, device="cuda") for _, N, K in sizes]
    calls = lambda: [L.linear_backward(*a, need=(False, True, False))[1] for a in zip(x, w, dy)]
    want = calls()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(2):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for t in x:
        t.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, 2 * b) for a, b in zip(outs, want))
