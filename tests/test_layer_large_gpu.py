"""Layer steps on tensors of more than 2^31 elements: what lies beyond the
32-bit offsets is what the same call gives for that part alone."""
import pytest
import torch

from layer_steps import library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return library()


def _fill(t, seed, scale=1.0):
    t.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
    return t.mul_(scale) if scale != 1.0 else t


def test_gated_scan(L):
    B, T, D = 1, 530_000, 4096        # 2.17e9 elements
    x = _fill(torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda"), 1)
    log_a = torch.empty_like(x).uniform_(-1.0, 0.0, generator=torch.Generator(device="cuda").manual_seed(2))
    y, state, chunks = L.gated_scan_forward(x, log_a, return_state=True, keep_chunks=True)
    # the last 1000 tokens, from the state that the kept chunk states give
    c = (T - 1000) // L.SCAN_CHUNK
    t0 = c * L.SCAN_CHUNK
    tail = lambda t: t[:, t0:].contiguous()
    y2, state2 = L.gated_scan_forward(tail(x), tail(log_a), state_in=chunks[:, c].contiguous(), return_state=True)
    assert torch.equal(y2, tail(y))
    torch.testing.assert_close(state2, state, rtol=1e-5, atol=1e-5)   # folded in other groups of chunks
    dy = y
    dx, dg, ds = L.gated_scan_backward(x, log_a, dy, chunks)
    dx2, dg2, _ = L.gated_scan_backward(tail(x), tail(log_a), tail(dy), chunks[:, c:].contiguous())
    assert torch.equal(dx2, tail(dx)) and torch.equal(dg2, tail(dg))
    assert torch.isfinite(ds).all() and L.device_status() == 0


def test_queries_and_keys(L):
    B, T, H, d = 1, 270_000, 64, 128   # 2.2e9 elements
    z = _fill(torch.empty(B, T, H * d, dtype=torch.bfloat16, device="cuda"), 3)
    sc, sh = torch.rand(4, H, d, device="cuda") + 0.5, torch.rand(4, H, d, device="cuda")
    out = L.qk_forward(z, sc, sh, rot_dim=128)
    t0 = T - 700
    part = L.qk_forward(z[:, t0:].contiguous(), sc, sh, rot_dim=128, pos0=t0)
    for a, b in zip(out, part):
        assert torch.equal(a[:, :, t0:], b)
    dz, dsc, dsh = L.qk_backward(z, sc, *out, rot_dim=128)
    dz2, _, _ = L.qk_backward(z[:, t0:].contiguous(), sc, *part, rot_dim=128, pos0=t0)
    assert torch.equal(dz[:, t0:], dz2)
    # dshift: column sums of the gradients (q_m, k_m are not turned), each within 270000 2^-24 of the sum of sizes
    for i in (2, 3):
        want = out[i].sum((0, 2), dtype=torch.float64)
        size = out[i].abs().sum((0, 2), dtype=torch.float64)
        assert ((dsh[i].double() - want).abs() <= T * 2.0 ** -24 * size).all()


def test_projection(L):
    M, N, K = 1_100_000, 2048, 64      # y: 2.25e9 elements
    x = _fill(torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), 4)
    w = _fill(torch.empty(N, K, dtype=torch.bfloat16, device="cuda"), 5, K ** -0.5)
    y = L.linear_forward(x, w)
    t0 = M - 4096
    assert torch.equal(y[t0:], L.linear_forward(x[t0:].contiguous(), w))
    dx, dw, db = L.linear_backward(x, w, y)
    dx2, _, _ = L.linear_backward(x[t0:].contiguous(), w, y[t0:].contiguous())
    # (fewer rows are summed in other parts: two sums cut by 2^-23 a step of 16, two roundings to bf16)
    mag = y[t0:].abs().double() @ w.abs().double()
    assert ((dx[t0:].double() - dx2.double()).abs() <= 2.0 ** -7 * dx2.abs().double() + N / 8 * 2.0 ** -23 * mag).all()
    want, size = y.sum(0, dtype=torch.float64), y.abs().sum(0, dtype=torch.float64)
    assert ((db.double() - want).abs() <= M * 2.0 ** -24 * size).all()
    # dw = y^T x on 8 of its rows, in fp64 (2^-24 a term, cut sums: 2^-23; one rounding to bf16)
    cols = torch.arange(0, N, N // 8, device="cuda")
    ref, mag = (torch.zeros(8, K, dtype=torch.float64, device="cuda") for _ in range(2))
    for a in range(0, M, 100_000):
        yc, xc = y[a:a + 100_000][:, cols].double(), x[a:a + 100_000].double()
        ref += yc.T @ xc
        mag += yc.abs().T @ xc.abs()
    assert ((dw[cols].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + M / 16 * 2.0 ** -23 * mag).all()
