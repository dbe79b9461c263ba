"""The layer steps as a user runs them: one whole layer with its gradients,
other streams, CUDA graphs, two calls at once."""
import numpy as np
import pytest
import torch

from layer_steps import library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return library()


def _layer_inputs(B, T, H, d, dtype, seed):
    D = H * d
    r = torch.Generator().manual_seed(seed)
    n = lambda *s, scale=1.0: torch.randn(*s, generator=r) * scale
    p = dict(x=n(B, T, D), log_a=-torch.exp(n(B, T, D) - 1.0), wz=n(D, D, scale=D ** -0.5), bz=n(D, scale=0.1),
             wv=n(D, D, scale=D ** -0.5), bv=n(D, scale=0.1), wo=n(D, D, scale=D ** -0.5), scale=1 + 0.1 * n(4, H, d),
             shift=0.1 * n(4, H, d))
    keep = ("bz", "bv", "scale", "shift")   # fp32 parameters
    return {k: v.cuda() if k in keep else v.to(dtype).cuda() for k, v in p.items()}


def _layer(L, p, c, rot):
    B, T, D = p["x"].shape
    H = p["scale"].shape[1]
    h, _ = L.GatedScanFunction.apply(p["x"], p["log_a"], None, None)
    z = L.LinearFunction.apply(h, p["wz"], p["bz"], None, "none", 0)
    v = L.LinearFunction.apply(h, p["wv"], p["bv"], None, "silu", H)
    q, k, qm, km = L.QkFunction.apply(z, p["scale"], p["shift"], None, dict(rot_dim=rot))
    o_sca, o_mem = L.ScaAwmFunction.apply(q, k, v, qm, km, c)
    o = (o_sca + o_mem).transpose(1, 2).reshape(B, T, D)
    return L.LinearFunction.apply(o, p["wo"], None, p["x"], "none", 0)


def _layer_fp64(p, c, rot):
    """The same layer in plain torch, fp64, differentiable."""
    B, T, D = p["x"].shape
    H, d = p["scale"].shape[1:]
    a = torch.exp(p["log_a"])
    h, hs = torch.zeros_like(p["x"][:, 0]), []
    for t in range(T):
        h = a[:, t] * h + p["x"][:, t]
        hs.append(h)
    h = torch.stack(hs, 1)
    heads = lambda t: t.view(B, T, H, d).transpose(1, 2)
    z = heads(h @ p["wz"].T + p["bz"])
    v = heads(torch.nn.functional.silu(h @ p["wv"].T + p["bv"]))
    z = z / z.norm(dim=-1, keepdim=True)
    q, k, qm, km = (z * p["scale"][i][:, None] + p["shift"][i][:, None] for i in range(4))
    if rot:
        ang = torch.arange(T, device=z.device).double()[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, device=z.device).double() / rot)
        cs, sn = ang.cos(), ang.sin()

        def turn(t):
            x1, x2 = t[..., :rot // 2], t[..., rot // 2:rot]
            return torch.cat([x1 * cs - x2 * sn, x2 * cs + x1 * sn, t[..., rot:]], -1)

        q, k = turn(q), turn(k)
    i = torch.arange(T, device=z.device)
    vis = (i[None] <= i[:, None]) & (i[None] // c >= i[:, None] // c - 1)
    o = torch.softmax((q @ k.transpose(-1, -2)).masked_fill(~vis, -torch.inf), -1) @ v
    S = T // c
    M = [torch.zeros(B, H, d, d, dtype=torch.float64, device=z.device)] * 2   # M'_0, M'_1
    logz, mem = torch.full((B, H, d), -torch.inf, dtype=torch.float64, device=z.device), []
    for s in range(S):
        sl = slice(s * c, (s + 1) * c)
        mem.append(torch.softmax(qm[:, :, sl], -1) @ M[s])       # chunk s + 1 reads M'_s
        nz = torch.logaddexp(logz, torch.logsumexp(km[:, :, sl], 2))
        phi = torch.exp(km[:, :, sl] - nz[:, :, None])
        psi = torch.softmax(km[:, :, sl], -1)
        M.append(torch.exp(logz - nz)[..., None] * M[-1] + phi.transpose(-1, -2) @ (v[:, :, sl] - psi @ M[-1]))
        logz = nz
    o = (o + torch.cat(mem, 2)).transpose(1, 2).reshape(B, T, D)
    return o @ p["wo"].T + p["x"]


# Relative 2-norm of each result against fp64.  fp32: every stage is within
# about 1e-6 of its own result, ten of them in a row; bf16: about 20 stored
# intermediates, each off by up to 2^-8 (2^-9.2 in the 2-norm), adding up as
# independent errors to 2^-9.2 sqrt(20) < 1e-2, twice that through the
# softmax's and the norm's amplification.
@pytest.mark.parametrize("dtype,H,d,bar", [(torch.float32, 2, 64, 2e-5), (torch.bfloat16, 2, 128, 2e-2)])
def test_layer_and_gradients(L, dtype, H, d, bar):
    c = 128
    p = _layer_inputs(2, 4 * c, H, d, dtype, seed=1)
    leaves = {k: v.requires_grad_() for k, v in p.items()}
    y = _layer(L, leaves, c, 32)
    gen = torch.Generator().manual_seed(2)
    dy = torch.randn(y.shape, generator=gen).cuda()
    y.backward(dy.to(dtype))
    assert L.device_status() == 0
    ref = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    want = _layer_fp64(ref, c, 32)
    want.backward(dy.to(dtype).double())
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    errs = {"y": rel(y.detach(), want.detach())}
    errs.update({k: rel(leaves[k].grad, ref[k].grad) for k in leaves})
    assert all(np.isfinite(e) and e <= bar for e in errs.values()), errs


def _all_calls(L, p):
    """Every entry point once; a flat list of its outputs."""
    H = p["scale"].shape[1]
    y, s, ch = L.gated_scan_forward(p["x"], p["log_a"], return_state=True, keep_chunks=True)
    outs = [y, s, ch, *L.gated_scan_backward(p["x"], p["log_a"], y, ch)]
    v, pre = L.linear_forward(y, p["wv"], bias=p["bv"], act="silu", heads=H, keep_pre=True)
    outs += [v, pre, *L.linear_backward(y, p["wv"], v, pre=pre, act="silu", heads=H)]
    qk = L.qk_forward(y, p["scale"], p["shift"], rot_dim=32)
    return outs + [*qk, *L.qk_backward(y, p["scale"], *qk, rot_dim=32)]


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 700])
def test_captured_and_replayed(L, T):
    """Two graphs of the whole set, replayed in turn on new inputs, between eager calls of other sizes."""
    p, q = (_layer_inputs(2, T, 2, 64, torch.bfloat16, seed=s) for s in (3, 4))
    other = _layer_inputs(1, 900, 4, 64, torch.bfloat16, seed=5)
    want_p, want_q = _all_calls(L, p), _all_calls(L, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all_calls(L, p)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for inp in (p, q):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _all_calls(L, inp)
        graphs.append((g, outs))
    for _ in range(2):
        for g, outs in graphs:
            for o in outs:
                o.zero_()
        _all_calls(L, other)
        for g, _outs in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert _equal(graphs[0][1], want_p) and _equal(graphs[1][1], want_q)
    swap = {k: p[k].clone() for k in p}
    for k in p:
        p[k].copy_(q[k])
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert _equal(graphs[0][1], want_q)
    for k in p:
        p[k].copy_(swap[k])


def test_two_streams_at_once(L):
    ps = [_layer_inputs(2, 3000, 4, 64, torch.bfloat16, seed=s) for s in (6, 7)]
    want = [_all_calls(L, p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[] for _ in ps]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_all_calls(L, ps[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(_equal(g, want[i]) for g in got[i])


def test_stream_argument(L):
    """stream= runs the call, and allocates its outputs, on that stream."""
    p = _layer_inputs(2, 300, 2, 64, torch.bfloat16, seed=8)
    want = L.linear_forward(p["x"], p["wz"], bias=p["bz"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y = L.linear_forward(p["x"], p["wz"], bias=p["bz"], stream=s)
        h = L.gated_scan_forward(y, p["log_a"], stream=s)
        qk = L.qk_forward(h, p["scale"], p["shift"], stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    assert _equal(qk, L.qk_forward(L.gated_scan_forward(want, p["log_a"]), p["scale"], p["shift"]))


def test_working_memory_needs_no_initial_contents(L):
    """Workspaces full of NaN patterns change nothing."""
    p = _layer_inputs(1, 600, 2, 64, torch.bfloat16, seed=9)
    want = _all_calls(L, p)
    real = torch.empty

    def dirty(*a, **kw):
        t = real(*a, **kw)
        return t.view(torch.uint8).fill_(255).view(t.dtype) if t.numel() and t.is_cuda else t

    L.torch.empty = dirty
    try:
        got = _all_calls(L, p)
    finally:
        L.torch.empty = real
    assert _equal(got, want)


def test_refusals(L):
    p = _layer_inputs(1, 64, 2, 64, torch.bfloat16, seed=10)
    x, w = p["x"], p["wz"]
    with pytest.raises(ValueError):
        L.linear_forward(x.transpose(1, 2), w)
    with pytest.raises(ValueError):
        L.linear_forward(x, w.float())
    with pytest.raises(ValueError):
        L.linear_forward(x, w, bias=p["bz"].bfloat16())
    with pytest.raises(ValueError):
        L.linear_forward(x, w, act="relu")
    with pytest.raises(ValueError):
        L.linear_forward(x, w, heads=3)
    with pytest.raises(ValueError):
        L.linear_forward(x, w, y=torch.empty(1, 64, 64, dtype=x.dtype, device="cuda"))
    with pytest.raises(L.GeckoError):
        L.linear_backward(x, w, x, act="silu")                       # no pre
    with pytest.raises(L.GeckoError):
        L.linear_backward(x, w, x, need=(False, False, False))
    with pytest.raises(L.GeckoError):
        L.linear_forward(x[..., :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(ValueError):
        L.gated_scan_forward(x, p["log_a"].float())
    with pytest.raises(ValueError):
        L.gated_scan_forward(x, p["log_a"], reset=torch.zeros(1, 64, device="cuda"))
    with pytest.raises(ValueError):
        L.gated_scan_forward(x.cpu(), p["log_a"])
    with pytest.raises(L.GeckoError):
        L.gated_scan_forward(x[..., :20].contiguous(), p["log_a"][..., :20].contiguous())
    with pytest.raises(L.GeckoError):
        L.gated_scan_forward(x[:, :0].contiguous(), p["log_a"][:, :0].contiguous())
    with pytest.raises(ValueError):
        L.gated_scan_backward(x, p["log_a"], x, torch.zeros(1, 2, 128, device="cuda"))
    with pytest.raises(ValueError):
        L.qk_forward(x, p["scale"][:, :1].contiguous(), p["shift"])
    with pytest.raises(ValueError):
        L.qk_forward(x, p["scale"], p["shift"], pos=torch.arange(64, device="cuda"))
    with pytest.raises(L.GeckoError):
        L.qk_forward(x, p["scale"], p["shift"], rot_dim=24)
    with pytest.raises(L.GeckoError):
        L.qk_forward(x, p["scale"].view(4, 4, 32).contiguous(), p["shift"].view(4, 4, 32).contiguous())
    odd = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view_as(x)
    with pytest.raises(L.GeckoError):
        L.gated_scan_forward(odd, p["log_a"])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_calls_without_a_pause(L, dtype, captured):
    """Inputs written right before a call and overwritten right after it, several
    calls in a row on one stream: a call's kernels overlap with each other, and with
    nothing else.  The results are those of calls with a pause, bit for bit."""
    n = 4
    ps = [_layer_inputs(2, 300, 2, 64, dtype, seed=20 + i) for i in range(n)]
    now = {k: torch.empty_like(v) for k, v in ps[0].items()}

    def calls(p):
        y, st, ch = L.gated_scan_forward(p["x"], p["log_a"], return_state=True, keep_chunks=True)
        dx, dg, ds = L.gated_scan_backward(p["x"], p["log_a"], y, ch, dstate_out=st)
        v, pre = L.linear_forward(p["x"], p["wv"], bias=p["bv"], act="silu", heads=2, keep_pre=True)
        du = L.linear_backward(p["x"], p["wv"], v, pre=pre, act="silu", heads=2)
        q = L.qk_forward(p["x"], p["scale"], p["shift"], rot_dim=64)
        return [y, st, ch, dx, dg, ds, v, pre, *du, *q, *L.qk_backward(p["x"], p["scale"], *q, rot_dim=64)]

    want = []
    for p in ps:
        want.append(calls(p))
        torch.cuda.synchronize()

    def row():
        got = []
        for p in ps:
            for k, v in now.items():
                v.copy_(p[k])
            got.append(calls(now))
            for v in now.values():
                v.fill_(float("nan"))
        return got

    if captured:
        with torch.cuda.stream(torch.cuda.Stream()):
            row()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = row()
        for _ in range(3):
            graph.replay()
    else:
        got = row()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for s, t in zip(a, b):
            assert torch.equal(s, t)
