"""Timed cases of the layer steps around the SCA + AWM path: the projection
(a matrix product with bias, activation and residual), the shared
query/key representation (per-head norm, affines and position rotation) and
the gated linear recurrence, each forward and as a training step.

``run`` computes a case either in plain torch operations in 32 bits
(``own = False``) or with the framework's calls (``own = True``); ``exact``
gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # value projection of one generated token for a batch of 8, written head by head
        dict(name="linear_token", op="linear", train=False, dtype="bf16", B=8, T=1, K=4096, N=4096, heads=32,
             act="silu", bias=True, residual=False),
        # value projection of a 32K-token prompt at the 7B width (32 heads of 128)
        dict(name="linear_prompt", op="linear", train=False, dtype="bf16", B=1, T=32768, K=4096, N=4096, heads=32,
             act="silu", bias=True, residual=False),
        # output projection with the layer's residual, three documents of odd length, odd widths
        dict(name="linear_residual_ragged", op="linear", train=False, dtype="bf16", B=3, T=1237, K=1288, N=1000,
             heads=0, act="none", bias=True, residual=True),
        # training step of the value projection on two 4096-token chunks
        dict(name="linear_train", op="linear", train=True, dtype="bf16", B=2, T=4096, K=4096, N=4096, heads=32,
             act="silu", bias=True, residual=False),
        # fp32 training step of a small feed-forward projection
        dict(name="linear_train_f32", op="linear", train=True, dtype="f32", B=1, T=777, K=1032, N=520, heads=0,
             act="gelu", bias=True, residual=True),
        # queries and keys of one generated token for a batch of 16, far into 4M-token sequences
        dict(name="qk_token", op="qk", train=False, dtype="bf16", B=16, T=1, H=32, d=128, rot=128,
             interleaved=False, far=True),
        # queries and keys of a 32K-token prompt at the 7B width
        dict(name="qk_prompt", op="qk", train=False, dtype="bf16", B=1, T=32768, H=32, d=128, rot=128,
             interleaved=False, far=False),
        # training step with half of each head rotated in interleaved pairs, odd length
        dict(name="qk_train", op="qk", train=True, dtype="bf16", B=2, T=5003, H=16, d=64, rot=32,
             interleaved=True, far=False),
        # one generated token for a batch of 32 with its carried state
        dict(name="scan_token", op="scan", train=False, dtype="bf16", B=32, L=1, D=4096, resets=False),
        # a 32K-token prompt at the 7B width
        dict(name="scan_prompt", op="scan", train=False, dtype="bf16", B=1, L=32768, D=4096, resets=False),
        # training step over packed documents, odd length
        dict(name="scan_train", op="scan", train=True, dtype="bf16", B=2, L=6007, D=2048, resets=True),
        # fp32 training step, short and narrow
        dict(name="scan_train_f32", op="scan", train=True, dtype="f32", B=3, L=1000, D=264, resets=True),
    ]


def _log_size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "qk", "scan"])
    train = rng.random() < 0.5
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "linear":
        limit = 2.0 ** (34 if dtype == "f32" else 37)    # products of one pass
        while True:
            hd = rng.choice([0, 64, 128])
            N = 8 * _log_size(rng, 8, 1024)
            heads = 0
            if hd:
                heads = max(1, N // hd)
                N = heads * hd
            c = dict(op=op, train=train, dtype=dtype, B=rng.choice([1, 1, 2, 3, 5]), T=_log_size(rng, 1, 16384),
                     K=8 * _log_size(rng, 8, 1024), N=N, heads=heads, act=rng.choice(["none", "silu", "gelu"]),
                     bias=rng.random() < 0.8, residual=rng.random() < 0.4)
            if c["B"] * c["T"] * c["K"] * c["N"] * (3 if train else 1) <= limit:
                return c
    if op == "qk":
        while True:
            d = rng.choice([64, 128])
            c = dict(op=op, train=train, dtype=dtype, B=rng.choice([1, 2, 3, 7]), T=_log_size(rng, 1, 30000),
                     H=rng.choice([1, 2, 5, 8, 16, 32]), d=d, rot=rng.choice([0, d // 4, d // 2, d]),
                     interleaved=rng.random() < 0.5, far=rng.random() < 0.3)
            if c["B"] * c["T"] * c["H"] * d * _BYTES[dtype] * (2 if train else 1) <= 1 << 28:
                return c
    while True:
        c = dict(op=op, train=train, dtype=dtype, B=rng.choice([1, 2, 3, 8]), L=_log_size(rng, 1, 30000),
                 D=8 * _log_size(rng, 2, 640), resets=rng.random() < 0.5)
        if c["B"] * c["L"] * c["D"] * _BYTES[dtype] * (2 if train else 1) <= 1 << 28:
            return c


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case=case)
    if case["op"] == "linear":
        B, T, K, N, H = (case[n] for n in ("B", "T", "K", "N", "heads"))
        out = (B, H, T, N // H) if H else (B, T, N)
        s["x"] = normal(B, T, K)
        s["w"] = normal(N, K, scale=K ** -0.5)
        s["bias"] = normal(N, scale=0.1, dtype=torch.float32) if case["bias"] else None
        s["residual"] = normal(*out) if case["residual"] else None
        s["dy"] = normal(*out) if case["train"] else None
    elif case["op"] == "qk":
        B, T, H, d = (case[n] for n in ("B", "T", "H", "d"))
        s["z"] = normal(B, T, H * d)
        s["scale"] = 1.0 + normal(4, H, d, scale=0.1, dtype=torch.float32)
        s["shift"] = normal(4, H, d, scale=0.1, dtype=torch.float32)
        s["pos"] = None
        if case["far"]:   # each sequence of the batch stands somewhere else in up to 4M tokens
            first = torch.randint(0, 4194304 - T, (B, 1), generator=g, device="cuda")
            s["pos"] = first + torch.arange(T, device="cuda")
        s["grads"] = [normal(B, H, T, d) for _ in range(4)] if case["train"] else None
    else:
        B, L, D = (case[n] for n in ("B", "L", "D"))
        # decays between a few tokens and some thousands of tokens, inputs scaled to keep the state near 1
        log_a = -torch.exp(1.5 * torch.randn(B, L, D, generator=g, device="cuda") - 3.0)
        s["x"] = (torch.randn(B, L, D, generator=g, device="cuda") * torch.sqrt(-torch.expm1(2.0 * log_a))).to(dt)
        s["log_a"] = log_a.to(dt)
        s["reset"] = None
        if case["resets"]:   # documents of about 700 tokens
            s["reset"] = (torch.rand(B, L, generator=g, device="cuda") < 1.0 / 700).to(torch.uint8)
        s["state"] = normal(B, D, dtype=torch.float32)
        s["dy"] = normal(B, L, D) if case["train"] else None
        s["dstate"] = normal(B, D, dtype=torch.float32) if case["train"] else None
    return s


# ------------------------------------------------------------- plain forms --

def _act(u, act):
    if act == "silu":
        return u * torch.sigmoid(u)
    if act == "gelu":
        return 0.5 * u * (1.0 + torch.erf(u * 0.5 ** 0.5))
    return u


def _act_slope(u, act):
    if act == "silu":
        sg = torch.sigmoid(u)
        return sg * (1.0 + u * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(u * 0.5 ** 0.5)) + u * torch.exp(-0.5 * u * u) * (2.0 * math.pi) ** -0.5
    return torch.ones_like(u)


def _split(t, B, T, H):
    return t.view(B, T, H, -1).transpose(1, 2) if H else t


def _merge(t, B, T, H):
    return t.transpose(1, 2).reshape(B, T, -1) if H else t


def _plain_linear(s):
    c = s["case"]
    B, T, H, dt = c["B"], c["T"], c["heads"], _DT[c["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    u = x @ w.t()
    if s["bias"] is not None:
        u = u + s["bias"]
    y = _split(_act(u, c["act"]), B, T, H)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(dt).contiguous()
    if not c["train"]:
        return y
    du = (_merge(s["dy"].float(), B, T, H) * _act_slope(u, c["act"])).reshape(B * T, -1)
    dx = (du @ w).to(dt).view_as(s["x"])
    dw = (du.t() @ x.reshape(B * T, -1)).to(dt)
    return [y, dx, dw, du.sum(0)]


def _rotation(s):
    """cos and sin of each position's angles [B or 1, 1, T, rot / 2]; the angles in 64 bits."""
    c = s["case"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["T"], device="cuda")[None]
    freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    ang = pos.double()[..., None] * freq
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]


def _pairs(t, c):
    r = t[..., :c["rot"]]
    return (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :c["rot"] // 2], r[..., c["rot"] // 2:])


def _rotate(t, cos, sin, c):
    if c["rot"] == 0:
        return t
    a, b = _pairs(t, c)
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if c["interleaved"] else torch.cat((u, v), -1)
    return torch.cat((r, t[..., c["rot"]:]), -1)


def _plain_qk(s):
    c = s["case"]
    B, T, H, d, dt = c["B"], c["T"], c["H"], c["d"], _DT[c["dtype"]]
    z = s["z"].float().view(B, T, H, d).transpose(1, 2)
    n = torch.clamp(torch.sqrt((z * z).sum(-1, keepdim=True)), min=1e-6)
    zn = z / n
    cos, sin = _rotation(s)
    kap, nu = s["scale"][:, None, :, None], s["shift"][:, None, :, None]
    q, k = _rotate(kap[0] * zn + nu[0], cos, sin, c), _rotate(kap[1] * zn + nu[1], cos, sin, c)
    outs = [q.to(dt).contiguous(), k.to(dt).contiguous(), (kap[2] * zn + nu[2]).to(dt).contiguous(),
            (kap[3] * zn + nu[3]).to(dt).contiguous()]
    if not c["train"]:
        return outs
    dq, dk, dqm, dkm = (t.float() for t in s["grads"])
    dq, dk = _rotate(dq, cos, -sin, c), _rotate(dk, cos, -sin, c)
    g = kap[0] * dq + kap[1] * dk + kap[2] * dqm + kap[3] * dkm
    dz = (g - zn * (zn * g).sum(-1, keepdim=True)) / n
    dz = dz.transpose(1, 2).reshape(B, T, H * d).to(dt)
    dscale = torch.stack([(t * zn).sum((0, 2)) for t in (dq, dk, dqm, dkm)])
    dshift = torch.stack([t.sum((0, 2)) for t in (dq, dk, dqm, dkm)])
    return outs + [dz, dscale, dshift]


def _doubling(a, h):
    """h_t + a_t h_{t-1} + a_t a_{t-1} h_{t-2} + ... along dim 1, by doubling the reach."""
    step = 1
    while step < h.shape[1]:
        h = torch.cat((h[:, :step], h[:, step:] + a[:, step:] * h[:, :-step]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return h


def _decay(s):
    a = torch.exp(s["log_a"].float())
    return a if s["reset"] is None else a * (s["reset"] == 0)[..., None]


def _plain_scan(s):
    c = s["case"]
    dt = _DT[c["dtype"]]
    a, x = _decay(s), s["x"].float()
    h0 = s["state"][:, None]
    first = x[:, :1] + a[:, :1] * h0
    h = _doubling(a, torch.cat((first, x[:, 1:]), 1))
    y = h.to(dt)
    if not c["train"]:
        return [y, h[:, -1].contiguous()]
    dy = s["dy"].float()
    last = dy[:, -1:] + s["dstate"][:, None]
    # the reverse recurrence: dh_t = dy_t + a_{t+1} dh_{t+1}
    back = torch.flip(torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1), (1,))
    dh = torch.flip(_doubling(back, torch.flip(torch.cat((dy[:, :-1], last), 1), (1,))), (1,))
    before = torch.cat((h0, h[:, :-1]), 1)
    return [y, h[:, -1].contiguous(), dh.to(dt), (dh * a * before).to(dt), a[:, 0] * dh[:, 0]]


# --------------------------------------------------------- framework calls --

def _own_linear(s):
    from long_context_sequence_sca_b200 import lib
    c = s["case"]
    kw = dict(act=c["act"], heads=c["heads"])
    if not c["train"]:
        return lib.linear_forward(s["x"], s["w"], bias=s["bias"], residual=s["residual"], **kw)
    y, pre = lib.linear_forward(s["x"], s["w"], bias=s["bias"], residual=s["residual"], keep_pre=True, **kw)
    return [y, *lib.linear_backward(s["x"], s["w"], s["dy"], pre=pre, **kw)]


def _own_qk(s):
    from long_context_sequence_sca_b200 import lib
    c = s["case"]
    kw = dict(rot_dim=c["rot"], interleaved=c["interleaved"], pos=s["pos"])
    outs = list(lib.qk_forward(s["z"], s["scale"], s["shift"], **kw))
    return outs + list(lib.qk_backward(s["z"], s["scale"], *s["grads"], **kw)) if c["train"] else outs


def _own_scan(s):
    from long_context_sequence_sca_b200 import lib
    c = s["case"]
    if not c["train"]:
        return list(lib.gated_scan_forward(s["x"], s["log_a"], reset=s["reset"], state_in=s["state"],
                                           return_state=True))
    y, state, chunks = lib.gated_scan_forward(s["x"], s["log_a"], reset=s["reset"], state_in=s["state"],
                                              return_state=True, keep_chunks=True)
    return [y, state, *lib.gated_scan_backward(s["x"], s["log_a"], s["dy"], chunks, reset=s["reset"],
                                               dstate_out=s["dstate"])]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "qk": _own_qk, "scan": _own_scan}[op](state)
    return {"linear": _plain_linear, "qk": _plain_qk, "scan": _plain_scan}[op](state)


def work(case):
    e, tr = _BYTES[case["dtype"]], case["train"]
    if case["op"] == "linear":
        M, N, K = case["B"] * case["T"], case["N"], case["K"]
        byts = e * (M * K + N * K + M * N * (2 if case["residual"] else 1)) + 4 * N * case["bias"]
        if tr:   # dy in; dx, dw, db out
            byts += e * (M * N + M * K + N * K) + 4 * N
        return {"bytes": byts, "flops": 2 * M * N * K * (3 if tr else 1)}
    if case["op"] == "qk":
        hd = case["H"] * case["d"]
        n = case["B"] * case["T"] * hd
        byts = 5 * n * e + 32 * hd + (8 * case["B"] * case["T"] if case["far"] else 0)
        if tr:   # four gradients in; dz, dscale, dshift out
            byts += 5 * n * e + 32 * hd
        return {"bytes": byts, "flops": n * (45 if tr else 17)}
    n, bd = case["B"] * case["L"] * case["D"], case["B"] * case["D"]
    byts = n * e * (6 if tr else 3) + 4 * bd * (4 if tr else 2) + (case["B"] * case["L"] if case["resets"] else 0)
    return {"bytes": byts, "flops": n * (7 if tr else 3)}


# ------------------------------------------------- the definitions, 64 bits --

def _exact_linear(s):
    """y[m, n] = f(sum_k x[m, k] w[n, k] + b[n]) + r[m, n]; gradients by the chain rule."""
    c = s["case"]
    B, T, N, K, H = c["B"], c["T"], c["N"], c["K"], c["heads"]
    X, W = s["x"].double().reshape(-1, K), s["w"].double()
    U = torch.einsum("mk,nk->mn", X, W)
    if s["bias"] is not None:
        U += s["bias"].double()
    f = {"none": lambda u: u, "silu": lambda u: u / (1 + torch.exp(-u)),
         "gelu": lambda u: u * torch.special.ndtr(u)}[c["act"]]
    Y = f(U).reshape(B, T, N)
    if H:
        Y = Y.reshape(B, T, H, N // H).permute(0, 2, 1, 3)
    if s["residual"] is not None:
        Y = Y + s["residual"].double()
    if not c["train"]:
        return Y
    G = s["dy"].double()
    G = (G.permute(0, 2, 1, 3) if H else G).reshape(-1, N)
    if c["act"] == "silu":
        e = torch.exp(-U)
        G = G * (1 / (1 + e) + U * e / (1 + e) ** 2)
    elif c["act"] == "gelu":
        G = G * (torch.special.ndtr(U) + U * torch.exp(-U ** 2 / 2) / math.sqrt(2 * math.pi))
    return [Y, torch.einsum("mn,nk->mk", G, W).reshape(B, T, K), torch.einsum("mn,mk->nk", G, X), G.sum(0)]


def _exact_qk(s):
    """z' = z / max(|z|, 1e-6) per head; q, k, qm, km = scale_i z' + shift_i, and q, k as complex
    numbers times e^(i angle) on the rotated pairs."""
    c = s["case"]
    B, T, H, d, R = c["B"], c["T"], c["H"], c["d"], c["rot"]
    Z = s["z"].double().reshape(B, T, H, d)
    norm = torch.linalg.vector_norm(Z, dim=-1, keepdim=True).clamp_min(1e-6)
    unit = Z / norm
    S, F = s["scale"].double(), s["shift"].double()
    turn = None
    if R:
        where = (s["pos"] if s["pos"] is not None else torch.arange(T, device="cuda").expand(B, T)).double()
        rate = torch.exp(-math.log(10000.0) * torch.arange(R // 2, device="cuda", dtype=torch.float64) * 2 / R)
        turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), where[:, :, None, None] * rate)
    even = torch.arange(0, R, 2) if c["interleaved"] else torch.arange(R // 2)
    odd = even + (1 if c["interleaved"] else R // 2)

    def turned(t, by):
        if not R:
            return t
        w = torch.complex(t[..., even], t[..., odd]) * by
        t = t.clone()
        t[..., even], t[..., odd] = w.real, w.imag
        return t

    outs = [unit * S[i] + F[i] for i in range(4)]
    outs[:2] = [turned(t, turn) for t in outs[:2]]
    outs = [t.permute(0, 2, 1, 3) for t in outs]
    if not c["train"]:
        return outs
    G = [t.double().permute(0, 2, 1, 3) for t in s["grads"]]
    if R:
        G[:2] = [turned(t, turn.conj()) for t in G[:2]]
    up = sum(G[i] * S[i] for i in range(4))
    dz = (up - unit * (up * unit).sum(-1, keepdim=True)) / norm
    return outs + [dz.reshape(B, T, H * d), torch.stack([(t * unit).sum((0, 1)) for t in G]),
                   torch.stack([t.sum((0, 1)) for t in G])]


def _exact_scan(s):
    """h_t = a_t h_{t-1} + x_t one token after another, and its reverse."""
    c = s["case"]
    L = c["L"]
    a = torch.exp(s["log_a"].double())
    if s["reset"] is not None:
        a[s["reset"] != 0] = 0.0
    h = torch.empty_like(a)
    prev = s["state"].double()
    for t in range(L):
        prev = torch.addcmul(s["x"][:, t].double(), a[:, t], prev)
        h[:, t] = prev
    if not c["train"]:
        return [h, prev]
    dh, carry = torch.empty_like(a), s["dstate"].double()
    for t in range(L - 1, -1, -1):
        dh[:, t] = s["dy"][:, t].double() + carry
        carry = a[:, t] * dh[:, t]
    before = torch.cat((s["state"].double()[:, None], h[:, :-1]), 1)
    return [h, prev, dh, dh * a * before, carry]


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "qk": _exact_qk, "scan": _exact_scan}[case["op"]](s)
