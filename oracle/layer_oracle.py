"""Plain fp64 CPU oracle for the layer steps around the SCA + AWM path: the
gated linear recurrence, the queries and keys from the shared representation,
and the projection, each with its gradients.

TEST INFRASTRUCTURE ONLY.  Only ``tests/`` and ``__graft_entry__.smoke()`` may
import this module.  The product path never calls it and shares no code with
it.  All arithmetic is float64; every function takes and returns NumPy arrays.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["decay", "gated_scan", "gated_scan_grad", "turns", "qk", "qk_grad", "act", "act_slope", "split_heads",
           "merge_heads", "linear", "linear_grad"]


# ------------------------------------------------------------- recurrence --

def decay(log_a, reset=None):
    """a = exp(log_a), 0 where a document starts."""
    a = np.exp(np.asarray(log_a, np.float64))
    return a if reset is None else np.where(np.asarray(reset)[..., None] != 0, 0.0, a)


def _times(a, h):
    """a h, with a zero gate dropping h whatever it holds."""
    return np.where(a == 0.0, 0.0, a * np.where(a == 0.0, 0.0, h))


def gated_scan(x, log_a, state=None, reset=None):
    """(h [B, L, D], last state): h_t = a_t h_{t-1} + x_t, token by token."""
    x, a = np.asarray(x, np.float64), decay(log_a, reset)
    B, L, D = x.shape
    h, prev = np.empty_like(x), np.zeros((B, D)) if state is None else np.asarray(state, np.float64)
    for t in range(L):
        prev = _times(a[:, t], prev) + x[:, t]
        h[:, t] = prev
    return h, prev


def gated_scan_grad(x, log_a, dy, state=None, reset=None, dstate=None):
    """(dx, dlog_a, dstate_in) for the gradients dy of h and dstate of the last state."""
    dy, a = np.asarray(dy, np.float64), decay(log_a, reset)
    h, _ = gated_scan(x, log_a, state, reset)
    B, L, D = dy.shape
    first = np.zeros((B, 1, D)) if state is None else np.asarray(state, np.float64)[:, None]
    before = np.concatenate([first, h[:, :-1]], 1)
    back = np.zeros((B, D)) if dstate is None else np.asarray(dstate, np.float64)
    dx, dg = np.empty_like(dy), np.empty_like(dy)
    for t in range(L - 1, -1, -1):
        dx[:, t] = dy[:, t] + back
        back = _times(a[:, t], dx[:, t])
        dg[:, t] = _times(a[:, t], dx[:, t] * before[:, t])
    return dx, dg, back


# --------------------------------------------------------- queries and keys --

def turns(pos, rot_dim, base):
    """Angles [..., rot_dim / 2] = pos base^(-2 i / rot_dim)."""
    rate = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    return np.asarray(pos, np.float64)[..., None] * rate


def _turn(p, ang, rot_dim, interleaved):
    """p [B, T, H, d] with the pairs of its first rot_dim features turned by ang [B, T, rot_dim / 2]."""
    if rot_dim == 0:
        return p
    ia = np.arange(0, rot_dim, 2) if interleaved else np.arange(rot_dim // 2)
    ib = ia + (1 if interleaved else rot_dim // 2)
    c, s = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None]
    out = p.copy()
    out[..., ia] = p[..., ia] * c - p[..., ib] * s
    out[..., ib] = p[..., ib] * c + p[..., ia] * s
    return out


def _heads(z, H):
    z = np.asarray(z, np.float64)
    return z.reshape(z.shape[0], z.shape[1], H, -1)


def qk(z, scale, shift, eps, rot_dim=0, base=10000.0, interleaved=False, pos=None):
    """[q, k, qm, km], each [B, H, T, d]; pos [B, T]."""
    scale, shift = np.asarray(scale, np.float64), np.asarray(shift, np.float64)
    zh = _heads(z, scale.shape[1])
    unit = zh / np.maximum(np.sqrt((zh * zh).sum(-1, keepdims=True)), eps)
    out = [unit * scale[i] + shift[i] for i in range(4)]
    if rot_dim:
        ang = turns(pos, rot_dim, base)
        out = [_turn(p, ang, rot_dim, interleaved) if i < 2 else p for i, p in enumerate(out)]
    return [p.transpose(0, 2, 1, 3) for p in out]


def qk_grad(z, scale, grads, eps, rot_dim=0, base=10000.0, interleaved=False, pos=None):
    """(dz, dscale, dshift) for the gradients [dq, dk, dqm, dkm] [B, H, T, d]."""
    scale = np.asarray(scale, np.float64)
    zh = _heads(z, scale.shape[1])
    norm = np.sqrt((zh * zh).sum(-1, keepdims=True))
    n = np.maximum(norm, eps)
    unit = zh / n
    g = [np.asarray(p, np.float64).transpose(0, 2, 1, 3) for p in grads]
    if rot_dim:
        ang = turns(pos, rot_dim, base)
        g = [_turn(p, -ang, rot_dim, interleaved) if i < 2 else p for i, p in enumerate(g)]
    up = sum(scale[i] * g[i] for i in range(4))
    along = np.where(norm > eps, (unit * up).sum(-1, keepdims=True), 0.0)
    dz = (up - unit * along) / n
    return (dz.reshape(dz.shape[0], dz.shape[1], -1), np.stack([(p * unit).sum((0, 1)) for p in g]),
            np.stack([p.sum((0, 1)) for p in g]))


# --------------------------------------------------------------- projection --

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(u, name):
    if name == "silu":
        return u / (1.0 + np.exp(-u))
    if name == "gelu":
        return 0.5 * u * _erfc(-u / math.sqrt(2.0))
    return u


def act_slope(u, name):
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-u))
        return s * (1.0 + u * (1.0 - s))
    if name == "gelu":
        return 0.5 * _erfc(-u / math.sqrt(2.0)) + u * np.exp(-0.5 * u * u) / math.sqrt(2.0 * math.pi)
    return np.ones_like(u)


def split_heads(y, H):
    """[B, T, N] -> [B, H, T, N / H] (H = 0: as it is)."""
    return y.reshape(*y.shape[:2], H, -1).transpose(0, 2, 1, 3) if H else y


def merge_heads(y, H):
    return y.transpose(0, 2, 1, 3).reshape(y.shape[0], y.shape[2], -1) if H else y


def linear(x, w, bias=None, residual=None, name="none", H=0):
    """(y, u), both in y's layout."""
    u = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        u = u + np.asarray(bias, np.float64)
    y = split_heads(act(u, name), H)
    return (y if residual is None else y + np.asarray(residual, np.float64)), split_heads(u, H)


def linear_grad(x, w, dy, bias=None, name="none", H=0):
    """(dx, dw, db, du [B, T, N])."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    u = x @ w.T + (0.0 if bias is None else np.asarray(bias, np.float64))
    du = merge_heads(np.asarray(dy, np.float64), H) * act_slope(u, name)
    return du @ w, np.einsum("btn,btk->nk", du, x), du.sum((0, 1)), du
