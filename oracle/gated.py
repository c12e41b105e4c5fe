"""float64 oracle of gated linear attention and of the head-row group norm
(NumPy, token by token, from the definitions).

Test infrastructure only: it shares no code with the CUDA path.  Every
function is pinned by tests/test_gated_oracle.py to something other than
itself (finite differences, the quadratic form, torch's library group norm).
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def forward(q, k, v, log_gate, scale=1.0, S_in=None):
    """(o, S): S_t = exp(log_gate_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.
    q [B, H, N, D]; k, v [B, Hkv, N, D]; log_gate [B, Hkv, N]."""
    q, k, v, S_in = (_f64(x) for x in (q, k, v, S_in))
    a = np.exp(_f64(log_gate))
    B, H, N, D = q.shape
    Hkv = k.shape[1]
    qg = q.reshape(B, Hkv, H // Hkv, N, D)
    S = np.zeros((B, Hkv, D, D)) if S_in is None else S_in.copy()
    o = np.zeros_like(qg)
    for t in range(N):
        S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, :, t] = scale * (qg[:, :, :, t] @ S)
    return o.reshape(B, H, N, D), S


def backward(q, k, v, log_gate, dO, scale=1.0, S_in=None, dS_out=None):
    """(dq, dk, dv, dlog_gate, dS_in) of sum(dO * o) + sum(dS_out * S): the
    chain rule through the recurrence, keeping every state."""
    q, k, v, dO, S_in, dS_out = (_f64(x) for x in (q, k, v, dO, S_in, dS_out))
    a = np.exp(_f64(log_gate))
    B, H, N, D = q.shape
    Hkv = k.shape[1]
    qg, dg = (x.reshape(B, Hkv, H // Hkv, N, D) for x in (q, dO))
    S = np.zeros((N + 1, B, Hkv, D, D))
    if S_in is not None:
        S[0] = S_in
    for t in range(N):
        S[t + 1] = a[:, :, t, None, None] * S[t] + k[:, :, t, :, None] * v[:, :, t, None, :]
    dq, dk, dv = np.zeros_like(qg), np.zeros_like(k), np.zeros_like(v)
    dl = np.zeros((B, Hkv, N))
    dS = np.zeros((B, Hkv, D, D)) if dS_out is None else dS_out.copy()
    for t in range(N - 1, -1, -1):
        qt, dt = qg[:, :, :, t], dg[:, :, :, t]
        dq[:, :, :, t] = scale * (dt @ S[t + 1].swapaxes(-1, -2))
        dS = dS + scale * (qt.swapaxes(-1, -2) @ dt)
        dk[:, :, t] = (dS @ v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (k[:, :, t, None, :] @ dS)[..., 0, :]
        dl[:, :, t] = a[:, :, t] * (S[t] * dS).sum((-1, -2))
        dS = a[:, :, t, None, None] * dS
    return dq.reshape(B, H, N, D), dk, dv, dl, dS


def decode_step(S, q, k, v, log_gate, scale=1.0):
    """(o, S) of one token: q [B, H, D], k, v [B, Hkv, D], log_gate [B, Hkv]."""
    q, k, v, lg = (_f64(x) for x in (q, k, v, log_gate))
    o, S = forward(q[:, :, None], k[:, :, None], v[:, :, None], lg[:, :, None], scale, S)
    return o[:, :, 0], S


def _act(x, act):
    return x / (1 + np.exp(-x)) if act == "silu" else x


def _dact(x, act):
    if act != "silu":
        return np.ones_like(x)
    s = 1 / (1 + np.exp(-x))
    return s + x * s * (1 - s)


def _rows(x, weight, bias, eps):
    B, H, N, D = x.shape
    x = x.transpose(0, 2, 1, 3)  # [B, N, H, D]
    c = x - x.mean(-1, keepdims=True)
    sd = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    xh = c / sd
    w = weight.reshape(H, D)
    return xh, sd, w, xh * w + (0 if bias is None else bias.reshape(H, D))


def group_norm(x, weight, bias=None, gate=None, act="silu", eps=1e-5):
    """y [B, N, H*D]: m = weight * x_hat + bias, y = m act(gate) or act(m)."""
    x, weight, bias, gate = (_f64(t) for t in (x, weight, bias, gate))
    B, H, N, D = x.shape
    m = _rows(x, weight, bias, eps)[3].reshape(B, N, H * D)
    return _act(m, act) if gate is None else m * _act(gate, act)


def group_norm_backward(x, weight, dy, bias=None, gate=None, act="silu", eps=1e-5):
    """(dx, dweight, dbias, dgate) of sum(dy * y); dgate None without a gate."""
    x, weight, bias, gate, dy = (_f64(t) for t in (x, weight, bias, gate, dy))
    B, H, N, D = x.shape
    xh, sd, w, m = _rows(x, weight, bias, eps)
    dy = dy.reshape(B, N, H, D)
    dgate = None
    if gate is None:
        dm = dy * _dact(m, act)
    else:
        g = gate.reshape(B, N, H, D)
        dgate = (dy * m * _dact(g, act)).reshape(B, N, H * D)
        dm = dy * _act(g, act)
    t = dm * w
    dx = (t - t.mean(-1, keepdims=True) - xh * (t * xh).mean(-1, keepdims=True)) / sd
    return (dx.transpose(0, 2, 1, 3), (dm * xh).sum((0, 1)).reshape(-1),
            dm.sum((0, 1)).reshape(-1), dgate)
