"""Pins of the float64 oracle of gated linear attention and of the head-row
group norm (oracle/gated.py), on the CPU: the quadratic form, finite
differences, special cases and torch's library group norm."""
import numpy as np
import pytest
import torch

from oracle import gated


def tensors(B, H, Hkv, N, D, seed=0):
    r = np.random.default_rng(seed)
    q, dO = r.standard_normal((2, B, H, N, D))
    k, v = r.standard_normal((2, B, Hkv, N, D))
    lg = -np.exp(r.standard_normal((B, Hkv, N)))
    S, dS = r.standard_normal((2, B, Hkv, D, D))
    return q, k, v, lg, dO, S, dS


def test_forward_is_the_quadratic_form():
    q, k, v, lg, _, S, _ = tensors(2, 4, 2, 9, 3)
    o, S_out = gated.forward(q, k, v, lg, 0.7, S)
    G = np.cumsum(lg, -1)
    for b in range(2):
        for h in range(4):
            c = h // 2
            for i in range(9):
                want = np.exp(G[b, c, i]) * q[b, h, i] @ S[b, c]
                for j in range(i + 1):
                    want = want + np.exp(G[b, c, i] - G[b, c, j]) * (q[b, h, i] @ k[b, c, j]) * v[b, c, j]
                np.testing.assert_allclose(o[b, h, i], 0.7 * want, rtol=1e-12, atol=1e-13)
    want = np.exp(G[..., -1])[..., None, None] * S
    want = want + np.einsum("bcn,bcnd,bcne->bcde", np.exp(G[..., -1:] - G), k, v)
    np.testing.assert_allclose(S_out, want, rtol=1e-12, atol=1e-13)


def test_a_gate_of_zero_starts_a_new_document():
    q, k, v, lg, dO, S, _ = tensors(1, 2, 2, 10, 4, 1)
    lg[:, :, 6] = -np.inf
    o, S_out = gated.forward(q, k, v, lg, 1.0, S)
    o2, S2 = gated.forward(q[:, :, 6:], k[:, :, 6:], v[:, :, 6:], lg[:, :, 6:])
    np.testing.assert_allclose(o[:, :, 6:], o2, rtol=1e-13)
    np.testing.assert_allclose(S_out, S2, rtol=1e-13)
    dq, dk, dv, dl, dS = gated.backward(q, k, v, lg, dO, 1.0, S)
    g2 = gated.backward(q[:, :, 6:], k[:, :, 6:], v[:, :, 6:], lg[:, :, 6:], dO[:, :, 6:])
    for a, b in zip((dq, dk, dv, dl), g2):
        np.testing.assert_allclose(a[:, :, 6:], b, rtol=1e-12, atol=1e-13)
    assert (dl[:, :, 6] == 0).all() and np.isfinite(dl).all()


def test_gates_of_one_are_plain_sums_and_pieces_join():
    q, k, v, lg, _, S, _ = tensors(1, 2, 1, 8, 4, 2)
    o, _ = gated.forward(q, k, v, np.zeros_like(lg))
    np.testing.assert_allclose(o[:, :, -1], q[:, :, -1] @ np.einsum("bcnd,bcne->bde", k, v)[:, None][:, 0],
                               rtol=1e-12)
    whole, S_all = gated.forward(q, k, v, lg, 1.0, S)
    a, Sa = gated.forward(q[:, :, :5], k[:, :, :5], v[:, :, :5], lg[:, :, :5], 1.0, S)
    for t in range(5, 8):
        ot, Sa = gated.decode_step(Sa, q[:, :, t], k[:, :, t], v[:, :, t], lg[:, :, t])
        np.testing.assert_allclose(ot, whole[:, :, t], rtol=1e-12)
    np.testing.assert_allclose(a, whole[:, :, :5], rtol=1e-13)
    np.testing.assert_allclose(Sa, S_all, rtol=1e-13)


@pytest.mark.parametrize("which", ["q", "k", "v", "lg", "S"])
def test_backward_by_differences(which):
    q, k, v, lg, dO, S, dS = tensors(1, 4, 2, 5, 3, 3)
    at = dict(q=q, k=k, v=v, lg=lg, S=S)
    grads = dict(zip(("q", "k", "v", "lg", "S"), gated.backward(q, k, v, lg, dO, 0.6, S, dS)))

    def loss():
        o, S_out = gated.forward(at["q"], at["k"], at["v"], at["lg"], 0.6, at["S"])
        return (dO * o).sum() + (dS * S_out).sum()

    x, g = at[which], grads[which]
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + 1e-6
        up = loss()
        x[i] = old - 1e-6
        down = loss()
        x[i] = old
        assert abs((up - down) / 2e-6 - g[i]) <= 1e-7 * (1 + abs(g[i])), (which, i)


def norm_tensors(seed=0, B=2, H=3, N=4, D=8):
    r = np.random.default_rng(seed)
    x = r.standard_normal((B, H, N, D)) * 2 + 0.5
    w, b = 1 + 0.2 * r.standard_normal(H * D), 0.3 * r.standard_normal(H * D)
    gate, dy = r.standard_normal((2, B, N, H * D))
    return x, w, b, gate, dy


def test_group_norm_is_torchs():
    x, w, b, gate, _ = norm_tensors()
    B, H, N, D = x.shape
    rows = torch.from_numpy(x).permute(0, 2, 1, 3).reshape(B * N, H * D)
    want = torch.nn.functional.group_norm(rows, H, torch.from_numpy(w), torch.from_numpy(b), 1e-3)
    want = want.reshape(B, N, H * D)
    np.testing.assert_allclose(gated.group_norm(x, w, b, None, "identity", 1e-3), want, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(gated.group_norm(x, w, b, None, "silu", 1e-3),
                               torch.nn.functional.silu(want), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(gated.group_norm(x, w, b, gate, "silu", 1e-3),
                               want * torch.nn.functional.silu(torch.from_numpy(gate)), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("act", ["identity", "silu"])
@pytest.mark.parametrize("gated_", [False, True])
def test_group_norm_backward_by_differences(act, gated_):
    x, w, b, gate, dy = norm_tensors(1, 1, 2, 2, 4)
    gate = gate if gated_ else None
    grads = gated.group_norm_backward(x, w, dy, b, gate, act, 1e-2)
    for t, g in zip((x, w, b, gate), grads):
        if t is None:
            assert g is None
            continue
        for i in np.ndindex(t.shape):
            old = t[i]
            t[i] = old + 1e-6
            up = (dy * gated.group_norm(x, w, b, gate, act, 1e-2)).sum()
            t[i] = old - 1e-6
            down = (dy * gated.group_norm(x, w, b, gate, act, 1e-2)).sum()
            t[i] = old
            assert abs((up - down) / 2e-6 - g[i]) <= 1e-7 * (1 + abs(g[i])), i
