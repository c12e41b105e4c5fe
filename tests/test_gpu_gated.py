"""Gated linear attention on the GPU against the float64 oracle: forward,
backward, one-token step, states carried in and out, shared heads, gates of
zero, streams, captured graphs, refusals."""
import math

import numpy as np
import pytest
import torch

from gated_util import MAX, REL, REL_STATE, close, tensors
from linear_attention_transformers_b200 import api
from oracle import gated

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
# B, H, Hkv, N, state, resets: lengths about the 64- and 128-token chunks
SHAPES = [
    (1, 1, 1, 1, False, False),
    (2, 2, 2, 1, True, False),
    (1, 2, 2, 2, False, True),
    (2, 3, 3, 63, False, False),
    (1, 2, 1, 64, True, True),
    (1, 2, 2, 65, False, False),
    (1, 4, 2, 127, True, False),
    (1, 2, 2, 128, False, True),
    (2, 3, 1, 129, True, False),
    (1, 3, 3, 256, True, True),
    (1, 2, 2, 257, False, False),
    (1, 4, 1, 511, True, True),
    (1, 5, 5, 777, False, True),
    (1, 2, 2, 1000, True, False),
    (1, 4, 1, 1500, True, True),
]


def check_fwd(dtype, ins, scale, state, what=""):
    q, k, v, lg, _, S, _ = ins
    S = S if state else None
    o, S_out = api.la_forward_gated(q, k, v, lg, scale, S, return_state=True)
    torch.cuda.synchronize()
    api.la_get_device_error()
    ro, rS = gated.forward(q, k, v, lg, scale, S)
    close(o, ro, REL[dtype], MAX[dtype], f"{what} o")
    close(S_out, rS, REL_STATE[dtype], 4 * REL_STATE[dtype], f"{what} S")
    o2, S2 = api.la_forward_gated(q, k, v, lg, scale, S, return_state=True)
    assert torch.equal(o, o2) and torch.equal(S_out, S2)
    close(api.la_forward_gated(q, k, v, lg, scale, S), ro, REL[dtype], MAX[dtype], f"{what} o alone")


def check_bwd(dtype, ins, scale, state, what=""):
    q, k, v, lg, dO, S, dS = ins
    if not state:
        S = dS = None
    got = api.la_backward_gated(q, k, v, lg, dO, scale, S, dS, return_dstate=True)
    torch.cuda.synchronize()
    api.la_get_device_error()
    ref = gated.backward(q, k, v, lg, dO, scale, S, dS)
    for n, g, r in zip(("dq", "dk", "dv"), got, ref):
        close(g, r, REL[dtype], MAX[dtype], f"{what} {n}")
    close(got[3], ref[3], REL[dtype] * (4 if dtype == torch.float32 else 1), MAX[dtype], f"{what} dlog_gate")
    close(got[4], ref[4], REL_STATE[dtype], 4 * REL_STATE[dtype], f"{what} dS_in")
    again = api.la_backward_gated(q, k, v, lg, dO, scale, S, dS, return_dstate=True)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    alone = api.la_backward_gated(q, k, v, lg, dO, scale, S, dS)
    for n, g, r in zip(("dq", "dk", "dv"), alone, ref):
        close(g, r, REL[dtype], MAX[dtype], f"{what} {n} alone")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(dtype, D, shape):
    B, H, Hkv, N, state, resets = shape
    check_fwd(dtype, tensors(B, H, Hkv, N, D, dtype, N + D, resets), D ** -0.5, state)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(dtype, D, shape):
    B, H, Hkv, N, state, resets = shape
    check_bwd(dtype, tensors(B, H, Hkv, N, D, dtype, 2 * N + D, resets), D ** -0.5, state)


@pytest.mark.parametrize("shape", [(32, 4, 4, 400), (20, 12, 6, 300), (1, 8, 8, 3000), (2, 32, 1, 2049),
                                   (150, 1, 1, 129)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_heads_and_long_ones(D, shape):
    # the ways the states are formed that the oracle's sizes do not reach, against the
    # float32 kernels (held to the oracle above) on the same values
    B, H, Hkv, N = shape
    bf, f32 = torch.bfloat16, torch.float32
    ins = tensors(B, H, Hkv, N, D, bf, N, resets=True)
    q, k, v, lg, dO, S, dS = ins
    wide = [x.float() for x in (q, k, v, lg, dO)]
    o, S_out = api.la_forward_gated(q, k, v, lg, 0.1, S, return_state=True)
    ro, rS = api.la_forward_gated(*wide[:4], 0.1, S, return_state=True)
    close(o, ro.cpu(), REL[bf], MAX[bf], "o")
    close(S_out, rS.cpu(), REL_STATE[bf], 4 * REL_STATE[bf], "S")
    got = api.la_backward_gated(q, k, v, lg, dO, 0.1, S, dS, return_dstate=True)
    ref = api.la_backward_gated(*wide, 0.1, S, dS, return_dstate=True)
    for n, g, r in zip(("dq", "dk", "dv", "dlog_gate"), got, ref):
        close(g, r.cpu(), REL[bf], MAX[bf], n)
    close(got[4], ref[4].cpu(), REL_STATE[bf], 4 * REL_STATE[bf], "dS_in")
    torch.cuda.synchronize()
    api.la_get_device_error()
    plain = api.la_forward_gated(q, k, v, lg, 0.1)
    close(plain, api.la_forward_gated(*wide[:4], 0.1).cpu(), REL[bf], MAX[bf], "o without a state")


@pytest.mark.parametrize("shape", [(2, 4, 4, 1), (1, 6, 2, 2), (1, 1, 1, 5), (2, 8, 1, 16), (1, 148, 148, 3),
                                   (1, 148, 37, 16)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_few_tokens_are_rounded_once(D, shape):
    # bf16 in, float32 within, one rounding out: half a step of each value, and what
    # float32 sums of D + 16 terms leave of the largest
    B, H, Hkv, N = shape
    ins = tensors(B, H, Hkv, N, D, torch.bfloat16, N + H, resets=True)
    q, k, v, lg, dO, *_ = ins
    scale = D ** -0.5
    got = (api.la_forward_gated(q, k, v, lg, scale), *api.la_backward_gated(q, k, v, lg, dO, scale))
    ref = (gated.forward(q, k, v, lg, scale)[0], *gated.backward(q, k, v, lg, dO, scale)[:4])
    for n, g, r in zip(("o", "dq", "dk", "dv", "dlog_gate"), got, ref):
        off = np.abs(g.double().cpu().numpy() - r)
        assert (off <= 2.0 ** -8 * np.abs(r) + 2.0 ** -16 * np.abs(r).max()).all(), n


@pytest.mark.parametrize("gate", [0.0, -1e-3, -5.0, -80.0, -300.0, -math.inf])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_gates_of_every_size(dtype, D, gate):
    ins = tensors(1, 2, 2, 300, D, dtype, 7, gate=gate)
    check_fwd(dtype, ins, 1.0, True, f"gate {gate}")
    check_bwd(dtype, ins, 1.0, True, f"gate {gate}")


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_what_lies_before_a_zero_gate_does_not_matter(dtype, D):
    q, k, v, lg, dO, S, _ = tensors(1, 2, 2, 400, D, dtype, 11)
    lg[:, :, 133] = -math.inf
    o = api.la_forward_gated(q, k, v, lg, 1.0, S)
    g = api.la_backward_gated(q, k, v, lg, dO, 1.0, S)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, :133] *= -3
    v2[:, :, :133] += 1
    o2 = api.la_forward_gated(q, k2, v2, lg, 1.0, 2 * S)
    g2 = api.la_backward_gated(q, k2, v2, lg, dO, 1.0, 2 * S)
    assert torch.equal(o[:, :, 133:], o2[:, :, 133:])
    for a, b in zip(g[:3], g2[:3]):
        assert torch.equal(a[:, :, 133:], b[:, :, 133:])


@pytest.mark.parametrize("dtype", TYPES)
def test_dlog_gate_by_differences(dtype):
    # the loss itself in float64 (the oracle's), stepped along one gate at a time
    q, k, v, lg, dO, S, dS = tensors(1, 2, 1, 200, 64, dtype, 13)
    got = api.la_backward_gated(q, k, v, lg, dO, 0.5, S, dS)[3].double().cpu().numpy()
    lg64 = lg.double().cpu().numpy()
    d64 = dO.double().cpu().numpy()
    for t in (0, 1, 63, 64, 127, 128, 199):
        f = []
        for h in (1e-5, -1e-5):
            x = lg64.copy()
            x[0, 0, t] += h
            o, S_out = gated.forward(q, k, v, x, 0.5, S)
            f.append((d64 * o).sum() + (dS.double().cpu().numpy() * S_out).sum())
        want = (f[0] - f[1]) / 2e-5
        # the difference quotient itself is good to about 1e-6 of the loss's terms
        tol = REL[dtype] * 8 * np.abs(got).max() + 1e-5 * np.abs(got).max()
        assert abs(got[0, 0, t] - want) <= tol, (t, got[0, 0, t], want)


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 4, 4), (2, 8, 2), (1, 6, 1), (5, 10, 2), (700, 2, 1)])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_step(dtype, D, shape):
    B, H, Hkv = shape
    q, k, v, lg, _, S, _ = tensors(B, H, Hkv, 3, D, dtype, D + H, resets=True)
    S = S.clone()
    ref_S = S.double().cpu().numpy()
    for t in range(3):
        at = [x[:, :, t].contiguous() for x in (q, k, v, lg)]
        o = api.la_decode_step_gated(S, *at, scale=0.3)
        ref_o, ref_S = gated.decode_step(ref_S, *at, 0.3)
        # one rounding of o, float32 sums of D terms
        close(o, ref_o, REL[dtype], MAX[dtype], f"o {t}")
        close(S, ref_S, REL_STATE[torch.float32], 2.0 ** -18, f"S {t}")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_pieces_and_steps_join(dtype, D):
    q, k, v, lg, _, S0, _ = tensors(2, 4, 2, 333, D, dtype, 17, resets=True)
    ro, rS = gated.forward(q, k, v, lg, 0.2, S0)
    S, outs, n = S0, [], 0
    for m in (200, 1, 130):
        o, S = api.la_forward_gated(*(x[:, :, n:n + m].contiguous() for x in (q, k, v, lg)), scale=0.2,
                                    S_in=S, return_state=True)
        outs.append(o)
        n += m
    for t in range(n, 333):
        o = api.la_decode_step_gated(S, *(x[:, :, t].contiguous() for x in (q, k, v, lg)), scale=0.2)
        outs.append(o[:, :, None])
    close(torch.cat(outs, 2), ro, REL[dtype], MAX[dtype], "o")
    close(S, rS, 2 * REL_STATE[dtype], 8 * REL_STATE[dtype], "S")


def test_no_tokens_pass_the_state_through():
    for dtype in TYPES:
        q, k, v, lg, dO, S, dS = tensors(2, 2, 2, 0, 64, dtype, 1)
        o, S_out = api.la_forward_gated(q, k, v, lg, 1.0, S, return_state=True)
        assert o.shape == q.shape and torch.equal(S_out, S)
        _, S_out = api.la_forward_gated(q, k, v, lg, return_state=True)
        assert not S_out.any()
        *_, dS_in = api.la_backward_gated(q, k, v, lg, dO, 1.0, S, dS, return_dstate=True)
        assert torch.equal(dS_in, dS)
        *_, dS_in = api.la_backward_gated(q, k, v, lg, dO, return_dstate=True)
        assert not dS_in.any()


@pytest.mark.parametrize("D", [32, 64, 128])
def test_rows_behind_the_last_are_left(D):
    # the outputs end inside larger buffers: what lies behind them stays
    dtype = torch.bfloat16
    q, k, v, lg, dO, S, dS = tensors(1, 2, 2, 200, D, dtype, 3)
    n = q.numel()
    bufs = [torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    o, dq, dk, dv = (b[:n].view_as(q) for b in bufs)
    api.la_forward_gated(q, k, v, lg, o=o)
    api.la_backward_gated(q, k, v, lg, dO, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    for b in bufs:
        assert (b[n:] == 7.0).all()


@pytest.mark.parametrize("D", [32, 64, 128])
def test_long_offsets(D):
    # tensors of more than 2^31 elements: the last heads are those of a call on them
    # alone (up to its own rounding: the states may be formed another way there)
    dtype = torch.bfloat16
    N, H = 4096, (1 << 31) // (4096 * D) + 3
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(1, H, N, D, generator=g, device="cuda", dtype=dtype)
    lg = torch.nn.functional.logsigmoid(torch.randn(1, H, N, generator=g, device="cuda") + 3).to(dtype)
    o, S = api.la_forward_gated(q, q, q, lg, return_state=True)
    a, b = (q[:, -2:].contiguous(), lg[:, -2:].contiguous())
    o2, S2 = api.la_forward_gated(a, a, a, b, return_state=True)
    close(o[:, -2:], o2.double().cpu(), 2 * REL[dtype], 2 * MAX[dtype], "o")
    close(S[:, -2:], S2.double().cpu(), 2 * REL_STATE[dtype], 8 * REL_STATE[dtype], "S")


@pytest.mark.parametrize("D", [32, 64, 128])
def test_another_stream_and_two_at_once(D):
    dtype = torch.bfloat16
    ins = [tensors(2, 2, 2, 500, D, dtype, s) for s in (1, 2)]
    want = [api.la_forward_gated(*x[:4]) for x in ins]
    grad = [api.la_backward_gated(*x[:5]) for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        got = [api.la_forward_gated(*x[:4], stream=s) for x, s in zip(ins, streams)]
        bwd = [api.la_backward_gated(*x[:5], stream=s) for x, s in zip(ins, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, b in zip(bwd, grad):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("D", [32, 64, 128])
def test_captured_and_replayed(D):
    dtype = torch.bfloat16
    q, k, v, lg, dO, S, dS = tensors(1, 4, 2, 300, D, dtype, 5)
    step = [x[:, :, 0].contiguous() for x in (q, k, v, lg)]
    w = torch.ones(4 * D, device="cuda")

    def work():
        o, S_out = api.la_forward_gated(q, k, v, lg, 0.5, S, return_state=True)
        y = api.la_group_norm(o, w)
        g = api.la_backward_gated(q, k, v, lg, dO, 0.5, S, dS)
        s = api.la_decode_step_gated(S_out, *step)
        return (o, y, *g, s, S_out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for seed in (5, 6):
        for t, n in zip((q, k, v, lg, dO, S, dS), tensors(1, 4, 2, 300, D, dtype, seed)):
            t.copy_(n)
        for t, n in zip(step, (q, k, v, lg)):
            t.copy_(n[:, :, 0])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, work()):
            assert torch.equal(a, b)


def test_a_layer_and_its_norm_through_autograd():
    # the run of them together: gated attention, the norm behind it, their
    # gradients, against the oracle chained by hand
    for dtype in TYPES:
        q, k, v, lg, _, S, _ = tensors(2, 4, 2, 150, 64, dtype, 23, resets=True)
        leaves = [t.requires_grad_() for t in (q, k, v, lg, S)]
        g = torch.Generator().manual_seed(2)
        w, b = (torch.randn(2, 256, generator=g) * 0.1 + 1).cuda().unbind(0)
        w, b = w.clone().requires_grad_(), b.clone().requires_grad_()
        gate = torch.randn(2, 150, 256, generator=g).to(dtype).cuda().requires_grad_()
        dy = torch.randn(2, 150, 256, generator=g).to(dtype).cuda()
        o, S_out = api.GatedLinearAttention.apply(q, k, v, lg, 0.125, S, True)
        y = api.HeadGroupNorm.apply(o, w, b, gate, "silu", 1e-5)
        (y.float() * dy.float()).sum().backward()
        # oracle: the norm on the attention's output as stored, then the chain
        o_st = o.detach().double().cpu().numpy()
        close(y, gated.group_norm(o, w, b, gate), REL[dtype], MAX[dtype], "y")
        dx, dw, db, dg = gated.group_norm_backward(o_st, w, dy, b, gate)
        close(w.grad, dw, 2.0 ** -17, 2.0 ** -15, "dweight")
        close(b.grad, db, 2.0 ** -17, 2.0 ** -15, "dbias")
        close(gate.grad, dg, REL[dtype], MAX[dtype], "dgate")
        ref = gated.backward(q, k, v, lg, dx, 0.125, S)
        for n, t, r in zip(("q", "k", "v", "log_gate", "S"), leaves, ref):
            # one more rounding than the bound counts: the norm's dx between the two
            close(t.grad, r, 4 * REL[dtype], 2 * MAX[dtype], n)


def test_autograd_leaves_what_is_not_asked():
    q, k, v, lg, dO, S, dS = tensors(1, 2, 2, 70, 32, torch.float32, 29)
    q.requires_grad_()
    o, S_out = api.GatedLinearAttention.apply(q, k, v, lg, 1.0, S, True)
    (S_out * dS).sum().backward()  # the output itself unused
    assert q.grad is not None and not q.grad.any() and k.grad is None
    k.requires_grad_()
    api.GatedLinearAttention.apply(q.detach(), k, v, lg).mul(dO).sum().backward()
    ref = gated.backward(q, k, v, lg, dO)
    close(k.grad, ref[1], REL[torch.float32], MAX[torch.float32], "dk")


def test_second_derivatives_raise():
    q, k, v, lg, dO, *_ = tensors(1, 2, 2, 70, 32, torch.float32, 30)
    q.requires_grad_()
    o = api.GatedLinearAttention.apply(q, k, v, lg)
    w = torch.ones(64, device="cuda")
    y = api.HeadGroupNorm.apply(q, w)
    for out in (o, y):
        (dq,) = torch.autograd.grad(out.pow(2).sum(), q, create_graph=True)
        with pytest.raises(RuntimeError):
            dq.sum().backward()


def test_refusals():
    q, k, v, lg, dO, S, dS = tensors(1, 4, 2, 32, 64, torch.bfloat16, 1)
    ok = (q, k, v, lg)
    for bad in ((q.cpu(), k, v, lg), (q, k.float(), v, lg), (q, k, v, lg.float()), (q, k, v, lg[:, :1]),
                (q, k, v[:, :1], lg), (q, k[:, :, :8], v[:, :, :8], lg), (q.transpose(1, 2), k, v, lg),
                (q[0], k[0], v[0], lg[0]), (q.half(), k.half(), v.half(), lg.half()),
                (q[:, :3].contiguous(), k, v, lg)):
        with pytest.raises((ValueError, api.LinearAttentionError)):
            api.la_forward_gated(*bad)
        with pytest.raises((ValueError, api.LinearAttentionError)):
            api.la_backward_gated(*bad, dO)
    with pytest.raises(ValueError):
        api.la_forward_gated(*ok, S_in=S.bfloat16())
    with pytest.raises(ValueError):
        api.la_forward_gated(*ok, S_in=S[:, :1])
    with pytest.raises(ValueError):
        api.la_forward_gated(*ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(api.LinearAttentionError):
        api.la_forward_gated(*ok, S_in=S, S_out=S, return_state=True)
    with pytest.raises(ValueError):
        api.la_backward_gated(*ok, dO, dk=torch.empty_like(q))
    x = torch.randn(1, 2, 8, 48, device="cuda")
    with pytest.raises(api.LinearAttentionError):  # a head size that is not offered
        api.la_forward_gated(x, x, x, x[..., 0].contiguous())
    with pytest.raises(ValueError):
        api.la_decode_step_gated(S, q, k, v, lg)
    with pytest.raises(ValueError):
        api.la_decode_step_gated(S[:, :1], q[:, :, 0].contiguous(), k[:, :, 0].contiguous(),
                                 v[:, :, 0].contiguous(), lg[:, :, 0].contiguous())


def test_what_a_call_writes_is_known_to_autograd():
    # the calls write through pointers; a tensor that a pending backward saved must
    # not change unseen
    q, k, v, lg, dO, S, dS = tensors(1, 4, 2, 70, 64, torch.bfloat16, 31)
    at = [x[:, :, 0].contiguous() for x in (q, k, v, lg)]
    q.requires_grad_()
    plain = q.detach()

    def stepped(S):
        api.la_decode_step_gated(S, *at)

    def returned(S):
        api.la_forward_gated(plain, k, v, lg, S_out=S, return_state=True)

    def differentiated(S):
        api.la_backward_gated(plain, k, v, lg, dO, dS_out=dS, dS_in=S, return_dstate=True)

    for write in (stepped, returned, differentiated):
        state = S.clone()
        o = api.GatedLinearAttention.apply(q, k, v, lg, 1.0, state)
        write(state)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            o.sum().backward()
        # the state that a step leaves starts a pass of its own
        api.GatedLinearAttention.apply(q, k, v, lg, 1.0, state).sum().backward()

    def bumped(call, **outs):
        before = {n: t._version for n, t in outs.items()}
        call(**outs)
        assert all(t._version > before[n] for n, t in outs.items()), outs.keys()

    e = torch.empty_like
    w = torch.ones(256, device="cuda")
    y = torch.empty(1, 70, 256, dtype=plain.dtype, device="cuda")
    gate = torch.randn_like(y)
    bumped(lambda **t: api.la_forward_gated(plain, k, v, lg, **t), o=e(plain), S_out=e(S))
    bumped(lambda **t: api.la_backward_gated(plain, k, v, lg, dO, **t), dq=e(plain), dk=e(k), dv=e(v),
           dlog_gate=e(lg), dS_in=e(S))
    bumped(lambda **t: api.la_decode_step_gated(q=at[0], k=at[1], v=at[2], log_gate=at[3], **t), S=S.clone(),
           o=e(at[0]))
    bumped(lambda **t: api.la_group_norm(plain, w, w, gate, **t), y=e(y))
    bumped(lambda **t: api.la_group_norm_backward(plain, w, y.zero_(), w, gate, **t), dx=e(plain), dweight=e(w),
           dbias=e(w), dgate=e(y))


@pytest.mark.parametrize("N", [13, 64, 300, 1500])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_gate_of_zero_has_no_gradient(dtype, D, N):
    # single gates of zero among gates near 1: nothing passes them, so their
    # gradient is 0, not what rounding leaves of the pairs around them
    for state in (False, True):
        q, k, v, lg, dO, S, dS = tensors(1, 4, 2, N, D, dtype, 37 + N, gate=-0.01)
        at = [0, 1, N // 3, N // 2, N // 2 + 1, N - 1]
        lg[:, 0, at] = -math.inf
        lg[:, 1, at[2:5]] = torch.tensor([-1000.0, -200.0, -88.0], dtype=dtype, device="cuda")  # below 2^-126
        S, dS = (S, dS) if state else (None, None)
        got = api.la_backward_gated(q, k, v, lg, dO, 0.3, S, dS)
        ref = gated.backward(q, k, v, lg, dO, 0.3, S, dS)[3]
        assert not got[3][:, 0, at].any() and not got[3][:, 1, at[2:5]].any()
        ref[:, 1, at[2:5]] = 0.0
        close(got[3], ref, REL[dtype] * (4 if dtype == torch.float32 else 1), MAX[dtype], "dlog_gate")


@pytest.mark.parametrize("shape", [(1, 2, 2, 17), (2, 3, 3, 64), (1, 4, 2, 100), (3, 8, 1, 128)])
@pytest.mark.parametrize("D", [64, 128])
def test_the_gates_gradient_inside_a_block_is_rounded_once(D, shape):
    # a block that no state enters or leaves.  The terms of dlog_gate are products of
    # float32 sums of exact products (2^-22 in all) and of weights whose exponents are
    # differences of sums up to 64, each rounded to float32 (2^-19 off at most, two of
    # them: 2^-18.5 of the weight) under an exponential good to 2^-22.  They are held and
    # added in float32; a partial sum is no larger than the largest output by more than
    # a few times, so 256 additions leave 16 * 2^-24.  Errors of independent terms add
    # like the terms themselves: 2^-18 and a little of the largest value, 2^-16 is four
    # times that, beside the half step of the output's own bf16
    B, H, Hkv, N = shape
    q, k, v, lg, dO, *_ = tensors(B, H, Hkv, N, D, torch.bfloat16, 41 + N)
    got = api.la_backward_gated(q, k, v, lg, dO, D ** -0.5)[3].double().cpu().numpy()
    ref = gated.backward(q, k, v, lg, dO, D ** -0.5)[3]
    off = np.abs(got - ref)
    assert (off <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * np.abs(ref).max()).all(), (
        off / np.abs(ref).max()).max()


@pytest.mark.parametrize("D", [32, 64])
def test_autograd_takes_any_strides(D):
    # transposed inputs, a sliced gate, a state and gradients that are expanded give
    # what their contiguous copies give
    q, k, v, lg, _, S, _ = tensors(2, 4, 2, 150, D, torch.bfloat16, 43)
    far = [x.transpose(1, 2).contiguous().transpose(1, 2).requires_grad_() for x in (q, k, v)]
    gate = torch.stack([lg, lg], -1)[..., 0].detach().requires_grad_()
    start = S[:1].expand(2, -1, -1, -1).detach().requires_grad_()
    assert not any(t.is_contiguous() for t in (*far, gate, start))
    o, S_out = api.GatedLinearAttention.apply(*far, gate, 0.5, start, True)
    S = S[:1].repeat(2, 1, 1, 1)
    want = api.la_forward_gated(q, k, v, lg, 0.5, S, return_state=True)
    assert torch.equal(o, want[0]) and torch.equal(S_out, want[1])
    dO = torch.full((), 0.25, dtype=o.dtype, device="cuda").expand_as(o)
    dS = torch.full((), 0.125, device="cuda").expand_as(S_out)
    torch.autograd.backward([o, S_out], [dO, dS])
    want = api.la_backward_gated(q, k, v, lg, dO.contiguous(), 0.5, S, dS.contiguous(), return_dstate=True)
    for t, r in zip((*far, gate, start), want):
        assert torch.equal(t.grad, r)


def test_two_host_threads():
    # each on a stream of its own, all calls at once
    from concurrent.futures import ThreadPoolExecutor

    def work(ins, stream=None):
        q, k, v, lg, dO, S, dS = ins
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            w = torch.ones(q.shape[1] * q.shape[3], device="cuda")
            o, S_out = api.la_forward_gated(q, k, v, lg, 0.5, S, return_state=True)
            y = api.la_group_norm(o, w)
            g = api.la_backward_gated(q, k, v, lg, dO, 0.5, S, dS, return_dstate=True)
            s = api.la_decode_step_gated(S_out, *(x[:, :, 0].contiguous() for x in (q, k, v, lg)))
        return (o, y, *g, s, S_out)

    ins = [tensors(2, 4, 2, 700, D, torch.bfloat16, D) for D in (64, 128)]
    want = [work(x) for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    with ThreadPoolExecutor(2) as pool:
        got = [pool.submit(lambda a, s: [work(a, s) for _ in range(20)], *p) for p in zip(ins, streams)]
        got = [f.result() for f in got]
    torch.cuda.synchronize()
    api.la_get_device_error()
    for runs, ref in zip(got, want):
        for outs in runs:
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))
