"""The head-row group norm on the GPU against the float64 oracle."""
import pytest
import torch

from gated_util import MAX, REL, close
from linear_attention_transformers_b200 import api
from oracle import gated

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
# B, H, N: fewer channels than a block, a block, several blocks; odd counts
SHAPES = [(1, 1, 1), (7, 16, 1), (1, 3, 5), (2, 6, 129), (3, 5, 333), (1, 40, 17), (2, 32, 1000), (1, 1, 4099)]


def tensors(B, H, N, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rows = torch.exp(torch.randn(B, H, N, 1, generator=g))
    x = ((torch.randn(B, H, N, D, generator=g) + 0.3) * rows).to(dtype).cuda()
    w = (1 + 0.2 * torch.randn(H * D, generator=g)).cuda()
    b = (0.2 * torch.randn(H * D, generator=g)).cuda()
    gate, dy = torch.randn(2, B, N, H * D, generator=g).to(dtype).cuda().unbind(0)
    return x, w, b, gate.contiguous(), dy.contiguous()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_forward_and_backward(dtype, D, shape):
    x, w, b, gate, dy = tensors(*shape, D, dtype, D)
    for bias, gt, act in ((b, gate, "silu"), (None, gate, "identity"), (b, None, "silu"),
                          (None, None, "identity")):
        y = api.la_group_norm(x, w, bias, gt, act, 1e-4)
        close(y, gated.group_norm(x, w, bias, gt, act, 1e-4), REL[dtype], MAX[dtype], "y")
        got = api.la_group_norm_backward(x, w, dy, bias, gt, act, 1e-4)
        ref = gated.group_norm_backward(x, w, dy, bias, gt, act, 1e-4)
        for n, g, r in zip(("dx", "dweight", "dbias", "dgate"), got, ref):
            if g is None:
                assert (n == "dbias" and bias is None) or (n == "dgate" and gt is None)
                continue
            # channel sums: float32 terms (each within 2^-20), added over at most
            # 4099 tokens with errors that add like a random walk
            rel, most = (2.0 ** -18, 2.0 ** -16) if n in ("dweight", "dbias") else (REL[dtype], MAX[dtype])
            close(g, r, rel, most, n)
        again = api.la_group_norm_backward(x, w, dy, bias, gt, act, 1e-4)
        for a, c in zip(got, again):
            assert (a is None and c is None) or torch.equal(a, c)


def test_rows_of_one_value_and_of_zeros():
    # no variance: x_hat is zero (or what rounding leaves over sqrt(eps)), never NaN
    x, w, b, gate, dy = tensors(1, 2, 6, 64, torch.float32, 3)
    x[0, 0, 1] = 0
    x[0, 1, 2] = 5.0
    y = api.la_group_norm(x, w, b, gate)
    close(y, gated.group_norm(x, w, b, gate), REL[torch.float32], MAX[torch.float32], "y")
    got = api.la_group_norm_backward(x, w, dy, b, gate)
    ref = gated.group_norm_backward(x, w, dy, b, gate)
    for g, r in zip(got, ref):
        close(g, r, REL[torch.float32], MAX[torch.float32], "gradient")


def test_a_row_that_is_not_finite_stays_alone():
    x, w, b, gate, _ = tensors(1, 3, 9, 32, torch.float32, 4)
    y = api.la_group_norm(x, w, b, gate)
    x2 = x.clone()
    x2[0, 1, 4, 7] = float("nan")
    x2[0, 2, 5, 0] = float("inf")
    y2 = api.la_group_norm(x2, w, b, gate)
    keep = torch.ones(1, 9, 96, dtype=torch.bool, device="cuda")
    keep[0, 4, 32:64] = False
    keep[0, 5, 64:96] = False
    assert torch.equal(y[keep], y2[keep]) and not torch.isfinite(y2[~keep]).any()


def test_no_rows():
    x = torch.empty(2, 3, 0, 64, device="cuda")
    w = torch.ones(192, device="cuda")
    e = torch.empty(2, 0, 192, device="cuda")
    assert api.la_group_norm(x, w).shape == (2, 0, 192)
    dx, dw, db, dg = api.la_group_norm_backward(x, w, e, bias=w, gate=e)
    assert dx.shape == x.shape and dg.shape == e.shape and not dw.any() and not db.any()


def test_long_offsets():
    # more than 2^31 elements: the last rows equal a call on them alone
    H, N, D = 64, (1 << 31) // (64 * 128) + 5, 128
    x = torch.randn(1, H, N, D, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(H * D, device="cuda")
    y = api.la_group_norm(x, w)
    y2 = api.la_group_norm(x[:, :, -7:].contiguous(), w)
    assert torch.equal(y[:, -7:], y2)


def test_streams_and_refusals():
    x, w, b, gate, dy = tensors(2, 4, 50, 64, torch.bfloat16, 9)
    want = api.la_group_norm(x, w, b, gate)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.la_group_norm(x, w, b, gate, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=-1.0), dict(eps=float("inf"))):
        with pytest.raises(api.LinearAttentionError):
            api.la_group_norm(x, w, b, gate, **kw)
    for args in ((x, w.bfloat16()), (x, w[:-1]), (x[0], w), (x.transpose(1, 2), w), (x, w, b, gate.float()),
                 (x, w, b, gate.transpose(0, 1)), (x, w, b[:-1])):
        with pytest.raises(ValueError):
            api.la_group_norm(*args)
    with pytest.raises(ValueError):
        api.la_group_norm(x, w, act="gelu")
    with pytest.raises(ValueError):
        api.la_group_norm_backward(x, w, dy, dbias=torch.empty_like(w))
    with pytest.raises(ValueError):
        api.la_group_norm_backward(x, w, dy.float())


def test_an_empty_batch_has_channel_sums_of_zero():
    # dweight and dbias have H*D elements whatever the batch is
    for N in (0, 5):
        x = torch.empty(0, 3, N, 64, device="cuda")
        w = torch.ones(192, device="cuda")
        e = torch.empty(0, N, 192, device="cuda")
        dw, db = torch.full((2, 192), 7.0, device="cuda").unbind(0)
        dx, dw2, db2, dg = api.la_group_norm_backward(x, w, e, bias=w, gate=e, dweight=dw, dbias=db)
        assert dw2 is dw and db2 is db and not dw.any() and not db.any()
        assert dx.shape == x.shape and dg.shape == e.shape
        wg, bg = w.clone().requires_grad_(), w.clone().requires_grad_()
        api.HeadGroupNorm.apply(x, wg, bg, e).sum().backward()
        assert not wg.grad.any() and not bg.grad.any()


def test_backward_on_another_stream_and_captured():
    x, w, b, gate, dy = tensors(2, 4, 500, 64, torch.bfloat16, 10)
    want = api.la_group_norm_backward(x, w, dy, b, gate)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.la_group_norm_backward(x, w, dy, b, gate, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(g, r) for g, r in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = api.la_group_norm_backward(x, w, dy, b, gate)
    for seed in (10, 11):
        for t, n in zip((x, w, b, gate, dy), tensors(2, 4, 500, 64, torch.bfloat16, seed)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, r) for g, r in zip(outs, api.la_group_norm_backward(x, w, dy, b, gate)))


def test_long_offsets_backward():
    # more than 2^31 elements: the last rows' dx and dgate equal a call's on them alone
    H, N, D = 64, (1 << 31) // (64 * 128) + 5, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, H, N, D, generator=g, device="cuda", dtype=torch.bfloat16)
    gate = torch.randn(1, N, H * D, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(H * D, device="cuda")
    dx, _, _, dg = api.la_group_norm_backward(x, w, gate, gate=gate)
    tail = gate[:, -7:].contiguous()
    dx2, _, _, dg2 = api.la_group_norm_backward(x[:, :, -7:].contiguous(), w, tail, gate=tail)
    assert torch.equal(dx[:, :, -7:], dx2) and torch.equal(dg[:, -7:], dg2)


def test_autograd_takes_any_strides():
    # a transposed input, a sliced gate and an expanded gradient give what their
    # contiguous copies give
    x, w, b, gate, _ = tensors(2, 4, 50, 64, torch.bfloat16, 12)
    far = x.transpose(1, 2).contiguous().transpose(1, 2).requires_grad_()
    wide = torch.cat([gate, gate], -1)[..., :256].detach().requires_grad_()
    wg, bg = w.clone().requires_grad_(), b.clone().requires_grad_()
    y = api.HeadGroupNorm.apply(far, wg, bg, wide)
    assert torch.equal(y, api.la_group_norm(x, w, b, gate))
    dy = torch.full((1, 1, 1), 0.5, dtype=y.dtype, device="cuda").expand_as(y)
    y.backward(dy)
    want = api.la_group_norm_backward(x, w, dy.contiguous(), b, gate)
    for got, ref in zip((far.grad, wg.grad, bg.grad, wide.grad), want):
        assert torch.equal(got, ref)
