"""The gated-attention and head-norm entry points refuse bad arguments before
anything is launched (no device is needed; the fake pointer is never read)."""
import pytest

from linear_attention_transformers_b200 import api, build

F = 0x100000
BF, F32 = api.LA_BF16, api.LA_F32
INVALID, UNSUPPORTED, WORKSPACE = api.LA_ERR_INVALID_ARG, api.LA_ERR_UNSUPPORTED, api.LA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def need(lib, op, B=1, H=2, Hkv=2, N=100, D=64, dt=BF):
    return lib.la_workspace_size_gated(op, B, H, Hkv, N, D, dt)


def fwd(lib, q=F, k=F, v=F, lg=F, o=F, S_in=None, S_out=None, B=1, H=2, Hkv=2, N=100, D=64, dt=BF, ws=F,
        ws_bytes=None):
    n = need(lib, api.LA_OP_FORWARD, B, H, Hkv, N, D, dt) if ws_bytes is None else ws_bytes
    return lib.la_forward_gated(q, k, v, lg, o, S_in, S_out, 1.0, B, H, Hkv, N, D, dt, ws, n, None)


def bwd(lib, q=F, lg=F, dO=F, S_in=None, dS_out=None, dq=F, dlg=F, dS_in=None, B=1, H=2, Hkv=2, N=100, D=64,
        dt=BF, ws=F, ws_bytes=None):
    n = need(lib, api.LA_OP_BACKWARD, B, H, Hkv, N, D, dt) if ws_bytes is None else ws_bytes
    return lib.la_backward_gated(q, F, F, lg, dO, S_in, dS_out, dq, F, F, dlg, dS_in, 1.0, B, H, Hkv, N, D, dt,
                                 ws, n, None)


def test_forward_refusals(lib):
    for kw in (dict(q=None), dict(k=F + 2), dict(v=None), dict(lg=None), dict(lg=F + 1), dict(o=F + 8),
               dict(S_in=F + 4), dict(S_out=F + 4), dict(S_in=F, S_out=F), dict(Hkv=0), dict(H=3, Hkv=2),
               dict(N=-1), dict(D=0), dict(dt=5), dict(ws=F + 8, ws_bytes=1 << 30)):
        assert fwd(lib, **kw) == INVALID, kw
    for kw in (dict(D=48), dict(D=256), dict(N=1 << 31), dict(B=1 << 16, H=1 << 14, Hkv=1 << 14, N=1 << 20)):
        assert fwd(lib, **kw) == UNSUPPORTED, kw
    n = need(lib, api.LA_OP_FORWARD)
    assert n > 0
    assert fwd(lib, ws=None) == WORKSPACE and fwd(lib, ws_bytes=n - 1) == WORKSPACE


def test_backward_refusals(lib):
    for kw in (dict(q=None), dict(lg=F + 1), dict(dO=None), dict(dq=None), dict(dlg=None), dict(dS_in=F + 4),
               dict(dS_out=F, dS_in=F), dict(S_in=F, dS_in=F), dict(H=4, Hkv=3), dict(dt=9)):
        assert bwd(lib, **kw) == INVALID, kw
    assert bwd(lib, D=40) == UNSUPPORTED
    n = need(lib, api.LA_OP_BACKWARD)
    assert n > need(lib, api.LA_OP_FORWARD)
    assert bwd(lib, ws=None) == WORKSPACE and bwd(lib, ws_bytes=n - 1) == WORKSPACE


def test_workspace_sizes(lib):
    for kw in (dict(D=48), dict(H=3, Hkv=2), dict(N=0), dict(B=0), dict(dt=7)):
        assert need(lib, api.LA_OP_FORWARD, **kw) == 0, kw
    assert lib.la_workspace_size_gated(7, 1, 2, 2, 100, 64, BF) == 0
    assert need(lib, api.LA_OP_FORWARD, B=2, N=5000) >= need(lib, api.LA_OP_FORWARD, B=1, N=5000)
    assert lib.la_workspace_size_group_norm(1, 2, 100, 48, BF) == 0
    assert lib.la_workspace_size_group_norm(1, 2, 100, 64, BF) > 0


def test_nothing_to_do(lib):
    assert fwd(lib, B=0) == api.LA_OK and fwd(lib, H=0, Hkv=0) == api.LA_OK and fwd(lib, N=0, ws=None) == api.LA_OK
    assert bwd(lib, B=0) == api.LA_OK and bwd(lib, N=0, ws=None) == api.LA_OK
    assert lib.la_decode_step_gated(F, F, F, F, F, F, 1.0, 0, 2, 2, 64, BF, None) == api.LA_OK
    assert lib.la_group_norm(F, None, F, None, F, 1e-5, 0, 1, 2, 0, 64, BF, None) == api.LA_OK


def test_step_refusals(lib):
    def step(S=F, lg=F, o=F, H=2, Hkv=2, D=64, dt=BF):
        return lib.la_decode_step_gated(S, F, F, F, lg, o, 1.0, 1, H, Hkv, D, dt, None)
    for kw in (dict(S=None), dict(S=F + 4), dict(lg=None), dict(o=None), dict(H=3), dict(dt=3)):
        assert step(**kw) == INVALID, kw
    assert step(D=96) == UNSUPPORTED
    assert step(lg=F + 2, dt=F32) == INVALID


def test_norm_refusals(lib):
    def norm(x=F, gate=None, w=F, b=None, y=F, eps=1e-5, act=1, H=2, D=64, dt=BF):
        return lib.la_group_norm(x, gate, w, b, y, eps, act, 1, H, 8, D, dt, None)
    for kw in (dict(x=None), dict(gate=F + 2), dict(w=None), dict(b=F + 4), dict(y=None), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(act=2), dict(dt=4)):
        assert norm(**kw) == INVALID, kw
    assert norm(D=48) == UNSUPPORTED and norm(H=1 << 19) == UNSUPPORTED

    def back(gate=None, dgate=None, dw=F, dx=F, ws=F, n=1 << 20):
        return lib.la_group_norm_backward(F, gate, F, None, F, dx, dgate, dw, None, 1e-5, 1, 1, 2, 8, 64, BF, ws, n,
                                          None)
    assert back(gate=F) == INVALID and back(dgate=F) == INVALID and back(dw=None) == INVALID
    assert back(dx=None) == INVALID and back(ws=None) == WORKSPACE and back(n=8) == WORKSPACE


def test_an_empty_batch_still_writes_the_channel_sums(lib):
    # so their pointers are needed, as with N = 0; without channels nothing is
    def back(B, H, N, w=F, dw=F):
        return lib.la_group_norm_backward(None, None, w, None, None, None, None, dw, None, 1e-5, 1, B, H, N, 64, BF,
                                          None, 0, None)
    for B, N in ((0, 8), (0, 0), (1, 0)):
        assert back(B, 2, N, dw=None) == INVALID and back(B, 2, N, w=None) == INVALID
        assert back(B, 0, N, w=None, dw=None) == api.LA_OK
