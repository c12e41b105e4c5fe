"""The ways in which the tensor-core kernels form the border states, each at
lengths where its rings and buffers go round more than once, against the float32
kernels (held to the oracle in test_gpu_gated.py) on the same values.  The names of
the launches show which way a call took: a size that the model of pick_chain no
longer sends there fails here instead of testing something else."""
import pytest
import torch

from gated_util import MAX, REL, REL_STATE, close, tensors
from linear_attention_transformers_b200 import api

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# B, Hkv, N by D.  The walks go over 12 blocks, three rounds of their ring of gates;
# the spans are more than three times as many as the blocks of the grid (148 SMs, two
# blocks on each at D = 64)
WALK64 = dict(D64=(16, 8, 1500), D128=(16, 8, 1500))
WALK32 = dict(D64=(8, 8, 1500), D128=(4, 8, 1500))
SPANS = dict(D64=(1, 8, 16300), D128=(1, 8, 16300))


def launched(call):
    """(what the call returns, the names of its launches)"""
    torch.cuda.synchronize()
    api.la_profile_collect()
    api.la_profile_enable(True)
    try:
        out = call()
        torch.cuda.synchronize()
    finally:
        api.la_profile_enable(False)
    api.la_get_device_error()
    return out, set(api.la_profile_collect())


def all_close(names, got, ref):
    for n, g, r in zip(names, got, ref):
        rel = REL_STATE[BF] if n in ("S", "dS_in") else REL[BF]
        close(g, r.cpu(), rel, 4 * rel if n in ("S", "dS_in") else MAX[BF], n)


@pytest.mark.parametrize("way,sizes", [("chain64", WALK64), ("chain32", WALK32), ("span", SPANS)])
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("D", [64, 128])
def test_every_way_to_the_states(D, group, way, sizes):
    B, Hkv, N = sizes[f"D{D}"]
    ins = tensors(B, Hkv * group, Hkv, N, D, BF, N + D + group, resets=True)
    q, k, v, lg, dO, S, dS = ins
    wide = [x.float() for x in (q, k, v, lg, dO)]
    scale = D ** -0.5
    s_way = {"span": {"gated_span", "gated_border"}}.get(way, {f"gated_{way}"})
    r_way = {n + "_rev" for n in s_way}

    # nothing carried in or out: the states only enter the blocks, in two parts
    o, names = launched(lambda: api.la_forward_gated(q, k, v, lg, scale))
    assert names == s_way | {"gated_o"}
    all_close(["o"], [o], [api.la_forward_gated(*wide[:4], scale)])
    got, names = launched(lambda: api.la_backward_gated(q, k, v, lg, dO, scale))
    assert names == s_way | r_way | {"gated_bwd"}
    all_close(["dq", "dk", "dv", "dlog_gate"], got, api.la_backward_gated(*wide, scale))
    again = api.la_backward_gated(q, k, v, lg, dO, scale)
    assert all(torch.equal(a, b) for a, b in zip(got, again))

    # a state in and out: three parts
    got, names = launched(lambda: api.la_forward_gated(q, k, v, lg, scale, S, return_state=True))
    assert names == s_way | {"gated_o"}
    all_close(["o", "S"], got, api.la_forward_gated(*wide[:4], scale, S, return_state=True))
    got, names = launched(lambda: api.la_backward_gated(q, k, v, lg, dO, scale, S, dS, return_dstate=True))
    assert names == s_way | r_way | {"gated_bwd"}
    all_close(["dq", "dk", "dv", "dlog_gate", "dS_in"], got,
              api.la_backward_gated(*wide, scale, S, dS, return_dstate=True))


@pytest.mark.parametrize("D", [32, 64, 128])
def test_long_offsets_in_the_same_way(D):
    # forward and backward on tensors of more than 2^31 elements: the last heads are
    # bitwise those of a call on them alone, which forms their states the same way
    N, H, last = 4096, (1 << 31) // (4096 * D) + 3, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(1, H, N, D, generator=g, device="cuda", dtype=BF)
    lg = torch.nn.functional.logsigmoid(torch.randn(1, H, N, generator=g, device="cuda") + 3).to(BF)
    a, b = q[:, -last:].contiguous(), lg[:, -last:].contiguous()
    for whole, part in ((lambda: (api.la_forward_gated(q, q, q, lg, 0.1),),
                         lambda: (api.la_forward_gated(a, a, a, b, 0.1),)),
                        (lambda: api.la_backward_gated(q, q, q, lg, q, 0.1),
                         lambda: api.la_backward_gated(a, a, a, b, a, 0.1))):
        x, names = launched(whole)
        x = [t[:, -last:].clone() for t in x]
        y, names_part = launched(part)
        assert names == names_part
        for s, t in zip(x, y):
            assert torch.equal(s, t)
