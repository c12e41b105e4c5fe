"""Inputs and bounds of the gated-attention and head-norm tests.

Bounds, for outputs compared with the float64 oracle on the same inputs:

float32.  Every output is a sum of at most 128 (head size) + 64 (chunk)
products and as many border states as the sequence has chunks (at most 16 in
these tests), each addition off by at most half a step, 2^-24 of the partial
sum; the weights carry two more (exp2f and its rounded argument).  The errors
are independent, so their 2-norm grows with the square root of the count,
about sqrt(210) * 2^-24 < 2^-20; REL = 2^-18 leaves four times that, and the
largest single one is a few times the typical one (MAX = 2^-16).  dlog_gate is
a running sum of differences whose terms are larger than itself: 4 REL.

bf16.  At most three roundings to bf16 lie behind an output: the weighted C x C
product, the state operand, and the output itself.  Each is off by at most
u = 2^-8 of the value, u / sqrt(3) in the root mean square; independent, they
give at most u in the 2-norm: REL = 2^-8.  The largest of 10^6 errors is about
six of the typical ones beside the output's own half step: 7 u < MAX = 2^-5 of
the largest value.  float32 outputs of bf16 inputs (states, channel sums) come
from products of exact bf16 values and of a scaled operand held as three bf16
parts (2^-24 of the value), added in float32 as above: REL = 2^-18.
"""
import math

import numpy as np
import torch

REL = {torch.float32: 2.0 ** -18, torch.bfloat16: 2.0 ** -8}
MAX = {torch.float32: 2.0 ** -16, torch.bfloat16: 2.0 ** -5}
REL_STATE = {torch.float32: 2.0 ** -18, torch.bfloat16: 2.0 ** -18}


def close(got, ref, rel, most, what):
    g = got.detach().double().cpu().numpy()
    r = np.asarray(ref, dtype=np.float64)
    # no float32 lies between 0 and 2^-149: an oracle value below half of that is 0 in
    # every type an output has
    r = np.where(np.abs(r) < 2.0 ** -150, 0.0, r)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert np.isfinite(g).all(), f"{what}: not finite"
    if r.size == 0:
        return
    err = np.abs(g - r)
    if not np.abs(r).max() > 0:
        assert not err.any(), f"{what}: {err.max()} where the oracle is zero"
        return
    a = np.linalg.norm(err) / np.linalg.norm(r)
    b = err.max() / np.abs(r).max()
    assert a <= rel and b <= most, f"{what}: {a:.3e} of {rel:.3e} in the 2-norm, {b:.3e} of {most:.3e} at most"


def tensors(B, H, Hkv, N, D, dtype, seed, resets=False, gate=None):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, size=1.0, dt=dtype):
        return (torch.randn(*shape, generator=g) * size).to(dt).cuda()

    q, dO = normal(B, H, N, D), normal(B, H, N, D)
    k, v = normal(B, Hkv, N, D), normal(B, Hkv, N, D)
    reach = torch.linspace(0.0, 6.0, max(Hkv, 1))[:Hkv].view(1, Hkv, 1)
    lg = torch.nn.functional.logsigmoid(torch.randn(B, Hkv, N, generator=g) + reach)
    if gate is not None:
        lg = torch.full_like(lg, gate)
    if resets:
        lg = torch.where(torch.rand(lg.shape, generator=g) < 0.05, -math.inf, lg)
    S = normal(B, Hkv, D, D, dt=torch.float32)
    dS = normal(B, Hkv, D, D, size=0.3, dt=torch.float32)
    return q, k, v, lg.to(dtype).cuda(), dO, S, dS
