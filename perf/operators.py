"""Cases of the gated linear-attention and head-norm operators, in plain form and
through this library's calls.

The operators, per batch b and key/value head (query head h reads key/value head
h // (H / Hkv)), with a_t = exp(log_gate_t) one gate per token and head:

    S_t = a_t S_{t-1} + k_t v_t^T        o_t = scale * S_t^T q_t

"forward" is the whole sequence from a state S_in (zero when absent), "backward"
its gradients, "step" one token against the state held in place.  "norm" is the
group norm of each head's output row with a gate's activation, written channels
last, and "norm_backward" its gradients:

    y[b, n, h*D + d] = (w x_hat + bias)[h*D + d] * act(gate[b, n, h*D + d])

(without a gate: act(w x_hat + bias)), x_hat the row x[b, h, n, :] less its mean
over its standard deviation.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a pretraining layer's forward at the benchmark's shape (8 sequences of
        # 8192 tokens, 16 heads of 64)
        dict(name="fwd_b8h16n8192d64", op="forward", B=8, H=16, Hkv=16, N=8192, D=64, dtype="bf16",
             state=False, resets=False),
        # one long document's prefill, 131072 tokens, keeping the state for decoding
        dict(name="fwd_b1h32n131072d128", op="forward", B=1, H=32, Hkv=32, N=131072, D=128,
             dtype="bf16", state=True, resets=False),
        # a piece of a prompt continued from the state of the pieces before it:
        # ragged length, four query heads per key/value head, packed documents
        dict(name="fwd_b2h16kv4n777d128", op="forward", B=2, H=16, Hkv=4, N=777, D=128, dtype="bf16",
             state=True, resets=True),
        # float32 at a small head size: the reference-quality path
        dict(name="fwd_b3h6n1000d32_f32", op="forward", B=3, H=6, Hkv=6, N=1000, D=32, dtype="f32",
             state=True, resets=False),
        # the same layer's gradients in training, at the benchmark's shape
        dict(name="bwd_b8h16n8192d64", op="backward", B=8, H=16, Hkv=16, N=8192, D=64, dtype="bf16",
             state=False, resets=False),
        # a 16 x 128 language-model layer's gradients, documents packed into rows
        dict(name="bwd_b4h16n4096d128", op="backward", B=4, H=16, Hkv=16, N=4096, D=128,
             dtype="bf16", state=False, resets=True),
        # gradients through a carried state (truncated back-propagation), shared
        # key/value heads, odd length, float32
        dict(name="bwd_b2h6kv2n333d64_f32", op="backward", B=2, H=6, Hkv=2, N=333, D=64, dtype="f32",
             state=True, resets=False),
        # decoding a large batch: the state of 256 requests is read and written
        dict(name="step_b256h32d128", op="step", B=256, H=32, Hkv=32, N=1, D=128, dtype="bf16",
             state=True, resets=False),
        # decoding one request: latency
        dict(name="step_b1h16kv4d64", op="step", B=1, H=16, Hkv=4, N=1, D=64, dtype="bf16",
             state=True, resets=False),
        # the norm behind the layer above, gated
        dict(name="norm_b4h16n4096d128", op="norm", B=4, H=16, Hkv=16, N=4096, D=128, dtype="bf16",
             gate=True, act="silu", bias=True),
        # the norm of one decoding step of a small batch: latency
        dict(name="norm_b7h16n1d64", op="norm", B=7, H=16, Hkv=16, N=1, D=64, dtype="bf16",
             gate=True, act="silu", bias=False),
        # its gradients in training
        dict(name="normbwd_b8h16n8192d64", op="norm_backward", B=8, H=16, Hkv=16, N=8192, D=64,
             dtype="bf16", gate=True, act="silu", bias=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "step", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128]) if dtype == "bf16" and rng.random() < 0.8 else rng.choice([16, 32, 64, 128])
    fast = dtype == "bf16" and D >= 64
    Hkv = _log_int(rng, 1, 32)
    H = Hkv * (rng.choice([1, 1, 1, 2, 4]) if op in ("forward", "backward", "step") else 1)
    case = dict(op=op, H=H, Hkv=Hkv, D=D, dtype=dtype)
    if op == "step":
        case.update(B=min(_log_int(rng, 1, 300), (256 * 32 * 128 * 128) // (Hkv * D * D)), N=1,
                    state=True, resets=rng.random() < 0.3)
        return case
    # elements of one [B, H, N, D] tensor: no more than the largest listed case's,
    # and fewer where the float32 products run on the plain cores
    room = {"forward": 1 << 28 if fast else 1 << 24, "backward": 1 << 26 if fast else 1 << 22,
            "norm": 1 << 25, "norm_backward": 1 << 26}[op]
    longest = {"forward": 65536 if fast else 8192, "backward": 16384 if fast else 4096, "norm": 16384,
               "norm_backward": 16384}[op]
    N = _log_int(rng, 1, max(1, min(longest, room // (H * D))))
    B = _log_int(rng, 1, max(1, min(16, room // (H * D * N))))
    case.update(B=B, N=N)
    if op in ("forward", "backward"):
        case.update(state=rng.random() < 0.5, resets=rng.random() < 0.3)
    else:
        case.update(gate=rng.random() < 0.7, act=rng.choice(["silu", "silu", "identity"]),
                    bias=rng.random() < 0.5)
    return case


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    B, H, Hkv, N, D = (case[x] for x in ("B", "H", "Hkv", "N", "D"))

    def normal(*shape, size=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)

    st = dict(case)
    if case["op"] in ("norm", "norm_backward"):
        # an unnormalised attention output: rows of very different sizes
        rows = torch.exp(torch.randn(B, H, N, 1, generator=g, device="cuda"))
        st["x"] = (torch.randn(B, H, N, D, generator=g, device="cuda") * rows + 0.1 * rows).to(dt)
        st["weight"] = 1.0 + 0.1 * normal(H * D, dtype=torch.float32)
        st["bias_"] = normal(H * D, size=0.1, dtype=torch.float32) if case["bias"] else None
        st["gate_"] = normal(B, N, H * D) if case["gate"] else None
        if case["op"] == "norm_backward":
            st["dy"] = normal(B, N, H * D)
        return st
    toks = (N,) if case["op"] != "step" else ()
    st["q"], st["k"], st["v"] = (normal(B, h, *toks, D) for h in (H, Hkv, Hkv))
    # gates: the log-sigmoid of a projection, each head with a memory of its own
    # (from about ten to about a thousand tokens)
    reach = torch.linspace(2.3, 7.0, Hkv, device="cuda").view(1, Hkv, *(1 for _ in toks))
    x = torch.randn(B, Hkv, *toks, generator=g, device="cuda")
    lg = torch.nn.functional.logsigmoid(x + reach)
    if case["resets"]:  # a new document starts: the state before it is dropped
        lg = torch.where(torch.rand(lg.shape, generator=g, device="cuda") < 0.005, -math.inf, lg)
    st["log_gate"] = lg.to(dt)
    st["scale"] = D ** -0.5
    st["S_in"] = normal(B, Hkv, D, D, size=3.0, dtype=torch.float32) if case["state"] else None
    if case["op"] == "backward":
        st["dO"] = normal(B, H, N, D)
        st["dS_out"] = normal(B, Hkv, D, D, size=0.3, dtype=torch.float32) if case["state"] else None
    return st


# ------------------------------------------------------------- the plain forms
def _chunked(x, C):
    """[B, H, N, ...] -> [B, H, N/C, C, ...] in float32, zeros behind the end."""
    n = x.shape[2]
    pad = (-n) % C
    x = x.float()
    if pad:
        x = torch.cat([x, x.new_zeros(*x.shape[:2], pad, *x.shape[3:])], dim=2)
    return x.reshape(*x.shape[:2], (n + pad) // C, C, *x.shape[3:])


def _gates(lg, C):
    """Sums of the log gates in 64 bits: within each chunk (inclusive) and over
    whole chunks; a gate of zero is one that no product survives."""
    n = lg.shape[2]
    lg = lg.double().clamp(min=-1e4)
    pad = (-n) % C
    if pad:
        lg = torch.cat([lg, lg.new_zeros(*lg.shape[:2], pad)], dim=2)
    within = lg.reshape(*lg.shape[:2], (n + pad) // C, C).cumsum(-1)
    return within, within[..., -1].cumsum(-1)


def _carry(parts, total, first, reverse):
    """States at the chunks' borders from the chunks' own parts [B, H, n, D, D]:
    returns what enters each chunk and what leaves the last one."""
    B, H, n, D, _ = parts.shape
    if reverse:
        parts = parts.flip(2)
        total = (total[..., -1:] - torch.cat([torch.zeros_like(total[..., :1]), total[..., :-1]], -1)).flip(-1)
    at = torch.cat([torch.zeros_like(total[..., :1]), total], -1)  # [B, H, n + 1]
    far = at[..., :, None] - total[..., None, :]  # border m, chunk c < m
    m = torch.arange(n + 1, device=far.device)
    far = far.masked_fill(m[:, None] <= m[None, :n], -math.inf)
    S = (torch.exp(far).float() @ parts.reshape(B, H, n, D * D)).reshape(B, H, n + 1, D, D)
    if first is not None:
        S = S + torch.exp(at).float()[..., None, None] * first.float()[:, :, None]
    enter, leave = S[:, :, :n], S[:, :, n]
    return (enter.flip(2) if reverse else enter), leave


def _per_query(x, G):
    return x if G == 1 else x.repeat_interleave(G, dim=1)


def _per_kv(x, G):
    return x if G == 1 else x.reshape(x.shape[0], x.shape[1] // G, G, *x.shape[2:]).sum(2)


def _sequence(x, N, dtype):
    return x.reshape(*x.shape[:2], -1, *x.shape[4:])[:, :, :N].to(dtype)


def _plain_forward(st):
    q, k, v, lg, scale = (st[x] for x in ("q", "k", "v", "log_gate", "scale"))
    G, C, N = q.shape[1] // k.shape[1], 128, q.shape[2]
    within, total = _gates(lg, C)
    Q, K, V = (_chunked(x, C) for x in (q, k, v))
    left = torch.exp(within[..., -1:] - within).float()[..., None]
    S, S_out = _carry((K * left).transpose(-1, -2) @ V, total, st["S_in"], False)
    if not st["state"]:
        S_out = None
    decay = torch.exp((within[..., :, None] - within[..., None, :]).masked_fill(
        ~torch.ones(C, C, dtype=torch.bool, device=q.device).tril(), -math.inf)).float()
    P = (Q @ _per_query(K, G).transpose(-1, -2)) * _per_query(decay, G)
    o = P @ _per_query(V, G)
    o = o + _per_query(torch.exp(within).float()[..., None], G) * (Q @ _per_query(S, G))
    o = _sequence(o * scale, N, q.dtype)
    return {"o": o} if S_out is None else {"o": o, "S": S_out}


def _plain_backward(st):
    q, k, v, lg, dO, scale = (st[x] for x in ("q", "k", "v", "log_gate", "dO", "scale"))
    G, C, N = q.shape[1] // k.shape[1], 128, q.shape[2]
    within, total = _gates(lg, C)
    Q, K, V, dO = (_chunked(x, C) for x in (q, k, v, dO))
    tail = torch.exp(within[..., -1:] - within).float()[..., None]
    head = torch.exp(within).float()[..., None]
    S, _ = _carry((K * tail).transpose(-1, -2) @ V, total, st["S_in"], False)
    R, dS_in = _carry(_per_kv((Q * _per_query(head, G)).transpose(-1, -2) @ dO, G) * scale, total,
                      st["dS_out"], True)
    decay = torch.exp((within[..., :, None] - within[..., None, :]).masked_fill(
        ~torch.ones(C, C, dtype=torch.bool, device=q.device).tril(), -math.inf)).float() * scale
    decay = _per_query(decay, G)
    Kq, Vq, hq = _per_query(K, G), _per_query(V, G), _per_query(head, G) * scale
    P, W = Q @ Kq.transpose(-1, -2), dO @ Vq.transpose(-1, -2)
    dq_far = hq * (dO @ _per_query(S, G).transpose(-1, -2))
    dq = (W * decay) @ Kq + dq_far
    dk_far, dv_far = tail * (V @ R.transpose(-1, -2)), tail * (K @ R)
    dk = _per_kv((W * decay).transpose(-1, -2) @ Q, G) + dk_far
    dv = _per_kv((P * decay).transpose(-1, -2) @ dO, G) + dv_far
    # the gate at t scales what passes from the tokens j < t to the tokens i >= t
    M = _per_kv(P * W * decay, G)
    M = M.flip(-2).cumsum(-2).flip(-2).cumsum(-1)  # sums over i >= t and j <= u
    dg = torch.cat([torch.zeros_like(M[..., :1, 0]), M.diagonal(offset=-1, dim1=-2, dim2=-1)], -1)
    dg = dg + _per_kv((Q * dq_far).sum(-1), G).flip(-1).cumsum(-1).flip(-1)
    passed = (K * dk_far).sum(-1)
    dg = dg + passed.cumsum(-1) - passed
    dg = dg + torch.exp(within[..., -1:]).float() * (S * R).sum((-1, -2))[..., None]
    out = {"dq": _sequence(dq, N, q.dtype), "dk": _sequence(dk, N, k.dtype),
           "dv": _sequence(dv, N, v.dtype),
           "dlog_gate": dg.reshape(*dg.shape[:2], -1)[:, :, :N].to(lg.dtype)}
    if st["state"]:
        out["dS_in"] = dS_in
    return out


def _plain_step(st):
    q, k, v, lg, S = (st[x] for x in ("q", "k", "v", "log_gate", "S_in"))
    G = q.shape[1] // k.shape[1]
    S.copy_(torch.exp(lg.float())[..., None, None] * S + k.float()[..., :, None] * v.float()[..., None, :])
    o = (q.float()[..., None, :] @ _per_query(S, G))[..., 0, :] * st["scale"]
    return {"o": o.to(q.dtype), "S": S}


def _act(x, act):
    return x * torch.sigmoid(x) if act == "silu" else x


def _dact(x, act):
    if act != "silu":
        return torch.ones_like(x)
    s = torch.sigmoid(x)
    return s * (1 + x * (1 - s))


def _normalised(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    rstd = torch.rsqrt(var + _EPS)
    return ((x - mean) * rstd).transpose(1, 2).flatten(2), rstd.transpose(1, 2)


def _plain_norm(st):
    n = _normalised(st)[0] * st["weight"]
    n = n if st["bias_"] is None else n + st["bias_"]
    y = _act(n, st["act"]) if st["gate_"] is None else n * _act(st["gate_"].float(), st["act"])
    return y.to(st["x"].dtype)


def _plain_norm_backward(st):
    B, H, N, D = st["x"].shape
    xh, rstd = _normalised(st)
    n = xh * st["weight"]
    n = n if st["bias_"] is None else n + st["bias_"]
    dy, out = st["dy"].float(), {}
    if st["gate_"] is None:
        dn = dy * _dact(n, st["act"])
    else:
        gate = st["gate_"].float()
        dn = dy * _act(gate, st["act"])
        out["dgate"] = (dy * n * _dact(gate, st["act"])).to(st["gate_"].dtype)
    out["dweight"] = (dn * xh).sum((0, 1))
    if st["bias_"] is not None:
        out["dbias"] = dn.sum((0, 1))
    dx = (dn * st["weight"]).reshape(B, N, H, D)
    xh = xh.reshape(B, N, H, D)
    dx = rstd * (dx - dx.mean(-1, keepdim=True) - xh * (dx * xh).mean(-1, keepdim=True))
    out["dx"] = dx.transpose(1, 2).to(st["x"].dtype).contiguous()
    return out


# ------------------------------------------------------------ the library's calls
def _own(st):
    from linear_attention_transformers_b200 import api

    op = st["op"]
    if op == "forward":
        r = api.la_forward_gated(st["q"], st["k"], st["v"], st["log_gate"], scale=st["scale"],
                                 S_in=st["S_in"], return_state=st["state"])
        return {"o": r[0], "S": r[1]} if st["state"] else {"o": r}
    if op == "backward":
        r = api.la_backward_gated(st["q"], st["k"], st["v"], st["log_gate"], st["dO"],
                                  scale=st["scale"], S_in=st["S_in"], dS_out=st["dS_out"],
                                  return_dstate=st["state"])
        return dict(zip(("dq", "dk", "dv", "dlog_gate", "dS_in"), r))
    if op == "step":
        o = api.la_decode_step_gated(st["S_in"], st["q"], st["k"], st["v"], st["log_gate"],
                                     scale=st["scale"])
        return {"o": o, "S": st["S_in"]}
    if op == "norm":
        return api.la_group_norm(st["x"], st["weight"], bias=st["bias_"], gate=st["gate_"],
                                 act=st["act"], eps=_EPS)
    dx, dw, db, dg = api.la_group_norm_backward(st["x"], st["weight"], st["dy"], bias=st["bias_"],
                                                gate=st["gate_"], act=st["act"], eps=_EPS)
    return {n: t for n, t in (("dgate", dg), ("dweight", dw), ("dbias", db), ("dx", dx)) if t is not None}


def run(state):
    if own:
        return _own(state)
    return {"forward": _plain_forward, "backward": _plain_backward, "step": _plain_step,
            "norm": _plain_norm, "norm_backward": _plain_norm_backward}[state["op"]](state)


# ---------------------------------------------------------- bytes and operations
def work(case):
    B, H, Hkv, N, D = (case[x] for x in ("B", "H", "Hkv", "N", "D"))
    es = 2 if case["dtype"] == "bf16" else 4
    q, kv, states = B * H * N * D, B * Hkv * N * D, B * Hkv * D * D * 4
    op = case["op"]
    if op == "forward":
        # q, k, v, gates and the state in, o and the state out; two products with
        # the state a token (its update and the readout)
        return {"bytes": es * (2 * q + 2 * kv + kv // D) + (2 * states if case["state"] else 0),
                "flops": 2 * D * (q + kv)}
    if op == "backward":
        # q, k, v, dO, gates (and two states) in, four gradients (and a state's) out;
        # S rebuilt, R built, and the readouts dq, dk, dv
        return {"bytes": es * (3 * q + 4 * kv + 2 * (kv // D)) + (3 * states if case["state"] else 0),
                "flops": 2 * D * (2 * q + 3 * kv)}
    if op == "step":
        return {"bytes": 2 * states + es * (2 * q + 2 * kv + kv // D), "flops": 2 * D * (q + kv)}
    gate, params = int(case["gate"]), H * D * 4 * (1 + int(case["bias"]))
    if op == "norm":
        return {"bytes": es * q * (2 + gate) + params, "flops": 12 * q}
    return {"bytes": es * q * (3 + 2 * gate) + 2 * params, "flops": 30 * q}


# ------------------------------------------------------------- in 64 bits, by definition
def exact(case, seed):
    st = prepare(case, seed)
    f = {n: t.double() for n, t in st.items() if isinstance(t, torch.Tensor)}
    if case["op"] in ("norm", "norm_backward"):
        return _exact_norm(case, f)
    G = case["H"] // case["Hkv"]
    q, k, v, a, S = f["q"], f["k"], f["v"], torch.exp(f["log_gate"]), f.get("S_in")
    B, Hkv, D, N, scale = case["B"], case["Hkv"], case["D"], case["N"], st["scale"]
    if case["op"] == "step":
        S = a[..., None, None] * S + torch.einsum("bhd,bhe->bhde", k, v)
        o = scale * torch.einsum("bhgd,bhde->bhge", q.reshape(B, Hkv, G, D), S)
        return {"o": o.reshape(B, Hkv * G, D), "S": S}
    if N * (1 if case["op"] == "forward" else 2) * (2 + B * Hkv * D * D / 2e6) > 6e5:
        return None  # the token-by-token recurrence would take too long
    # time first; one state per key/value head
    W = B * Hkv
    q = q.reshape(W, G, N, D).permute(2, 0, 1, 3).contiguous()
    k, v = (x.reshape(W, N, D).permute(1, 0, 2).contiguous() for x in (k, v))
    a = a.reshape(W, N).t().contiguous()[..., None, None]
    S = torch.zeros(W, D, D, dtype=torch.float64, device=q.device) if S is None else S.reshape(W, D, D)
    back = lambda x: x.permute(1, 2, 0, 3).reshape(B, Hkv * x.shape[2], N, D)  # noqa: E731
    if case["op"] == "forward":
        o = torch.empty_like(q)
        for t in range(N):
            S = torch.baddbmm(a[t] * S, k[t][:, :, None], v[t][:, None, :])
            torch.bmm(q[t], S, out=o[t])
        out = {"o": back(o * scale)}
        if case["state"]:
            out["S"] = S.reshape(B, Hkv, D, D)
        return out
    dO = f["dO"].reshape(W, G, N, D).permute(2, 0, 1, 3).contiguous()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(N):
        S = torch.baddbmm(a[t] * S, k[t][:, :, None], v[t][:, None, :])
        torch.bmm(dO[t], S.transpose(1, 2), out=dq[t])
    dq *= scale
    dS = f.get("dS_out")
    dS = torch.zeros_like(S) if dS is None else dS.reshape(W, D, D)
    end = (S * dS).sum((1, 2))
    for t in range(N - 1, -1, -1):  # dS: the gradient with respect to S_t
        dS = torch.baddbmm(dS, q[t].transpose(1, 2), dO[t], alpha=scale)
        dk[t] = torch.bmm(dS, v[t][:, :, None])[..., 0]
        dv[t] = torch.bmm(k[t][:, None, :], dS)[:, 0]
        dS = a[t] * dS
    # the loss's derivative along each sum of log gates, then their sums from t on
    dg = (q * dq).sum((-1, -2)) - (k * dk).sum(-1)
    dg[-1] += end
    dg = dg.flip(0).cumsum(0).flip(0)
    if not case["state"]:
        dg[0] = 0  # nothing stands before the first token
    out = {"dq": back(dq), "dk": back(dk[:, :, None]), "dv": back(dv[:, :, None]),
           "dlog_gate": dg.t().reshape(B, Hkv, N)}
    if case["state"]:
        out["dS_in"] = dS.reshape(B, Hkv, D, D)
    return out


def _exact_norm(case, f):
    B, H, N, D = (case[x] for x in ("B", "H", "N", "D"))
    x = f["x"].permute(0, 2, 1, 3)  # [B, N, H, D]
    w = f["weight"].reshape(H, D)
    b = f["bias_"].reshape(H, D) if case["bias"] else torch.zeros_like(w)
    sd = torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + _EPS)
    xh = (x - x.mean(-1, keepdim=True)) / sd
    n = xh * w + b
    silu = case["act"] == "silu"
    at = f["gate_"].reshape(B, N, H, D) if case["gate"] else n
    e = 1 / (1 + torch.exp(-at))
    act, dact = (at * e, e + at * e * (1 - e)) if silu else (at, torch.ones_like(at))
    if case["op"] == "norm":
        return (n * act if case["gate"] else act).reshape(B, N, H * D)
    dy = f["dy"].reshape(B, N, H, D)
    out = {}
    if case["gate"]:
        out["dgate"] = (dy * n * dact).reshape(B, N, H * D)
        dn = dy * act
    else:
        dn = dy * dact
    out["dweight"] = torch.einsum("bnhd,bnhd->hd", dn, xh).reshape(-1)
    if case["bias"]:
        out["dbias"] = dn.sum((0, 1)).reshape(-1)
    t = dn * w
    # dx_i = (t_i - sum_j t_j (1 + xh_i xh_j) / D) / sd
    dx = (t - (t.sum(-1, keepdim=True) + xh * torch.einsum("bnhd,bnhd->bnh", t, xh)[..., None]) / D) / sd
    out["dx"] = dx.permute(0, 2, 1, 3).contiguous()
    return out
