"""The operators that join the attention chain: the per-head norm of queries
and keys with the position rotation in the same pass (forward and backward,
positions of one or several axes), and linear attention with a decay for each
head (chunked forward, backward, and the recurrent form for single tokens).

A case names the operator and its sizes.  ``run`` makes one pass, in the plain
form (elementary torch operations in 32 bits) or, where ``own`` is set,
through the framework's entry points.  ``exact`` evaluates the definitions in
64 bits.

Layouts: q [B][T][Hq][D], k, v [B][T][Hkv][D]; query head h reads KV head
h / (Hq / Hkv); recurrent state [B][Hkv][D][D] fp32 (key component, value
component); positions [axes][B][T] int32.
"""
import math

import torch

own = False

_BF, _F = torch.bfloat16, torch.float32
_CHUNK = 64          # tokens per chunk of the plain chunked form


# --------------------------------------------------------------------- cases
def _qk(name, op, B, T, Hq, Hkv, D, rotary, base, interleaved, axes, dtype="bf16", dy="f32", far=0):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rotary": rotary, "base": base,
            "interleaved": interleaved, "axes": axes, "dtype": dtype, "dy": dy, "far": far}


def _lin(name, op, B, T, Hq, Hkv, D, state=False, padded=False):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "state": state, "padded": padded}


def listed():
    return [
        # one new token for each of 64 sequences at positions of their own, beside the decode attention (20/5 heads)
        _qk("qk_fwd_decode", "qk_norm_rope_fwd", 64, 1, 20, 5, 128, 128, 500000.0, True, 1, far=1000000),
        # the queries and keys of a training step, T = 2048, read out of a packed projection
        _qk("qk_fwd_train", "qk_norm_rope_fwd", 4, 2048, 20, 20, 128, 128, 10000.0, False, 1),
        # image and video tokens: three axes over the rotated part of the head, odd length, fp32 activations
        _qk("qk_fwd_axes_f32", "qk_norm_rope_fwd", 2, 1025, 20, 5, 80, 48, 10000.0, False, 3, dtype="f32"),
        # one layer of the 30-layer chain: fp32 gradients from the softmax attention's backward
        _qk("qk_bwd_layer", "qk_norm_rope_bwd", 2, 512, 20, 5, 128, 128, 500000.0, True, 1),
        # a training step on video tokens: bf16 gradients from the linear attention's backward
        _qk("qk_bwd_axes", "qk_norm_rope_bwd", 4, 2048, 20, 20, 128, 96, 10000.0, False, 3, dy="bf16"),
        # one layer of the chain with shared KV heads
        _lin("lin_fwd_layer", "lin_attn_fwd", 2, 512, 20, 5, 128),
        # a long prompt that continues from a state and hands its state on
        _lin("lin_fwd_long_state", "lin_attn_fwd", 1, 8192, 32, 32, 128, state=True),
        # a short ragged batch of prompts, padded on the right, small heads
        _lin("lin_fwd_padded", "lin_attn_fwd", 3, 777, 16, 4, 64, state=True, padded=True),
        # one layer of the chain, backward
        _lin("lin_bwd_layer", "lin_attn_bwd", 2, 512, 20, 5, 128),
        # a training step's backward, T = 2048, with the states' gradients
        _lin("lin_bwd_train", "lin_attn_bwd", 4, 2048, 20, 20, 128, state=True),
        # one token for one sequence: latency
        _lin("lin_decode_one", "lin_attn_decode", 1, 1, 20, 5, 128),
        # one token for each of 64 sequences in a pool of states, some rows of the batch empty
        _lin("lin_decode_pool", "lin_attn_decode", 64, 1, 20, 20, 128, padded=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope_fwd", "qk_norm_rope_bwd", "lin_attn_fwd", "lin_attn_bwd", "lin_attn_decode"])
    Hkv, G = rng.choice([1, 2, 4, 5, 8, 20, 32]), rng.choice([1, 1, 2, 4, 8])
    G = min(G, max(1, 32 // Hkv))
    Hq = Hkv * G
    if op.startswith("qk"):
        D = rng.choice([64, 80, 96, 128, 128, 256])
        rotary = rng.choice([D, D, 2 * (D // 4), 2 * (3 * D // 8)])
        most = max(2, 4 * 2048 * 40 * 128 // ((Hq + Hkv) * D))          # tokens
        T = _log_int(rng, 1, most)
        B = _log_int(rng, 1, max(1, min(64, most // T)))
        case = _qk("", op, B, T, Hq, Hkv, D, rotary, rng.choice([10000.0, 500000.0]), rng.random() < 0.5,
                   rng.choice([1, 1, 2, 3]), dtype=rng.choice(["bf16", "bf16", "f32"]), dy=rng.choice(["f32", "bf16"]),
                   far=rng.choice([0, 0, 100000]))
    elif op == "lin_attn_decode":
        D = rng.choice([64, 128])
        most = max(1, 64 * 20 * 128 * 128 // (Hkv * D * D))
        case = _lin("", op, _log_int(rng, 1, min(256, most)), 1, Hq, Hkv, D, padded=rng.random() < 0.5)
    else:
        D = rng.choice([64, 128])
        most = max(2, 4 * 2048 * 20 * 128 // (Hq * D))
        T = _log_int(rng, 1, min(8192, most))
        B = _log_int(rng, 1, max(1, min(32, most // T)))
        case = _lin("", op, B, T, Hq, Hkv, D, state=rng.random() < 0.5, padded=B > 1 and rng.random() < 0.4)
    del case["name"]
    return case


# -------------------------------------------------------------------- inputs
def _sections(pairs, axes):
    """Pairs of each axis: the first axis takes what an even split leaves over."""
    if axes == 1:
        return [pairs]
    each = pairs // axes
    return [pairs - each * (axes - 1)] + [each] * (axes - 1)


def _log_decays(heads):
    """Slopes as the heads of a linear attention have them: from fast to slow."""
    h = torch.arange(1, heads + 1, dtype=torch.float64, device="cuda")
    return (-(2.0 ** (-8.0 * h / heads))).to(_F)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]

    def normal(*shape, dtype=_F):
        return torch.randn(*shape, generator=g, device="cuda", dtype=_F).to(dtype)

    s = dict(case)
    if case["op"].startswith("qk"):
        dtype = _BF if case["dtype"] == "bf16" else _F
        qkv = normal(B, T, Hq + 2 * Hkv, D, dtype=dtype)     # the projection's packed output
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], eps=1e-6,
                 gamma_q=1.0 + 0.1 * normal(D), gamma_k=1.0 + 0.1 * normal(D),
                 sections=_sections(case["rotary"] // 2, case["axes"]), positions=None)
        if case["axes"] > 1:
            t = torch.arange(T, device="cuda", dtype=torch.int32)
            side = max(1, int(math.isqrt(max(T // 4, 1))))
            planes = torch.stack([t // (side * side), (t // side) % side, t % side][:case["axes"]])
            start = torch.randint(0, 64 + case["far"], (case["axes"], B, 1), generator=g, device="cuda", dtype=torch.int32)
            s["positions"] = (planes[:, None, :] + start).contiguous()
        elif case["far"]:
            start = torch.randint(0, case["far"], (1, B, 1), generator=g, device="cuda", dtype=torch.int32)
            s["positions"] = (start + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        if case["op"].endswith("bwd"):
            dyt = _BF if case["dy"] == "bf16" else _F
            s.update(dq_out=normal(B, T, Hq, D, dtype=dyt), dk_out=normal(B, T, Hkv, D, dtype=dyt))
        return s
    s["scale"] = 1.0 / math.sqrt(D)
    s["log_decay"] = _log_decays(Hkv)
    if case["op"] == "lin_attn_decode":
        s.update(q=normal(B, Hq, D, dtype=_BF), k=normal(B, Hkv, D, dtype=_BF), v=normal(B, Hkv, D, dtype=_BF))
        s["slots"], pool = None, B
        if case["padded"]:                                   # a pool with spare states; a few rows of the batch are empty
            pool = B + 3
            slots = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
            empty = torch.rand(B, generator=g, device="cuda") < 0.1
            s["slots"] = torch.where(empty, torch.full_like(slots, -1), slots)
        s["recurrent"] = normal(pool, Hkv, D, D)
        return s
    s.update(q=normal(B, T, Hq, D, dtype=_BF), k=normal(B, T, Hkv, D, dtype=_BF), v=normal(B, T, Hkv, D, dtype=_BF),
             initial=None, dfinal=None, lengths=None)
    if case["state"]:
        s["initial"] = normal(B, Hkv, D, D)
    if case["padded"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
        s["lengths"] = n
    if case["op"] == "lin_attn_bwd":
        s["dout"] = normal(B, T, Hq, D, dtype=_BF)
        if case["state"]:
            s["dfinal"] = normal(B, Hkv, D, D)
    return s


# --------------------------------------------------- the framework's own calls
def _own(s):
    import transformer_attention_backward_gb300 as abw
    op = s["op"]
    if op.startswith("qk"):
        how = dict(eps=s["eps"], rope_base=s["base"], rotary_dim=s["rotary"], interleaved=s["interleaved"],
                   positions=s["positions"], sections=s["sections"])
        if op == "qk_norm_rope_fwd":
            return abw.qk_norm_rope_fwd(s["q"], s["k"], s["gamma_q"], s["gamma_k"], **how)
        return abw.qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["gamma_q"], s["gamma_k"], **how)
    if op == "lin_attn_decode":
        o = abw.lin_attn_decode(s["q"], s["k"], s["v"], s["recurrent"], s["log_decay"], s["scale"], slots=s["slots"])
        return o, s["recurrent"]
    if op == "lin_attn_fwd":
        return abw.lin_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], initial_state=s["initial"],
                                lengths=s["lengths"], want_final_state=s["state"])
    return abw.lin_attn_bwd(s["q"], s["k"], s["v"], s["dout"], s["log_decay"], s["scale"], initial_state=s["initial"],
                            dfinal_state=s["dfinal"], lengths=s["lengths"], want_dinitial_state=s["state"])


# -------------------------------------------------------------- the plain form
def _cos_sin(s):
    """cos, sin of the angles, [B or 1][T][1][rotary / 2]; formed in 64 bits."""
    pairs = s["rotary"] // 2
    freq = s["base"] ** (-2.0 * torch.arange(pairs, device="cuda", dtype=torch.float64) / s["rotary"])
    if s["positions"] is None:
        pos = torch.arange(s["T"], device="cuda", dtype=torch.float64)[None, :, None]
    else:
        axis = torch.repeat_interleave(torch.arange(s["axes"], device="cuda"),
                                       torch.tensor(s["sections"], device="cuda"), output_size=pairs)
        pos = s["positions"].double()[axis].permute(1, 2, 0)
    angle = (pos * freq)[:, :, None, :]
    return angle.cos().float(), angle.sin().float()


def _turn(x, cos, sin, s):
    """Rotates the pairs of the first `rotary` components by the angles."""
    R = s["rotary"]
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_qk_fwd(x, gamma, cos, sin, s):
    y = x.float()
    inv = 1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"])
    return _turn(y * inv * gamma, cos, sin, s).to(x.dtype)


def _plain_qk_bwd(x, dy, gamma, cos, sin, s):
    y, dn = x.float(), _turn(dy.float(), cos, -sin, s)
    inv = 1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"])
    c = (dn * gamma * y).mean(-1, keepdim=True)
    dx = (dn * gamma - y * c * inv * inv) * inv
    return dx.to(x.dtype), (dn * y * inv).sum((0, 1, 2))


def _chunks(x, heads):
    """[B][T][..][D] as fp32 chunks [B][N][C][heads][-1][D], zero behind T."""
    B, T, D = x.shape[0], x.shape[1], x.shape[-1]
    pad = -T % _CHUNK
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad))
    return x.reshape(B, (T + pad) // _CHUNK, _CHUNK, heads, -1, D)


def _powers(log_decay, n):
    """decay^0 .. decay^(n - 1) for each head, [heads][n]."""
    return torch.exp(log_decay[:, None] * torch.arange(n, device="cuda", dtype=_F))


def _within(log_decay):
    """decay^(i - j) for j <= i inside a chunk, [heads][C][C]."""
    i = torch.arange(_CHUNK, device="cuda")
    gap = i[:, None] - i[None, :]
    return torch.where(gap >= 0, torch.exp(log_decay[:, None, None] * gap.clamp(min=0)), torch.zeros((), device="cuda"))


def _across(log_decay, n):
    """decay^(C (n - 1 - m)) for chunks m < n, [heads][N][N]."""
    i = torch.arange(n, device="cuda")
    gap = i[:, None] - 1 - i[None, :]
    return torch.where(gap >= 0, torch.exp(log_decay[:, None, None] * (_CHUNK * gap.clamp(min=0))),
                       torch.zeros((), device="cuda"))


def _masked(x, s):
    if s["lengths"] is None:
        return x
    live = torch.arange(s["T"], device="cuda")[None, :] < s["lengths"][:, None]
    return torch.where(live[:, :, None, None], x, torch.zeros((), device="cuda", dtype=x.dtype))


def _to_end(s):
    """decay^(length - 1 - t) for t < length, else 0, [B][T][Hkv]; and
    decay^length, [B][Hkv]."""
    T, ld = s["T"], s["log_decay"]
    n = torch.full((s["B"],), T, device="cuda") if s["lengths"] is None else s["lengths"]
    gap = n[:, None] - 1 - torch.arange(T, device="cuda")[None, :]
    w = torch.where((gap >= 0)[:, :, None], torch.exp(ld * gap.clamp(min=0)[:, :, None]), torch.zeros((), device="cuda"))
    return w, torch.exp(ld * n[:, None])


def _states(k, v, s):
    """The state that enters each chunk, [B][N][Hkv][D][D]."""
    ld, n = s["log_decay"], k.shape[1]
    w = _powers(ld, _CHUNK).flip(1)
    add = torch.einsum("hc,bnchd,bnche->bnhde", w, k, v)
    into = torch.einsum("hnm,bmhde->bnhde", _across(ld, n), add)
    if s["initial"] is not None:
        into = into + torch.exp(ld * _CHUNK * torch.arange(n, device="cuda")[:, None])[None, :, :, None, None] * s["initial"][:, None]
    return into


def _joined(x, s, heads):
    """Chunks [B][N][C][Hkv][..][D] as the first T rows [B][T][heads][D]."""
    return x.reshape(s["B"], -1, heads, s["D"])[:, :s["T"]]


def _plain_lin_fwd(s):
    H, ld = s["Hkv"], s["log_decay"]
    q, k, v = (_chunks(_masked(s[x], s), H) for x in "qkv")
    k, v = k[:, :, :, :, 0], v[:, :, :, :, 0]
    p = torch.einsum("bnchgd,bnkhd->bnhgck", q, k) * _within(ld)[:, None]
    o = torch.einsum("bnhgck,bnkhe->bnchge", p, v)
    o = o + torch.einsum("hc,bnchgd,bnhde->bnchge", _powers(ld, _CHUNK + 1)[:, 1:], q, _states(k, v, s))
    o = _joined(o * s["scale"], s, s["Hq"]).to(_BF)
    if not s["state"]:
        return o, None
    w, all_ = _to_end(s)
    final = torch.einsum("bth,bthd,bthe->bhde", w, _masked(s["k"], s).float(), _masked(s["v"], s).float())
    return o, final + all_[:, :, None, None] * s["initial"]


def _plain_lin_bwd(s):
    H, ld, scale = s["Hkv"], s["log_decay"], s["scale"]
    q, k, v, do = (_chunks(_masked(s[x], s), H) for x in ("q", "k", "v", "dout"))
    k, v = k[:, :, :, :, 0], v[:, :, :, :, 0]
    inside, up = _within(ld)[:, None], _powers(ld, _CHUNK + 1)[:, 1:]
    p = torch.einsum("bnchgd,bnkhd->bnhgck", q, k) * inside * scale
    dp = torch.einsum("bnchge,bnkhe->bnhgck", do, v) * inside * scale
    dq = torch.einsum("bnhgck,bnkhd->bnchgd", dp, k)
    dk = torch.einsum("bnhgck,bnchgd->bnkhd", dp, q)
    dv = torch.einsum("bnhgck,bnchge->bnkhe", p, do)
    dq = dq + scale * torch.einsum("hc,bnchge,bnhde->bnchgd", up, do, _states(k, v, s))
    add = scale * torch.einsum("hc,bnchgd,bnchge->bnhde", up, q, do)
    back = torch.einsum("hmn,bmhde->bnhde", _across(ld, q.shape[1]), add)     # what later chunks hand back
    down = _powers(ld, _CHUNK).flip(1)
    dk = dk + torch.einsum("hc,bnche,bnhde->bnchd", down, v, back)
    dv = dv + torch.einsum("hc,bnchd,bnhde->bnche", down, k, back)
    dq, dk, dv = _joined(dq, s, s["Hq"]), _joined(dk, s, H), _joined(dv, s, H)
    if not s["state"]:
        return dq.to(_BF), dk.to(_BF), dv.to(_BF), None
    w, all_ = _to_end(s)
    dk = dk + torch.einsum("bth,bthe,bhde->bthd", w, _masked(s["v"], s).float(), s["dfinal"])
    dv = dv + torch.einsum("bth,bthd,bhde->bthe", w, _masked(s["k"], s).float(), s["dfinal"])
    chunk = torch.exp(ld * _CHUNK * torch.arange(q.shape[1], device="cuda")[:, None])
    dinit = torch.einsum("nh,bnhde->bhde", chunk, add) + all_[:, :, None, None] * s["dfinal"]
    return dq.to(_BF), dk.to(_BF), dv.to(_BF), dinit


def _plain_decode(s):
    H, D, state = s["Hkv"], s["D"], s["recurrent"]
    q, k, v = s["q"].float().reshape(s["B"], H, -1, D), s["k"].float(), s["v"].float()
    rows = torch.arange(s["B"], device="cuda") if s["slots"] is None else s["slots"].long()
    live = rows >= 0
    at = torch.where(live, rows, torch.full_like(rows, state.shape[0]))   # an empty row works on a spare state
    if s["slots"] is None:
        state.mul_(torch.exp(s["log_decay"])[:, None, None]).add_(k[..., :, None] * v[..., None, :])
        new = state
    else:
        spare = torch.cat([state, torch.zeros_like(state[:1])])
        new = spare[at] * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
        spare[at] = new
        state.copy_(spare[:-1])
    o = torch.einsum("bhgd,bhde->bhge", q, new) * s["scale"]
    o = torch.where(live[:, None, None, None], o, torch.zeros((), device="cuda"))
    return o.reshape(s["B"], s["Hq"], D).to(_BF), state


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"].startswith("qk"):
        cos, sin = _cos_sin(s)
        if s["op"] == "qk_norm_rope_fwd":
            return _plain_qk_fwd(s["q"], s["gamma_q"], cos, sin, s), _plain_qk_fwd(s["k"], s["gamma_k"], cos, sin, s)
        dq, dgq = _plain_qk_bwd(s["q"], s["dq_out"], s["gamma_q"], cos, sin, s)
        dk, dgk = _plain_qk_bwd(s["k"], s["dk_out"], s["gamma_k"], cos, sin, s)
        return dq, dk, dgq, dgk
    return {"lin_attn_fwd": _plain_lin_fwd, "lin_attn_bwd": _plain_lin_bwd, "lin_attn_decode": _plain_decode}[s["op"]](s)


# ------------------------------------------------------------------------ work
def work(case):
    """Inputs read once, outputs written once; products of the recurrence
    (one D x D update and one D x D read for each head and token)."""
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    n = B * T
    if case["op"].startswith("qk"):
        e = 2 if case["dtype"] == "bf16" else 4
        el = n * (Hq + Hkv) * D
        pos = 4 * n * case["axes"] if case["axes"] > 1 or case["far"] else 0
        if case["op"].endswith("fwd"):
            return {"bytes": 2 * el * e + pos + 8 * D, "flops": 9 * el}
        return {"bytes": el * (2 * e + (2 if case["dy"] == "bf16" else 4)) + pos + 16 * D, "flops": 16 * el}
    state = 4 * B * Hkv * D * D
    if case["op"] == "lin_attn_decode":
        return {"bytes": 2 * state + 2 * n * (2 * Hq + 2 * Hkv) * D, "flops": n * D * D * (3 * Hkv + 2 * Hq)}
    extra = 2 * state if case["state"] else 0
    if case["op"] == "lin_attn_fwd":
        return {"bytes": 2 * n * (2 * Hq + 2 * Hkv) * D + extra, "flops": 2 * n * D * D * (Hq + Hkv)}
    return {"bytes": 2 * n * (3 * Hq + 4 * Hkv) * D + (extra + 4 * B * Hkv * D * D if case["state"] else 0),
            "flops": 2 * n * D * D * (2 * Hq + 3 * Hkv)}


# ----------------------------------------------------- the definitions, 64 bits
def _exact_rotation(case, s, b, t0, t1):
    """One complex number per pair for the tokens t0 .. t1 - 1 of sequence b."""
    pairs = case["rotary"] // 2
    turn = torch.empty(t1 - t0, pairs, dtype=torch.float64, device="cuda")
    first = 0
    for axis, count in enumerate(s["sections"]):
        where = torch.arange(t0, t1, device="cuda") if s["positions"] is None else s["positions"][axis, b, t0:t1]
        for i in range(first, first + count):
            turn[:, i] = where.double() / case["base"] ** (2.0 * i / case["rotary"])
        first += count
    return torch.polar(torch.ones_like(turn), turn)


def _exact_qk(case, s):
    R, half = case["rotary"], case["rotary"] // 2
    bwd = case["op"].endswith("bwd")

    def rotated(x, z):
        y = x.clone()
        if case["interleaved"]:
            w = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) * z[:, None, :]
            y[..., 0:R:2], y[..., 1:R:2] = w.real, w.imag
        else:
            w = torch.complex(x[..., :half], x[..., half:R]) * z[:, None, :]
            y[..., :half], y[..., half:R] = w.real, w.imag
        return y

    outs, scales = [], []
    for x, gamma, dy in ((s["q"], s["gamma_q"], s.get("dq_out")), (s["k"], s["gamma_k"], s.get("dk_out"))):
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dg = torch.zeros(case["D"], dtype=torch.float64, device="cuda")
        g = gamma.double()
        for b in range(case["B"]):
            z = _exact_rotation(case, s, b, 0, case["T"])
            xb = x[b].double()
            rms = torch.sqrt(xb.pow(2).sum(-1, keepdim=True) / case["D"] + s["eps"])
            if not bwd:
                out[b] = rotated(g * (xb / rms), z)
                continue
            dn = rotated(dy[b].double(), z.conj())
            unit = xb / rms
            du = dn * g
            out[b] = (du - unit * (du * unit).sum(-1, keepdim=True) / case["D"]) / rms
            dg += (dn * unit).sum((0, 1))
        outs.append(out)
        scales.append(dg)
    return outs + scales if bwd else outs


def _exact_lin(case, s):
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    G, scale, bwd = Hq // Hkv, s["scale"], case["op"] == "lin_attn_bwd"
    f64 = dict(dtype=torch.float64, device="cuda")
    o, dq = torch.zeros(B, T, Hq, D, **f64), torch.zeros(B, T, Hq, D, **f64)
    dk, dv = torch.zeros(B, T, Hkv, D, **f64), torch.zeros(B, T, Hkv, D, **f64)
    end = torch.zeros(B, Hkv, D, D, **f64)
    for h in range(Hkv):
        ld = float(s["log_decay"][h])
        for b in range(B):
            n = T if s["lengths"] is None else int(s["lengths"][b])
            t = torch.arange(n, **f64)
            weight = torch.tril(torch.exp(torch.clamp(t[:, None] - t[None, :], min=0.0).mul_(ld)))
            k, v = s["k"][b, :n, h].double(), s["v"][b, :n, h].double()
            rise, fall = torch.exp(ld * (t + 1))[:, None], torch.exp(ld * (n - 1 - t))[:, None]
            s0 = s["initial"][b, h].double() if case["state"] else None
            if not bwd:
                for hq in range(h * G, (h + 1) * G):
                    q = s["q"][b, :n, hq].double()
                    y = (weight * (q @ k.T)) @ v
                    o[b, :n, hq] = scale * (y + (rise * q) @ s0 if s0 is not None else y)
                if case["state"]:
                    end[b, h] = (fall * k).T @ v + math.exp(ld * n) * s0
                continue
            if case["state"]:
                df = s["dfinal"][b, h].double()
                end[b, h] = math.exp(ld * n) * df
                dk[b, :n, h] += fall * (v @ df.T)
                dv[b, :n, h] += fall * (k @ df)
            for hq in range(h * G, (h + 1) * G):
                q, do = s["q"][b, :n, hq].double(), s["dout"][b, :n, hq].double() * scale
                dw = weight * (do @ v.T)
                dq[b, :n, hq] = dw @ k
                dk[b, :n, h] += dw.T @ q
                dv[b, :n, h] += (weight * (q @ k.T)).T @ do
                if case["state"]:
                    dq[b, :n, hq] += rise * (do @ s0.T)
                    end[b, h] += (rise * q).T @ do
    state = end if case["state"] else None
    return (dq, dk, dv, state) if bwd else (o, state)


def _exact_decode(case, s):
    G, state = case["Hq"] // case["Hkv"], s["recurrent"].double()
    o = torch.zeros(case["B"], case["Hq"], case["D"], dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        at = b if s["slots"] is None else int(s["slots"][b])
        if at < 0:
            continue
        for h in range(case["Hkv"]):
            state[at, h] = math.exp(float(s["log_decay"][h])) * state[at, h] + torch.outer(s["k"][b, h].double(), s["v"][b, h].double())
            o[b, h * G:(h + 1) * G] = s["scale"] * (s["q"][b, h * G:(h + 1) * G].double() @ state[at, h])
    return o, state


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("qk"):
        return _exact_qk(case, s)
    return _exact_decode(case, s) if case["op"] == "lin_attn_decode" else _exact_lin(case, s)
