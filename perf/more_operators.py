"""Softmax attention over a sliding window with a few first tokens that stay
visible (forward and backward), and what serves it: keys and values written
into a paged cache, attention of one new token over that cache, and the
eviction of the tokens that got the least attention.

A case names the operator and its sizes.  ``run`` makes one pass, in the plain
form (elementary torch operations in 32 bits) or, where ``own`` is set,
through the framework's entry points.  ``exact`` evaluates the definitions in
64 bits.

Layouts: q [B][T][Hq][D], k, v [B][T][Hkv][D]; query head h reads KV head
h / (Hq / Hkv); pages [n_pages][page_size][Hkv][D]; block_table [B][max_pages]
int32 (position p of a sequence stands in row p % page_size of page
block_table[b][p / page_size]; an entry that is no page's number is an absent
page); weight sums [B][Hkv][max_pages * page_size] fp32.
"""
import math

import torch

own = False

_BF, _F = torch.bfloat16, torch.float32


# --------------------------------------------------------------------- cases
def _win(name, op, B, T, Hq, Hkv, D, window, sinks, padded=False, packed=False):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "window": window, "sinks": sinks,
            "padded": padded, "packed": packed}


def _dec(name, B, tokens, Hq, Hkv, D, page, window=0, sinks=0, weights=False, ragged=False, dtype="bf16"):
    return {"name": name, "op": "attn_decode_paged", "B": B, "tokens": tokens, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "window": window, "sinks": sinks, "weights": weights, "ragged": ragged, "dtype": dtype}


def _write(name, B, T, Hkv, D, page, start, ragged=False):
    return {"name": name, "op": "kv_pages_write", "B": B, "T": T, "Hkv": Hkv, "D": D, "page": page, "start": start,
            "ragged": ragged}


def _evict(name, B, tokens, Hkv, D, page, budget, sinks, recent, ragged=False):
    return {"name": name, "op": "kv_pages_evict", "B": B, "tokens": tokens, "Hkv": Hkv, "D": D, "page": page,
            "budget": budget, "sinks": sinks, "recent": recent, "ragged": ragged}


def listed():
    return [
        # one layer of the 30-layer chain with shared KV heads: latency counts
        _win("win_fwd_layer", "attn_fwd_window", 2, 512, 20, 5, 128, 128, 4),
        # a long prompt, T = 8192
        _win("win_fwd_long", "attn_fwd_window", 1, 8192, 32, 32, 128, 1024, 4),
        # a short ragged batch of prompts, padded on the right, small heads, out of a packed projection
        _win("win_fwd_padded", "attn_fwd_window", 3, 777, 16, 4, 64, 200, 0, padded=True, packed=True),
        # one layer of the chain, backward
        _win("win_bwd_layer", "attn_bwd_window", 2, 512, 20, 5, 128, 128, 4),
        # a training step's backward, T = 2048
        _win("win_bwd_train", "attn_bwd_window", 4, 2048, 20, 20, 128, 512, 4),
        # one sequence: latency
        _dec("decode_one", 1, 1000, 20, 5, 128, 16),
        # a decode step of 64 sequences of different lengths, 20/5 heads, some rows of the batch empty
        _dec("decode_batch", 64, 1024, 20, 5, 128, 16, ragged=True),
        # long caches, whose attention weights are summed for the eviction
        _dec("decode_long_weights", 8, 32768, 32, 8, 128, 64, weights=True, ragged=True),
        # the new token of each of 64 sequences
        _write("write_step", 64, 1, 5, 128, 16, 1000),
        # a batch of prompts
        _write("write_prompt", 4, 2048, 20, 128, 16, 0, ragged=True),
        # one sequence that outgrew its budget
        _evict("evict_one", 1, 1025, 5, 128, 16, 512, 4, 128),
        # a batch of long ones
        _evict("evict_batch", 16, 8192, 8, 128, 64, 2048, 4, 256, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_fwd_window", "attn_bwd_window", "attn_decode_paged", "attn_decode_paged", "kv_pages_write",
                     "kv_pages_evict"])
    Hkv, D = rng.choice([1, 2, 4, 5, 8, 20]), rng.choice([64, 128])
    G = min(rng.choice([1, 1, 2, 4, 8]), max(1, 32 // Hkv))
    page = rng.choice([1, 16, 16, 24, 32, 64, 128])
    if op.endswith("window"):
        Hq = Hkv * G
        T = _log_int(rng, 1, 8192 if op == "attn_fwd_window" else 4096)
        most = 32 * 8192 * 8192 * 128 if op == "attn_fwd_window" else 80 * 2048 * 2048 * 128
        if T * T * Hq * D > most:
            T = int(math.isqrt(most // (Hq * D)))
        B = _log_int(rng, 1, max(1, min(16, most // (T * T * Hq * D))))
        window = _log_int(rng, 1, 1024 if op == "attn_fwd_window" else 512)
        while B > 1 and B * T * min(T, window) * Hq * D > most // 8:
            B -= 1
        case = _win("", op, B, T, Hq, Hkv, D, window, rng.choice([0, 1, 4, 4, 16, 130]),
                    padded=B > 1 and rng.random() < 0.4, packed=rng.random() < 0.3)
    elif op == "attn_decode_paged":
        tokens = _log_int(rng, 1, 65536)
        B = _log_int(rng, 1, max(1, min(128, 8 * 16384 * 8 * 128 // (tokens * Hkv * D))))
        window = _log_int(rng, 1, tokens) if rng.random() < 0.3 else 0
        case = _dec("", B, tokens, Hkv * min(rng.choice([1, 3, 4, 4, 8, 16]), max(1, 64 // Hkv)), Hkv, D, page, window=window,
                    sinks=rng.choice([0, 4, 20]) if window else 0, weights=rng.random() < 0.4,
                    ragged=B > 1 and rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "f32"]))
    elif op == "kv_pages_write":
        T = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(128, 4 * 2048 * 20 * 128 // (T * Hkv * D))))
        case = _write("", B, T, Hkv, D, page, rng.choice([0, 0, 17, 1000]), ragged=B > 1 and rng.random() < 0.5)
    else:
        tokens = _log_int(rng, 16, 16384)
        budget = _log_int(rng, 8, max(8, min(4096, tokens)))
        B = _log_int(rng, 1, max(1, min(32, 16 * 2048 * 8 * 128 // (tokens * Hkv * D))))
        sinks = min(rng.choice([0, 4, 16]), budget // 2)
        case = _evict("", B, tokens, Hkv, D, page, budget, sinks, _log_int(rng, 1, budget - sinks),
                      ragged=B > 1 and rng.random() < 0.5)
    del case["name"]
    return case


# -------------------------------------------------------------------- inputs
def _lengths(count, most, ragged):
    """Tokens of each sequence: all, or spread between half and all of them,
    with the second sequence empty."""
    if not ragged:
        return [most] * count
    n = [most - (b * 7919) % (most // 2 + 1) for b in range(count)]
    n[1] = 0
    return n


def _pages(tokens, page):
    return (tokens + page - 1) // page


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, dtype=_F):
        return torch.randn(*shape, generator=g, device="cuda", dtype=_F).to(dtype)

    def int32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    s = dict(case)
    B, Hkv, D, op = case["B"], case["Hkv"], case["D"], case["op"]
    s["scale"] = 1.0 / math.sqrt(D)
    if op.endswith("window"):
        T, Hq = case["T"], case["Hq"]
        if case["packed"]:                                   # parts of the projection's packed output
            qkv = normal(B, T, Hq + 2 * Hkv, D, dtype=_BF)
            s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:])
        else:
            s.update(q=normal(B, T, Hq, D, dtype=_BF), k=normal(B, T, Hkv, D, dtype=_BF), v=normal(B, T, Hkv, D, dtype=_BF))
        s["lengths"] = int32(_lengths(B, T, True)) if case["padded"] else None
        if op == "attn_bwd_window":                          # what the forward left, and the gradient that comes back
            o, lse = _plain_win_fwd(s)
            s.update(o=o, lse=lse, dout=normal(B, T, Hq, D, dtype=_BF))
        return s
    page = case["page"]
    if op == "kv_pages_write":
        T = case["T"]
        each = _pages(case["start"] + T, page)
        n = B * each + 3
        kv = normal(B, T, 2 * Hkv, D, dtype=_BF)
        s.update(k=kv[:, :, :Hkv], v=kv[:, :, Hkv:], starts=int32([case["start"]] * B),
                 lengths=int32(_lengths(B, T, True)) if case["ragged"] else None)
    else:
        each = _pages(case["tokens"], page)
        n = B * each + 3
        if op == "kv_pages_evict":
            fresh = _pages(case["budget"], page)
            n += B * fresh
        s["lengths"] = int32(_lengths(B, case["tokens"], case["ragged"]))
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    s["block_table"] = order[:B * each].reshape(B, each).contiguous()
    if op == "kv_pages_write":
        s["k_pages"] = torch.zeros(n, page, Hkv, D, dtype=_BF, device="cuda")
        s["v_pages"] = torch.zeros(n, page, Hkv, D, dtype=_BF, device="cuda")
        return s
    s["k_pages"], s["v_pages"] = normal(n, page, Hkv, D, dtype=_BF), normal(n, page, Hkv, D, dtype=_BF)
    first = torch.arange(each, device="cuda") * page         # a page behind the last token has not been taken yet
    unused = first[None, :] >= s["lengths"][:, None]
    if op == "attn_decode_paged":
        if case["window"]:                                   # and one that the window has left was given back
            unused |= (first + page <= s["lengths"][:, None] - case["window"]) & (first >= case["sinks"])[None, :]
        s["q"] = normal(B, case["Hq"], D, dtype=_BF if case["dtype"] == "bf16" else _F)
    else:
        s["new_table"] = order[B * each:B * (each + fresh)].reshape(B, fresh).contiguous()
    s["block_table"] = torch.where(unused, torch.full_like(s["block_table"], -1), s["block_table"])
    s["weight_sums"] = None
    if op == "kv_pages_evict" or case["weights"]:            # a few tokens hold most of the weight
        s["weight_sums"] = torch.exp(2.0 * normal(B, Hkv, each * page) - 4.0)
    return s


# --------------------------------------------------- the framework's own calls
def _own(s):
    import transformer_attention_backward_gb300 as abw
    op = s["op"]
    if op == "attn_fwd_window":
        return abw.attn_fwd_window(s["q"], s["k"], s["v"], s["window"], s["sinks"], s["scale"], lengths=s["lengths"])
    if op == "attn_bwd_window":
        return abw.attn_bwd_window(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["window"], s["sinks"],
                                   s["scale"], lengths=s["lengths"])
    if op == "attn_decode_paged":
        o = abw.attn_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["lengths"], s["scale"],
                                  window=s["window"] or None, sinks=s["sinks"], weight_sums=s["weight_sums"])
        return (o, s["weight_sums"]) if s["weights"] else (o,)
    if op == "kv_pages_write":
        abw.kv_pages_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["starts"], lengths=s["lengths"])
        return s["k_pages"], s["v_pages"]
    kept, n, sums = abw.kv_pages_evict(s["k_pages"], s["v_pages"], s["block_table"], s["lengths"], s["weight_sums"],
                                       s["budget"], s["new_table"], sinks=s["sinks"], recent=s["recent"])
    return s["k_pages"], s["v_pages"], kept, n, sums


# -------------------------------------------------------------- the plain form
def _visible(T, s):
    """[query][key]: key <= query, and inside the window or among the first."""
    i = torch.arange(T, device="cuda")
    gap = i[:, None] - i[None, :]
    return (gap >= 0) & ((gap < s["window"]) | (i < s["sinks"])[None, :])


def _win_parts(s):
    """The parts (sequence, KV head) of a batch, with q [G][n][D], k, v [n][D]
    of the sequence's tokens in 32 bits."""
    G = s["Hq"] // s["Hkv"]
    for b in range(s["B"]):
        n = s["T"] if s["lengths"] is None else _lengths(s["B"], s["T"], True)[b]
        for h in range(s["Hkv"]):
            at = (b, slice(0, n), slice(h * G, h * G + G))
            yield at, (b, slice(0, n), h), n, s["q"][at].float().transpose(0, 1), s["k"][b, :n, h].float(), s["v"][b, :n, h].float()


def _plain_win_fwd(s):
    o = torch.zeros(s["B"], s["T"], s["Hq"], s["D"], dtype=_BF, device="cuda")
    lse = torch.full((s["B"], s["Hq"], s["T"]), -math.inf, device="cuda")
    seen = _visible(s["T"], s)
    for at, _, n, q, k, v in _win_parts(s):
        if n == 0:
            continue
        score = (q @ k.T * s["scale"]).masked_fill(~seen[:n, :n], -math.inf)
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        o[at] = ((p @ v) / total).transpose(0, 1).to(_BF)
        lse[at[0], at[2], :n] = (top + torch.log(total))[..., 0]
    return o, lse


def _plain_win_bwd(s):
    dq = torch.zeros(s["B"], s["T"], s["Hq"], s["D"], dtype=_BF, device="cuda")
    dk = torch.zeros(s["B"], s["T"], s["Hkv"], s["D"], dtype=_BF, device="cuda")
    dv = torch.zeros_like(dk)
    seen = _visible(s["T"], s)
    for at, kv, n, q, k, v in _win_parts(s):
        if n == 0:
            continue
        o, do = s["o"][at].float().transpose(0, 1), s["dout"][at].float().transpose(0, 1)
        p = torch.exp(q @ k.T * s["scale"] - s["lse"][at[0], at[2], :n, None]) * seen[:n, :n]
        ds = p * (do @ v.T - (do * o).sum(-1, keepdim=True)) * s["scale"]
        dq[at] = (ds @ k).transpose(0, 1).to(_BF)
        dk[kv] = torch.einsum("gij,gid->jd", ds, q).to(_BF)
        dv[kv] = torch.einsum("gij,gid->jd", p, do).to(_BF)
    return dq, dk, dv


def _places(s):
    """Page and row of every position of every sequence, and whether a page
    stands there: [B][positions] each."""
    table, page = s["block_table"], s["page"]
    at = torch.arange(table.shape[1] * page, device="cuda")
    where = table[:, at // page].long()
    present = (where >= 0) & (where < s["k_pages"].shape[0])
    return torch.where(present, where, torch.zeros_like(where)), at % page, present, at


def _plain_decode(s):
    where, row, present, at = _places(s)
    n = s["lengths"][:, None]
    seen = present & (at < n)
    if s["window"]:
        seen &= (at >= n - s["window"]) | (at < s["sinks"])
    B, Hkv, D = s["B"], s["Hkv"], s["D"]
    o = torch.zeros(B, s["Hq"], D, device="cuda")
    for b in range(B):
        k, v = s["k_pages"][where[b], row].float(), s["v_pages"][where[b], row].float()
        q = s["q"][b].float().reshape(Hkv, -1, D)
        score = torch.einsum("hgd,jhd->hgj", q, k) * s["scale"]
        score = torch.where(seen[b], score, torch.full((), -math.inf, device="cuda"))
        top = score.amax(-1, keepdim=True)
        p = torch.where(seen[b], torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top))), torch.zeros_like(score))
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, torch.zeros_like(p))
        o[b] = torch.einsum("hgj,jhd->hgd", p, torch.where(seen[b, :, None, None], v, torch.zeros_like(v))).reshape(-1, D)
        if s["weights"]:
            s["weight_sums"][b] += p.sum(1)
    return (o.to(s["q"].dtype), s["weight_sums"]) if s["weights"] else (o.to(s["q"].dtype),)


def _plain_write(s):
    B, T, page = s["B"], s["T"], s["page"]
    t = torch.arange(T, device="cuda")
    pos = s["starts"].long()[:, None] + t
    live = torch.ones(B, T, dtype=torch.bool, device="cuda") if s["lengths"] is None else t[None, :] < s["lengths"][:, None]
    b, t = torch.nonzero(live, as_tuple=True)
    p = pos[b, t]
    where = s["block_table"][b, p // page].long()
    s["k_pages"][where, p % page] = s["k"][b, t]
    s["v_pages"][where, p % page] = s["v"][b, t]
    return s["k_pages"], s["v_pages"]


def _plain_evict(s):
    where, row, present, at = _places(s)
    n, budget, page, H = s["lengths"][:, None], s["budget"], s["page"], s["Hkv"]
    live = present & (at < n)
    held = live & ((at < s["sinks"]) | (at >= n - s["recent"]))
    kind = live.int() + held.int()
    w = torch.where(s["weight_sums"].isnan(), torch.full((), -math.inf, device="cuda"), s["weight_sums"])
    by_weight = torch.sort(w, dim=-1, descending=True, stable=True).indices
    kinds = torch.gather(kind[:, None, :].expand_as(by_weight), 2, by_weight)
    order = torch.gather(by_weight, 2, torch.sort(kinds, dim=-1, descending=True, stable=True).indices)
    total = torch.clamp(live.sum(-1), max=budget)
    first = torch.arange(budget, device="cuda")
    pad = budget - min(budget, order.shape[-1])
    order = torch.nn.functional.pad(order[..., :budget], (0, pad), value=at.shape[0])
    kept = torch.where(first < total[:, None, None], order, torch.full_like(order, at.shape[0]))
    kept = torch.sort(kept, dim=-1).values
    there = first < total[:, None, None]
    src = torch.where(there, kept, torch.zeros_like(kept))
    sums = torch.zeros(s["B"], H, s["new_table"].shape[1] * page, device="cuda")
    sums[..., :budget] = torch.where(there, torch.gather(s["weight_sums"], 2, src), torch.zeros((), device="cuda"))
    b, h, i = torch.nonzero(there.expand(-1, H, -1), as_tuple=True)
    j = src[b, h, i]
    to = s["new_table"][b, i // page].long()
    for pages in (s["k_pages"], s["v_pages"]):
        pages[to, i % page, h] = pages[where[b, j], row[j], h]
    return s["k_pages"], s["v_pages"], torch.where(there, src, torch.full_like(src, -1)).int(), total.int(), sums


def run(state):
    if own:
        return _own(state)
    return {"attn_fwd_window": _plain_win_fwd, "attn_bwd_window": _plain_win_bwd, "attn_decode_paged": _plain_decode,
            "kv_pages_write": _plain_write, "kv_pages_evict": _plain_evict}[state["op"]](state)


# ------------------------------------------------------------------------ work
def _pairs(n, window, sinks):
    """Visible (query, key) pairs of a sequence of n tokens."""
    full = min(n, window)
    inside = full * (full + 1) // 2 + (n - full) * window
    for j in range(min(sinks, n)):                           # a first token that the window has left
        inside += max(0, n - window - j)
    return inside


def work(case):
    """Inputs read once, outputs written once; the products of the visible
    pairs."""
    B, Hkv, D, op = case["B"], case["Hkv"], case["D"], case["op"]
    if op.endswith("window"):
        T, Hq = case["T"], case["Hq"]
        lens = _lengths(B, T, case["padded"])
        n = sum(lens)
        pairs = Hq * sum(_pairs(x, case["window"], case["sinks"]) for x in lens)
        if op == "attn_fwd_window":
            return {"bytes": 2 * n * (Hq + 2 * Hkv) * D + B * T * Hq * (2 * D + 4), "flops": 4 * D * pairs}
        return {"bytes": 2 * n * (3 * Hq + 2 * Hkv) * D + 4 * n * Hq + 2 * B * T * (Hq + 2 * Hkv) * D, "flops": 10 * D * pairs}
    if op == "kv_pages_write":
        n = sum(_lengths(B, case["T"], case["ragged"]))
        return {"bytes": 8 * n * Hkv * D, "flops": 0}
    lens = _lengths(B, case["tokens"], case["ragged"])
    if op == "attn_decode_paged":
        seen = sum(n if not case["window"] else n - max(0, n - case["window"]) + min(case["sinks"], max(0, n - case["window"]))
                   for n in lens)
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 4 * seen * Hkv * D + 2 * e * B * case["Hq"] * D + (8 * seen * Hkv if case["weights"] else 0),
                "flops": 4 * seen * case["Hq"] * D}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": 4 * sum(lens) * Hkv + kept * Hkv * (8 * D + 4) + 4 * B * Hkv * _pages(case["budget"], case["page"]) * case["page"],
            "flops": 0}


# ----------------------------------------------------- the definitions, 64 bits
def _exact_win(case, s):
    """Blocks of queries, each with the columns that any of them sees."""
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    G, W, S, bwd = Hq // Hkv, case["window"], case["sinks"], case["op"] == "attn_bwd_window"
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(B, T, Hq, D, **f64), torch.full((B, Hq, T), -math.inf, **f64)
    dk, dv = torch.zeros(B, T, Hkv, D, **f64), torch.zeros(B, T, Hkv, D, **f64)
    for b in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][b])
        for t0 in range(0, n, 256):
            t1 = min(n, t0 + 256)
            lo = max(0, t0 - W + 1)
            cols = torch.cat([torch.arange(0, min(S, lo), device="cuda"), torch.arange(lo, t1, device="cuda")])
            rows = torch.arange(t0, t1, device="cuda")
            hidden = (cols[None, :] > rows[:, None]) | ((cols[None, :] <= rows[:, None] - W) & (cols[None, :] >= S))
            for hq in range(Hq):
                h = hq // G
                q, k, v = s["q"][b, t0:t1, hq].double(), s["k"][b, cols, h].double(), s["v"][b, cols, h].double()
                z = torch.matmul(q, k.transpose(0, 1)) * s["scale"]
                z[hidden] = -math.inf
                if not bwd:
                    norm = torch.logsumexp(z, 1)
                    lse[b, hq, t0:t1] = norm
                    out[b, t0:t1, hq] = torch.matmul(torch.exp(z - norm[:, None]), v)
                    continue
                p = torch.exp(z - s["lse"][b, hq, t0:t1, None].double())
                do = s["dout"][b, t0:t1, hq].double()
                delta = torch.einsum("id,id->i", do, s["o"][b, t0:t1, hq].double())
                g = s["scale"] * p * (torch.matmul(do, v.transpose(0, 1)) - delta[:, None])
                out[b, t0:t1, hq] = torch.matmul(g, k)
                dk[b].index_put_((cols, torch.full_like(cols, h)), torch.matmul(g.transpose(0, 1), q), accumulate=True)
                dv[b].index_put_((cols, torch.full_like(cols, h)), torch.matmul(p.transpose(0, 1), do), accumulate=True)
    return (out, dk, dv) if bwd else (out, lse)


def _positions(case, s, b, n):
    """Positions below n of sequence b whose page is there, and the pages."""
    table, total = s["block_table"][b].tolist(), s["k_pages"].shape[0]
    pos, pages = [], []
    for i, entry in enumerate(table):
        if 0 <= entry < total:
            here = range(i * case["page"], min(n, (i + 1) * case["page"]))
            pos.extend(here)
            pages.extend([entry] * len(here))
    return torch.tensor(pos, dtype=torch.long, device="cuda"), torch.tensor(pages, dtype=torch.long, device="cuda")


def _exact_decode(case, s):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    sums = s["weight_sums"].double() if case["weights"] else None
    for b in range(B):
        n = int(s["lengths"][b])
        pos, pages = _positions(case, s, b, n)
        if case["window"]:
            stay = (pos < case["sinks"]) | (pos >= n - case["window"])
            pos, pages = pos[stay], pages[stay]
        if pos.numel() == 0:
            continue
        k, v = (s[x][pages, pos % case["page"]].double() for x in ("k_pages", "v_pages"))
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            p = torch.softmax(torch.mv(k[:, h], s["q"][b, hq].double()) * s["scale"], 0)
            o[b, hq] = torch.mv(v[:, h].transpose(0, 1), p)
            if case["weights"]:
                sums[b, h, pos] += p
    return (o, sums) if case["weights"] else (o,)


def _exact_write(case, s):
    pages = [s["k_pages"].double(), s["v_pages"].double()]
    for b in range(case["B"]):
        start, n = int(s["starts"][b]), case["T"] if s["lengths"] is None else int(s["lengths"][b])
        p = start
        while p < start + n:                                 # page by page
            end = min(start + n, (p // case["page"] + 1) * case["page"])
            at, r = int(s["block_table"][b, p // case["page"]]), p % case["page"]
            for x, y in zip(pages, (s["k"], s["v"])):
                x[at, r:r + end - p] = y[b, p - start:end - start].double()
            p = end
    return tuple(pages)


def _exact_evict(case, s):
    B, H, page, budget = case["B"], case["Hkv"], case["page"], case["budget"]
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    kept = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(B, dtype=torch.int32, device="cuda")
    sums = torch.zeros(B, H, s["new_table"].shape[1] * page, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lengths"][b])
        pos, pages = _positions(case, s, b, n)
        count[b] = m = min(budget, pos.numel())
        if m == 0:
            continue
        to = s["new_table"][b].long().repeat_interleave(page)[:m]
        rows = torch.arange(m, device="cuda") % page
        for h in range(H):
            w = s["weight_sums"][b, h, pos].double()
            w[(pos < case["sinks"]) | (pos >= n - case["recent"])] = math.inf
            pick = torch.argsort(-w, stable=True)[:m].sort().values
            kept[b, h, :m] = pos[pick].int()
            sums[b, h, :m] = s["weight_sums"][b, h, pos[pick]].double()
            for x, y in ((kp, s["k_pages"]), (vp, s["v_pages"])):
                x[to, rows, h] = y[pages[pick], pos[pick] % page, h].double()
    return kp, vp, kept, count, sums


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].endswith("window"):
        return _exact_win(case, s)
    return {"attn_decode_paged": _exact_decode, "kv_pages_write": _exact_write, "kv_pages_evict": _exact_evict}[case["op"]](case, s)
