"""Measured cases of the decode-layer operators: rotation with the append to a paged key-value
cache, attention of one new token over that cache, and the residual step with its norms.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` makes
one pass through the operator, `work` counts what the pass has to read, write and compute, and
`exact` computes the same outputs in 64 bits. With `own` false `run` computes the plain form in
elementary torch operations; with `own` true it makes the calls of the library's binding.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
_ELEM = {"bf16": 2, "e4m3": 1}
_TYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------- the cases

def _append(name, n_seq, per_seq, pad, heads, kv_heads, head_dim, rot, inter, cache, page, hnd,
            start):
    return {"name": name, "op": "append", "n_seq": n_seq, "per_seq": per_seq, "pad": pad,
            "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rot": rot,
            "inter": inter, "cache": cache, "page": page, "hnd": hnd, "start": start}


def _attn(name, n_seq, ctx, ragged, heads, kv_heads, head_dim, cache, page, hnd, window, softcap):
    return {"name": name, "op": "attention", "n_seq": n_seq, "ctx": ctx, "ragged": ragged,
            "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "cache": cache,
            "page": page, "hnd": hnd, "window": window, "softcap": softcap}


def _norm(name, rows, d, kind, wtype, post, gate, scaled):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "kind": kind, "wtype": wtype,
            "post": post, "gate": gate, "scaled": scaled}


def listed():
    return [
        # one decoded token of a 32-head, 128-wide block (4096): the batch-one step
        _append("append_token_mha", 1, 1, 0, 32, 32, 128, 128, False, "bf16", 16, False, 1000),
        # a serving batch: one token of each of 96 sequences far into their contexts, 8-bit cache
        _append("append_batch_e4m3", 96, 1, 0, 64, 8, 128, 128, False, "e4m3", 64, True, 100003),
        # odd widths: part of each head rotated, interleaved pairs, padded rows behind the batch
        _append("append_partial_odd", 7, 73, 6, 12, 3, 80, 32, True, "bf16", 24, False, 11),
        # the prompts of five sequences, 8000 tokens in all, written at once
        _append("append_prompts", 5, 1600, 0, 32, 8, 128, 128, False, "bf16", 16, False, 0),

        # batch one, a short context, one key head for each query head
        _attn("attn_token_mha", 1, 517, False, 32, 32, 128, "bf16", 16, False, 0, 0.0),
        # batch one, a very long context, four query heads on each key head
        _attn("attn_token_long", 1, 131071, False, 32, 8, 128, "bf16", 16, False, 0, 0.0),
        # a serving batch of unlike lengths, from empty to 8192
        _attn("attn_batch_ragged", 64, 8192, True, 32, 8, 128, "bf16", 16, False, 0, 0.0),
        # an 8-bit cache, eight query heads on each key head, heads before tokens in a page
        _attn("attn_batch_e4m3", 33, 4099, False, 64, 8, 128, "e4m3", 64, True, 0, 0.0),
        # wide heads with a sliding window and capped scores, pages of an odd size
        _attn("attn_window_cap", 48, 9001, True, 16, 2, 256, "bf16", 21, False, 2048, 50.0),

        # batch one: the residual sum and the next norm between two projections of a 4096 block
        _norm("norm_token", 1, 4096, "rms", "bf16", False, "none", False),
        # a serving batch at width 8192 with norms on both sides and a learned gate
        _norm("norm_batch_sandwich", 150, 8192, "rms", "bf16", True, "row", True),
        # prompt rows of an odd width with mean-subtracting norms and a gate for each token
        _norm("norm_prompt_odd", 4001, 5003, "layer", "fp32", True, "token", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "norm"])
    if op == "norm":
        rows = _log(rng, 1, 6000)
        d = _log(rng, 64, min(28672, max(256, 20_000_000 // rows)))
        d = d if rng.random() < 0.3 else max(64, d // 64 * 64)
        c = _norm("", rows, d, rng.choice(["rms", "layer"]), rng.choice(["bf16", "fp32"]),
                  rng.random() < 0.5, rng.choice(["none", "row", "token"]), rng.random() < 0.5)
    else:
        kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
        group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
        while kv_heads * group > 128:
            group = rng.choice([1, 2, 3, 4])
        head_dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        cache = rng.choice(["bf16", "bf16", "e4m3"])
        page = rng.choice([1, 8, 16, 16, 21, 32, 64, 128, 256])
        hnd = rng.random() < 0.4
        if op == "append":
            budget = 8000 * 48 * 128
            most = max(1, min(8000, budget // ((group + 2) * kv_heads * head_dim)))
            n_seq = _log(rng, 1, min(200, most))
            per_seq = _log(rng, 1, max(1, most // n_seq))
            rot = rng.choice([head_dim, head_dim, head_dim // 2, 0])
            c = _append("", n_seq, per_seq, rng.choice([0, 0, 1, 9]), kv_heads * group, kv_heads,
                        head_dim, rot, rng.random() < 0.4, cache, page, hnd,
                        _log(rng, 1, 100000) - 1)
        else:
            n_seq = _log(rng, 1, 128)
            row = 2 * kv_heads * head_dim * _ELEM[cache]
            tokens = 500_000_000 // row
            ctx = _log(rng, 1, max(2, min(131072, tokens // n_seq)))
            window = rng.choice([0, 0, 0, 1, 127, 1024, 4096])
            c = _attn("", n_seq, ctx, rng.random() < 0.6, kv_heads * group, kv_heads, head_dim,
                      cache, page, hnd, window, rng.choice([0.0, 0.0, 0.0, 30.0]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ the inputs

def _lengths(c):
    """The cached tokens of each sequence, in no particular order: all alike, or spread over
    [0, ctx] with an empty one (when there is more than one sequence)."""
    n, ctx = c["n_seq"], c["ctx"]
    if not c["ragged"] or n == 1:
        return [ctx] * n
    return [int(round(ctx * (i / (n - 1)) ** 2)) for i in range(n)]


def _seen(c, n):
    return min(n, c["window"]) if c["window"] > 0 else n


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _make_cache(c, n_pages, g):
    """Key and value pools as [page][token][head][dim] views, heads or tokens outermost in a page."""
    shape = ((n_pages, c["kv_heads"], c["page"], c["head_dim"]) if c["hnd"]
             else (n_pages, c["page"], c["kv_heads"], c["head_dim"]))
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).to(_TYPE[c["cache"]])
        out.append(t.transpose(1, 2) if c["hnd"] else t)
    return out


def _scales(c):
    """Per-cache scales of the 8-bit type; 1 for bf16."""
    return (0.02, 0.015) if c["cache"] == "e4m3" else (1.0, 1.0)


def _freq(c):
    """Rotation frequencies of the pairs, base 500000."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV)
    return 500000.0 ** (-i / max(1, c["rot"]))


def _prepare_append(c, seed):
    g = _gen(seed)
    n_seq, per = c["n_seq"], c["per_seq"]
    n_tok = n_seq * per + c["pad"]
    max_pages = -(-(c["start"] % (4 * c["page"]) + per) // c["page"])
    # the pool holds the pages that the call reaches; earlier pages of a sequence are elsewhere
    first = (c["start"] // (4 * c["page"])) * 4  # pages before these are not in this pool
    n_pages = n_seq * max_pages + 3
    k, v = _make_cache(c, n_pages, g)
    perm = torch.randperm(n_pages, generator=g, device=DEV)[: n_seq * max_pages]
    table = torch.zeros(n_seq, first + max_pages, dtype=torch.int32, device=DEV)
    table[:, first:] = perm.reshape(n_seq, max_pages).to(torch.int32)
    seq = torch.arange(n_seq, device=DEV, dtype=torch.int32).repeat_interleave(per)
    pos = torch.arange(per, device=DEV, dtype=torch.int32).repeat(n_seq) + c["start"]
    pad = torch.full((c["pad"],), -1, dtype=torch.int32, device=DEV)
    H, K, D = c["heads"], c["kv_heads"], c["head_dim"]
    # one row of q, k and v for each token, as one projection writes them
    qkv = torch.randn(n_tok, (H + 2 * K) * D, generator=g, device=DEV)
    s = {"c": c, "k": k, "v": v, "table": table, "seq": torch.cat([seq, pad]),
         "pos": torch.cat([pos, pad]), "qkv": qkv, "freq": _freq(c),
         "q": qkv[:, : H * D].view(n_tok, H, D),
         "kn": qkv[:, H * D: (H + K) * D].view(n_tok, K, D),
         "vn": qkv[:, (H + K) * D:].view(n_tok, K, D),
         "q_out": torch.zeros(n_tok, H, D, device=DEV),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if own:
        from tiered_weight_gemv_b200 import spax

        ks, vs = _scales(c)
        s["cache"] = spax.KvCache(k, v, k_scale=ks, v_scale=vs)
        s["rope"] = spax.Rope(s["freq"], interleaved=c["inter"]) if c["rot"] else None
    return s


def _prepare_attention(c, seed):
    g = _gen(seed)
    lens = _lengths(c)
    n_seq, page = c["n_seq"], c["page"]
    max_pages = max(1, -(-c["ctx"] // page))
    used = [-(-n // page) for n in lens]
    n_pages = max(1, sum(used)) + 2
    k, v = _make_cache(c, n_pages, g)
    order = torch.randperm(n_seq, generator=g, device=DEV)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)[order]
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    # each sequence takes the next run of the shuffled pages; entries past its pages stay 0
    used_t = (lens_t.long() + page - 1) // page
    first = torch.cumsum(used_t, 0) - used_t
    j = torch.arange(max_pages, device=DEV)
    at = (first[:, None] + j[None, :]).clamp(max=n_pages - 1)
    table = torch.where(j[None, :] < used_t[:, None], perm[at], torch.zeros_like(perm[at]))
    H, D = c["heads"], c["head_dim"]
    ks, vs = _scales(c)
    q = torch.randn(n_seq, H, D, generator=g, device=DEV) * (1.5 / ks)
    s = {"c": c, "k": k, "v": v, "table": table.contiguous(), "lens": lens_t, "q": q,
         "scale": 1.0 / math.sqrt(D)}
    if own:
        from tiered_weight_gemv_b200 import spax

        s["cache"] = spax.KvCache(k, v, k_scale=ks, v_scale=vs)
        s["out"] = torch.empty(n_seq, H, D, device=DEV)
        s["lse"] = torch.empty(n_seq, H, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["ws"] = spax.alloc_attention_workspace(s["cache"], H)
    return s


def _prepare_norm(c, seed):
    g = _gen(seed)
    n, d = c["rows"], c["d"]
    wt = torch.bfloat16 if c["wtype"] == "bf16" else torch.float32

    def vec(scale, shift):
        return (torch.randn(d, generator=g, device=DEV) * scale + shift).to(wt)

    bias = c["kind"] == "layer"
    s = {"c": c, "h": torch.randn(n, d, generator=g, device=DEV) * 3.0,
         "y": torch.randn(n, d, generator=g, device=DEV),
         "pre_w": vec(0.1, 1.0), "pre_b": vec(0.1, 0.0) if bias else None,
         "post_w": vec(0.1, 1.0) if c["post"] else None,
         "post_b": vec(0.1, 0.0) if c["post"] and bias else None,
         "gate": {"none": None, "row": torch.randn(d, generator=g, device=DEV),
                  "token": torch.randn(n, d, generator=g, device=DEV)}[c["gate"]],
         "res_scale": 0.75 if c["scaled"] else 1.0, "out_scale": 0.5 if c["scaled"] else 1.0}
    if own:
        from tiered_weight_gemv_b200 import spax

        kind = spax.NORM_RMS if c["kind"] == "rms" else spax.NORM_LAYER
        s["pre"] = spax.Norm(s["pre_w"], s["pre_b"], eps=1e-5, kind=kind)
        s["post"] = spax.Norm(s["post_w"], s["post_b"], eps=1e-5, kind=kind) if c["post"] else None
        s["r"] = torch.empty(n, d, device=DEV)
        s["x"] = torch.empty(n, d, device=DEV)
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "attention": _prepare_attention,
            "norm": _prepare_norm}[case["op"]](case, seed)


# ---------------------------------------------------------------------------- one pass, plain form

def _rotate(x, cos, sin, c):
    """The pairs of the first `rot` entries of each head turned by their angles."""
    rot = c["rot"]
    if rot == 0:
        return x
    if c["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _store(pool, at, off, val, scale):
    val = val if pool.dtype == torch.bfloat16 else (val / scale).clamp(-_E4M3_MAX, _E4M3_MAX)
    val = val.to(pool.dtype)
    if pool.dtype != torch.bfloat16:  # indexed writes take bytes
        pool, val = pool.view(torch.uint8), val.view(torch.uint8)
    pool[at, off] = val


def _plain_append(s):
    c = s["c"]
    live = s["pos"] >= 0
    pos, seq = s["pos"][live].long(), s["seq"][live].long()
    angle = pos.double()[:, None] * s["freq"][None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    at = s["table"][seq, pos // c["page"]].long()
    off = pos % c["page"]
    ks, vs = _scales(c)
    s["q_out"][live] = _rotate(s["q"][live], cos, sin, c)
    _store(s["k"], at, off, _rotate(s["kn"][live], cos, sin, c), ks)
    _store(s["v"], at, off, s["vn"][live], vs)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_attention(s):
    c = s["c"]
    n, H, K, D, page = c["n_seq"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    ks, vs = _scales(c)
    table = s["table"].long()
    L = table.shape[1] * page
    lens = s["lens"].long()

    def gather(pool, scale):  # [n, K, L, D] in 32 bits
        if pool.dtype == torch.bfloat16:
            rows = pool[table]
        else:
            rows = pool.view(torch.uint8)[table].view(pool.dtype)
        return rows.reshape(n, L, K, D).transpose(1, 2).float() * scale

    q = s["q"].view(n, K, H // K, D)
    score = torch.matmul(q, gather(s["k"], ks).transpose(2, 3)) * s["scale"]  # [n, K, G, L]
    if c["softcap"] > 0:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    j = torch.arange(L, device=DEV)
    seen = j[None, :] < lens[:, None]
    if c["window"] > 0:
        seen &= j[None, :] >= (lens - c["window"])[:, None]
    seen = seen[:, None, None, :]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)  # an empty row: every exponential is 0
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, gather(s["v"], vs)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + total.log(), torch.full_like(top, -math.inf))
    return {"out": out.reshape(n, H, D), "lse": lse.reshape(n, H)}


def _plain_normed(z, w, b, kind):
    if kind == "layer":
        z = z - z.mean(-1, keepdim=True)
    z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + 1e-5)
    z = z if w is None else z * w.float()
    return z if b is None else z + b.float()


def _plain_norm(s):
    c = s["c"]
    y = _plain_normed(s["y"], s["post_w"], s["post_b"], c["kind"]) if c["post"] else s["y"]
    y = y if s["gate"] is None else y * s["gate"]
    r = s["res_scale"] * s["h"] + s["out_scale"] * y
    return {"r": r, "x": _plain_normed(r, s["pre_w"], s["pre_b"], c["kind"])}


# ------------------------------------------------------------------------ one pass, the library's

def _own_append(s):
    from tiered_weight_gemv_b200 import spax

    spax.spax_kv_append(s["cache"], s["q"], s["kn"], s["vn"], s["pos"], s["table"], s["status"],
                        rope=s["rope"], seq=s["seq"], q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_attention(s):
    from tiered_weight_gemv_b200 import spax

    c = s["c"]
    spax.spax_paged_attention(s["cache"], s["q"], s["table"], s["lens"], s["out"], s["status"],
                              s["ws"], scale=s["scale"], window=c["window"],
                              softcap=c["softcap"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_norm(s):
    from tiered_weight_gemv_b200 import spax

    spax.spax_residual_norm(s["h"], s["y"], s["r"], s["x"], pre=s["pre"], post=s["post"],
                            gate=s["gate"], res_scale=s["res_scale"], out_scale=s["out_scale"])
    return {"r": s["r"], "x": s["x"]}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "norm": _own_norm}[op](state)
    return {"append": _plain_append, "attention": _plain_attention, "norm": _plain_norm}[op](state)


# -------------------------------------------------------------------------------- the work of a pass

def work(case):
    c = case
    if c["op"] == "append":
        n = c["n_seq"] * c["per_seq"]
        H, K, D = c["heads"], c["kv_heads"], c["head_dim"]
        read = n * (H + 2 * K) * D * 4 + n * 12 + 4 * c["rot"]
        write = n * H * D * 4 + n * 2 * K * D * _ELEM[c["cache"]]
        return {"bytes": read + write, "flops": n * 3 * (H + K) * c["rot"]}
    if c["op"] == "attention":
        H, K, D = c["heads"], c["kv_heads"], c["head_dim"]
        tokens = sum(_seen(c, n) for n in _lengths(c))
        pages = sum(-(-_seen(c, n) // c["page"]) for n in _lengths(c))
        kv = tokens * 2 * K * D * _ELEM[c["cache"]]
        return {"bytes": kv + c["n_seq"] * (2 * H * D * 4 + H * 4 + 4) + pages * 4,
                "flops": tokens * 4 * H * D}
    n, d = c["rows"], c["d"]
    wb = 2 if c["wtype"] == "bf16" else 4
    vectors = (1 + (c["kind"] == "layer")) * (1 + c["post"]) * d * wb
    gate = {"none": 0, "row": 4 * d, "token": 4 * n * d}[c["gate"]]
    return {"bytes": 16 * n * d + vectors + gate, "flops": n * d * (8 + 6 * c["post"])}


# -------------------------------------------------------------------------- the definition, 64 bits

def _exact_append(c, s):
    """q and k as complex numbers times e^(i pos freq), token by token in 64 bits; the pools with
    the new rows before their rounding, everything else as it was."""
    D, rot = c["head_dim"], c["rot"]
    pos, seq = s["pos"].double(), s["seq"].long()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                       pos[:, None] * s["freq"][None, :])[:, None, :]

    def turned(x):
        x = x.double().clone()
        if rot:
            ia = torch.arange(rot // 2, device=DEV) * (2 if c["inter"] else 1)
            ib = ia + (1 if c["inter"] else rot // 2)
            z = torch.complex(x[..., ia], x[..., ib]) * turn
            x[..., ia], x[..., ib] = z.real.clone(), z.imag.clone()
        return x

    q = turned(s["q"])
    q[s["pos"] < 0] = 0.0
    pools = []
    for pool, x, scale in ((s["k"], turned(s["kn"]), _scales(c)[0]),
                           (s["v"], s["vn"].double(), _scales(c)[1])):
        wide = pool.double().reshape(-1, c["kv_heads"], D)
        slot = (s["table"].long()[seq, s["pos"].long().clamp(min=0) // c["page"]] * c["page"]
                + s["pos"].long() % c["page"])
        live = s["pos"] >= 0
        if c["cache"] == "e4m3":
            x = (x / scale).clamp(-_E4M3_MAX, _E4M3_MAX)
        wide.index_copy_(0, slot[live], x[live])
        pools.append(wide.reshape(pool.shape))
    return {"q": q, "k": pools[0], "v": pools[1]}


def _exact_attention(c, s):
    """One sequence at a time: the tokens that it sees, their scores, a softmax and the mean."""
    ks, vs = _scales(c)
    K, D, page = c["kv_heads"], c["head_dim"], c["page"]
    G = c["heads"] // K
    out = torch.zeros(c["n_seq"], c["heads"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((c["n_seq"], c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] > 0 else 0
        if n == 0:
            continue
        t = torch.arange(lo, n, device=DEV)
        at, off = s["table"][i].long()[t // page], t % page
        raw = ((lambda p: p[at, off]) if c["cache"] == "bf16" else
               (lambda p: p.view(torch.uint8)[at, off].view(p.dtype)))
        key, val = raw(s["k"]).double() * ks, raw(s["v"]).double() * vs  # [t, K, D]
        q = s["q"][i].double().view(K, G, D)
        score = torch.einsum("kgd,tkd->kgt", q, key) * s["scale"]
        if c["softcap"] > 0:
            score = c["softcap"] * torch.tanh(score / c["softcap"])
        out[i] = torch.einsum("kgt,tkd->kgd", torch.softmax(score, -1), val).reshape(-1, D)
        lse[i] = torch.logsumexp(score, -1).reshape(-1)
    return {"out": out, "lse": lse}


def _exact_norm(c, s):
    def normed(z, w, b):
        if c["kind"] == "layer":
            var, mean = torch.var_mean(z, -1, unbiased=False, keepdim=True)
            z = (z - mean) * torch.rsqrt(var + 1e-5)
        else:
            z = z * torch.rsqrt((z * z).sum(-1, keepdim=True) / z.shape[-1] + 1e-5)
        z = z * w.double()
        return z if b is None else z + b.double()

    y = s["y"].double()
    if c["post"]:
        y = normed(y, s["post_w"], s["post_b"])
    if s["gate"] is not None:
        y = y * s["gate"].double()
    r = s["h"].double() * s["res_scale"] + y * s["out_scale"]
    return {"r": r, "x": normed(r, s["pre_w"], s["pre_b"])}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention,
            "norm": _exact_norm}[case["op"]](case, s)
