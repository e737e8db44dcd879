"""The serving step's paged operators, as cases to measure: appending a batch's new keys and values to a paged cache
(with the query/key normalisation and the position rotation on the way), attention of those new tokens over the paged
cache, and sampling the next tokens from the output head's logits.

`run` computes each operator in elementary torch operations, or, with `own` true, through the framework's entry
points. Heads, vocabulary, contexts and batch sizes are those of the framework's own model (32 query and 4 key/value
heads of dimension 128, a vocabulary of 150,144, contexts up to 32,768, calls of up to 8,192 tokens) or generic."""
import math
import random

import torch

own = False

DH = 128
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of each of 64 conversations: the append in front of a batched decode step
        {"name": "append_decode_64", "op": "append", "B": 64, "n_lo": 1, "n_hi": 1, "ctx_lo": 0, "ctx_hi": 700,
         "hq": 32, "hkv": 4, "page": 16, "cache": "bf16", "rope": True, "norm": True, "layout": 1},
        # five prompts filled in one call of about 8,192 tokens
        {"name": "append_prefill_8k", "op": "append", "B": 5, "n_lo": 1500, "n_hi": 1777, "ctx_lo": 0, "ctx_hi": 0,
         "hq": 32, "hkv": 4, "page": 64, "cache": "bf16", "rope": True, "norm": True, "layout": 2},
        # a mixed step (decodes and prompt pieces) into an 8-bit cache
        {"name": "append_mixed_e4m3", "op": "append", "B": 23, "n_lo": 1, "n_hi": 129, "ctx_lo": 0, "ctx_hi": 900,
         "hq": 32, "hkv": 4, "page": 32, "cache": "e4m3", "rope": True, "norm": True, "layout": 3},
        # one conversation's next token over 4K of context: the latency of a single user
        {"name": "attn_decode_1x4k", "op": "attn", "B": 1, "n_lo": 1, "n_hi": 1, "ctx_lo": 4096, "ctx_hi": 4096,
         "hq": 32, "hkv": 4, "page": 16, "cache": "bf16", "window": 0, "layout": 4},
        # a decode step of 64 conversations of all lengths up to 8K
        {"name": "attn_decode_64_ragged", "op": "attn", "B": 64, "n_lo": 1, "n_hi": 1, "ctx_lo": 1, "ctx_hi": 8191,
         "hq": 32, "hkv": 4, "page": 16, "cache": "bf16", "window": 0, "layout": 5},
        # eight long contexts in an 8-bit cache
        {"name": "attn_decode_8x32k_e4m3", "op": "attn", "B": 8, "n_lo": 1, "n_hi": 1, "ctx_lo": 30001,
         "ctx_hi": 32767, "hq": 32, "hkv": 4, "page": 64, "cache": "e4m3", "window": 0, "layout": 6},
        # a step of prompt pieces beside decodes, on a sliding-window layer
        {"name": "attn_mixed_window", "op": "attn", "B": 11, "n_lo": 1, "n_hi": 300, "ctx_lo": 0, "ctx_hi": 6000,
         "hq": 32, "hkv": 4, "page": 32, "cache": "bf16", "window": 1024, "layout": 7},
        # a whole prompt of 8,192 tokens at once
        {"name": "attn_prefill_8k", "op": "attn", "B": 1, "n_lo": 8192, "n_hi": 8192, "ctx_lo": 0, "ctx_hi": 0,
         "hq": 32, "hkv": 4, "page": 64, "cache": "bf16", "window": 0, "layout": 8},
        # the last piece of a long prompt over an 8-bit cache
        {"name": "attn_chunk_1k_over_31k_e4m3", "op": "attn", "B": 1, "n_lo": 1024, "n_hi": 1024, "ctx_lo": 31000,
         "ctx_hi": 31000, "hq": 32, "hkv": 4, "page": 128, "cache": "e4m3", "window": 0, "layout": 9},
        # one user's sampling with the usual filters
        {"name": "sample_1_topk_topp", "op": "sample", "rows": 1, "vocab": 150144, "dtype": "f32", "mode": "topk_topp",
         "layout": 10},
        # eight rows of the head's largest call, no filter: the whole vocabulary counts
        {"name": "sample_8_plain", "op": "sample", "rows": 8, "vocab": 150144, "dtype": "f32", "mode": "plain",
         "layout": 11},
        # a large batch whose users chose different filters
        {"name": "sample_128_mixed", "op": "sample", "rows": 128, "vocab": 150144, "dtype": "f32", "mode": "mixed",
         "layout": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "sample"])
    layout = rng.randrange(1, 1 << 30)
    hq, hkv = rng.choice([(32, 4), (32, 4), (8, 8), (14, 2), (16, 1), (12, 4)])
    page, cache = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "e4m3"])
    if op == "append":
        n_hi = _log_int(rng, 1, 2000)
        B = _log_int(rng, 1, max(1, min(128, 8192 // n_hi)))
        return {"op": op, "B": B, "n_lo": 1, "n_hi": n_hi, "ctx_lo": 0, "ctx_hi": _log_int(rng, 1, 1500), "hq": hq,
                "hkv": hkv, "page": page, "cache": cache, "rope": rng.random() < 0.8, "norm": rng.random() < 0.8,
                "layout": layout}
    if op == "attn":
        window = rng.choice([0, 0, _log_int(rng, 17, 4096)])
        if rng.random() < 0.5:  # decode steps (one to two new tokens)
            B = _log_int(rng, 1, 64)
            return {"op": op, "B": B, "n_lo": 1, "n_hi": rng.choice([1, 1, 2]), "ctx_lo": 0,
                    "ctx_hi": _log_int(rng, 1, min(32768, 262144 // B)), "hq": hq, "hkv": hkv, "page": page,
                    "cache": cache, "window": window, "layout": layout}
        n_hi = _log_int(rng, 3, 2500)
        ctx_hi = _log_int(rng, 1, 16000)
        most = max(1, int(1.5e9 / (hq * n_hi * (n_hi + ctx_hi))))
        return {"op": op, "B": _log_int(rng, 1, min(24, most)), "n_lo": rng.choice([1, max(1, n_hi // 2)]),
                "n_hi": n_hi, "ctx_lo": 0, "ctx_hi": ctx_hi, "hq": hq, "hkv": hkv, "page": page, "cache": cache,
                "window": window, "layout": layout}
    return {"op": op, "rows": _log_int(rng, 1, 128), "vocab": _log_int(rng, 1000, 150144),
            "dtype": rng.choice(["f32", "f32", "bf16"]), "mode": rng.choice(["topk_topp", "plain", "minp", "mixed"]),
            "layout": layout}


def _lengths(case):
    """(new tokens, context before them) of each sequence: the same for every seed of a case."""
    r = random.Random(case["layout"])
    return [(r.randint(case["n_lo"], case["n_hi"]), r.randint(case["ctx_lo"], case["ctx_hi"]))
            for _ in range(case["B"])]


# ------------------------------------------------------------------ inputs
def _pool(case, g, n_pages, gain):
    shape = (n_pages, case["page"], case["hkv"], DH)
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * gain
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if case["cache"] == "bf16":
        return k, v, None, None
    ks = torch.rand(case["hkv"], generator=g, device="cuda") * 0.02 + 0.02
    vs = torch.rand(case["hkv"], generator=g, device="cuda") * 0.02 + 0.01
    to8 = lambda x, s: (x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    return to8(k, ks), to8(v, vs), ks, vs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + int(case["layout"]))
    if case["op"] == "sample":
        return _prepare_sample(case, g)
    lens = _lengths(case)
    B, page, hq, hkv = case["B"], case["page"], case["hq"], case["hkv"]
    n = [a for a, _ in lens]
    kv = [a + c for a, c in lens]
    T = sum(n)
    used = [-(-x // page) for x in kv]
    n_pages = sum(used) + max(2, sum(used) // 16)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(used)), dtype=torch.int32)
    at = torch.arange(max(used))[None, :] < torch.tensor(used)[:, None]
    table[at] = order[:sum(used)].cpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = [0]
    for a in n:
        starts.append(starts[-1] + a)
    k, v, ks, vs = _pool(case, g, n_pages, 1.5)
    s = {"case": dict(case), "T": T, "B": B, "table": table.cuda(), "q_start": i32(starts), "kv_len": i32(kv),
         "k": k, "v": v, "ks": ks, "vs": vs, "n_pages": n_pages, "max_n": max(n), "max_kv": max(kv),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "append":
        s["qkv"] = torch.randn((T, hq + 2 * hkv, DH), generator=g, device="cuda", dtype=torch.bfloat16)
        w = lambda: (torch.rand(DH, generator=g, device="cuda") + 0.5).to(torch.bfloat16)  # noqa: E731
        s["qw"], s["kw"] = (w(), w()) if case["norm"] else (None, None)
        s["max_pos"] = max(kv)
        if case["rope"]:
            inv = THETA ** (-torch.arange(0, DH, 2, dtype=torch.float64, device="cuda") / DH)
            ang = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * inv
            s["cs"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        else:
            s["cs"] = None
        s["q_out"] = torch.zeros((T, hq, DH), dtype=torch.bfloat16, device="cuda")
        return s
    s["q"] = torch.randn((T, hq, DH), generator=g, device="cuda", dtype=torch.bfloat16)
    s["out"] = torch.zeros((T, hq, DH), dtype=torch.bfloat16, device="cuda")
    if own:
        import nvfp4_weight_only_flint_b200 as fm
        nb = fm.flint_paged_attention_workspace_bytes(T, B, hq, hkv, s["max_n"])
        s["ws"] = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
    return s


def _prepare_sample(case, g):
    R, V = case["rows"], case["vocab"]
    # a head's logits: a broad bulk, a few hundred likely tokens above it, some tokens masked away
    x = torch.randn((R, V), generator=g, device="cuda") * 2.0
    likely = torch.randint(0, V, (R, 200), generator=g, device="cuda")
    lift = 8.0 + 5.0 * torch.rand((R, 200), generator=g, device="cuda") ** 3
    x.scatter_add_(1, likely, lift)
    x.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < 0.01, -math.inf)
    x = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    r = random.Random(case["layout"])
    kinds = {"topk_topp": ["topk_topp"], "plain": ["plain"], "minp": ["minp"],
             "mixed": ["topk_topp", "plain", "topk", "topp", "topp_hi", "minp", "greedy", "all"]}[case["mode"]]
    row = {"topk_topp": (0.8, 50, 0.9, 0.0), "plain": (1.0, 0, 1.0, 0.0), "topk": (0.7, 40, 1.0, 0.0),
           "topp": (1.0, 0, 0.9, 0.0), "topp_hi": (1.3, 0, 0.99, 0.0), "minp": (1.2, 0, 1.0, 0.05),
           "greedy": (0.0, 0, 1.0, 0.0), "all": (0.9, 1000, 0.95, 0.02)}
    p = [row[kinds[r.randrange(len(kinds))]] for _ in range(R)]
    f = lambda i, dt: torch.tensor([q[i] for q in p], dtype=dt, device="cuda")  # noqa: E731
    return {"case": dict(case), "logits": x, "temperature": f(0, torch.float32), "top_k": f(1, torch.int32),
            "top_p": f(2, torch.float32), "min_p": f(3, torch.float32),
            "u": torch.rand(R, generator=g, device="cuda"),
            "tokens": torch.zeros(R, dtype=torch.int32, device="cuda"),
            "logprobs": torch.zeros(R, dtype=torch.float32, device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------------ one pass
def run(s):
    if s["case"]["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    if s["case"]["op"] == "attn":
        return _attn_own(s) if own else _attn_plain(s)
    return _sample_own(s) if own else _sample_plain(s)


def _append_own(s):
    import nvfp4_weight_only_flint_b200 as fm
    c = s["case"]
    fm.flint_qk_norm_rope_paged_kv(
        s["qkv"], s["T"], c["hq"], c["hkv"], s["qw"], s["kw"], s["cs"], s["max_pos"], c["rope"], EPS, s["q_start"],
        s["kv_len"], s["B"], s["table"], s["table"].shape[1], c["page"], s["n_pages"],
        fm.FLINT_KV_BF16 if c["cache"] == "bf16" else fm.FLINT_KV_E4M3, s["ks"], s["vs"], s["q_out"], s["k"], s["v"],
        s["status"])
    return s["q_out"], s["k"], s["v"]


def _attn_own(s):
    import nvfp4_weight_only_flint_b200 as fm
    c = s["case"]
    fm.flint_paged_attention(
        s["q"], s["T"], s["q_start"], s["kv_len"], s["B"], s["table"], s["table"].shape[1], c["page"], s["n_pages"],
        s["k"], s["v"], fm.FLINT_KV_BF16 if c["cache"] == "bf16" else fm.FLINT_KV_E4M3, s["ks"], s["vs"], c["hq"],
        c["hkv"], s["max_n"], c["window"], DH ** -0.5, s["out"], s["ws"], s["status"])
    return s["out"]


def _sample_own(s):
    import nvfp4_weight_only_flint_b200 as fm
    c = s["case"]
    fm.flint_sample(s["logits"], c["rows"], c["vocab"], c["vocab"],
                    fm.FLINT_LOGITS_F32 if c["dtype"] == "f32" else fm.FLINT_LOGITS_BF16, s["temperature"],
                    s["top_k"], s["top_p"], s["min_p"], s["u"], s["tokens"], s["logprobs"], s["status"])
    return s["tokens"], s["logprobs"]


def _token_places(s):
    """Sequence and position of each new token."""
    t = torch.arange(s["T"], device="cuda")
    seq = torch.bucketize(t, s["q_start"][1:].long(), right=True)
    end = s["q_start"].long()[seq + 1]
    return seq, s["kv_len"].long()[seq] - end + t


def _append_plain(s):
    c = s["case"]
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    x = s["qkv"].float()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    seq, pos = _token_places(s)
    if c["norm"]:
        norm = lambda y, w: y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * w.float()  # noqa: E731
        q, k = norm(q, s["qw"]), norm(k, s["kw"])
    if c["rope"]:
        row = s["cs"][pos]
        cos, sin = row[:, None, :DH // 2], row[:, None, DH // 2:]
        turn = lambda y: torch.cat([y[..., :DH // 2] * cos - y[..., DH // 2:] * sin,  # noqa: E731
                                    y[..., DH // 2:] * cos + y[..., :DH // 2] * sin], -1)
        q, k = turn(q), turn(k)
    rows = s["table"].long()[seq, pos // page] * page + pos % page
    s["q_out"].copy_(q)
    if c["cache"] == "bf16":
        s["k"].view(-1, hkv, DH)[rows] = k.to(torch.bfloat16)
        s["v"].view(-1, hkv, DH)[rows] = v.to(torch.bfloat16)
    else:
        to8 = lambda y, sc: (y / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
        s["k"].view(torch.uint8).view(-1, hkv, DH)[rows] = to8(k, s["ks"]).view(torch.uint8)
        s["v"].view(torch.uint8).view(-1, hkv, DH)[rows] = to8(v, s["vs"]).view(torch.uint8)
    return s["q_out"], s["k"], s["v"]


def _attn_plain(s):
    c = s["case"]
    hq, hkv, page, B, N, L = c["hq"], c["hkv"], c["page"], s["B"], s["max_n"], s["max_kv"]
    G = hq // hkv
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    kv = s["kv_len"].long()
    i, j = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    live = i[None, :] < n[:, None]  # [B][N]: a query
    at = (s["q_start"][:-1].long()[:, None] + i).clamp_max(s["T"] - 1)
    q = s["q"].float()[at].view(B, N, hkv, G, DH).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * N, DH)
    rows = s["table"].long()[:, j // page] * page + j % page
    rows = torch.where(j[None, :] < kv[:, None], rows, 0)
    k = _values(s["k"], s["ks"], hkv)[rows] if c["cache"] == "bf16" else _gather8(s["k"], s["ks"], rows, hkv)
    v = _values(s["v"], s["vs"], hkv)[rows] if c["cache"] == "bf16" else _gather8(s["v"], s["vs"], rows, hkv)
    pos = (kv - n)[:, None] + i  # [B][N]
    sees = (j <= pos[..., None]) & live[..., None]
    if c["window"] > 0:
        sees &= j > pos[..., None] - c["window"]
    x = torch.matmul(q, k.float().permute(0, 2, 3, 1)).view(B, hkv, G, N, L)
    x = x.mul_(DH ** -0.5).masked_fill_(~sees[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, G * N, L), v.float().permute(0, 2, 1, 3)).view(B, hkv, G, N, DH)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, hq, DH)
    s["out"][at[live]] = o[live].to(torch.bfloat16)
    return s["out"]


def _values(pool, scale, hkv):
    return pool.view(-1, hkv, DH)


def _gather8(pool, scale, rows, hkv):
    x = pool.view(torch.uint8).view(-1, hkv, DH)[rows].view(torch.float8_e4m3fn).float()
    return x * scale[:, None]


def _sample_plain(s):
    x = s["logits"].double()
    V = x.shape[1]
    t = s["temperature"].double()[:, None]
    greedy = t == 0
    z, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = ((z - z[:, :1]) / torch.where(greedy, 1.0, t)).exp()
    rank = torch.arange(V, device="cuda")[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"], V).long()[:, None]
    k = torch.where(greedy, 1, k)
    w = torch.where(rank < k, w, 0.0)
    before = w.cumsum(1) - w
    p = s["top_p"].double()[:, None]
    keep = (p >= 1) | (rank == 0) | (before < p * w.sum(1, keepdim=True))
    keep &= w >= s["min_p"].double()[:, None]
    w = torch.where(keep, w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)  # back into the vocabulary's order
    c = w.cumsum(1)
    # a token's end of the unit interval: the first one above u
    first = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1).clamp_max(V - 1)
    s["tokens"].copy_(first)
    s["logprobs"].copy_((w.gather(1, first[:, None])[:, 0] / c[:, -1]).log())
    return s["tokens"], s["logprobs"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["rows"] * 28, "flops": 4 * n}
    lens = _lengths(case)
    hq, hkv, T = case["hq"], case["hkv"], sum(a for a, _ in lens)
    e = 2 if case["cache"] == "bf16" else 1
    if case["op"] == "append":
        b = T * (hq + 2 * hkv) * DH * 2 + T * hq * DH * 2 + T * 2 * hkv * DH * e
        if case["rope"]:  # rows of the angle table that some token needs
            b += 4 * DH * min(T, max(a + c for a, c in lens))
        return {"bytes": b, "flops": 10 * T * (hq + hkv) * DH}
    b, pairs = 2 * T * hq * DH * 2, 0
    w = case["window"]
    for a, c in lens:
        reach = a + c if w == 0 else min(a + c, a + w - 1)
        b += reach * hkv * DH * 2 * e
        if w == 0:
            pairs += a * c + a * (a + 1) // 2
        else:
            full = max(0, min(a, w - 1 - c))  # queries that still see everything before them
            pairs += full * c + full * (full + 1) // 2 + (a - full) * w
    return {"bytes": b, "flops": 4 * pairs * hq * DH}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _sample_exact(s)
    return _append_exact(s) if case["op"] == "append" else _attn_exact(s)


def _pool_exact(pool, hkv):
    return pool.double().view(-1, hkv, DH)


def _append_exact(s):
    c = s["case"]
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    shape = s["k"].shape
    q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
    k_out, v_out = _pool_exact(s["k"], hkv), _pool_exact(s["v"], hkv)
    one = torch.ones(hkv, dtype=torch.float64, device="cuda")
    ks, vs = (one, one) if s["ks"] is None else (s["ks"].double(), s["vs"].double())
    t0 = 0
    for b, (n, ctx) in enumerate(_lengths(c)):
        x = s["qkv"][t0:t0 + n].double()
        pos = torch.arange(ctx, ctx + n, device="cuda")
        rows = s["table"][b].long()[pos // page] * page + pos % page
        for lo, hi, w in ((0, hq, s["qw"]), (hq, hq + hkv, s["kw"])):
            y = x[:, lo:hi]
            if c["norm"]:
                y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / DH + EPS) * w.double()
            if c["rope"]:
                z = torch.view_as_complex(torch.stack([y[..., :64], y[..., 64:]], -1).contiguous())
                turn = torch.complex(s["cs"][pos, :64].double(), s["cs"][pos, 64:].double())
                z = torch.view_as_real(z * turn[:, None])
                y = torch.cat([z[..., 0], z[..., 1]], -1)
            if lo == 0:
                q_out[t0:t0 + n] = y
            else:
                k_out[rows] = y / ks[:, None]
        v_out[rows] = x[:, hq + hkv:] / vs[:, None]
        t0 += n
    return q_out, k_out.view(shape), v_out.view(shape)


def _attn_exact(s):
    c = s["case"]
    hq, hkv, page, w = c["hq"], c["hkv"], c["page"], c["window"]
    G = hq // hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, ctx) in enumerate(_lengths(c)):
        j = torch.arange(ctx + n, device="cuda")
        rows = s["table"][b].long()[j // page] * page + j % page
        for h in range(hkv):
            k, v = (x.view(torch.uint8 if c["cache"] != "bf16" else torch.bfloat16).view(-1, hkv, DH)[rows, h]
                    for x in (s["k"], s["v"]))
            if c["cache"] != "bf16":
                k = k.view(torch.float8_e4m3fn).double() * s["ks"][h].double()
                v = v.view(torch.float8_e4m3fn).double() * s["vs"][h].double()
            k, v = k.double(), v.double()
            for i0 in range(0, n, 1024):
                i = torch.arange(i0, min(n, i0 + 1024), device="cuda")
                far = j[None, :] - (ctx + i)[:, None]
                gone = far > 0 if w == 0 else (far > 0) | (far <= -w)
                q = s["q"][t0 + i, h * G:(h + 1) * G].double().transpose(0, 1)
                x = torch.softmax(((q @ k.T) / math.sqrt(DH)).masked_fill(gone, -math.inf), -1)
                out[t0 + i, h * G:(h + 1) * G] = (x @ v).transpose(0, 1)
        t0 += n
    return out


def _sample_exact(s):
    import numpy as np
    host = lambda x: x.double().cpu().numpy()  # noqa: E731
    x, t, p, m, u = (host(s[k]) for k in ("logits", "temperature", "top_p", "min_p", "u"))
    top_k = s["top_k"].cpu().numpy()
    R, V = x.shape
    tokens, logs = np.zeros(R, np.int32), np.zeros(R)
    for r in range(R):
        if t[r] == 0:
            tokens[r] = int(np.argmax(x[r]))
            continue
        w = np.exp((x[r] - x[r].max()) / t[r])
        order = np.argsort(-x[r], kind="stable")
        n = V if top_k[r] <= 0 else min(V, int(top_k[r]))
        if p[r] < 1:
            mass = np.concatenate([[0.0], np.cumsum(w[order[:n]])])
            n = max(1, int(np.searchsorted(mass[:-1], p[r] * mass[-1], side="left")))
        kept = np.sort(order[:n])
        kept = kept[w[kept] >= m[r]]
        c = np.cumsum(w[kept])
        at = min(len(kept) - 1, int(np.searchsorted(c, u[r] * c[-1], side="right")))
        tokens[r] = kept[at]
        logs[r] = math.log(w[kept[at]] / c[-1])
    return torch.from_numpy(tokens), torch.from_numpy(logs)
