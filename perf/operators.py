"""What is measured of the operators beside decode attention: writing the KV cache (append_kv) and
attention of a batch whose rows share prompts (decode_attention_shared_prefix).

append        q, k and v of new tokens (views of one fused projection output) are rotated by their
              positions; k and v go to their slots of the cache, q to its own buffer.
shared        one decode step: every row attends to the prompt its group shares and to its own
              cache; out and the log-sum-exp come back.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def listed():
    a = {"op": "append", "B": 16, "tokens": "one", "T": 16, "Hq": 32, "Hkv": 8, "d": 128,
         "dtype": "bf16", "cache": "bf16", "page": 16, "cap": 8192, "rot": 128, "style": "half"}
    s = {"op": "shared", "B": 8, "Q": 1, "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16",
         "cache": "bf16", "groups": 1, "prefix": 1000, "own": 129, "page": 0}
    return [
        # the smallest call: one decode step of a small batch over 16-token pages
        {**a, "name": "append_step"},
        # one step of a large serving batch over an FP8 cache
        {**a, "name": "append_step_fp8", "B": 256, "T": 256, "cache": "fp8", "page": 32,
         "cap": 2048},
        # f32, five tokens a row (speculative verification), partial interleaved rotation, odd sizes
        {**a, "name": "append_verify_f32", "B": 33, "tokens": "many", "T": 165, "Hq": 16,
         "Hkv": 16, "d": 64, "dtype": "f32", "cache": "f32", "page": 0, "cap": 257, "rot": 32,
         "style": "interleaved"},
        # prompts of different lengths packed into one prefill
        {**a, "name": "append_prefill", "B": 7, "tokens": "ragged", "T": 8191, "Hq": 64},
        # a large packed prefill into an FP8 cache
        {**a, "name": "append_prefill_fp8", "B": 12, "tokens": "ragged", "T": 32768, "Hq": 64,
         "cache": "fp8", "page": 64},
        # a few rows on a short system prompt: latency
        {**s, "name": "shared_small"},
        # a serving batch on one prompt, everything in 16-token pages
        {**s, "name": "shared_paged", "B": 32, "prefix": 8192, "own": 1024, "page": 16},
        # three prompts of different lengths in one batch
        {**s, "name": "shared_groups", "B": 48, "groups": 3, "prefix": 4001, "own": 512},
        # four draft tokens a row verified against a long document
        {**s, "name": "shared_verify", "B": 16, "Q": 4, "Hq": 64, "prefix": 16384, "own": 300},
        # a large batch on one long prompt over an FP8 cache
        {**s, "name": "shared_fp8", "B": 128, "cache": "fp8", "prefix": 32768, "own": 256,
         "page": 64},
        # f32, one query head per kv head, head dim 64, odd sizes
        {**s, "name": "shared_f32", "B": 33, "Hq": 16, "Hkv": 16, "d": 64, "dtype": "f32",
         "cache": "f32", "prefix": 2049, "own": 65},
        # the largest: 64 rows on a 128K-token document
        {**s, "name": "shared_128k", "B": 64, "Hq": 64, "prefix": 131072, "own": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "shared", "shared"])
    cache = rng.choice(["bf16", "bf16", "bf16", "fp8", "fp8", "f32"])
    dtype = "f32" if cache == "f32" else "bf16"
    d = 128 if cache == "fp8" else rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 2, 4, 4, 8])
    page = rng.choice([0, 8, 16, 16, 32, 64, 128, 256])
    if op == "append":
        B = _log(rng, 1, 300)
        tokens = rng.choice(["one", "many", "ragged", "ragged"])
        T = {"one": B, "many": B * rng.randint(2, 8), "ragged": max(B, _log(rng, 1, 32768))}[tokens]
        while T * (G + 2) * Hkv * d > 32768 * 80 * 128:
            T //= 2
        rot = rng.choice([d, d, d // 2, 0])
        cap = _log(rng, 16, 8192)
        while B * cap * Hkv * d > 1 << 29:
            cap //= 2
        return {"op": op, "B": B, "tokens": tokens, "T": max(T, B), "Hq": Hkv * G, "Hkv": Hkv,
                "d": d, "dtype": dtype, "cache": cache, "page": page,
                "cap": max(cap, 16), "rot": rot,
                "style": rng.choice(["half", "half", "interleaved"])}
    B = _log(rng, 2, 256)
    Q = rng.choice([1, 1, 1, 2, 4]) if G <= 4 else 1
    groups = min(B, rng.choice([1, 1, 1, 2, 3, 5]))
    prefix = _log(rng, 16, 131072)
    while (B * Q * G * Hkv * prefix * d > (64 * 64 * 131072 * 128 if dtype == "bf16" else 1 << 36)
           or (groups > 1 and B * Hkv * prefix * d > 1 << 31)):
        prefix //= 2
    return {"op": op, "B": B, "Q": Q, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "dtype": dtype,
            "cache": cache, "groups": groups, "prefix": max(prefix, 3),
            "own": _log(rng, 8, 1024), "page": page}


# ------------------------------------------------------------------ lengths and layouts


def _spread(n, lo, hi, salt):
    """n whole numbers over [lo, hi], the first of them hi: fixed for a case, like a batch's lengths."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * (((i + salt) * 0.6180339887498949) % 1.0))
            for i in range(n)]


def _new_tokens(c):
    """New tokens of each row (append)."""
    if c["tokens"] != "ragged":
        return [c["T"] // c["B"]] * c["B"]
    rest, n = c["T"] - c["B"], c["B"]
    w = _spread(n, 1, 1000, 3)
    got = [1 + rest * x // sum(w) for x in w]
    got[0] += c["T"] - sum(got)
    return got


def _append_lengths(c):
    """Row lengths after the append: the new tokens and what was there before."""
    return [m + x for m, x in zip(_new_tokens(c), _spread(c["B"], 0, c["cap"] // 2, 1))]


def _group_sizes(c):
    w = _spread(c["groups"], 1, 7, 2)
    got = [max(1, c["B"] * x // sum(w)) for x in w]
    got[0] += c["B"] - sum(got)
    return got


def _prefix_lengths(c):
    return _spread(c["groups"], min(c["prefix"], 3), c["prefix"], 5)


def _own_lengths(c):
    return _spread(c["B"], c["Q"], max(c["own"], c["Q"]), 7)


def _fill(g, shape, dtype):
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16 if dtype == "fp8" else _T[dtype])
    x.normal_(generator=g)
    return x.to(_T[dtype]) if dtype == "fp8" else x


def _scales(g, H, cache):
    if cache != "fp8":
        return None, None
    s = torch.rand((2, H), device="cuda", generator=g) * 0.01 + 0.01   # amax / 448 of such rows
    return s[0].contiguous(), s[1].contiguous()


def _table(g, lens, page):
    """(pages in the pool, block table with -1 past each row's pages), in a random order."""
    n = torch.tensor([-(-x // page) for x in lens], device="cuda")
    width = max(1, max(-(-x // page) for x in lens))
    total = max(1, sum(-(-x // page) for x in lens))
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = n.cumsum(0) - n
    at = (first[:, None] + col[None, :]).clamp(max=total - 1)
    return total, torch.where(col[None, :] < n[:, None], perm[at], -1).to(torch.int32).contiguous()


def _ints(v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (_prepare_append if case["op"] == "append" else _prepare_shared)(case, g)


def _prepare_append(c, g):
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    lens, new = _append_lengths(c), _new_tokens(c)
    if c["tokens"] == "many":
        T = c["T"] // B * B
    qkv = _fill(g, (T, (Hq + 2 * Hkv) * d), c["dtype"])
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = qkv[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    if c["tokens"] == "many":
        q, k, v = (x.unflatten(0, (B, T // B)) for x in (q, k, v))
    most = max(lens)
    pages, table = _table(g, lens, c["page"]) if c["page"] else (0, None)
    shape = (pages, Hkv, c["page"], d) if c["page"] else (B, Hkv, most, d)
    k_cache, v_cache = _fill(g, shape, c["cache"]), _fill(g, shape, c["cache"])
    cos_sin = None
    if c["rot"]:
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * freq[None, :]
        cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ks, vs = _scales(g, Hkv, c["cache"])
    return {"case": c, "q": q, "k": k, "v": v, "k_cache": k_cache, "v_cache": v_cache,
            "seq_lens": _ints(lens), "cu": _ints(cu) if c["tokens"] == "ragged" else None,
            "table": table, "cos_sin": cos_sin, "k_scale": ks, "v_scale": vs,
            "q_out": torch.empty(q.shape, device="cuda", dtype=q.dtype),
            "workspace": torch.zeros(256, device="cuda", dtype=torch.uint8)}


def _prepare_shared(c, g):
    B, Q, Hq, Hkv, d, P, page = (c[x] for x in ("B", "Q", "Hq", "Hkv", "d", "groups", "page"))
    plens, lens, sizes = _prefix_lengths(c), _own_lengths(c), _group_sizes(c)
    q = _fill(g, (B, Q, Hq, d) if Q > 1 else (B, Hq, d), c["dtype"])
    ks, vs = _scales(g, Hkv, c["cache"])
    if page:   # prompts and rows in one pool of pages
        pages, table = _table(g, plens + lens, page)
        k_cache, v_cache = (_fill(g, (pages, Hkv, page, d), c["cache"]) for _ in range(2))
        k_prefix, v_prefix = k_cache, v_cache
        width = lambda v: max(1, max(-(-x // page) for x in v))  # noqa: E731
        prefix_table = table[:P, :width(plens)].contiguous()
        table = table[P:, :width(lens)].contiguous()
    else:
        k_prefix, v_prefix = (_fill(g, (P, Hkv, max(plens), d), c["cache"]) for _ in range(2))
        k_cache, v_cache = (_fill(g, (B, Hkv, max(lens), d), c["cache"]) for _ in range(2))
        prefix_table = table = None
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    workspace = None
    if own:
        import decode_attention_05_gb300 as fd
        cap = lambda cache, t: cache.shape[2] * (1 if t is None else t.shape[1])  # noqa: E731
        workspace = torch.zeros(fd.shared_prefix_workspace_size(
            B, Q, Hq, Hkv, d, P, cap(k_prefix, prefix_table), cap(k_cache, table)),
            device="cuda", dtype=torch.uint8)
    return {"case": c, "q": q, "k_prefix": k_prefix, "v_prefix": v_prefix,
            "prefix_lens": _ints(plens), "prefix_table": prefix_table, "k_cache": k_cache,
            "v_cache": v_cache, "seq_lens": _ints(lens), "table": table,
            "group_start": _ints(starts) if P > 1 else None,
            "group_of": torch.repeat_interleave(torch.arange(P), torch.tensor(sizes)).cuda(),
            "k_scale": ks, "v_scale": vs, "workspace": workspace,
            "out": torch.empty_like(q),
            "lse": torch.empty(q.shape[:-1], device="cuda", dtype=torch.float32)}


# ------------------------------------------------------------------ one pass


def run(s):
    return (_run_append if s["case"]["op"] == "append" else _run_shared)(s)


def _run_append(s):
    c = s["case"]
    if own:
        import decode_attention_05_gb300 as fd
        fd.append_kv(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["seq_lens"],
                     s["cos_sin"],
                     rope_style=fd.FD_ROPE_HALF if c["style"] == "half" else fd.FD_ROPE_INTERLEAVED,
                     cu_tokens=s["cu"], block_table=s["table"], page_size=c["page"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"],
                     workspace=s["workspace"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    q, k, v = s["q"], s["k"], s["v"]
    shape = q.shape
    if q.dim() == 4:
        q, k, v = (x.flatten(0, 1) for x in (q, k, v))
    row, pos = _places(s, q.shape[0])
    q, k = _rotate(q, pos, s["cos_sin"], c), _rotate(k, pos, s["cos_sin"], c)
    at = (row, slice(None), pos)
    if c["page"]:
        at = (s["table"][row, pos // c["page"]].long(), slice(None), pos % c["page"])
    s["k_cache"][at] = _stored(k, s["k_scale"], s["k_cache"].dtype)
    s["v_cache"][at] = _stored(v, s["v_scale"], s["v_cache"].dtype)
    return {"q": q.to(s["q"].dtype).view(shape), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _places(s, T):
    """Each new token's row and position in that row's cache."""
    B = s["seq_lens"].shape[0]
    t = torch.arange(T, device="cuda")
    if s["cu"] is None:
        row, end = t // (T // B), (t // (T // B) + 1) * (T // B)
    else:
        row = (t[:, None] >= s["cu"][None, 1:]).sum(1)
        end = s["cu"][row + 1].long()
    return row, s["seq_lens"][row].long() - end + t


def _rotate(x, pos, cos_sin, c):
    x, r = x.float(), c["rot"]
    if not r:
        return x
    cos, sin = cos_sin[pos][:, None, :r // 2], cos_sin[pos][:, None, r // 2:]
    if c["style"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _stored(x, scale, dtype):
    if dtype != torch.float8_e4m3fn:
        return x.to(dtype)
    return (x.float() / scale[None, :, None]).clamp(-448.0, 448.0).to(dtype)


def _gathered(cache, table, scale):
    """[rows, Hkv, capacity, d] in f32 of a contiguous cache or of a block table's pages."""
    if table is not None:
        cache = cache.view(torch.uint8) if cache.element_size() == 1 else cache
        x = cache[table.clamp(min=0).long()]                   # [rows, pages, Hkv, page, d]
        x = x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x
        x = x.float().transpose(1, 2).flatten(2, 3)
    else:
        x = cache.float()
    return x if scale is None else x * scale[None, :, None, None]


def _run_shared(s):
    c = s["case"]
    if own:
        import decode_attention_05_gb300 as fd
        fd.decode_attention_shared_prefix(
            s["q"], s["k_prefix"], s["v_prefix"], s["prefix_lens"], s["k_cache"], s["v_cache"],
            s["seq_lens"], group_start=s["group_start"], prefix_table=s["prefix_table"],
            block_table=s["table"], page_size=c["page"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], out=s["out"], lse_out=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Q, Hq, Hkv, d, P = (c[x] for x in ("B", "Q", "Hq", "Hkv", "d", "groups"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Q, Hkv, G, d).permute(2, 0, 1, 3, 4) / math.sqrt(d)
    kp = _gathered(s["k_prefix"], s["prefix_table"], s["k_scale"])
    vp = _gathered(s["v_prefix"], s["prefix_table"], s["v_scale"])
    ko = _gathered(s["k_cache"], s["table"], s["k_scale"])
    vo = _gathered(s["v_cache"], s["table"], s["v_scale"])
    Lp, Lo = kp.shape[2], ko.shape[2]
    if P == 1:       # one product per kv head for all rows
        xp = (q.reshape(Hkv, B * Q * G, d) @ kp[0].transpose(1, 2)).view(Hkv, B, Q * G, Lp)
    else:            # each row with its group's prompt
        kp, vp = kp[s["group_of"]].transpose(0, 1), vp[s["group_of"]].transpose(0, 1)
        xp = q.reshape(Hkv, B, Q * G, d) @ kp.transpose(2, 3)
    xo = q.reshape(Hkv, B, Q * G, d) @ ko.transpose(0, 1).transpose(2, 3)
    tp, to = torch.arange(Lp, device="cuda"), torch.arange(Lo, device="cuda")
    xp = xp.masked_fill_((tp[None, :] >= s["prefix_lens"][s["group_of"]][:, None])[None, :, None, :],
                         -math.inf)
    last = s["seq_lens"][:, None] - Q + torch.arange(Q, device="cuda")[None, :]
    seen = (to[None, None, :] <= last[:, :, None])[:, :, None, :].expand(B, Q, G, Lo)
    xo = xo.masked_fill_(~seen.reshape(1, B, Q * G, Lo), -math.inf)
    m = torch.maximum(xp.amax(-1), xo.amax(-1))[..., None]
    ep, eo = xp.sub_(m).exp_(), xo.sub_(m).exp_()
    l = ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True)
    y = eo @ vo.transpose(0, 1)
    if P == 1:
        y = y + (ep.view(Hkv, B * Q * G, Lp) @ vp[0]).view(Hkv, B, Q * G, d)
    else:
        y = y + ep @ vp
    y = (y / l).view(Hkv, B, Q, G, d).permute(1, 2, 0, 3, 4)
    lse = (m + l.log()).view(Hkv, B, Q, G).permute(1, 2, 0, 3)
    return {"out": y.reshape(s["q"].shape).to(s["q"].dtype),
            "lse": lse.reshape(s["q"].shape[:-1]).contiguous()}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c = case
    e, ec, Hq, Hkv, d = _T[c["dtype"]].itemsize, _T[c["cache"]].itemsize, c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "append":
        T = sum(_new_tokens(c))
        rows = T * (Hq + 2 * Hkv) * d * e + T * Hq * d * e + 2 * T * Hkv * d * ec
        return {"bytes": rows + 4 * T * c["rot"], "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    B, Q = c["B"], c["Q"]
    plens, lens, sizes = _prefix_lengths(c), _own_lengths(c), _group_sizes(c)
    kv = 2 * Hkv * d * ec * (sum(plens) + sum(lens))
    keys = sum(n * p for n, p in zip(sizes, plens)) + sum(lens)
    return {"bytes": kv + B * Q * Hq * (2 * d * e + 4), "flops": 4 * d * Hq * Q * keys}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_shared)(case, s)


def _exact_append(c, s):
    B, page, r = c["B"], c["page"], c["rot"]
    new, lens = _new_tokens(c), _append_lengths(c)
    rows = [b for b in range(B) for _ in range(new[b])]
    places = [lens[b] - new[b] + i for b in range(B) for i in range(new[b])]
    row, pos = torch.tensor(rows, device="cuda"), torch.tensor(places, device="cuda")

    def turned(x):
        x = x.reshape(len(rows), -1, c["d"]).double()
        if not r:
            return x
        cos = s["cos_sin"].double()[pos, :r // 2][:, None, :]
        sin = s["cos_sin"].double()[pos, r // 2:][:, None, :]
        first = torch.arange(r // 2, device="cuda") * (1 if c["style"] == "half" else 2)
        second = first + (r // 2 if c["style"] == "half" else 1)
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(cos, sin)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def filled(cache, x, scale):
        y = cache.double()
        if scale is not None:
            x = (x / scale.double().view(1, -1, 1)).clamp(-448.0, 448.0)
        if page:
            y.index_put_((s["table"].long()[row, pos.div(page, rounding_mode="floor")],
                          torch.arange(c["Hkv"], device="cuda")[:, None], pos.remainder(page)),
                         x.transpose(0, 1))
        else:
            y.index_put_((row, torch.arange(c["Hkv"], device="cuda")[:, None], pos),
                         x.transpose(0, 1))
        return y

    return {"q": turned(s["q"]).view(s["q"].shape), "k_cache": filled(s["k_cache"], turned(s["k"]), s["k_scale"]),
            "v_cache": filled(s["v_cache"], s["v"].reshape(len(rows), c["Hkv"], c["d"]).double(), s["v_scale"])}


def _exact_shared(c, s):
    B, Q, Hq, Hkv, d, page = (c[x] for x in ("B", "Q", "Hq", "Hkv", "d", "page"))
    G, plens, lens, sizes = Hq // Hkv, _prefix_lengths(c), _own_lengths(c), _group_sizes(c)
    q = s["q"].view(B, Q, Hkv, G, d)
    out = torch.zeros((B, Q, Hkv, G, d), device="cuda", dtype=torch.float64)
    lse = torch.zeros((B, Q, Hkv, G), device="cuda", dtype=torch.float64)

    def keys(cache, table, i, h, n, scale):
        if page:
            ids = table[i, :-(-n // page)].long()
            x = cache[:, h][ids].double().flatten(0, 1)[:n]
        else:
            x = cache[i, h, :n].double()
        return x if scale is None else x * scale[h].double()

    for h in range(Hkv):
        b = 0
        for p, n in enumerate(sizes):
            kp = keys(s["k_prefix"], s["prefix_table"], p, h, plens[p], s["k_scale"])
            vp = keys(s["v_prefix"], s["prefix_table"], p, h, plens[p], s["v_scale"])
            x = q[b:b + n, :, h].double().reshape(n * Q * G, d) @ kp.T / math.sqrt(d)
            part = torch.logsumexp(x, -1)
            o = torch.softmax(x, -1) @ vp
            part, o = part.view(n, Q, G), o.view(n, Q, G, d)
            for i in range(n):
                ko = keys(s["k_cache"], s["table"], b + i, h, lens[b + i], s["k_scale"])
                vo = keys(s["v_cache"], s["table"], b + i, h, lens[b + i], s["v_scale"])
                y = q[b + i, :, h].double() @ ko.T / math.sqrt(d)                 # [Q, G, L]
                for j in range(Q - 1):
                    y[j, :, lens[b + i] - Q + j + 1:] = -math.inf
                mine = torch.logsumexp(y, -1)
                total = torch.logaddexp(part[i], mine)
                lse[b + i, :, h] = total
                w = (mine - total).exp()[..., None] * torch.softmax(y, -1).nan_to_num(0.0)
                out[b + i, :, h] = (part[i] - total).exp()[..., None] * o[i] + w @ vo
            b += n
    return {"out": out.reshape(s["q"].shape), "lse": lse.reshape(s["q"].shape[:-1])}
