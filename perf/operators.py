"""Measured cases of the paged-cache operators: page_map, page_append, page_select + page_attn.

A batch of R rows (requests) keeps its keys and values in pages of P tokens, [N, P, Hkv, d], that a block
table [R, W] names.  One serving step maps the new tokens to slots (``map``), writes their keys and values
(``append``), and attends from one query per row over its cache, in full or over a sink and a window
(``attn``), or over the pages that a score of the page means selects (``sparse``: selection and attention).

``own`` False runs the plain form in elementary torch operations, True the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _attn(name, R, H, Hkv, d, P, lo, hi, q="bf16", kv="bf16", sink=0, window=0, idle=False):
    return {"name": name, "kind": "attn", "R": R, "H": H, "Hkv": Hkv, "d": d, "P": P, "lo": lo, "hi": hi, "q": q,
            "kv": kv, "sink": sink, "window": window, "idle": idle}


def _sparse(name, R, H, Hkv, d, P, lo, hi, topk, first, last, q="bf16", kv="bf16", idle=False):
    return {"name": name, "kind": "sparse", "R": R, "H": H, "Hkv": Hkv, "d": d, "P": P, "lo": lo, "hi": hi,
            "topk": topk, "first": first, "last": last, "q": q, "kv": kv, "idle": idle}


def _append(name, R, Hkv, d, P, lo, hi, new_lo, new_hi, x="bf16", kv="bf16", means=True):
    return {"name": name, "kind": "append", "R": R, "Hkv": Hkv, "d": d, "P": P, "lo": lo, "hi": hi,
            "new_lo": new_lo, "new_hi": new_hi, "x": x, "kv": kv, "means": means}


def _map(name, R, P, lo, hi, new_lo, new_hi):
    return {"name": name, "kind": "map", "R": R, "P": P, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi}


def listed():
    return [
        # one rollout's next token over a single cached frame: nothing but latency
        _attn("attn_one_frame", 1, 40, 8, 128, 64, 1560, 1560),
        # a served batch of short and long requests, small pages, one row free and one just started
        _attn("attn_ragged", 24, 32, 4, 128, 16, 1, 16384, q="fp16", kv="fp16", idle=True),
        # a batch over an 8-bit cache
        _attn("attn_e4m3", 64, 40, 8, 128, 64, 4096, 12288, kv="e4m3"),
        # every head its own cache, 24 frames of 1560 tokens: the whole cache ...
        _attn("attn_24_frames", 8, 12, 12, 128, 128, 37440, 37440),
        # ... and the sink frame with the last five
        _attn("attn_sink_window", 8, 12, 12, 128, 128, 37440, 37440, sink=1560, window=7800),
        # two very long rollouts that attend to 64 of about 2000 pages
        _sparse("sparse_long", 2, 40, 8, 128, 64, 120000, 131071, 64, 1, 2),
        # a batch over an 8-bit cache of small pages, an odd selection
        _sparse("sparse_e4m3", 32, 32, 8, 128, 32, 16001, 48000, 97, 2, 4, q="fp16", kv="e4m3"),
        # one token for each of 64 requests, page means kept
        _append("append_decode", 64, 8, 128, 64, 0, 4096, 1, 1),
        # prompts of a few requests enter the cache
        _append("append_prompts", 6, 8, 128, 64, 0, 700, 1000, 4680),
        # prompts into an 8-bit cache, 12 key heads
        _append("append_e4m3", 9, 12, 128, 16, 3, 600, 200, 1560, x="fp16", kv="e4m3"),
        # a decoding step of 256 requests, some ending and some starting
        _map("map_decode", 256, 64, 0, 8192, 1, 1),
        # long prompts mixed with decoding requests
        _map("map_prompts", 48, 16, 0, 4096, 1, 4680),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["attn"] * 4 + ["sparse"] * 3 + ["append"] * 3 + ["map"] * 2)
    P = rng.choice([16, 32, 64, 128])
    if kind == "map":
        R = _log(rng, 1, 256)
        new_hi = rng.choice([1, _log(rng, 2, max(2, 200000 // R // 2))])
        return _map("", R, P, 0, _log(rng, 16, 8192), 1, min(new_hi, 4680))
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    q = rng.choice(["bf16", "fp16"])
    kv = rng.choice([q, q, "e4m3"])
    if kind == "append":
        R = _log(rng, 1, 128)
        new_hi = rng.choice([1, _log(rng, 2, max(2, 16000 // R))])
        hi = _log(rng, 16, max(16, 60000 // R))
        return _append("", R, Hkv, d, P, 0, hi, rng.choice([1, new_hi]), new_hi, x=q, kv=kv, means=rng.random() < 0.7)
    H = Hkv * rng.choice([1, 2, 4, 5, 8, 12, 16])
    R = _log(rng, 1, 64)
    cap = 250_000_000 // (R * Hkv * d)
    if kind == "attn":
        hi = _log(rng, 1, max(1, min(131072, cap)))
        sink, window = rng.choice([(0, 0), (0, 0), (rng.randint(0, hi), rng.randint(1, hi))])
        return _attn("", R, H, Hkv, d, P, rng.choice([1, hi, (hi + 1) // 2]), hi, q=q, kv=kv, sink=sink,
                     window=window, idle=R > 2 and rng.random() < 0.4)
    hi = _log(rng, 1000, max(1000, min(131072, cap)))
    first, last = rng.randint(0, 2), rng.randint(1, 4)
    topk = rng.randint(first + last, 128)
    return _sparse("", R, H, Hkv, d, P, (hi + 1) // 2, hi, topk, first, last, q=q, kv=kv,
                   idle=R > 2 and rng.random() < 0.4)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], both ends among them (n > 1), in no order."""
    if n == 1:
        return [hi]
    return [lo + int((hi - lo) * (i * 0.6180339887498949 % 1.0)) if i not in (0, n - 1) else (hi if i else lo)
            for i in range(n)]


def _lengths(case):
    """Cached tokens of each row; -1 is a row without a request."""
    ln = _spread(case["R"], case["lo"], case["hi"])
    if case.get("idle"):
        ln[1] = -1
        ln[2] = 0
    return ln


def _map_lengths(case):
    """(cached, new) of each row: mostly running requests, some ending (-1), some starting, some free rows."""
    ln = _spread(case["R"], case["lo"], case["hi"])
    new = _spread(case["R"], case["new_lo"], case["new_hi"])
    for r in range(case["R"]):
        if r % 16 == 7:
            new[r] = -1  # ends
        elif r % 16 == 11:
            ln[r] = -1  # starts
        elif r % 32 == 13:
            ln[r], new[r] = -1, 0  # free
        elif r % 32 == 14:
            new[r] = 0  # waits
    return ln, new


def _order(n, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()


def _cache(shape, kind, g):
    x = torch.empty(shape, dtype=TYPES[kind], device=DEV)
    if kind == "e4m3":
        for part in x.split(max(1, shape[0] // 8)):
            part.copy_(torch.randn(part.shape, dtype=torch.bfloat16, device=DEV, generator=g) * 2.0)
    else:
        x.normal_(generator=g)
    return x


def _means(k_pages, k_scale):
    out = torch.empty((k_pages.shape[0],) + tuple(k_pages.shape[2:]), dtype=torch.float32, device=DEV)
    for o, k in zip(out.split(4096), k_pages.split(4096)):
        o.copy_(k.float().mean(1))
    return out if k_scale is None else out * k_scale[None, :, None]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    R, P = case["R"], case["P"]
    order = _order(R, seed)
    if case["kind"] == "map":
        ln, new = _map_lengths(case)
        ln, new = [ln[i] for i in order], [new[i] for i in order]
        W = max(-(-(max(a, 0) + max(b, 0)) // P) for a, b in zip(ln, new)) or 1
        used = sum(-(-max(a, 0) // P) for a in ln)
        total = sum(max(b, 0) for b in new)
        N = used + sum(-(-max(b, 0) // P) + 1 for b in new) + 8
        pages = torch.randperm(N, device=DEV, generator=g).to(torch.int32)
        kv_len = torch.tensor(ln, dtype=torch.int32, device=DEV)
        table = torch.full((R, W), -1, dtype=torch.int32, device=DEV)
        held = torch.arange(W, device=DEV)[None] < ((kv_len.clamp(min=0) + P - 1) // P)[:, None]
        table[held] = pages[:used]
        free = torch.where(torch.arange(N, device=DEV) < used, -1, pages).to(torch.int32)
        cap = max(1, total + 5)  # the step's buffers hold a few tokens more than it brings
        s.update(kv_len=kv_len, new_len=torch.tensor(new, dtype=torch.int32, device=DEV), table=table, free=free,
                 ring=torch.tensor([3 * N + used, 4 * N], dtype=torch.int64, device=DEV), cap=cap,
                 out={"kv_len": torch.empty(R, dtype=torch.int32, device=DEV),
                      "ring": torch.empty(2, dtype=torch.int64, device=DEV),
                      "slot": torch.empty(cap, dtype=torch.int64, device=DEV),
                      "row": torch.empty(cap, dtype=torch.int32, device=DEV),
                      "pos": torch.empty(cap, dtype=torch.int32, device=DEV),
                      "cu": torch.empty(R + 1, dtype=torch.int32, device=DEV)})
        return s
    Hkv, d, kv = case["Hkv"], case["d"], case["kv"]
    if case["kind"] == "append":
        ln, new = _spread(R, case["lo"], case["hi"]), _spread(R, case["new_lo"], case["new_hi"])
        ln, new = [ln[i] for i in order], [new[i] for i in order]
        upto = [a + b for a, b in zip(ln, new)]
    else:
        ln = _lengths(case)
        ln = [ln[i] for i in order]
        upto = [max(a, 0) for a in ln]
    W = max(1, max(-(-n // P) for n in upto))
    used = sum(-(-n // P) for n in upto)
    N = used + 3
    pages = torch.randperm(N, device=DEV, generator=g).to(torch.int32)
    held = torch.arange(W, device=DEV)[None] < ((torch.tensor(upto, device=DEV) + P - 1) // P)[:, None]
    table = torch.full((R, W), -1, dtype=torch.int32, device=DEV)
    table[held] = pages[:used]
    s["table"] = table
    s["k_scale"] = s["v_scale"] = None
    if kv == "e4m3":
        s["k_scale"], s["v_scale"] = (torch.rand(Hkv, device=DEV, generator=g) * 0.5 + 0.25 for _ in range(2))
    s["k"], s["v"] = (_cache((N, P, Hkv, d), kv, g) for _ in range(2))
    if case["kind"] == "append":
        T = sum(new)
        row = torch.repeat_interleave(torch.arange(R), torch.tensor(new))
        first = torch.tensor(new).cumsum(0) - torch.tensor(new)
        pos = (torch.arange(T) - first[row] + torch.tensor(ln)[row]).to(DEV)
        s["slot"] = table[row.to(DEV), pos // P].long() * P + pos % P
        s["k_new"], s["v_new"] = (torch.randn((T, Hkv, d), dtype=TYPES[case["x"]], device=DEV, generator=g)
                                  for _ in range(2))
        s["kbar"] = _means(s["k"], s["k_scale"]) if case["means"] else None
        return s
    H = case["H"]
    s["kv_len"] = torch.tensor(ln, dtype=torch.int32, device=DEV)
    s["scale"] = d ** -0.5
    s["qx"] = (torch.randn((R, H, d), device=DEV, generator=g) * 1.5).to(TYPES[case["q"]])
    s["o"] = torch.zeros((R, H, d), dtype=TYPES[case["q"]], device=DEV)
    s["lse"] = torch.zeros((R, H), dtype=torch.float32, device=DEV)
    if case["kind"] == "sparse":
        s["kbar"] = _means(s["k"], s["k_scale"])
        s["sel"] = torch.empty((R, Hkv, case["topk"]), dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _plain_map(s):
    P, table, free, cap = s["P"], s["table"], s["free"], s["cap"]
    N, W = free.shape[0], table.shape[1]
    new = s["new_len"]
    base, add = s["kv_len"].clamp(min=0), new.clamp(min=0)
    ends = new < 0
    had, has = (base + P - 1) // P, (base + add + P - 1) // P
    need, back = torch.where(ends, 0, has - had), torch.where(ends, had, 0)
    need_at, back_at = need.cumsum(0) - need, back.cumsum(0) - back
    taken, returned = s["ring"][0], s["ring"][1]
    j = torch.arange(W, device=table.device)[None]
    gone = ends[:, None] & (j < had[:, None])
    to = (returned + back_at[:, None] + j) % N
    free[to[gone]] = table[gone]
    fresh = ~ends[:, None] & (j >= had[:, None]) & (j < has[:, None])
    at = (taken + need_at[:, None] + j - had[:, None]) % N
    table.copy_(torch.where(fresh, free[at], table))
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)]).to(torch.int32)
    t = torch.arange(cap, device=table.device)
    live = t < cu[-1]
    row = torch.searchsorted(cu[1:], t, right=True).clamp(max=table.shape[0] - 1)
    pos = base[row] + t - cu[row]
    page = torch.where(live, pos // P, 0)
    slot = table[row, page].long() * P + pos % P
    ln = torch.where(ends | ((s["kv_len"] < 0) & (add == 0)), -1, base + add)
    return {"kv_len": ln.to(torch.int32), "ring": torch.stack([taken + need.sum(), returned + back.sum()]),
            "slot": torch.where(live, slot, -1), "row": torch.where(live, row, -1).to(torch.int32),
            "pos": torch.where(live, pos, -1).to(torch.int32), "cu": cu, "table": table, "free": free}


def _stored(x, scale, to):
    x = x.float()
    if to != torch.float8_e4m3fn:
        return x.to(to)
    return (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(to)


def _plain_append(s):
    P, k, v, slot = s["P"], s["k"], s["v"], s["slot"]
    page, off = slot // P, slot % P
    k[page, off] = _stored(s["k_new"], s["k_scale"], k.dtype)
    v[page, off] = _stored(s["v_new"], s["v_scale"], v.dtype)
    if s["kbar"] is None:
        return {"k": k, "v": v}
    ends = torch.cat([page[1:] != page[:-1], page.new_ones(1, dtype=torch.bool)])
    pages, n = page[ends], off[ends] + 1
    rows = k[pages].float()
    inside = torch.arange(P, device=k.device)[None] < n[:, None]
    mean = torch.where(inside[:, :, None, None], rows, 0).sum(1) / n[:, None, None]
    if s["k_scale"] is not None:
        mean = mean * s["k_scale"][None, :, None]
    s["kbar"][pages] = mean
    return {"k": k, "v": v, "kbar": s["kbar"]}


def _softmax_v(sc, seen, v):
    """sc [..., G, L] scores, seen [..., 1, L], v [..., L, d]: (softmax(sc) v, log-sum-exp)."""
    sc = torch.where(seen, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return o, (m + torch.log(total))[..., 0]


def _finish(s, o, lse):
    R, H, d = s["qx"].shape
    kept = (s["kv_len"] < 0)[:, None]
    o = torch.where(kept[:, :, None], s["o"], o.reshape(R, H, d).to(s["o"].dtype))
    return o, torch.where(kept, s["lse"], lse.reshape(R, H))


def _values(x, scale, at):
    """Cached rows as 32-bit values, [R, Hkv, L, d]; `at` says which of them count."""
    x = x.float()
    if scale is not None:
        x = x * scale[:, None, None]
    return torch.where(at, x, 0.0)


def _plain_attn(s):
    R, H, d = s["qx"].shape
    Hkv, P, W = s["Hkv"], s["P"], s["table"].shape[1]
    q = s["qx"].float().view(R, Hkv, H // Hkv, d)
    pages = s["table"].clamp(min=0).long()
    pos = torch.arange(W * P, device=q.device)[None]
    n = s["kv_len"][:, None]
    seen = pos < n
    if s["window"]:
        seen = seen & ((pos < s["sink"]) | (pos >= n - s["window"]))
    seen = seen[:, None, :, None]
    k = _values(s["k"][pages].view(R, W * P, Hkv, d).transpose(1, 2), s["k_scale"], seen)
    sc = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    v = _values(s["v"][pages].view(R, W * P, Hkv, d).transpose(1, 2), s["v_scale"], seen)
    return dict(zip(("o", "lse"), _finish(s, *_softmax_v(sc, seen.transpose(2, 3), v))))


def _plain_select(s):
    R, H, d = s["qx"].shape
    Hkv, P, W, topk = s["Hkv"], s["P"], s["table"].shape[1], s["topk"]
    q = s["qx"].double().view(R, Hkv, H // Hkv, d).sum(2)
    kbar = s["kbar"][s["table"].clamp(min=0).long()].double()
    score = (kbar * q[:, None]).sum(-1).transpose(1, 2)  # [R, Hkv, W]
    n = ((s["kv_len"].clamp(min=0) + P - 1) // P)[:, None, None]
    j = torch.arange(W, device=q.device).expand(R, Hkv, W)
    score = torch.where((j < s["first"]) | (j >= n - s["last"]), math.inf, score)
    score = torch.where(j < n, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :topk]
    best = torch.where(best < n, best, W)
    if best.shape[-1] < topk:
        best = torch.cat([best, best.new_full((R, Hkv, topk - best.shape[-1]), W)], -1)
    best = best.sort(-1).values
    return torch.where(best < W, best, -1).to(torch.int32)


def _plain_sparse(s):
    R, H, d = s["qx"].shape
    Hkv, P, topk = s["Hkv"], s["P"], s["topk"]
    sel = _plain_select(s)
    q = s["qx"].float().view(R, Hkv, H // Hkv, d)
    pages = torch.gather(s["table"][:, None].expand(R, Hkv, -1), 2, sel.clamp(min=0).long()).clamp(min=0).long()
    heads = torch.arange(Hkv, device=q.device)[None, :, None]
    pos = sel[..., None] * P + torch.arange(P, device=q.device)
    seen = ((sel[..., None] >= 0) & (pos < s["kv_len"][:, None, None, None])).view(R, Hkv, topk * P, 1)
    k = _values(s["k"][pages, :, heads].view(R, Hkv, topk * P, d), s["k_scale"], seen)
    v = _values(s["v"][pages, :, heads].view(R, Hkv, topk * P, d), s["v_scale"], seen)
    sc = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    o, lse = _finish(s, *_softmax_v(sc, seen.transpose(2, 3), v))
    return {"sel": sel, "o": o, "lse": lse}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _own(s):
    from kv_cache_attention_chunk_b200 import vkv

    kind = s["kind"]
    if kind == "map":
        out = vkv.page_map(s["kv_len"], s["new_len"], s["table"], s["free"], s["ring"], s["P"], s["cap"], out=s["out"])
        return {**out, "table": s["table"], "free": s["free"]}
    if kind == "append":
        vkv.page_append(s["k_new"], s["v_new"], s["slot"], s["k"], s["v"], k_scale=s["k_scale"],
                        v_scale=s["v_scale"], kbar=s["kbar"])
        return {"k": s["k"], "v": s["v"]} if s["kbar"] is None else {"k": s["k"], "v": s["v"], "kbar": s["kbar"]}
    if kind == "attn":
        o, lse = vkv.page_attn(s["qx"], s["k"], s["v"], s["table"], s["kv_len"], scale=s["scale"], sink=s["sink"],
                               window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=(s["o"], s["lse"]))
        return {"o": o, "lse": lse}
    sel = vkv.page_select(s["qx"], s["kbar"], s["table"], s["kv_len"], s["P"], s["topk"], sink_pages=s["first"],
                          local_pages=s["last"], out=s["sel"])
    o, lse = vkv.page_attn(s["qx"], s["k"], s["v"], s["table"], s["kv_len"], scale=s["scale"], sel=sel,
                           k_scale=s["k_scale"], v_scale=s["v_scale"], out=(s["o"], s["lse"]))
    return {"sel": sel, "o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"map": _plain_map, "append": _plain_append, "attn": _plain_attn, "sparse": _plain_sparse}[state["kind"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    R, P, kind = case["R"], case["P"], case["kind"]
    pages = lambda n: -(-max(n, 0) // P)  # noqa: E731
    if kind == "map":
        ln, new = _map_lengths(case)
        tokens = sum(max(b, 0) for b in new)
        moved = sum(pages(a) if b < 0 else pages(max(a, 0) + b) - pages(a) for a, b in zip(ln, new))
        return {"bytes": 16 * tokens + 8 * moved + 16 * R + 36, "flops": 0}
    Hkv, d, e = case["Hkv"], case["d"], BYTES[case["kv"]]
    if kind == "append":
        ln, new = _spread(R, case["lo"], case["hi"]), _spread(R, case["new_lo"], case["new_hi"])
        tokens = sum(new)
        b = tokens * (8 + 2 * Hkv * d * (2 + e))
        if case["means"]:  # the earlier rows of each row's first page, and a mean for each page written
            b += Hkv * d * sum(e * (a % P) + 4 * (pages(a + n) - a // P) for a, n in zip(ln, new))
        return {"bytes": b, "flops": 2 * tokens * Hkv * d}
    H, ln = case["H"], _lengths(case)
    b = sum(4 + (H * (2 * d * 2 + 4) if n >= 0 else 0) for n in ln)
    if kind == "attn":
        seen = [max(n, 0) for n in ln]
        if case["window"]:
            seen = [min(n, case["sink"] + case["window"]) for n in seen]
        tokens = sum(seen)
        b += sum(4 * -(-n // P) for n in seen) + tokens * Hkv * 2 * d * e
        return {"bytes": b, "flops": 4 * tokens * H * d}
    tokens = 0
    for n in ln:
        k = min(case["topk"], pages(n))
        tokens += k * P - (pages(n) * P - max(n, 0))
        b += 4 * pages(n) + 4 * case["topk"] * Hkv
        b += pages(n) * Hkv * d * 4 if pages(n) > case["topk"] else 0
    return {"bytes": b + tokens * Hkv * 2 * d * e, "flops": 4 * tokens * H * d}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, row by row
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["kind"] == "map":
        return None  # whole numbers only
    s = prepare(case, seed)
    P, Hkv, d = case["P"], case["Hkv"], case["d"]
    one = torch.ones(Hkv, dtype=torch.float64, device=DEV)
    ks, vs = (one if s[x] is None else s[x].double() for x in ("k_scale", "v_scale"))
    if case["kind"] == "append":
        k, v = s["k"].double(), s["v"].double()
        kn, vn = s["k_new"].double() / ks[:, None], s["v_new"].double() / vs[:, None]
        if case["kv"] == "e4m3":
            kn, vn = kn.clamp(-E4M3_MAX, E4M3_MAX), vn.clamp(-E4M3_MAX, E4M3_MAX)
        slot = s["slot"]
        k.view(-1, Hkv, d)[slot] = kn
        v.view(-1, Hkv, d)[slot] = vn
        if not case["means"]:
            return {"k": k, "v": v}
        mean = s["kbar"].double()
        held = s["k"].double()
        held.view(-1, Hkv, d)[slot] = kn.to(TYPES[case["kv"]]).double()  # the mean is of what the cache holds
        last = {}
        for x in slot.tolist():
            last[x // P] = x % P
        for page, off in last.items():
            mean[page] = held[page, :off + 1].mean(0) * ks[:, None]
        return {"k": k, "v": v, "kbar": mean}
    R, H = case["R"], case["H"]
    o = torch.zeros((R, H, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((R, H), dtype=torch.float64, device=DEV)
    sel = torch.full((R, Hkv, case.get("topk", 1)), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate(s["kv_len"].tolist()):
        if n < 0:
            continue
        if n == 0:
            lse[r] = -math.inf
            continue
        count = -(-n // P)
        pages = s["table"][r, :count].long()
        q = s["qx"][r].double().view(Hkv, H // Hkv, d)
        if case["kind"] == "attn":
            pos = torch.arange(n, device=DEV)
            if case["window"]:
                pos = pos[(pos < case["sink"]) | (pos >= n - case["window"])]
            flat = pages[pos // P] * P + pos % P
            rows = [flat] * Hkv
        else:
            points = torch.einsum("gad,pgd->gp", q, s["kbar"][pages].double())
            rows = []
            for h in range(Hkv):
                free = [j for j in range(count) if case["first"] <= j < count - case["last"]]
                forced = [j for j in range(count) if not case["first"] <= j < count - case["last"]]
                value = points[h].tolist()
                best = sorted(free, key=lambda j: (-value[j], j))
                kept = sorted((forced + best)[:case["topk"]])
                sel[r, h, :len(kept)] = torch.tensor(kept, dtype=torch.int32, device=DEV)
                pos = (torch.tensor(kept, device=DEV)[:, None] * P + torch.arange(P, device=DEV)).view(-1)
                pos = pos[pos < n]
                rows.append(pages[pos // P] * P + pos % P)
        for h in range(Hkv):
            k = s["k"].view(-1, Hkv, d)[rows[h], h].double() * ks[h]
            v = s["v"].view(-1, Hkv, d)[rows[h], h].double() * vs[h]
            z = q[h] @ k.T * s["scale"]
            w = torch.softmax(z, -1)
            o[r].view(Hkv, H // Hkv, d)[h] = w @ v
            lse[r].view(Hkv, H // Hkv)[h] = torch.logsumexp(z, -1)
    out = {"o": o, "lse": lse}
    return out if case["kind"] == "attn" else {"sel": sel, **out}
