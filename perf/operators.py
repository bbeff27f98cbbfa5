"""The operators of a serving step around the NVFP4 projections, as measured cases.

* plan: page tables and slot maps of a paged cache, built on the GPU from
  request lengths (nvfp4_kv_release, nvfp4_kv_plan);
* append: K and V rows quantized into the 4-bit cache and read back as the
  values they stand for (nvfp4_kv_append, nvfp4_kv_read);
* attention: softmax(q K^T scale) V over the 4-bit cache, causal within a
  request, optionally within a window (nvfp4_kv_attention);
* logits: penalties for repeated tokens, biases and grammar masks in front of
  the sampler (nvfp4_process_logits).

Cache layout, shared by all cases (D the head size, 64 or 128): pages are
uint8 [pages, kv heads, page/16 groups, 18 D]; a group holds 16 tokens of one
head as K codes (8 D bytes), K scales (D), V codes (8 D), V scales (D).  An
E2M1 code is 4 bits (the even element in the low nibble), a scale is E4M3, one
per 16 elements, and x = code * scale * global.  Token t of a group stands at

* K codes   [pos][D/2 bytes], pos = 8 (t/2 mod 2) + 2 (t/4) + t mod 2
* K scales  [r 8][c 4][i 2][D/64], pos = 8 i + r, block = c D/64 + last
* V codes   D = 128: [4][i 2][2][c 4][2][8 bytes], t = 4 c + 2 i + last but one,
            bytes of elements 16 r .. 16 r + 15 at r = 2 first + third;
            D = 64: [r 8][t 16][4 bytes], elements 8 r .. 8 r + 7
* V scales  [block][t]
"""
import math

import numpy as np
import torch

own = False

QWEN3_32B_HEADS = (64, 8)      # query and kv heads behind the qkv projection 5120 -> 10240
QWEN3_14B_HEADS = (40, 8)
QWEN3_8B_HEADS = (32, 8)
VOCAB = 151936


# ---- the cases ------------------------------------------------------------------
def listed():
    h32, k32 = QWEN3_32B_HEADS
    h14, k14 = QWEN3_14B_HEADS
    h8, k8 = QWEN3_8B_HEADS
    return [
        # a decode step's bookkeeping for the library's largest decode batch
        {"name": "plan-decode", "op": "plan", "batch": 8, "page": 64, "ctx": 4096, "prefill_every": 0, "chunk": 0,
         "done": 0},
        # a loaded server: hundreds of requests, every second one prefilling a chunk, some ended and replaced
        {"name": "plan-mixed", "op": "plan", "batch": 1024, "page": 32, "ctx": 32768, "prefill_every": 2,
         "chunk": 512, "done": 64},
        # one decode step's rows, a slice of the FP32 qkv output
        {"name": "append-decode", "op": "append", "tokens": 8, "heads": k32, "dim": 128, "page": 64, "dtype": "f32",
         "query_heads": h32, "pad": 0},
        # a long prompt in one call
        {"name": "append-prefill", "op": "append", "tokens": 16384, "heads": k32, "dim": 128, "page": 64,
         "dtype": "bf16", "query_heads": h32, "pad": 100},
        # one user, a short conversation: latency
        {"name": "attention-one", "op": "attention", "batch": 1, "heads": h32, "kv_heads": k32, "dim": 128, "page": 64,
         "shortest": 1000, "longest": 1000, "query": 1, "window": 0, "dtype": "bf16"},
        # a decode batch of very different lengths, one request empty, five query heads to a kv head
        {"name": "attention-ragged", "op": "attention", "batch": 8, "heads": h14, "kv_heads": k14, "dim": 128,
         "page": 32, "shortest": 0, "longest": 8191, "query": 1, "window": 0, "dtype": "f32"},
        # long reasoning traces
        {"name": "attention-long", "op": "attention", "batch": 8, "heads": h32, "kv_heads": k32, "dim": 128,
         "page": 64, "shortest": 131000, "longest": 131072, "query": 1, "window": 0, "dtype": "bf16"},
        # many requests, small heads that share nothing, a sliding window over small pages
        {"name": "attention-window", "op": "attention", "batch": 64, "heads": 16, "kv_heads": 16, "dim": 64,
         "page": 16, "shortest": 17, "longest": 4097, "query": 1, "window": 1024, "dtype": "bf16"},
        # drafted tokens verified: up to 8 query rows a request
        {"name": "attention-verify", "op": "attention", "batch": 16, "heads": h8, "kv_heads": k8, "dim": 128,
         "page": 64, "shortest": 500, "longest": 16384, "query": 8, "window": 0, "dtype": "bf16"},
        # prompt chunks over what is cached already
        {"name": "attention-prefill", "op": "attention", "batch": 2, "heads": h32, "kv_heads": k32, "dim": 128,
         "page": 64, "shortest": 4096, "longest": 8192, "query": 1024, "window": 0, "dtype": "bf16"},
        # one user's logits
        {"name": "logits-one", "op": "logits", "rows": 1, "vocab": VOCAB, "history": 700, "bias": 16, "masked": 0,
         "dtype": "f32"},
        # the sampler's largest batch after long outputs, half of it under a grammar
        {"name": "logits-batch", "op": "logits", "rows": 64, "vocab": VOCAB, "history": 16384, "bias": 300,
         "masked": 32, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.25 / hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "logits"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        batch = _log(rng, 1, 1024)
        return {"op": op, "batch": batch, "page": max(32, page), "ctx": _log(rng, 16, 32768),
                "prefill_every": rng.choice([0, 0, 1, 2, 5]), "chunk": _log(rng, 2, 256), "done": rng.randint(0, batch // 4)}
    if op == "append":
        heads = rng.choice([1, 2, 4, 8])
        tokens = _log(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "heads": heads, "dim": rng.choice([64, 128]), "page": page,
                "dtype": rng.choice(["bf16", "f32"]) if tokens <= 8192 else "bf16", "query_heads": heads * rng.randint(1, 8),
                "pad": rng.randint(0, tokens // 4)}
    if op == "attention":
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        case = {"op": op, "kv_heads": kv_heads, "heads": kv_heads * group, "dim": rng.choice([64, 128]), "page": page,
                "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "dtype": rng.choice(["bf16", "f32"])}
        kind = rng.choice(["decode", "decode", "verify", "prefill"])
        if kind == "decode":
            batch, query = _log(rng, 1, 64), 1
            longest = _log(rng, 1, min(131072, 1048576 // batch))
        elif kind == "verify":
            batch, query = _log(rng, 1, 32), rng.randint(2, 8)
            longest = _log(rng, query, 262144 // batch)
        else:
            query, group = _log(rng, 9, 1024), min(group, 8)
            batch = rng.randint(1, max(1, min(4, 1024 // query)))
            longest = _log(rng, query, 8192)
            case["heads"] = kv_heads * group
        return {**case, "batch": batch, "query": query, "longest": longest,
                "shortest": min(longest, rng.choice([0, query, longest // 2, longest]))}
    rows = _log(rng, 1, 64)
    vocab = _log(rng, 1000, 200000)
    return {"op": op, "rows": rows, "vocab": vocab, "history": _log(rng, 1, 16384), "bias": rng.randint(0, 300),
            "masked": rng.choice([0, rng.randint(0, rows), rows]), "dtype": rng.choice(["f32", "bf16"])}


# ---- lengths, fixed by the case (the seed only shuffles them) ----------------------
def _spread(lo, hi, n):
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _plan_lens(case):
    """Per request: tokens held, whether it has ended, tokens in the cache and new tokens of this step.  The row
    of a request that has ended stays empty in this step; the row behind it starts a new prompt."""
    n, every = case["batch"], case["prefill_every"]
    ends = {i * n // case["done"] for i in range(case["done"])}
    starts = {i + 1 for i in ends} - ends
    held = [0 if i in starts else h + (7 * i) % 13 for i, h in enumerate(_spread(1, case["ctx"], n))]
    new = [0 if i in ends else 1 + case["ctx"] // 9 if i in starts else
           1 if not every or i % every else 1 + (case["chunk"] * (3 + i % 5)) // 7 for i in range(n)]
    return held, [int(i in ends) for i in range(n)], [0 if i in ends else h for i, h in enumerate(held)], new


def _attention_lens(case):
    """Per request: keys and query rows."""
    keys = _spread(case["shortest"], case["longest"], case["batch"])
    if case["query"] == 1:
        return keys, [1] * case["batch"]
    return keys, [case["query"] - (i * 3) % (1 + case["query"] // 2) for i in range(case["batch"])]


def _pairs(case):
    """(visible query-key pairs of one query head, keys of one kv head that are read)."""
    keys, rows = (np.array(v, dtype=np.int64) for v in _attention_lens(case))
    i = np.arange(rows.max())
    seen = np.clip((keys - rows)[:, None] + i + 1, 0, None) * (i < rows[:, None])
    first = np.zeros_like(keys)
    if case["window"]:
        seen = np.minimum(seen, case["window"])
        first = np.clip(keys - rows - case["window"] + 1, 0, None)
    return int(seen.sum()), int(np.clip(keys - first, 0, None).sum())


def work(case):
    if case["op"] == "plan":
        held, ended, ctx, new = _plan_lens(case)
        pg = case["page"]
        taken = sum(-(-(c + q) // pg) - -(-c // pg) for c, q in zip(ctx, new))
        freed = sum(-(-h // pg) for h, e in zip(held, ended) if e)
        # the lengths; pages given back (read from the table, pushed); pages taken (popped, written to the table);
        # the cached part's last page of each request; slot and position of each new token; row starts and lengths
        return {"bytes": 4 * (4 * case["batch"] + 2 * freed + 2 * taken + case["batch"] + 2 * sum(new) + 2 * case["batch"])}
    if case["op"] == "append":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        live = t - case["pad"]
        size = 4 if case["dtype"] == "f32" else 2
        # rows in, 9/16 byte an element written and read back, BF16 rows out
        return {"bytes": 4 * t + 2 * live * h * d * size + 2 * (2 * live * h * d * 9 // 16) + 2 * t * h * d * 2}
    if case["op"] == "attention":
        pairs, read = _pairs(case)
        rows = sum(_attention_lens(case)[1])
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": read * case["kv_heads"] * case["dim"] * 18 // 16 + rows * case["heads"] * case["dim"] * (size + 2),
                "flops": 4 * case["heads"] * case["dim"] * pairs}
    m, v = case["rows"], case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": m * v * (size + 4) + case["masked"] * ((v + 31) // 32) * 4 + m * case["history"] * 4 + m * case["bias"] * 8}


# ---- inputs ---------------------------------------------------------------------
def _round_e2m1(a):
    """E2M1 code (0..7) of non-negative values, ties to the even code, saturating."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _quantize(x, glob):
    """FP32 [..., D] -> code bytes [..., D/2], scale bytes [..., D/16], in FP32 step by step."""
    b = x.unflatten(-1, (-1, 16))
    most = b.abs().amax(-1)
    s8 = (most / (6.0 * glob)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s8.float() * glob).unsqueeze(-1)
    code = torch.where(step > 0, _round_e2m1(b.abs() / step), 0) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), s8.view(torch.uint8)


def _sections(pages, dim):
    """Views of the pages' four sections, cut as the layout above says."""
    k, ks, v, vs = pages.split([8 * dim, dim, 8 * dim, dim], dim=-1)
    v = v.unflatten(-1, (4, 2, 2, 4, 2, 8)) if dim == 128 else v.unflatten(-1, (8, 16, 4))
    return (k.unflatten(-1, (16, dim // 2)), ks.unflatten(-1, (8, 4, 2, dim // 64)), v,
            vs.unflatten(-1, (dim // 16, 16)))


def _store(pages, dim, page, slots, k, v, k_glob, v_glob):
    """Quantizes rows [T, heads, dim] into the pages at their slots."""
    kc, ks, vc, vs = _sections(pages, dim)
    pg, at = slots // page, slots % page
    g, t = at // 16, at % 16
    c, i, lo = t // 4, t // 2 % 2, t % 2
    r = 2 * c + lo
    codes, scales = _quantize(k, k_glob)
    kc[pg, :, g, 8 * i + r] = codes
    ks[pg, :, g, r, :, i] = scales.unflatten(-1, (4, -1))
    codes, scales = _quantize(v, v_glob)
    if dim == 128:
        vc[pg, :, g, :, i, :, c, lo] = codes.unflatten(-1, (4, 2, 8))
    else:
        vc[pg, :, g, :, t] = codes.unflatten(-1, (8, 4))
    vs[pg, :, g, :, t] = scales


def _load(pages, dim, page, slots, k_glob, v_glob):
    """The FP32 values [..., heads, dim] of K and V at slots [...]."""
    kc, ks, vc, vs = _sections(pages, dim)
    pg, at = slots // page, slots % page
    g, t = at // 16, at % 16
    c, i, lo = t // 4, t // 2 % 2, t % 2
    r = 2 * c + lo
    k = _values(kc[pg, :, g, 8 * i + r], ks[pg, :, g, r, :, i].flatten(-2), k_glob)
    vcode = vc[pg, :, g, :, i, :, c, lo].flatten(-3) if dim == 128 else vc[pg, :, g, :, t].flatten(-2)
    return k, _values(vcode, vs[pg, :, g, :, t], v_glob)


def _values(codes, scales, glob):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    x = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 16))
    return (x * (scales.view(torch.float8_e4m3fn).float() * glob).unsqueeze(-1)).flatten(-2)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g, torch.Generator().manual_seed(seed)


def _rows(g, shape, spread=1.0):
    """Activations: normal, one channel in a hundred twelve times as large, magnitudes changing from token to token."""
    x = torch.randn(shape, generator=g, device="cuda") * spread
    x[..., 5::100] *= 12.0
    return x * torch.exp(0.5 * torch.randn((shape[0],) + (1,) * (len(shape) - 1), generator=g, device="cuda"))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, host = _gen(seed)
    s = dict(case)
    if case["op"] == "plan":
        held, ended, ctx, new = _plan_lens(case)
        order = torch.randperm(case["batch"], generator=host).tolist()
        held, ended, ctx, new = ([v[i] for i in order] for v in (held, ended, ctx, new))
        pg = case["page"]
        used = [-(-h // pg) for h in held]
        need = sum(-(-(c + q) // pg) - -(-c // pg) for c, q in zip(ctx, new))
        total = sum(used) + need + 17
        width = max(-(-max(h, c + q) // pg) for h, c, q in zip(held, ctx, new)) + 1
        pages = torch.randperm(total, generator=host).int()
        table = torch.full((case["batch"], width), -1, dtype=torch.int32)
        # the first pages are held, request after request; the rest are free
        live = torch.arange(width)[None] < torch.tensor(used)[:, None]
        table[live] = pages[:sum(used)]
        stack = torch.full((total,), -1, dtype=torch.int32)
        stack[:total - sum(used)] = pages[sum(used):]
        n = sum(new)
        s.update(held=_ints(held), ended=torch.tensor(ended, dtype=torch.uint8, device="cuda"), ctx_lens=_ints(ctx),
                 new_lens=_ints(new), table=table.cuda(), stack=stack.cuda(), count=_ints([total - sum(used)]), n=n,
                 out=[torch.empty(k, dtype=torch.int32, device="cuda")
                      for k in (n, n, case["batch"] + 1, case["batch"], 1, 1, 2)])
        return s
    if case["op"] == "append":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        s["dt"] = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # K and V are column slices of one projection's output, behind the query columns
        cols = case["query_heads"] * d
        x = torch.zeros((t, cols + 2 * h * d), dtype=s["dt"], device="cuda")
        x[:, cols:] = _rows(g, (t, 2 * h * d)).to(s["dt"])
        live = t - case["pad"]
        # request after request from the start of a page, the pages in no order; padding at the end
        per = -(-live // 3)
        starts = -(-per // case["page"]) * case["page"]
        n_pages = max(1, 3 * starts // case["page"])
        pos = torch.arange(live)
        logical = pos // per * starts + pos % per
        perm = torch.randperm(n_pages, generator=host)
        slots = torch.full((t,), -1, dtype=torch.int64)
        slots[:live] = perm[logical // case["page"]] * case["page"] + logical % case["page"]
        s.update(k=x[:, cols:cols + h * d].unflatten(-1, (h, d)), v=x[:, cols + h * d:].unflatten(-1, (h, d)),
                 slots=slots.int().cuda(), n_pages=n_pages, k_global=torch.tensor([0.5], device="cuda"),
                 v_global=torch.tensor([0.125], device="cuda"),
                 # one page more than the cache has: the plain form writes its padding there
                 pages=torch.zeros((n_pages + 1, h, case["page"] // 16, 18 * d), dtype=torch.uint8, device="cuda"))
        return s
    if case["op"] == "attention":
        d, h, hk, pg = case["dim"], case["heads"], case["kv_heads"], case["page"]
        keys, rows = _attention_lens(case)
        order = torch.randperm(case["batch"], generator=host).tolist()
        keys, rows = [keys[i] for i in order], [rows[i] for i in order]
        used = [-(-n // pg) for n in keys]
        width = max(1, max(used))
        perm = torch.randperm(sum(used) + 3, generator=host)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32)
        table[torch.arange(width)[None] < torch.tensor(used)[:, None]] = perm[:sum(used)].int()
        pages = torch.empty((sum(used) + 3, hk, pg // 16, 18 * d), dtype=torch.uint8, device="cuda")
        s.update(k_global=torch.tensor([0.25], device="cuda"), v_global=torch.tensor([0.125], device="cuda"))
        step = max(1, (1 << 25) // (hk * d) // pg)                       # pages filled at a time
        for a in range(0, pages.shape[0], step):
            part = pages[a:a + step]
            at = torch.arange(part.shape[0] * pg, device="cuda")
            _store(part, d, pg, at, _rows(g, (at.numel(), hk, d)), torch.randn((at.numel(), hk, d), generator=g, device="cuda"),
                   s["k_global"], s["v_global"])
        total = sum(rows)
        # queries are the first columns of the projection's output
        x = torch.zeros((total, (h + 2 * hk) * d), device="cuda")
        x[:, :h * d] = 1.5 * torch.randn((total, h * d), generator=g, device="cuda")
        x = x if case["dtype"] == "f32" else x.bfloat16()
        starts = [0] + np.cumsum(rows).tolist()
        s.update(q=x[:, :h * d].unflatten(-1, (h, d)), pages=pages, table=table.cuda(), lens=_ints(keys),
                 starts=_ints(starts), most_keys=max(keys), most_rows=max(rows), scale=1.0 / math.sqrt(d),
                 out=torch.empty((total, h, d), dtype=torch.bfloat16, device="cuda"))
        return s
    m, v, n = case["rows"], case["vocab"], case["history"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    s["logits"] = (3.0 * torch.randn((m, v), generator=g, device="cuda")).to(dt)
    # tokens repeat as in text: a few are frequent
    s["tokens"] = (v * torch.rand((m, n), generator=g, device="cuda") ** 4).int().clamp(max=v - 1)
    used = [max(1, n - (i * n) // (2 * m)) for i in range(m)]
    s["n_tokens"], s["n_prompt"] = _ints(used), _ints([u // 3 for u in used])
    s["repetition"] = 1.0 + 0.3 * torch.rand(m, generator=g, device="cuda")
    s["presence"] = torch.rand(m, generator=g, device="cuda")
    s["frequency"] = 0.2 * torch.rand(m, generator=g, device="cuda")
    b = min(case["bias"], v)
    at = (torch.arange(b, device="cuda")[None] * (v // max(1, b)) + torch.randint(0, v // max(1, b), (m, b), generator=g, device="cuda"))
    at[:, b - b // 5:] = -1                                            # rows with fewer biases than others
    s["bias_ids"], s["bias_values"] = at.int(), 4.0 * torch.randn((m, b), generator=g, device="cuda")
    words = (v + 31) // 32
    # grammars allow few tokens: about one in eight
    w = [torch.randint(-2**31, 2**31, (max(1, case["masked"]), words), generator=g, device="cuda") for _ in range(3)]
    s["mask"] = (w[0] & w[1] & w[2]).int()
    rows = torch.randperm(m, generator=host)
    s["mask_rows"] = torch.where(rows < case["masked"], rows, -1).int().cuda()
    s["out"] = torch.empty((m, v), device="cuda")
    return s


# ---- one pass -------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "plan":
        return _plain_plan(s)
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "attention":
        return _plain_attention(s)
    return _plain_logits(s)


def _plain_plan(s):
    pg, width = s["page"], s["table"].shape[1]
    cols = torch.arange(width, device="cuda")
    # pages of ended requests go back on the stack, request after request
    held = torch.where(s["ended"] > 0, -(-s["held"] // pg), 0)
    before = held.cumsum(0) - held
    back = torch.where(cols < held[:, None], s["count"] + before[:, None] + cols, s["stack"].numel()).long()
    stack = torch.cat([s["stack"], s["stack"][:1]]).scatter(0, back.flatten(), s["table"].flatten())[:-1]
    count = s["count"] + held.sum()
    # new pages come from its top
    old, now = -(-s["ctx_lens"] // pg), -(-(s["ctx_lens"] + s["new_lens"]) // pg)
    need = now - old
    last = need.cumsum(0)
    refused = (need > 0) & (last > count)
    take = (count - 1 - (last - need)[:, None] - (cols - old[:, None])).clamp(0, s["stack"].numel() - 1).long()
    fresh = (cols >= old[:, None]) & (cols < now[:, None]) & ~refused[:, None]
    table = torch.where(fresh, stack[take], s["table"])
    starts = torch.cat([torch.zeros_like(count), s["new_lens"].cumsum(0)])
    row = torch.repeat_interleave(torch.arange(s["batch"], device="cuda"), s["new_lens"], output_size=s["n"])
    pos = torch.arange(s["n"], device="cuda") - starts[row] + s["ctx_lens"][row]
    slots = torch.where(refused[row], -1, table[row, pos // pg] * pg + pos % pg)
    kv = torch.where(refused, s["ctx_lens"], s["ctx_lens"] + s["new_lens"])
    left = count - torch.where(refused, 0, need).sum()
    return [t.int() for t in (stack, table, slots, pos, starts, kv, left, torch.stack([refused.sum(), starts[-1]]))]


def _plain_append(s):
    # what is written for padding goes to the page behind the cache's own
    at = torch.where(s["slots"] < 0, s["n_pages"] * s["page"], s["slots"])
    _store(s["pages"], s["dim"], s["page"], at, s["k"].bfloat16().float(), s["v"].bfloat16().float(), s["k_global"],
           s["v_global"])
    k, v = _load(s["pages"], s["dim"], s["page"], at, s["k_global"], s["v_global"])
    gone = (s["slots"] < 0)[:, None, None]
    return [torch.where(gone, 0.0, x).bfloat16() for x in (k, v)]


def _plain_attention(s):
    pg, hk, n, m = s["page"], s["kv_heads"], s["most_keys"], s["most_rows"]
    col = torch.arange(n, device="cuda")
    slot = (s["table"][:, col // pg].long().clamp(min=0) * pg + col % pg)                       # [B, n]
    k, v = _load(s["pages"], s["dim"], pg, slot, s["k_global"], s["v_global"])
    rows = s["starts"][1:] - s["starts"][:-1]
    row = torch.arange(m, device="cuda")
    live = row < rows[:, None]                                                                  # [B, m]
    at = torch.where(live, s["starts"][:-1, None] + row, 0).long()
    q = s["q"].bfloat16().float()[at].unflatten(2, (hk, -1))                                    # [B, m, hk, G, D]
    groups = q.shape[3]
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                                                  # [B, hk, m G, D]
    score = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).unflatten(2, (m, groups))              # [B, hk, m, G, n]
    pos = (s["lens"] - rows)[:, None] + row                                                     # [B, m]
    hidden = (col > pos[..., None]) | (col >= s["lens"][:, None, None])
    if s["window"]:
        hidden |= col <= pos[..., None] - s["window"]
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    most = score.amax(-1, keepdim=True).clamp(min=-1e30) if n else score.new_zeros(score.shape[:-1] + (1,))
    p = score.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((col < s["lens"][:, None])[..., None, None], v, 0.0)
    out = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (m, groups)) / torch.where(total > 0, total, 1.0)
    out = out.permute(0, 2, 1, 3, 4).flatten(2, 3).bfloat16()                                   # [B, m, h, D]
    # each live row to its place; the others to a row that is cut off
    to = torch.where(live, s["starts"][:-1, None] + row, s["q"].shape[0]).long().flatten()
    flat = torch.empty((s["q"].shape[0] + 1,) + out.shape[2:], dtype=out.dtype, device="cuda")
    return flat.index_copy(0, to, out.flatten(0, 1))[:-1]


def _plain_logits(s):
    m, v = s["logits"].shape
    x = s["logits"].float()
    col = torch.arange(s["tokens"].shape[1], device="cuda")
    ids = s["tokens"].long()
    zero = torch.zeros((m, v), device="cuda")
    seen = zero.scatter_add(1, ids, (col < s["n_tokens"][:, None]).float()) > 0
    count = zero.scatter_add(1, ids, ((col >= s["n_prompt"][:, None]) & (col < s["n_tokens"][:, None])).float())
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count
    x = torch.where(count > 0, x - s["presence"][:, None], x)
    x = x.scatter_add(1, s["bias_ids"].long().clamp(min=0), torch.where(s["bias_ids"] >= 0, s["bias_values"], 0.0))
    col = torch.arange(v, device="cuda")
    allowed = (s["mask"][s["mask_rows"].long().clamp(min=0)][:, col // 32] >> (col % 32)) & 1
    return x.masked_fill((allowed == 0) & (s["mask_rows"] >= 0)[:, None], -math.inf)


def _run_own(s):
    from nvfp4_w4a4_decode_gemv_gb300 import api
    if s["op"] == "plan":
        slots, pos, starts, kv, back, left, info = s["out"]
        api.nvfp4_kv_release(s["held"], s["ended"], s["table"], s["stack"], s["count"], s["page"], free_count_out=back)
        api.nvfp4_kv_plan(s["ctx_lens"], s["new_lens"], s["table"], s["stack"], back, s["page"],
                          out=api.KVPlan(slots, pos, starts, kv, left, info))
        return [s["stack"], s["table"], slots, pos, starts, kv, left, info]
    if "cache" not in s:                                               # the handle that a program keeps
        if s["op"] == "append":
            s["cache"] = api.NVFP4KVCache(s["pages"][:s["n_pages"]], s["k_global"], s["v_global"])
        elif s["op"] == "attention":
            s["cache"] = api.NVFP4KVCache(s["pages"], s["k_global"], s["v_global"])
    if s["op"] == "append":
        api.nvfp4_kv_append(s["k"], s["v"], s["slots"], s["cache"])
        return list(api.nvfp4_kv_read(s["cache"], s["slots"]))
    if s["op"] == "attention":
        return api.nvfp4_kv_attention(s["q"], s["cache"], s["table"], s["lens"], s["starts"] if s["query"] > 1 else None,
                                      max_q=s["most_rows"], scale=s["scale"], window=s["window"], out=s["out"])
    return api.nvfp4_process_logits(s["logits"], s["tokens"], s["n_tokens"], s["n_prompt"], s["repetition"],
                                    s["presence"], s["frequency"], s["bias_ids"], s["bias_values"], s["mask"],
                                    s["mask_rows"], out=s["out"])


# ---- the definitions, in 64 bits ---------------------------------------------------
_E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
_E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def _nearest(a, grid):
    """Index of the nearest grid value, ties to the even index; above the grid, the last."""
    hi = np.searchsorted(grid, a).clip(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _exact_rows(x, glob):
    """What rows of values stand for after quantization."""
    b = x.reshape(-1, 16)
    step = _E4M3[_nearest(np.abs(b).max(1) / (6 * glob), _E4M3)] * glob
    safe = np.where(step > 0, step, 1.0)[:, None]
    return (np.copysign(_E2M1[_nearest(np.abs(b) / safe, _E2M1)], b) * step[:, None]).reshape(x.shape)


def _exact_cache(s, slots):
    """K and V [n, heads, D] in FP64 at slots, byte by byte from the layout's offsets."""
    d, hk = s["dim"], s["kv_heads"]
    flat, per = s["pages"].view(-1), s["page"] // 16
    grid = torch.tensor(np.concatenate([_E2M1, -_E2M1]), device="cuda")
    e4m3 = torch.tensor(np.concatenate([_E4M3, [math.nan], -_E4M3, [math.nan]]), device="cuda")
    t = (slots % 16)[:, None, None]
    base = ((slots // s["page"])[:, None] * hk + torch.arange(hk, device="cuda")) * per + (slots % s["page"] // 16)[:, None]
    base = (base * (18 * d))[..., None]                                    # [n, heads, 1]
    e = torch.arange(d, device="cuda")
    pos = 8 * (t // 2 % 2) + 2 * (t // 4) + t % 2
    byte = flat[base + pos * (d // 2) + e // 2]
    block = e // 16
    nb = d // 64
    sc = flat[base + 8 * d + ((pos % 8) * 4 + block // nb) * 2 * nb + (pos // 8) * nb + block % nb]
    k = grid[((byte >> (4 * (e % 2)).to(torch.uint8)) & 15).long()] * e4m3[sc.long()] * s["k_global"].double()
    if d == 128:
        r = e // 16
        off = (((r // 2 * 2 + t // 2 % 2) * 2 + r % 2) * 4 + t // 4) * 16 + t % 2 * 8 + e % 16 // 2
    else:
        off = (e // 8 * 16 + t) * 4 + e % 8 // 2
    byte = flat[base + 9 * d + off]
    sc = flat[base + 17 * d + block * 16 + t]
    v = grid[((byte >> (4 * (e % 2)).to(torch.uint8)) & 15).long()] * e4m3[sc.long()] * s["v_global"].double()
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                                        # whole numbers, compared as they are
    if case["op"] == "append":
        gone = (s["slots"] < 0).cpu().numpy()[:, None, None]
        return [np.where(gone, 0.0, _exact_rows(s[n].bfloat16().double().cpu().numpy(), float(s[n + "_global"])))
                for n in ("k", "v")]
    if case["op"] == "attention":
        out = torch.zeros((s["q"].shape[0], case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
        lens, starts = s["lens"].tolist(), s["starts"].tolist()
        group = case["heads"] // case["kv_heads"]
        for b, n in enumerate(lens):
            if n == 0:
                continue
            col = torch.arange(n, device="cuda")
            k, v = _exact_cache(s, s["table"][b][col // case["page"]].long() * case["page"] + col % case["page"])
            q = s["q"][starts[b]:starts[b + 1]].bfloat16().double()
            pos = n - q.shape[0] + torch.arange(q.shape[0], device="cuda")[:, None]
            seen = col <= pos
            if case["window"]:
                seen &= col > pos - case["window"]
            some = seen.any(1)
            for h in range(case["heads"]):
                p = (q[:, h] @ k[:, h // group].T * s["scale"]).masked_fill(~seen, -math.inf)
                p = torch.softmax(torch.where(some[:, None], p, 0.0), -1)
                out[starts[b]:starts[b + 1], h] = torch.where(some[:, None], p @ v[:, h // group], 0.0)
        return out
    m, v = s["logits"].shape
    x = s["logits"].double().cpu().numpy()
    tokens, n_tokens, n_prompt = (s[k].cpu().numpy() for k in ("tokens", "n_tokens", "n_prompt"))
    rep, pres, freq, values = (s[k].double().cpu().numpy() for k in ("repetition", "presence", "frequency", "bias_values"))
    ids, mask, mask_rows = (s[k].cpu().numpy() for k in ("bias_ids", "mask", "mask_rows"))
    for i in range(m):
        every = np.bincount(tokens[i, :n_tokens[i]], minlength=v)
        count = np.bincount(tokens[i, n_prompt[i]:n_tokens[i]], minlength=v)
        row = np.where(every > 0, np.where(x[i] > 0, x[i] / rep[i], x[i] * rep[i]), x[i])
        row = row - freq[i] * count - pres[i] * (count > 0)
        some = ids[i] >= 0
        row[ids[i][some]] += values[i][some]
        if mask_rows[i] >= 0:
            bits = np.unpackbits(mask[mask_rows[i]].view(np.uint8), bitorder="little")[:v]
            row[bits == 0] = -np.inf
        x[i] = row
    return torch.tensor(x)
