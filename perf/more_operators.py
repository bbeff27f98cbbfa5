"""Operators of a decoder layer with experts and positions, as measured cases.

* route: scores of a token's experts, the choice of the best of them, their
  weights, and the order of the (token, expert) pairs by expert
  (nvfp4_moe_route);
* up: the chosen experts' gate and up products on NVFP4 activations and
  weights, joined to SiLU(gate) up (nvfp4_moe_gate_up);
* down: their down products, summed over a token's experts with its weights
  (nvfp4_moe_down);
* rope: q and k rotated by their positions, k and v quantized into the 4-bit
  paged cache, and read back as the values they stand for
  (nvfp4_kv_append_rope, nvfp4_kv_read).

A pair is a token t and its j-th expert, number t k + j.  A plan of the pairs
is their order by expert (pairs, equal experts in the order of their numbers),
offsets (where an expert's pairs begin) and places (where a pair stands).

NVFP4: an E2M1 code is 4 bits (the even element in the low nibble), a scale is
E4M3, one per 16 elements, x = code * scale * global.  Packed expert weights
are blocks of 18432 bytes, one per expert, 128 rows and 256 elements of K, K
fastest: the 16-byte piece j of row r at 128 r + 16 (j xor r mod 8), then the
scales of blocks 4 q .. 4 q + 3 of row r at 16384 + 512 q + 16 (r mod 32) +
4 (r / 32).  Rows of gate and up alternate: 2 i is gate row i, 2 i + 1 up row i.
"""
import math

import numpy as np
import torch

own = False

QWEN3_32B_HEADS = (64, 8)      # query and kv heads behind the qkv projection 5120 -> 10240
QWEN3_14B_HEADS = (40, 8)
MAX_POSITIONS = 32768


# ---- the cases ------------------------------------------------------------------
def listed():
    h32, k32 = QWEN3_32B_HEADS
    h14, k14 = QWEN3_14B_HEADS
    return [
        # one user's token: latency
        {"name": "route-one", "op": "route", "tokens": 1, "experts": 128, "top": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_best": 1, "renormalize": True, "scale": 1.0, "dtype": "f32"},
        # a decode batch over experts that live in groups, BF16 logits, weights as they are
        {"name": "route-batch", "op": "route", "tokens": 64, "experts": 64, "top": 6, "score": "softmax", "bias": False,
         "groups": 8, "top_groups": 3, "group_best": 1, "renormalize": False, "scale": 16.0, "dtype": "bf16"},
        # a long prompt, sigmoid scores with a bias that balances the experts, groups by their two best
        {"name": "route-prefill", "op": "route", "tokens": 8192, "experts": 256, "top": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True, "scale": 2.5, "dtype": "f32"},
        # one user's token through its eight experts
        {"name": "up-one", "op": "up", "tokens": 1, "experts": 128, "top": 8, "hidden": 4096, "inter": 1024},
        # the library's largest decode batch: about fifty small experts, one or two rows each
        {"name": "up-batch", "op": "up", "tokens": 8, "experts": 128, "top": 8, "hidden": 5120, "inter": 768},
        # a ragged batch over few large experts
        {"name": "up-few", "op": "up", "tokens": 33, "experts": 8, "top": 2, "hidden": 4096, "inter": 8192},
        # a prompt: every expert has rows, from a handful to hundreds
        {"name": "up-prefill", "op": "up", "tokens": 2048, "experts": 128, "top": 8, "hidden": 4096, "inter": 768},
        # the ways back of the same
        {"name": "down-one", "op": "down", "tokens": 1, "experts": 128, "top": 8, "hidden": 4096, "inter": 1024},
        {"name": "down-batch", "op": "down", "tokens": 64, "experts": 128, "top": 8, "hidden": 5120, "inter": 768},
        {"name": "down-prefill", "op": "down", "tokens": 2048, "experts": 128, "top": 8, "hidden": 4096, "inter": 768},
        # one decode step's rows, slices of the FP32 qkv output
        {"name": "rope-decode", "op": "rope", "tokens": 8, "heads": h32, "kv_heads": k32, "dim": 128, "rotated": 128,
         "style": "halves", "page": 64, "dtype": "f32", "pad": 0},
        # a long prompt in one call
        {"name": "rope-prefill", "op": "rope", "tokens": 8192, "heads": h14, "kv_heads": k14, "dim": 128, "rotated": 128,
         "style": "halves", "page": 64, "dtype": "bf16", "pad": 100},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.25 / hi)))))


def draw(rng):
    op = rng.choice(["route", "up", "up", "down", "down", "rope"])
    if op == "route":
        groups, each = rng.choice([(1, 8), (1, 31), (1, 60), (1, 128), (1, 160), (4, 16), (8, 8), (8, 20), (8, 32), (16, 24)])
        top_groups = rng.randint(1, groups) if groups > 1 else 1
        return {"op": op, "tokens": _log(rng, 1, 8192) if groups * each <= 256 else _log(rng, 1, 4096),
                "experts": groups * each, "top": rng.randint(1, min(10, top_groups * each)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "group_best": rng.choice([1, 2]), "renormalize": rng.random() < 0.5,
                "scale": rng.choice([1.0, 1.0, 2.5]), "dtype": rng.choice(["f32", "bf16"])}
    if op in ("up", "down"):
        experts = rng.choice([1, 4, 8, 16, 40, 64, 96, 128])
        top = rng.randint(1, min(experts, 8))
        hidden, inter = 64 * _log(rng, 4, 80), 64 * _log(rng, 1, 32)
        while experts * hidden * inter > 128 * 4096 * 768:
            hidden, inter = 64 * _log(rng, 4, 80), 64 * _log(rng, 1, 32)
        return {"op": op, "tokens": _log(rng, 1, 2048 * 8 // max(8, top)), "experts": experts, "top": top, "hidden": hidden,
                "inter": inter}
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    tokens = _log(rng, 1, 8192)
    return {"op": op, "tokens": tokens, "heads": kv_heads * rng.randint(1, 5), "kv_heads": kv_heads, "dim": dim,
            "rotated": rng.choice([32, 64, dim, dim]), "style": rng.choice(["halves", "pairs"]),
            "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["f32", "bf16"]) if tokens <= 4096 else "bf16",
            "pad": rng.randint(0, tokens // 4)}


# ---- what a case fixes (the seed only shuffles it) ---------------------------------
def _choices(case):
    """Experts of each token [T, k]: some are more popular than others."""
    n, e, k = case["tokens"], case["experts"], case["top"]
    r = np.random.RandomState(n * 7919 + e * 31 + k)
    score = 0.6 * r.standard_normal(e) + r.gumbel(size=(n, e))
    return np.argsort(-score, axis=1, kind="stable")[:, :k]


def work(case):
    t, e = case["tokens"], case.get("experts", 0)
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "route":
        # the logits; ids, weights, order and places of the pairs; where the experts begin
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 16 * t * case["top"] + 4 * (e + 1)}
    if case["op"] == "rope":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        live = t - case["pad"]
        # rows in, cosines and sines of the positions, q out; 9/16 byte an element written and read back, BF16 out
        return {"bytes": 8 * t + live * (h + 2 * hk) * d * size + -(-live // 3) * case["rotated"] * 4 + t * h * d * 2
                + 2 * (2 * live * hk * d * 9 // 16) + 2 * t * hk * d * 2}
    used, pairs, k, i = len(np.unique(_choices(case))), t * case["top"], case["hidden"], case["inter"]
    plan = 4 * pairs + 4 * (e + 1)
    if case["op"] == "up":
        return {"bytes": used * 2 * i * k * 9 // 16 + t * k * 9 // 16 + plan + pairs * i * 2, "flops": 4 * pairs * i * k}
    return {"bytes": used * i * k * 9 // 16 + pairs * i * 9 // 16 + plan + 8 * pairs + t * k * 4, "flops": 2 * pairs * i * k}


# ---- inputs ---------------------------------------------------------------------
def _round_e2m1(a):
    """E2M1 code (0..7) of non-negative values, ties to the even code, saturating."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _quantize(x, glob):
    """FP32 [..., K] -> code bytes [..., K/2], scale bytes [..., K/16], in FP32 step by step; glob [] or [..., 1]."""
    b = x.unflatten(-1, (-1, 16))
    most = b.abs().amax(-1)
    s8 = (most / (6.0 * glob)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s8.float() * glob).unsqueeze(-1)
    code = torch.where(step > 0, _round_e2m1(b.abs() / step), 0) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), s8.view(torch.uint8)


def _values(codes, scales, glob):
    """What NVFP4 tensors stand for, FP32; glob [] or [..., 1]."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    x = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 16))
    return (x * (scales.view(torch.float8_e4m3fn).float() * glob).unsqueeze(-1)).flatten(-2)


def _pack(codes, scales, gated):
    """Row-major codes [E, N, K/2] and scales [E, N, K/16] -> blocks [E, N/128, K/256, 18432]; short ends are zeros."""
    if gated:
        codes, scales = (t.unflatten(1, (2, -1)).transpose(1, 2).flatten(1, 2) for t in (codes, scales))
    e, n, half = codes.shape
    tiles, chunks = -(-n // 128), -(-half // 128)
    codes = torch.nn.functional.pad(codes, (0, chunks * 128 - half, 0, tiles * 128 - n))
    scales = torch.nn.functional.pad(scales, (0, chunks * 16 - half // 8, 0, tiles * 128 - n))
    codes = codes.view(e, tiles, 128, chunks, 8, 16).permute(0, 1, 3, 2, 4, 5)
    row, piece = torch.arange(128, device=codes.device)[:, None], torch.arange(8, device=codes.device)
    codes = codes[:, :, :, row, piece ^ (row % 8)]                       # [E, tiles, chunks, 128, 8, 16]
    scales = scales.view(e, tiles, 4, 32, chunks, 4, 4).permute(0, 1, 4, 5, 3, 2, 6)
    return torch.cat([codes.reshape(e, tiles, chunks, -1), scales.reshape(e, tiles, chunks, -1)], -1)


def _experts(g, case, n, k):
    """Weights [E, n, k] of normal values, one global scale an expert."""
    e = case["experts"]
    codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((e, n, k // 16), dtype=torch.uint8, device="cuda")
    glob = torch.empty(e, device="cuda")
    step = max(1, (1 << 26) // (n * k))                                  # experts made at a time
    for a in range(0, e, step):
        w = 0.02 * torch.randn((min(step, e - a), n, k), generator=g, device="cuda")
        glob[a:a + step] = w.abs().amax((1, 2)) / 2688.0
        codes[a:a + step], scales[a:a + step] = _quantize(w, glob[a:a + step, None, None])
    return codes, scales, glob


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g, torch.Generator().manual_seed(seed)


def _rows(g, shape):
    """Activations: normal, one channel in a hundred twelve times as large, magnitudes changing from token to token."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 5::100] *= 12.0
    return x * torch.exp(0.5 * torch.randn((shape[0],) + (1,) * (len(shape) - 1), generator=g, device="cuda"))


def _plan(ids, experts):
    """offsets, pairs and places of the experts [T, k] of the tokens."""
    flat = ids.flatten().long()
    order = torch.sort(flat, stable=True).indices
    count = torch.zeros(experts, dtype=torch.int64, device=ids.device).scatter_add(0, flat, torch.ones_like(flat))
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    places = torch.empty_like(order).scatter(0, order, torch.arange(order.numel(), device=ids.device))
    return offsets.int(), order.int(), places.view(ids.shape).int()


def prepare(case, seed):
    g, host = _gen(seed)
    s = dict(case)
    t = case["tokens"]
    if case["op"] == "route":
        e = case["experts"]
        x = 1.5 * torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        s["logits"] = x if case["dtype"] == "f32" else x.bfloat16()
        s["bias_values"] = 0.1 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")
        s["out"] = (i32(t, case["top"]), torch.empty((t, case["top"]), device="cuda"), i32(e + 1), i32(t * case["top"]),
                    i32(t, case["top"]))
        return s
    if case["op"] == "rope":
        h, hk, d, pg = case["heads"], case["kv_heads"], case["dim"], case["page"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # q, K and V are column slices of one projection's output
        x = _rows(g, (t, (h + 2 * hk) * d)).to(dt)
        live = t - case["pad"]
        # three requests from the start of a page each, behind what they hold; the pages in no order; padding at the end
        per = -(-live // 3)
        at = torch.arange(live)
        held = torch.randint(0, MAX_POSITIONS - per, (3,), generator=host)
        room = -(-(per + pg) // pg) * pg
        n_pages = 3 * room // pg
        perm = torch.randperm(n_pages, generator=host)
        logical = at // per * room + held[at // per] % pg + at % per
        slots, positions = torch.full((t,), -1, dtype=torch.int64), torch.zeros(t, dtype=torch.int64)
        slots[:live] = perm[logical // pg] * pg + logical % pg
        positions[:live] = held[at // per] + at % per
        half = case["rotated"] // 2
        angle = torch.arange(MAX_POSITIONS, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
            -torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s.update(q=x[:, :h * d].unflatten(-1, (h, d)), k=x[:, h * d:(h + hk) * d].unflatten(-1, (hk, d)),
                 v=x[:, (h + hk) * d:].unflatten(-1, (hk, d)), slots=slots.int().cuda(), positions=positions.int().cuda(),
                 table=torch.stack([angle.cos(), angle.sin()], -1).float(), n_pages=n_pages,
                 k_global=torch.tensor([0.5], device="cuda"), v_global=torch.tensor([0.125], device="cuda"),
                 q_out=torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda"),
                 pages=torch.zeros((n_pages, hk, pg // 16, 18 * d), dtype=torch.uint8, device="cuda"),
                 # the plain form's cache: codes and scales by slot, one more for its padding
                 plain=[torch.zeros((n_pages * pg + 1, hk, w), dtype=torch.uint8, device="cuda")
                        for w in (d // 2, d // 16, d // 2, d // 16)])
        return s
    up = case["op"] == "up"
    ids = torch.from_numpy(_choices(case))
    ids = torch.randperm(case["experts"], generator=host)[ids][torch.randperm(t, generator=host)].cuda()
    pairs, k, n = t * case["top"], case["hidden"], case["inter"]
    if up:
        codes, scales, s["w_global"] = _experts(g, case, 2 * n, k)
        x = _rows(g, (t, k))
    else:
        codes, scales, s["w_global"] = _experts(g, case, k, n)
        a = _rows(g, (pairs, n))
        x = a * torch.sigmoid(a) * torch.randn((pairs, n), generator=g, device="cuda")
        p = torch.softmax(torch.randn((t, case["top"]), generator=g, device="cuda"), -1)
        s["weights"] = p / p.sum(-1, keepdim=True)
    x = x.bfloat16().float()
    s["x_global"] = (x.abs().amax() / 2688.0).view(1)
    s["x_codes"], s["x_scales"] = _quantize(x, s["x_global"])
    s["packed"] = _pack(codes, scales, up).flatten()
    s["codes"], s["scales"] = codes, scales
    s["ids"] = ids.int()
    s["offsets"], s["pairs"], s["places"] = _plan(ids, case["experts"])
    # for the plain form: which experts have rows, and how many at most
    count = torch.bincount(ids.flatten(), minlength=case["experts"])
    s["used"], s["most"] = count.nonzero().flatten(), int(count.max())
    s["out"] = torch.empty((pairs, n), dtype=torch.bfloat16, device="cuda") if up else torch.empty((t, k), device="cuda")
    return s


# ---- one pass -------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "rope":
        return _plain_rope(s)
    return _plain_up(s) if s["op"] == "up" else _plain_down(s)


def _plain_route(s):
    # in 64 bits: the choice goes by values that may lie close together
    x = s["logits"].double()
    t, e = x.shape
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    value = p if s["bias_values"] is None else p + s["bias_values"].double()
    if s["groups"] > 1:
        best = torch.sort(value.view(t, s["groups"], -1), descending=True).values[..., :s["group_best"]].sum(-1)
        order = torch.sort(best, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(best).scatter(1, order, 1.0).bool().repeat_interleave(e // s["groups"], 1)
        value = torch.where(keep, value, -math.inf)
    ids = torch.sort(value, descending=True, stable=True).indices[:, :s["top"]]
    w = p.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return [ids.int(), (w * s["scale"]).float(), *_plan(ids, e)]


def _by_expert(s, rows):
    """FP32 rows [pairs, K] in the order of the plan -> [used, most, K], zeros behind an expert's rows, and their places."""
    offsets = s["offsets"].long()
    first = offsets[s["used"]]
    count = offsets[s["used"] + 1] - first
    at = torch.arange(s["most"], device="cuda")
    live = at < count[:, None]
    x = torch.where(live[..., None], rows[torch.where(live, first[:, None] + at, 0)], 0.0)
    where = torch.arange(rows.shape[0], device="cuda")
    a = torch.searchsorted(first, where, right=True) - 1
    return x, a, where - first[a]


def _plain_up(s):
    token = s["pairs"].long() // s["top"]
    x, a, r = _by_expert(s, _values(s["x_codes"], s["x_scales"], s["x_global"])[token])
    w = _values(s["codes"][s["used"]], s["scales"][s["used"]], s["w_global"][s["used"], None, None])
    gate, up = (x @ w.transpose(1, 2)).chunk(2, -1)
    return (gate / (1.0 + torch.exp(-gate)) * up).bfloat16()[a, r]


def _plain_down(s):
    x, a, r = _by_expert(s, _values(s["x_codes"], s["x_scales"], s["x_global"]))
    w = _values(s["codes"][s["used"]], s["scales"][s["used"]], s["w_global"][s["used"], None, None])
    y = x @ w.transpose(1, 2)
    at = s["places"].long()
    return (y[a[at], r[at]] * s["weights"][..., None]).sum(1)


def _rotate(s, x):
    """Rows [T, heads, D] turned by their positions, each step rounded to the type of x."""
    cs = s["table"].to(x.dtype)[s["positions"].long()][:, None]                # [T, 1, rotated / 2, 2]
    c, sn = cs[..., 0], cs[..., 1]
    turned, rest = x[..., :s["rotated"]], x[..., s["rotated"]:]
    if s["style"] == "halves":
        a, b = turned.chunk(2, -1)
        return torch.cat([a * c - b * sn, b * c + a * sn, rest], -1)
    a, b = turned[..., 0::2], turned[..., 1::2]
    return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), rest], -1)


def _plain_rope(s):
    # what is written for padding goes behind the cache's own slots
    gone = (s["slots"] < 0)[:, None, None]
    at = torch.where(s["slots"] < 0, s["n_pages"] * s["page"], s["slots"]).long()
    q = torch.where(gone, 0.0, _rotate(s, s["q"].float())).bfloat16()
    k, v = _rotate(s, s["k"].float()).bfloat16().float(), s["v"].bfloat16().float()
    kc, ks, vc, vs = s["plain"]
    kc[at], ks[at] = _quantize(k, s["k_global"])
    vc[at], vs[at] = _quantize(v, s["v_global"])
    return [q] + [torch.where(gone, 0.0, _values(c[at], z[at], gl)).bfloat16()
                  for c, z, gl in ((kc, ks, s["k_global"]), (vc, vs, s["v_global"]))]


def _run_own(s):
    from nvfp4_w4a4_decode_gemv_gb300 import api
    if s["op"] == "route":
        if "routing" not in s:                                             # the handle that a program keeps
            s["routing"] = api.MoERouting(*s["out"])
        r = api.nvfp4_moe_route(s["logits"], s["top"], score=s["score"], bias=s["bias_values"], groups=s["groups"],
                                top_groups=s["top_groups"], group_best=s["group_best"], renormalize=s["renormalize"],
                                scale=s["scale"], out=s["routing"])
        return [r.ids, r.weights, r.offsets, r.pairs, r.places]
    if s["op"] == "rope":
        if "cache" not in s:
            s["cache"] = api.NVFP4KVCache(s["pages"], s["k_global"], s["v_global"])
        q = api.nvfp4_kv_append_rope(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cache"], s["table"],
                                     style=s["style"], q_out=s["q_out"])
        return [q, *api.nvfp4_kv_read(s["cache"], s["slots"])]
    if "x" not in s:
        up = s["op"] == "up"
        n, k = (2 * s["inter"], s["hidden"]) if up else (s["hidden"], s["inter"])
        s["x"] = api.NVFP4Tensor(s["x_codes"], s["x_scales"], s["x_global"])
        s["w"] = api.NVFP4MoEWeight(s["packed"], s["w_global"], s["experts"], n, k, gated=up)
        s["routing"] = api.MoERouting(s["ids"], s.get("weights"), s["offsets"], s["pairs"], s["places"])
    if s["op"] == "up":
        return api.nvfp4_moe_gate_up(s["x"], s["w"], s["routing"], out=s["out"])
    return api.nvfp4_moe_down(s["x"], s["w"], s["routing"], y=s["out"])


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


def _exact_matrix(codes, scales, glob):
    """FP64 values of a row-major NVFP4 matrix [rows, K], element by element."""
    grid = torch.tensor(np.concatenate([_E2M1, -_E2M1]), device="cuda")
    e4m3 = torch.tensor(np.concatenate([_E4M3, [math.nan], -_E4M3, [math.nan]]), device="cuda")
    e = torch.arange(2 * codes.shape[1], device="cuda")
    code = (codes[:, e // 2] >> (4 * (e % 2)).to(torch.uint8)) & 15
    return grid[code.long()] * e4m3[scales.long()][:, e // 16] * glob.double()


def _exact_route(s):
    x = s["logits"].double().cpu().numpy()
    bias = None if s["bias_values"] is None else s["bias_values"].double().cpu().numpy()
    out = np.zeros((x.shape[0], s["top"]))
    each = x.shape[1] // s["groups"]
    for t, row in enumerate(x):
        p = np.exp(row - row.max()) if s["score"] == "softmax" else 1.0 / (1.0 + np.exp(-row))
        p = p / p.sum() if s["score"] == "softmax" else p
        v = p if bias is None else p + bias
        allowed = np.arange(len(row))
        if s["groups"] > 1:
            score = [np.sort(v[i * each:(i + 1) * each])[::-1][:s["group_best"]].sum() for i in range(s["groups"])]
            kept = np.argsort(-np.array(score), kind="stable")[:s["top_groups"]]
            allowed = allowed[np.isin(allowed // each, kept)]
        ids = allowed[np.argsort(-v[allowed], kind="stable")[:s["top"]]]
        out[t] = p[ids] / (p[ids].sum() if s["renormalize"] else 1.0) * s["scale"]
    return [None, torch.tensor(out), None, None, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "rope":
        gone = (s["slots"] < 0).cpu().numpy()[:, None, None]
        half = case["rotated"] // 2
        cs = s["table"].double().cpu().numpy()[s["positions"].long().cpu().numpy()]
        out = []
        for name in ("q", "k", "v"):
            x = s[name].double().cpu().numpy()
            if name != "v":
                first = np.arange(half) if case["style"] == "halves" else 2 * np.arange(half)
                second = first + half if case["style"] == "halves" else first + 1
                z = (x[..., first] + 1j * x[..., second]) * (cs[:, None, :, 0] + 1j * cs[:, None, :, 1])
                x = x.copy()
                x[..., first], x[..., second] = z.real, z.imag
            if name != "q":
                x = _exact_rows(torch.from_numpy(x).bfloat16().double().numpy(), float(s[name + "_global"]))
            out.append(np.where(gone, 0.0, x))
        return out
    offsets, pairs, top = s["offsets"].tolist(), s["pairs"].long(), case["top"]
    x = _exact_matrix(s["x_codes"], s["x_scales"], s["x_global"])
    if case["op"] == "up":
        out = torch.zeros((pairs.numel(), case["inter"]), dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        w = _exact_matrix(s["codes"][e], s["scales"][e], s["w_global"][e])
        if case["op"] == "up":
            gate, up = (x[pairs[a:b] // top] @ w.T).chunk(2, -1)
            out[a:b] = gate * torch.sigmoid(gate) * up
        else:
            out.index_add_(0, pairs[a:b] // top, s["weights"].double().flatten()[pairs[a:b]][:, None] * (x[a:b] @ w.T))
    return out
