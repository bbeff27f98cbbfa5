"""The serving step around the projections, plain: page tables and slot maps,
the NVFP4 KV cache, attention over it (FP64) and rules on the logits (FP64).

The ReSET pages run their kernels inside a serving engine that owns these parts
(reading note §4.3, §5.2) and keep the KV cache in BF16 (§6.1); the 4-bit cache
is this library's, in the format of §2.1 and with the quantizer's recipe.

Test infrastructure only (see the package docstring).
"""
import numpy as np

from .formats import e2m1_decode, e2m1_encode, e4m3_decode, e4m3_encode_nonneg


# ---- pages ------------------------------------------------------------------------
def kv_release(lens, ended, table, stack, count, page):
    """One request after the other: (stack, count) afterwards."""
    stack = np.array(stack, copy=True)
    for b in range(len(lens)):
        if not ended[b]:
            continue
        for j in range(min(-(-max(int(lens[b]), 0) // page), table.shape[1])):
            if count < len(stack):
                stack[count] = table[b, j]
                count += 1
    return stack, count


def kv_plan(ctx, new, table, stack, count, page, max_tokens):
    """One request after the other.  Returns table, slots, positions, cu_q, kv_lens, count, (refused, tokens)."""
    table = np.array(table, copy=True)
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    cu, kv, refused, asked, taken, tok = [0], [], 0, 0, 0, 0
    for b in range(len(ctx)):
        c, q = int(ctx[b]), int(new[b])
        bad = c < 0 or q < 0
        c, q = max(c, 0), max(q, 0)
        have, end = -(-c // page), -(-(c + q) // page)
        bad = bad or end > table.shape[1]
        need = 0 if bad else end - have
        asked += need
        refuse = bad or (need > 0 and asked > count)
        if not refuse:
            for j in range(need):
                table[b, have + j] = stack[count - 1 - (asked - need + j)]
            taken = max(taken, asked if need else 0)
        for i in range(q):
            if tok + i < max_tokens:
                pos = c + i
                positions[tok + i] = pos
                if not refuse:
                    slots[tok + i] = int(table[b, pos // page]) * page + pos % page
        tok += q
        cu.append(tok)
        kv.append(c if refuse else c + q)
        refused += refuse
    return table, slots, positions, np.array(cu), np.array(kv), count - taken, (refused, tok)


# ---- the cache ---------------------------------------------------------------------
def quantize_rows(x, glob):
    """FP32 values [..., D] (BF16-representable) -> codes [..., D] (one a byte), scale bytes [..., D/16]; FP32 IEEE
    at each step, as the quantizer's recipe with a given global scale."""
    x = np.asarray(x, np.float32)
    g = np.float32(glob)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    s = e4m3_encode_nonneg((np.abs(b).max(-1) / (np.float32(6.0) * g)).astype(np.float32))
    step = (e4m3_decode(s).astype(np.float32) * g)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(step > 0, b / np.where(step > 0, step, np.float32(1)), np.float32(0) * np.sign(b))
    t = np.where(step > 0, t, np.copysign(np.float32(0), b)).astype(np.float32)
    return e2m1_encode(t).reshape(x.shape), s


def dequantize_rows(codes, scales, glob):
    """FP64 values of codes [..., D] and scale bytes [..., D/16]."""
    v = e2m1_decode(codes).reshape(codes.shape[:-1] + (scales.shape[-1], 16))
    return (v * e4m3_decode(scales)[..., None] * float(np.float32(glob))).reshape(codes.shape)


class GroupOffsets:
    """Byte offsets within a 16-token group of head size D (nvfp4_kv_cache in nvfp4.h)."""

    def __init__(self, D):
        self.D, self.bytes = D, 18 * D
        t, e = np.arange(16)[:, None], np.arange(D)[None]
        blk = np.arange(D // 16)[None]
        nb = D // 64
        pos = 8 * (t // 2 % 2) + 2 * (t // 4) + t % 2
        self.k_codes = pos * (D // 2) + e // 2                                    # [16, D]
        self.k_scales = 8 * D + (pos % 8) * 8 * nb + blk // nb * 2 * nb + pos // 8 * nb + blk % nb
        if D == 128:
            r = e // 16
            self.v_codes = 9 * D + r // 2 * 256 + t // 2 % 2 * 128 + r % 2 * 64 + t // 4 * 16 + t % 2 * 8 + e % 16 // 2
        else:
            self.v_codes = 9 * D + e // 8 * 64 + t * 4 + e % 8 // 2
        self.v_scales = 17 * D + blk * 16 + t
        self.nibble = (4 * (e % 2)).astype(np.uint8)


def read_slots(pages, slots, page, D):
    """pages uint8 [num_pages, heads, page/16, 18 D]; slots [n] -> K codes, K scales, V codes, V scales
    ([n, heads, D] one code a byte, [n, heads, D/16])."""
    o = GroupOffsets(D)
    slots = np.asarray(slots)
    rows = pages[slots // page, :, slots % page // 16]                            # [n, heads, 18 D]
    t = slots % 16
    take = lambda off: np.take_along_axis(rows, np.broadcast_to(off[t][:, None], rows.shape[:2] + off.shape[1:]), 2)
    return ((take(o.k_codes) >> o.nibble) & 15, take(o.k_scales), (take(o.v_codes) >> o.nibble) & 15, take(o.v_scales))


def write_slots(pages, slots, page, D, kc, ks, vc, vs):
    """The reverse of read_slots, in place."""
    o = GroupOffsets(D)
    for i, s in enumerate(np.asarray(slots)):
        g = pages[s // page, :, s % page // 16]                                   # [heads, 18 D], a view
        t = s % 16
        g[:, o.k_codes[t][::2]] = kc[i][:, ::2] | (kc[i][:, 1::2] << 4)
        g[:, o.v_codes[t][::2]] = vc[i][:, ::2] | (vc[i][:, 1::2] << 4)
        g[:, o.k_scales[t]] = ks[i]
        g[:, o.v_scales[t]] = vs[i]


# ---- attention ---------------------------------------------------------------------
def attention(q, k, v, scale, window=0, n_keys=None):
    """One request: q [m, heads, D] at the last m positions, k, v [n, kv_heads, D], FP64.  Returns out, lse, and
    what bounds a kernel's rounding: the weighted magnitude of V (A), the plain one over the weights' sum (B) and
    the largest scale * sum |q k| and scale * max|q| * sum|k| of a row's visible keys."""
    m, heads, D = q.shape
    n, kvh = k.shape[0], k.shape[1]
    out, A, B = (np.zeros((m, heads, D)) for _ in range(3))
    lse = np.full((m, heads), -np.inf)
    S, Q = np.zeros((m, heads)), np.zeros((m, heads))
    for i in range(m):
        p = n - m + i
        lo = max(0, p - window + 1) if window else 0
        if p < lo:
            continue
        for h in range(heads):
            K, V = k[lo:p + 1, h // (heads // kvh)], v[lo:p + 1, h // (heads // kvh)]
            s = scale * (K @ q[i, h])
            w = np.exp(s - s.max())
            out[i, h] = w @ V / w.sum()
            A[i, h] = w @ np.abs(V) / w.sum()
            B[i, h] = np.abs(V).sum(0) / w.sum()
            lse[i, h] = s.max() + np.log(w.sum())
            S[i, h] = scale * (np.abs(K) @ np.abs(q[i, h])).max()
            Q[i, h] = scale * np.abs(q[i, h]).max() * np.abs(K).sum(1).max()
    return out, lse, A, B, S, Q


# ---- logits ------------------------------------------------------------------------
def process_logits(x, tokens=None, n_tokens=None, n_prompt=None, repetition=None, presence=None, frequency=None,
                   bias_ids=None, bias_values=None, mask=None, mask_rows=None, fill=-np.inf):
    """Token by token.  Returns the rules' result and the sum of the magnitudes of what was added up (FP64)."""
    x = np.array(x, dtype=np.float64)
    size = np.abs(np.where(np.isfinite(x), x, 0.0))
    M, V = x.shape
    for r in range(M):
        if tokens is not None:
            used = min(max(int(n_tokens[r]), 0), tokens.shape[1])
            prompt = min(max(int(n_prompt[r]), 0), used) if n_prompt is not None else 0
            rep = float(repetition[r]) if repetition is not None else 1.0
            pres = float(presence[r]) if presence is not None else 0.0
            freq = float(frequency[r]) if frequency is not None else 0.0
            seen, count = set(), {}
            for i in range(used):
                t = int(tokens[r, i])
                if 0 <= t < V:
                    seen.add(t)
                    if i >= prompt:
                        count[t] = count.get(t, 0) + 1
            for t in seen:
                x[r, t] = x[r, t] / rep if x[r, t] > 0 else x[r, t] * rep
                size[r, t] = abs(x[r, t]) if np.isfinite(x[r, t]) else 0.0
            for t, c in count.items():
                x[r, t] = x[r, t] - freq * c - pres
                size[r, t] += abs(freq * c) + abs(pres)
        if bias_ids is not None:
            last = {int(t): float(w) for t, w in zip(bias_ids[r], bias_values[r])}
            for t, w in last.items():
                if 0 <= t < V:
                    x[r, t] += w
                    size[r, t] += abs(w)
        if mask is not None:
            m = int(mask_rows[r]) if mask_rows is not None else r
            if 0 <= m < mask.shape[0]:
                bits = np.unpackbits(np.ascontiguousarray(mask[m]).view(np.uint8), bitorder="little")[:V]
                x[r, bits == 0] = fill
                size[r, bits == 0] = 0.0
    return x, size
