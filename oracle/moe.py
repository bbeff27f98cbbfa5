"""A layer with experts and positions, plain: routing and its plan, the experts'
products (FP64 after dequantization) and the rotation of q and k rows.

The ReSET pages' models are dense and keep their positions inside the serving
engine; these parts are the library's own, on the format of the reading note
§2.1 and the quantizer's recipe.

Test infrastructure only (see the package docstring).
"""
import numpy as np

from .formats import e2m1_decode, e4m3_decode
from .nvfp4 import unpack_codes


# ---- routing ----------------------------------------------------------------------
def route(x, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0,
          rows=None):
    """Token by token.  ids [T, k] (-1: none), weights [T, k] FP64, and how many tokens had no choice."""
    T, E = x.shape
    ids, weights, bad = np.full((T, top_k), -1), np.zeros((T, top_k)), 0
    for t in range(T):
        if rows is not None and not rows[t]:
            continue
        z = np.asarray(x[t], np.float64)
        m = z.max() if not np.isnan(z).any() else np.nan
        if np.isnan(m) or (score == "softmax" and np.isinf(m)):
            bad += 1
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                s = np.exp(z - m)
                s = s / s.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-z))
        v = s if bias is None else s + np.asarray(bias, np.float64)
        if np.isnan(v).any():
            bad += 1
            continue
        by = z if bias is None else v                        # without a bias: the order of the logits
        allowed = list(range(E))
        if top_groups < groups:
            per = E // groups
            gv = v if bias is not None or group_best == 2 else z
            rank = [sum(sorted(gv[g * per:(g + 1) * per], reverse=True)[:group_best]) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            allowed = [e for e in allowed if e // per in kept]
        best = sorted(allowed, key=lambda e: (-by[e], e))[:top_k]
        ids[t] = best
        w = s[best]
        if renormalize:
            zb = z[best]
            zm = zb.max()
            if zm == -np.inf:
                w = np.zeros(top_k)
            else:                                            # relative to the largest: no underflow
                r = (np.exp(zb - zm) if score == "softmax"
                     else np.exp(np.minimum(zb, 0) - min(zm, 0)) / (1.0 + np.exp(-np.abs(zb))))
                w = r / r.sum()
        weights[t] = w * scale
    return ids, weights, bad


def plan(ids, experts):
    """offsets [E + 1], pairs [T k] (-1 behind the last) and places [T, k] (-1: none), by appending to lists."""
    lists = [[] for _ in range(experts)]
    for p, e in enumerate(np.asarray(ids).ravel()):
        if 0 <= e < experts:
            lists[e].append(p)
    offsets = np.cumsum([0] + [len(v) for v in lists])
    pairs = np.full(np.asarray(ids).size, -1)
    places = np.full(np.asarray(ids).size, -1)
    for e, v in enumerate(lists):
        for i, p in enumerate(v):
            pairs[offsets[e] + i] = p
            places[p] = offsets[e] + i
    return offsets, pairs, places.reshape(np.asarray(ids).shape)


# ---- experts ----------------------------------------------------------------------
BLOCK = 18432


def pack(codes, scales, gated):
    """Row-major [E, N, K/2], [E, N, K/16] -> the packed image, byte by byte from the offsets of nvfp4_moe_pack_weights."""
    E, N, half = codes.shape
    K, I = 2 * half, N // 2
    tiles, chunks = -(-N // 128), -(-K // 256)
    out = np.zeros((E, tiles, chunks, BLOCK), np.uint8)
    for g in range(N):
        row = (g % 2) * I + g // 2 if gated else g
        r = g % 128
        for c in range(chunks):
            b = out[:, g // 128, c]
            part = codes[:, row, c * 128:(c + 1) * 128]
            for j in range(part.shape[1] // 16):
                at = r * 128 + ((j ^ (r % 8)) * 16)
                b[:, at:at + 16] = part[:, j * 16:(j + 1) * 16]
            part = scales[:, row, c * 16:(c + 1) * 16]
            for q in range(part.shape[1] // 4):
                at = 16384 + q * 512 + (r % 32) * 16 + (r // 32) * 4
                b[:, at:at + 4] = part[:, 4 * q:4 * q + 4]
    return out.ravel()


def values(codes, scales, glob):
    """FP64 values of NVFP4 rows."""
    return e2m1_decode(unpack_codes(codes)) * np.repeat(e4m3_decode(scales), 16, axis=-1) * np.float64(np.float32(glob))


def gate_up(x, w, offsets, pairs, top_k):
    """x [T, K], w [E, 2 I, K] FP64.  h [T k, I] by place, and what bounds a kernel's rounding of each: the magnitudes
    that are summed up in the gate and in the up (B_g, B_u), g and u."""
    I = w.shape[1] // 2
    h, Bg, Bu, G, U = (np.zeros((len(pairs), I)) for _ in range(5))
    for e in range(w.shape[0]):
        for q in range(offsets[e], offsets[e + 1]):
            row = x[pairs[q] // top_k]
            G[q], U[q] = w[e, :I] @ row, w[e, I:] @ row
            Bg[q], Bu[q] = np.abs(w[e, :I]) @ np.abs(row), np.abs(w[e, I:]) @ np.abs(row)
            with np.errstate(over="ignore"):
                h[q] = G[q] / (1.0 + np.exp(-G[q])) * U[q]
    return h, Bg, Bu, G, U


def down(h, w, weights, places, offsets):
    """h [T k, K] by place, w [E, N, K] FP64.  y [T, N] and the magnitudes that are summed up."""
    T, k = places.shape
    y, B = np.zeros((T, w.shape[1])), np.zeros((T, w.shape[1]))
    for t in range(T):
        for j in range(k):
            q = places[t, j]
            if q < 0:
                continue
            e = int(np.searchsorted(offsets, q, side="right")) - 1
            y[t] += float(weights[t, j]) * (w[e] @ h[q])
            B[t] += abs(float(weights[t, j])) * (np.abs(w[e]) @ np.abs(h[q]))
    return y, B


# ---- positions --------------------------------------------------------------------
def rope_table(positions, rotated, base=10000.0):
    """FP64 angles' cosines and sines, rounded to FP32 [positions, rotated / 2, 2]."""
    m = np.arange(rotated // 2)
    a = np.arange(positions)[:, None] * base ** (-2.0 * m / rotated)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate(x, positions, table, style):
    """FP32 rows [T, heads, D], each product and sum rounded to FP32."""
    x = np.asarray(x, np.float32).copy()
    half = table.shape[1]
    first = np.arange(half) if style == "halves" else 2 * np.arange(half)
    second = first + half if style == "halves" else first + 1
    c, s = table[positions][:, None, :, 0], table[positions][:, None, :, 1]
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    x[..., second] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return x
