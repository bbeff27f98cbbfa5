"""Rows rotated on the way into the NVFP4 cache: q's bits and the cache's bytes are those of the formula, each step rounded
to FP32, and of the append's recipe."""
import numpy as np
import pytest
import torch

from oracle import moe as O
from oracle import nvfp4 as Q
from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, bits, to_np
from tests.test_gpu_kv_cache import _cache

pytestmark = pytest.mark.gpu

BF = lambda x: Q.bf16_bits_to_f32(Q.f32_to_bf16_bits(x))


def _case(tokens, heads, kv_heads, D, rotated, style, dtype, slots, positions, page, n_pages, limit=4000, seed=0):
    rng = np.random.default_rng(seed)
    c = _cache(n_pages, page, kv_heads, D)
    want = to_np(c.pages).copy()
    wide = torch.from_numpy((rng.standard_normal((tokens, (heads + 2 * kv_heads) * D + 16)) * 3).astype(np.float32)).to(dtype)
    dev = wide.cuda()
    cut = [8, 8 + heads * D, 8 + (heads + kv_heads) * D, 8 + (heads + 2 * kv_heads) * D]
    rows = lambda t, i: t[:, cut[i]:cut[i + 1]].unflatten(-1, (-1, D))
    table = O.rope_table(limit, rotated)
    slots, positions = np.asarray(slots, np.int32), np.asarray(positions, np.int32)
    out = Guarded((tokens, heads, D), torch.bfloat16)
    api.nvfp4_kv_append_rope(rows(dev, 0), rows(dev, 1), rows(dev, 2), torch.from_numpy(positions).cuda(),
                             torch.from_numpy(slots).cuda(), c, torch.from_numpy(table).cuda(), style=style, q_out=out.t)
    live = (slots >= 0) & (slots < n_pages * page) & (positions >= 0) & (positions < limit)
    q, k, v = (rows(wide.float(), i).numpy()[live] for i in range(3))
    got = Q.bf16_bits_to_f32(bits(out.t))
    assert not got[~live].any()
    assert np.array_equal(got[live], BF(O.rotate(q, positions[live], table, style)))
    kc, ks = S.quantize_rows(BF(O.rotate(k, positions[live], table, style)), float(c.k_global))
    vc, vs = S.quantize_rows(BF(v), float(c.v_global))
    S.write_slots(want, slots[live], page, D, kc, ks, vc, vs)
    assert np.array_equal(to_np(c.pages), want)
    out.check("q_out")
    bad = (slots != -1) & ~live
    assert api.device_status() == (api.DEVERR_KV_RANGE if bad.any() else 0)


@pytest.mark.parametrize("D,rotated", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 96), (128, 128)])
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,kv_heads,page", [(1, 1, 1, 16), (8, 10, 2, 64), (70, 3, 3, 48)])
def test_few_tokens(D, rotated, style, dtype, tokens, heads, kv_heads, page):
    rng = np.random.default_rng(tokens)
    n_pages = -(-tokens // page) + 2
    slots = rng.permutation(n_pages * page)[:tokens]
    slots[3::7] = -1
    _case(tokens, heads, kv_heads, D, rotated, style, dtype, slots, rng.integers(0, 4000, tokens), page, n_pages)


def _windows(tokens, page, offset, rng):
    """Three requests' runs of slots from odd offsets, pages in no order, padding at the end."""
    per = -(-tokens // 3)
    at = np.arange(tokens)
    room = -(-(per + page) // page) * page
    logical = at // per * room + offset + at % per
    n_pages = 3 * room // page + 1
    order = rng.permutation(n_pages)
    slots = order[logical // page] * page + logical % page
    slots[tokens - tokens // 50:] = -1
    return slots, at % per + 100, n_pages


@pytest.mark.parametrize("D,rotated", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens(D, rotated, style, dtype):
    """More than a thread for every pair of blocks: windows of 16 tokens."""
    tokens, kv_heads = 4321, 4
    slots, positions, n_pages = _windows(tokens, 32, 5, np.random.default_rng(1))
    _case(tokens, 9, kv_heads, D, rotated, style, dtype, slots, positions, 32, n_pages)


@pytest.mark.parametrize("tokens", [40, 4200])
def test_slots_and_positions_outside(tokens):
    slots, positions, n_pages = _windows(tokens, 64, 0, np.random.default_rng(2))
    slots, positions = slots.copy(), positions.copy()
    slots[5], slots[21], slots[30] = n_pages * 64, -2, 2 ** 31 - 1
    positions[9], positions[17], positions[33] = -1, 4000, 2 ** 31 - 1
    slots[12], positions[12] = -1, 99999                        # padding: its position is not looked at
    _case(tokens, 2, 4, 128, 128, "halves", torch.bfloat16, slots, positions, 64, n_pages)


def test_strides_of_one_token_and_one_head():
    c = api.NVFP4KVCache.empty(2, 16, 1, 64)
    base = torch.randn(1000, device="cuda")
    row = base.as_strided((1, 1, 64), (3, 5, 1))                # the strides of a single row are used in no address
    table = api.rope_table(10, 64)
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    got = api.nvfp4_kv_append_rope(row, row, row, i32(7), i32(3), c, table)
    want = BF(O.rotate(to_np(base[:64]).reshape(1, 1, 64), np.array([7]), to_np(table), "halves"))
    assert np.array_equal(Q.bf16_bits_to_f32(bits(got)), want)


@pytest.mark.parametrize("tokens", [5, 4200])
def test_keys_and_values_alone(tokens):
    """The same cache as with q; bad slots are reported."""
    rng = np.random.default_rng(4)
    slots, positions, n_pages = _windows(tokens, 16, 3, rng)
    s, p = (torch.from_numpy(a.astype(np.int32)).cuda() for a in (slots, positions))
    q, k, v = torch.randn((3, tokens, 4, 128), device="cuda").bfloat16()
    table = api.rope_table(4000, 64)
    caches = [api.NVFP4KVCache.empty(n_pages, 16, 4, 128) for _ in range(2)]
    for c in caches:
        c.pages.zero_()
    api.nvfp4_kv_append_rope(q, k, v, p, s, caches[0], table)
    assert api.nvfp4_kv_append_rope(None, k, v, p, s, caches[1], table) is None
    assert torch.equal(caches[0].pages, caches[1].pages) and api.device_status() == 0
    s[1] = -5
    api.nvfp4_kv_append_rope(None, k, v, p, s, caches[1], table)
    assert api.device_status() == api.DEVERR_KV_RANGE
    with pytest.raises(ValueError):
        api.nvfp4_kv_append_rope(None, k, v, p, s, caches[1], table, q_out=q)


@pytest.mark.parametrize("rotated,base,scale", [(64, 10000.0, 1.0), (128, 1e6, 0.25), (32, 500.0, 1.0)])
def test_table(rotated, base, scale):
    """Off by half an FP32 step, and by what the angle (64 bits, positions up to 131072) is off: 2^-52 131072."""
    got = to_np(api.rope_table(131072, rotated, base, scale)).astype(np.float64)
    angle = np.arange(131072)[:, None] * scale * base ** (-2.0 * np.arange(rotated // 2) / rotated)
    want = np.stack([np.cos(angle), np.sin(angle)], -1)
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -24 + 131072 * 2.0 ** -50)


def test_far_positions_of_a_long_cache():
    """q and k of the same position turned alike: their product does not depend on the position, far ones included."""
    D, n = 128, 64
    table = api.rope_table(131072, D, 1e6)
    c = api.NVFP4KVCache.empty(8, 16, 1, D)
    x = torch.randn((1, 1, D), device="cuda").expand(n, 1, D).contiguous()
    pos = torch.linspace(0, 131071, n, device="cuda").int()
    q = api.nvfp4_kv_append_rope(x, x, x, pos, torch.arange(n, dtype=torch.int32, device="cuda"), c, table).float()[:, 0]
    norm = (q * q).sum(1)
    # BF16 rounds each of 128 elements by 2^-8 at most: 2^-7 of the sum of squares
    assert torch.all((norm - (x[0, 0] ** 2).sum()).abs() <= 2.0 ** -7 * (x[0, 0] ** 2).sum())


@pytest.mark.parametrize("tokens", [3, 4200])
def test_replayed_and_without_an_output(tokens):
    rng = np.random.default_rng(3)
    slots, positions, n_pages = _windows(tokens, 16, 3, rng)
    q = torch.randn((tokens, 6, 128), device="cuda").bfloat16()
    k, v = torch.randn((tokens, 2, 4, 128), device="cuda").bfloat16().unbind(1)
    table = api.rope_table(4000, 128)
    s, p = (torch.from_numpy(a.astype(np.int32)).cuda() for a in (slots, positions))
    caches = [api.NVFP4KVCache.empty(n_pages, 16, 4, 128) for _ in range(2)]
    for c in caches:
        c.pages.zero_()
    want = api.nvfp4_kv_append_rope(q, k, v, p, s, caches[0], table)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = api.nvfp4_kv_append_rope(q, k, v, p, s, caches[1], table)
    for _ in range(2):
        caches[1].pages.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(caches[0].pages, caches[1].pages)
