"""Append and read of prompts, where a warp takes a window of 16 tokens: bytes and values equal to the recipe's.

Calls of up to 2^21 elements of K go block by block; everything here is larger.
"""
import numpy as np
import pytest
import torch

from oracle import nvfp4 as Q
from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, bits, to_np
from tests.test_gpu_kv_cache import _bf16_values, _cache, _rows

pytestmark = pytest.mark.gpu

FEW = 1 << 21


def _put(pages, slots, page, D, kc, ks, vc, vs):
    """S.write_slots for distinct slots, all at once."""
    o = S.GroupOffsets(D)
    rows = pages[slots // page, :, slots % page // 16]
    t = slots % 16
    for off, val in ((o.k_codes[:, ::2], kc[:, :, ::2] | (kc[:, :, 1::2] << 4)),
                     (o.v_codes[:, ::2], vc[:, :, ::2] | (vc[:, :, 1::2] << 4)), (o.k_scales, ks), (o.v_scales, vs)):
        # tokens of one group hit the same row of `pages` in different bytes
        p, g = slots // page, slots % page // 16
        h = np.arange(rows.shape[1])
        pages[p[:, None, None], h[None, :, None], g[:, None, None], off[t][:, None]] = val


def _check_append(cache, before, k, v, slots):
    want = before.copy()
    slots = np.asarray(slots, np.int64)
    at = np.flatnonzero((slots >= 0) & (slots < cache.num_pages * cache.page_size))
    kc, ks = S.quantize_rows(_bf16_values(k)[at], float(cache.k_global))
    vc, vs = S.quantize_rows(_bf16_values(v)[at], float(cache.v_global))
    _put(want, slots[at], cache.page_size, cache.head_dim, kc, ks, vc, vs)
    assert np.array_equal(to_np(cache.pages), want)


def _check_read(cache, slots):
    n, H, D = len(slots), cache.kv_heads, cache.head_dim
    gk, gv = Guarded((n, H, D), torch.bfloat16), Guarded((n, H, D), torch.bfloat16)
    api.nvfp4_kv_read(cache, torch.from_numpy(slots).cuda(), gk.t, gv.t)
    live = (slots >= 0) & (slots < cache.num_pages * cache.page_size)
    kc, ks, vc, vs = S.read_slots(to_np(cache.pages), slots[live].astype(np.int64), cache.page_size, D)
    for g, codes, scales, glob in ((gk, kc, ks, cache.k_global), (gv, vc, vs, cache.v_global)):
        g.check("read output")
        got = bits(g.t)
        assert not got[~live].any()
        step = (S.e4m3_decode(scales & 127).astype(np.float32) * np.float32(float(glob))).astype(np.float32)
        want = S.e2m1_decode(codes).astype(np.float32).reshape(scales.shape + (16,)) * step[..., None]
        fine = np.repeat((scales & 127) != 127, 16, axis=-1)
        want = Q.f32_to_bf16_bits(np.where(fine, want.reshape(codes.shape), 0).astype(np.float32))
        assert np.array_equal(got[live][fine], want[fine])


def _runs(rng, tokens, n_pages, page, lens):
    """Slots of requests of these lengths one after the other, each from its own offset, pages in no order."""
    order = rng.permutation(n_pages)
    out, p = [], 0
    for i, n in enumerate(lens):
        start = int(rng.integers(0, page)) if i % 3 else 0
        pos = np.arange(start, start + n)
        out.append(order[p + pos // page] * page + pos % page)
        p += (start + n - 1) // page + 1
    return np.concatenate(out)[:tokens].astype(np.int32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,page,lens", [(160, 16, (33, 16, 1, 100, 15, 17, 48)), (37, 48, (500, 1, 1, 7, 300, 95)),
                                             (1024, 32, (33,)), (8, 64, (2100, 2000, 31))])
def test_append_and_read_of_prompts(D, dtype, heads, page, lens):
    """Whole groups that start anywhere in a window, parts of groups, padding and bad slots inside runs, a token
    count that is no multiple of 16."""
    rng = np.random.default_rng(heads + page)
    tokens = sum(lens)
    while tokens * heads * D <= FEW:
        lens += lens
        tokens = sum(lens)
    n_pages = sum(-(-n // page) + 1 for n in lens) + 2
    slots = _runs(rng, tokens, n_pages, page, lens)
    bad = rng.integers(0, tokens, max(4, tokens // 60))
    slots[bad[::2]] = -1
    slots[bad[1::4]] = n_pages * page + 5
    slots[bad[3::4]] = -7
    c = _cache(n_pages, page, heads, D)
    before = to_np(c.pages).copy()
    k, v = _rows(rng, tokens, heads, D, dtype), _rows(rng, tokens, heads, D, dtype)
    k[3, 0, :16], v[5, 0, 16:32] = 0, 0
    assert api.device_status() == 0
    api.nvfp4_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), c)
    assert api.device_status() == api.DEVERR_KV_RANGE
    _check_append(c, before, k, v, slots)
    _check_read(c, slots)
    assert api.device_status() == api.DEVERR_KV_RANGE


@pytest.mark.parametrize("D", [64, 128])
def test_append_and_read_of_scattered_tokens_and_padding(D):
    """No run at all, and a window's worth of padding in between: the same kernels, block by block."""
    rng = np.random.default_rng(D)
    heads, page = 64, 32
    tokens = FEW // (heads * D) + 45
    n_pages = -(-tokens // page) + 3
    slots = rng.permutation(n_pages * page)[:tokens].astype(np.int32)
    slots[100:150] = -1
    c = _cache(n_pages, page, heads, D)
    before = to_np(c.pages).copy()
    k, v = _rows(rng, tokens, heads, D, torch.bfloat16), _rows(rng, tokens, heads, D, torch.bfloat16)
    api.nvfp4_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), c)
    _check_append(c, before, k, v, slots)
    _check_read(c, slots)
    assert api.device_status() == 0


def test_append_of_strided_prompts():
    """K and V as column slices of one projection's output, FP32 and BF16."""
    rng = np.random.default_rng(12)
    H, D, page = 8, 128, 64
    tokens = FEW // (H * D) + 77
    for dtype in (torch.float32, torch.bfloat16):
        x = _rows(rng, tokens, 3 * H, D, dtype).reshape(tokens, 3 * H * D).cuda()
        k, v = x[:, H * D:2 * H * D].unflatten(-1, (H, D)), x[:, 2 * H * D:].unflatten(-1, (H, D))
        c = _cache(tokens // page + 2, page, H, D)
        before = to_np(c.pages).copy()
        slots = np.arange(tokens, dtype=np.int32) + 9
        api.nvfp4_kv_append(k, v, torch.from_numpy(slots).cuda(), c)
        _check_append(c, before, k.cpu(), v.cpu(), slots)


def test_windows_and_blocks_give_the_same_bytes():
    rng = np.random.default_rng(13)
    H, D, page = 8, 128, 64
    tokens = FEW // (H * D) + 300
    k, v = _rows(rng, tokens, H, D, torch.bfloat16).cuda(), _rows(rng, tokens, H, D, torch.bfloat16).cuda()
    slots = torch.arange(tokens, dtype=torch.int32, device="cuda") + 3
    a, b = (_cache(tokens // page + 2, page, H, D) for _ in range(2))
    api.nvfp4_kv_append(k, v, slots, a)
    for i in range(0, tokens, 500):
        api.nvfp4_kv_append(k[i:i + 500], v[i:i + 500], slots[i:i + 500], b)
    assert torch.equal(a.pages, b.pages)
