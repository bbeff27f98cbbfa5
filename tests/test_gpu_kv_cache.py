"""Rows into the NVFP4 KV cache and back: bytes equal to the recipe's, read values equal to what they stand for."""
import numpy as np
import pytest
import torch

from oracle import nvfp4 as Q
from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, bits, to_np

pytestmark = pytest.mark.gpu


def _rows(rng, n, heads, D, dtype):
    x = rng.standard_normal((n, heads, D)).astype(np.float32) * rng.choice([0.01, 1.0, 30.0], (n, heads, 1))
    x[:, :, 5::50] *= 20
    x = torch.from_numpy(x.astype(np.float32))
    return x if dtype == torch.float32 else x.to(dtype)


def _bf16_values(t):
    return Q.bf16_bits_to_f32(bits(t.to(torch.bfloat16)))


def _check_bytes(cache, pages_before, k, v, slots):
    want = pages_before.copy()
    live = [(s, i) for i, s in enumerate(slots) if 0 <= s < cache.num_pages * cache.page_size]
    kc, ks = S.quantize_rows(_bf16_values(k), float(cache.k_global))
    vc, vs = S.quantize_rows(_bf16_values(v), float(cache.v_global))
    at = [i for _, i in live]
    S.write_slots(want, [s for s, _ in live], cache.page_size, cache.head_dim, kc[at], ks[at], vc[at], vs[at])
    assert np.array_equal(to_np(cache.pages), want)


def _cache(num_pages, page, heads, D, kg=0.37, vg=0.011, seed=0):
    c = api.NVFP4KVCache.empty(num_pages, page, heads, D, kg, vg)
    c.pages.copy_(torch.from_numpy(np.random.default_rng(seed).integers(0, 256, c.pages.shape).astype(np.uint8)))
    return c


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,page,tokens", [(1, 16, 1), (8, 64, 8), (3, 48, 70), (2, 128, 300), (5, 32, 17), (1, 1024, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_bytes(D, heads, page, tokens, dtype):
    rng = np.random.default_rng(heads * page + tokens)
    n_pages = -(-tokens // page) + 3
    c = _cache(n_pages, page, heads, D)
    before = to_np(c.pages).copy()
    slots = rng.permutation(n_pages * page)[:tokens].astype(np.int32)
    slots[::7] = -1
    k, v = _rows(rng, tokens, heads, D, dtype), _rows(rng, tokens, heads, D, dtype)
    api.nvfp4_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), c)
    _check_bytes(c, before, k, v, slots)
    assert api.device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("start,tokens", [(0, 16), (0, 64), (5, 100), (15, 1), (3, 13), (16, 32), (1, 160)])
def test_append_runs_of_slots(D, start, tokens):
    """Consecutive slots (prompts) from any offset, whole groups and parts of them."""
    rng = np.random.default_rng(start * 1000 + tokens)
    c = _cache(4, 64, 2, D)
    before = to_np(c.pages).copy()
    slots = (np.arange(tokens) + start).astype(np.int32)
    k, v = _rows(rng, tokens, 2, D, torch.bfloat16), _rows(rng, tokens, 2, D, torch.bfloat16)
    api.nvfp4_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), c)
    _check_bytes(c, before, k, v, slots)


def test_append_long_run_and_padding():
    rng = np.random.default_rng(3)
    n, heads, D, page = 3000, 4, 128, 32
    c = _cache(110, page, heads, D)
    before = to_np(c.pages).copy()
    order = rng.permutation(110)
    pos = np.arange(n)
    slots = (order[pos // page] * page + pos % page).astype(np.int32)
    slots[2900:] = -1
    k, v = _rows(rng, n, heads, D, torch.bfloat16), _rows(rng, n, heads, D, torch.bfloat16)
    api.nvfp4_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), c)
    _check_bytes(c, before, k, v, slots)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_strided_rows(dtype):
    """K and V as column slices of one projection output, and with heads outermost."""
    rng = np.random.default_rng(4)
    T, H, D = 21, 2, 128
    x = _rows(rng, T, 3 * H, D, dtype).reshape(T, 3 * H * D).cuda()
    k, v = x[:, H * D:2 * H * D].unflatten(-1, (H, D)), x[:, 2 * H * D:].unflatten(-1, (H, D))
    slots = torch.arange(T, dtype=torch.int32, device="cuda") + 3
    c = _cache(3, 16, H, D)
    before = to_np(c.pages).copy()
    api.nvfp4_kv_append(k, v, slots, c)
    _check_bytes(c, before, k.cpu(), v.cpu(), to_np(slots))
    c2 = _cache(3, 16, H, D)
    api.nvfp4_kv_append(k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(0, 1).contiguous().transpose(0, 1),
                        slots, c2)
    assert torch.equal(c.pages, c2.pages)
    with pytest.raises(RuntimeError, match="ALIGN"):
        y = torch.zeros(T * (H * D + 1), dtype=dtype, device="cuda")
        bad = y.as_strided((T, H, D), (H * D + 1, D, 1))
        api.nvfp4_kv_append(bad, bad, slots, c)


def test_append_zero_and_extreme_blocks():
    c = _cache(1, 16, 1, 64, 1.0, 2.0 ** -9)
    before = to_np(c.pages).copy()
    k = torch.zeros((3, 1, 64))
    k[1, 0, 3], k[1, 0, 20], k[2, 0, :16] = -1e-30, 1e5, 1e30          # underflowing and saturating scales
    k[0, 0, 1] = -0.0
    slots = np.array([0, 7, 15], np.int32)
    api.nvfp4_kv_append(k.cuda(), k.cuda(), torch.from_numpy(slots).cuda(), c)
    _check_bytes(c, before, k, k, slots)


def test_slots_outside_the_cache_are_skipped_and_reported():
    rng = np.random.default_rng(6)
    c = _cache(2, 16, 2, 128)
    before = to_np(c.pages).copy()
    slots = np.array([3, 32, -2, 31, 2 ** 31 - 1, -2 ** 31, -1], np.int32)
    k, v = _rows(rng, 7, 2, 128, torch.bfloat16), _rows(rng, 7, 2, 128, torch.bfloat16)
    s = torch.from_numpy(slots).cuda()
    assert api.device_status() == 0
    api.nvfp4_kv_append(k.cuda(), v.cuda(), s, c)
    assert api.device_status() == api.DEVERR_KV_RANGE
    _check_bytes(c, before, k, v, slots)
    ko, vo = api.nvfp4_kv_read(c, s)
    assert api.device_status() == api.DEVERR_KV_RANGE
    gone = torch.tensor([1, 2, 4, 5, 6])
    assert not ko.cpu()[gone].any() and not vo.cpu()[gone].any() and ko.cpu()[0].any()


@pytest.mark.parametrize("D", [64, 128])
def test_read_values(D):
    """Any bytes: BF16 of the FP32 product code * (scale * global), exactly; NaN scales give NaN."""
    rng = np.random.default_rng(D)
    c = _cache(3, 32, 3, D, 0.37, 1.7, seed=D)
    slots = rng.permutation(96)[:77]
    gk, gv = Guarded((77, 3, D), torch.bfloat16), Guarded((77, 3, D), torch.bfloat16)
    api.nvfp4_kv_read(c, torch.from_numpy(slots.astype(np.int32)).cuda(), gk.t, gv.t)
    kc, ks, vc, vs = S.read_slots(to_np(c.pages), slots, 32, D)
    for g, codes, scales, glob in ((gk, kc, ks, 0.37), (gv, vc, vs, 1.7)):
        g.check("read output")
        step = (S.e4m3_decode(scales & 127).astype(np.float32) * np.float32(glob)).astype(np.float32)
        want = (S.e2m1_decode(codes).astype(np.float32).reshape(77, 3, -1, 16) * step[..., None]).reshape(77, 3, D)
        got = Q.bf16_bits_to_f32(bits(g.t))
        fine = np.repeat((scales & 127) != 127, 16, axis=-1).reshape(77, 3, D)
        ref = Q.bf16_bits_to_f32(Q.f32_to_bf16_bits(np.where(fine, want, 0).astype(np.float32)))
        assert np.array_equal(got[fine], ref[fine])


def test_append_beyond_four_gigabytes():
    """Byte offsets past 32 bits: the last pages of a cache of more than 4 GB."""
    heads, D, page = 8, 128, 64
    n_pages = (1 << 32) // (64 * 8 * 144) + 50
    c = api.NVFP4KVCache.empty(n_pages, page, heads, D)
    rng = np.random.default_rng(8)
    slots = (n_pages * page - 1 - np.arange(20) * 7).astype(np.int32)
    k, v = _rows(rng, 20, heads, D, torch.bfloat16), _rows(rng, 20, heads, D, torch.bfloat16)
    s = torch.from_numpy(slots).cuda()
    api.nvfp4_kv_append(k.cuda(), v.cuda(), s, c)
    ko, vo = api.nvfp4_kv_read(c, s)
    kc, ks = S.quantize_rows(_bf16_values(k), 1.0)
    want = S.dequantize_rows(kc, ks, 1.0)
    assert np.array_equal(Q.bf16_bits_to_f32(bits(ko)).astype(np.float64), want)
    tail = to_np(c.pages[-3:])
    got = S.read_slots(tail, slots - (n_pages - 3) * page, page, D)
    assert np.array_equal(got[0], kc) and np.array_equal(got[1], ks)
    assert api.device_status() == 0


def test_another_stream():
    rng = np.random.default_rng(10)
    c = _cache(4, 16, 2, 128)
    before = to_np(c.pages).copy()
    k, v = _rows(rng, 40, 2, 128, torch.bfloat16), _rows(rng, 40, 2, 128, torch.bfloat16)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    kd, vd = k.cuda(), v.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.nvfp4_kv_append(kd, vd, slots, c, stream=st)
    st.synchronize()
    _check_bytes(c, before, k, v, to_np(slots))
