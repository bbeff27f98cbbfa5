"""Attention over the NVFP4 cache against FP64.

What the kernels round (u = 2^-24, half an FP32 step):
* the dequantized keys and values are exact, FP32 queries are first rounded to BF16 (the oracle's queries are);
* queries enter the matrix instructions as FP16 of q / max|q|: exact above 2^-14 of the maximum, else off by at
  most 2^-25 of it, so a score is off by at most u Q with Q = scale max|q| sum|k|;
* a score is an FP32 sum of D products: off by at most (D + 8) u S, S = scale sum|q k|;
* so a weight exp(s - m) is off by the factor e = u ((D + 8) S + Q) plus a few u (the exponential and its
  argument, whose rounding grows with |s|, at most S), and by a rounding to FP16 that it may get before it
  multiplies V: 2^-11 relative, or 2^-25 absolute below 2^-14;
* the sums over n keys are FP32: (n + 64) u each, numerator and denominator;
* the result is rounded to BF16: 2^-8 of its magnitude.
With A = sum w|v| / sum w and B = sum|v| / sum w:
  |out - ref| <= 2^-8 (|ref| + t) + t,  t = A (2^-11 + 2 e + 2 (n + 64) u + 8 u (S + 1)) + 2^-24 B
  |lse - ref| <= e + (n + 64) u + 8 u (S + 1) + u |ref|
"""
import numpy as np
import pytest
import torch

from oracle import nvfp4 as Q
from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, bits, to_np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _cache(rng, num_pages, page, heads, D, kg=0.25, vg=0.05):
    """A cache of random codes with scales of all magnitudes around 1."""
    c = api.NVFP4KVCache.empty(num_pages, page, heads, D, kg, vg)
    shape = (num_pages * page, heads)
    put = []
    for _ in range(2):
        put.append(rng.integers(0, 16, shape + (D,)).astype(np.uint8))
        put.append(rng.integers(40, 72, shape + (D // 16,)).astype(np.uint8))
    pages = np.zeros(c.pages.shape, np.uint8)
    S.write_slots(pages, np.arange(num_pages * page), page, D, *put)
    c.pages.copy_(torch.from_numpy(pages))
    k = S.dequantize_rows(put[0], put[1], kg)
    v = S.dequantize_rows(put[2], put[3], vg)
    return c, k, v, pages


def _table(rng, lens, page, num_pages, width=None):
    used = [-(-n // page) for n in lens]
    width = width or max(1, max(used))
    ids = rng.permutation(num_pages)
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(used):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


def _queries(rng, tokens, heads, D, dtype, spread):
    q = torch.from_numpy((rng.standard_normal((tokens, heads, D)) * spread).astype(np.float32)).to(dtype)
    return q, Q.bf16_bits_to_f32(bits(q.to(torch.bfloat16))).astype(np.float64)


def _check(out, lse, b0, q64, k, v, scale, window):
    m = q64.shape[0]
    ref, ref_lse, A, B, Sx, Qx = S.attention(q64, k, v, scale, window)
    n, D = k.shape[0], q64.shape[2]
    e = (U * ((D + 8) * Sx + Qx))[..., None]
    few = (8 * U * (Sx + 1))[..., None]
    t = A * (2.0 ** -11 + 2 * e + 2 * (n + 64) * U + few) + 2.0 ** -24 * B
    got = Q.bf16_bits_to_f32(bits(out[b0:b0 + m])).astype(np.float64)
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + t) + t)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], got[bad][:3], ref[bad][:3])
    if lse is not None:
        g = to_np(lse[b0:b0 + m]).astype(np.float64)
        none = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(g), none)
        tol = e[..., 0] + (n + 64) * U + few[..., 0] + U * np.abs(np.where(none, 0, ref_lse))
        assert np.all(np.abs(g - ref_lse)[~none] <= tol[~none])


def _run(seed, lens, rows, heads, kvh, D, page, window=0, dtype=torch.bfloat16, spread=1.0, scale=None, max_q=None,
         with_lse=True, poison=True):
    rng = np.random.default_rng(seed)
    num_pages = sum(-(-n // page) for n in lens) + 2
    c, k, v, pages = _cache(rng, num_pages, page, kvh, D)
    t = _table(rng, lens, page, num_pages)
    if poison:
        # what lies behind a request's last key (in its own last page, and in pages of nobody) is NaN and garbage
        for b, n in enumerate(lens):
            if n % page:
                p = t[b, n // page]
                full = np.full((1, kvh, page // 16, 18 * D), 0xFF, np.uint8)
                slots = p * page + np.arange(n % page)
                S.write_slots(full, np.arange(n % page), page, D, *S.read_slots(pages, slots, page, D))
                pages[p] = full[0]
        c.pages.copy_(torch.from_numpy(pages))
    total = sum(rows)
    q, q64 = _queries(rng, total, heads, D, dtype, spread)
    scale = scale or D ** -0.5
    g = Guarded((total, heads, D), torch.bfloat16)
    gl = Guarded((total, heads), torch.float32)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    decode = all(r == 1 for r in rows)
    api.nvfp4_kv_attention(q.cuda(), c, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           None if decode else torch.from_numpy(cu).cuda(), max_q=max_q, scale=scale, window=window,
                           out=g.t, lse=gl.t if with_lse else None)
    g.check("attention out")
    gl.check("attention lse")
    for b, n in enumerate(lens):
        at = np.arange(n)
        slots = t[b, at // page] * page + at % page
        _check(g.t, gl.t if with_lse else None, cu[b], q64[cu[b]:cu[b + 1]], k[slots], v[slots], scale, window)
    assert api.device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 1000])
def test_decode_lengths(D, n):
    _run(n + D, [n], [1], 8, 2, D, 64)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16, 24, 33, 64])
def test_decode_groups(D, group):
    _run(group, [100, 37], [1, 1], group * 2, 2, D, 32, dtype=torch.float32)


@pytest.mark.parametrize("page", [16, 32, 48, 112, 128, 1024])
def test_decode_pages_and_ragged_batch(page):
    _run(page, [0, 1, 500, 77, 2049, 0, 16], [1] * 7, 5, 1, 128, page)


@pytest.mark.parametrize("batch,kvh,n", [(64, 1, 40), (130, 2, 9), (3, 16, 300), (1, 1, 9000), (2, 3, 5000), (300, 1, 3)])
def test_decode_batches(batch, kvh, n):
    _run(batch, [max(0, n - 3 * (i % 5)) for i in range(batch)], [1] * batch, 4 * kvh, kvh, 64, 16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 16, 50, 64, 65, 1000])
def test_windows(D, window):
    _run(window, [1, 64, 333, 40, 0], [1] * 5, 6, 2, D, 32, window=window)
    _run(window + 1, [90, 333, 5], [9, 3, 5], 6, 2, D, 32, window=window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,lens", [((2,), (2,)), ((8, 5, 1, 3), (70, 5, 1, 200)), ((3, 4), (1, 0)), ((7,), (400,)),
                                       ((0, 6, 0, 2), (9, 44, 0, 300)), ((17, 40), (17, 130)), ((33,), (600,))])
def test_several_rows_a_request(D, rows, lens):
    """Causal rows, requests without rows, rows that see nothing (fewer keys than rows)."""
    _run(sum(rows), list(lens), list(rows), 8, 2, D, 16)
    _run(sum(rows) + 1, list(lens), list(rows), 5, 1, D, 64, dtype=torch.float32)


@pytest.mark.parametrize("group", [1, 3, 8, 16, 20])
def test_prefill_chunks(group):
    _run(group, [130, 257, 64], [130, 100, 64], group, 1, 128, 64)
    _run(group + 1, [300], [129], 2 * group, 2, 64, 32, window=100)


def test_max_q_chooses_nothing_but_speed():
    """Any max_q gives results within the same bounds."""
    for max_q in (1, 2, 8, 200, 10 ** 6):
        _run(7, [200, 33, 5], [20, 1, 9], 8, 2, 128, 32, max_q=max_q)


@pytest.mark.parametrize("spread", [1e-3, 6.0, 40.0])
def test_flat_and_peaked_weights(spread):
    _run(21, [700, 65], [1, 1], 8, 2, 128, 64, spread=spread)
    _run(22, [300], [12], 8, 2, 64, 64, spread=spread, scale=0.7)


def test_growing_scores():
    """Scores that rise along the keys, so that the running maximum changes at every step."""
    rng = np.random.default_rng(1)
    D, page, n = 128, 64, 1500
    c, k, v, pages = _cache(rng, 24, page, 1, D)
    codes, scales = np.full((n, 1, D), 2, np.uint8), np.zeros((n, 1, D // 16), np.uint8)
    scales[:] = np.minimum(8 + np.arange(n) // 15, 118)[:, None, None]
    _, _, vc, vs = S.read_slots(pages, np.arange(n), page, D)
    S.write_slots(pages, np.arange(n), page, D, codes, scales, vc, vs)
    c.pages.copy_(torch.from_numpy(pages))
    k[:n] = S.dequantize_rows(codes, scales, 0.25)
    t = np.arange(24, dtype=np.int32)[None]
    q, q64 = _queries(rng, 1, 4, D, torch.bfloat16, 0.02)
    q = torch.abs(q)
    q64 = np.abs(q64)
    lse = torch.empty((1, 4), device="cuda")
    out = api.nvfp4_kv_attention(q.cuda(), c, torch.from_numpy(t).cuda(), torch.tensor([n], dtype=torch.int32).cuda(), lse=lse)
    _check(out, lse, 0, q64, k[:n], v[:n], D ** -0.5, 0)


def test_queries_of_very_different_magnitudes():
    """Rows of one call whose queries differ by 2^40, a zero row, and elements far below their row's maximum."""
    rng = np.random.default_rng(2)
    D, page, n = 64, 16, 90
    c, k, v, _ = _cache(rng, 8, page, 2, D)
    t = _table(rng, [n], page, 8)
    q, _ = _queries(rng, 1, 12, D, torch.bfloat16, 1.0)
    q = q.float() * (2.0 ** torch.linspace(-30, 4, 12))[None, :, None]
    q[:, 3] = 0
    q[:, 5, ::2] *= 2.0 ** -20
    q = q.to(torch.bfloat16)
    q64 = Q.bf16_bits_to_f32(bits(q)).astype(np.float64)
    out = api.nvfp4_kv_attention(q.cuda(), c, torch.from_numpy(t).cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    at = np.arange(n)
    slots = t[0, at // page] * page + at % page
    _check(out, None, 0, q64, k[slots], v[slots], D ** -0.5, 0)


def test_strided_queries_and_shared_output():
    """Queries as the first columns of the projection output; the same bits as dense queries."""
    rng = np.random.default_rng(3)
    D, H, kvh, page = 128, 8, 2, 32
    lens = [77, 200]
    c, k, v, _ = _cache(rng, 12, page, kvh, D)
    t = torch.from_numpy(_table(rng, lens, page, 12)).cuda()
    x = torch.from_numpy(rng.standard_normal((2, (H + 2 * kvh) * D)).astype(np.float32)).cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    for y in (x, x.to(torch.bfloat16)):
        q = y[:, :H * D].unflatten(-1, (H, D))
        a = api.nvfp4_kv_attention(q, c, t, kv)
        b = api.nvfp4_kv_attention(q.contiguous(), c, t, kv)
        h = api.nvfp4_kv_attention(q.transpose(0, 1).contiguous().transpose(0, 1), c, t, kv)
        assert torch.equal(a, b) and torch.equal(a, h)
    # FP32 queries are rounded to BF16 first
    q = x[:, :H * D].unflatten(-1, (H, D))
    assert torch.equal(api.nvfp4_kv_attention(q, c, t, kv), api.nvfp4_kv_attention(q.to(torch.bfloat16), c, t, kv))


def test_bad_pages_and_lengths_are_skipped_and_reported():
    """Table entries outside the cache count as unseen keys, lengths beyond the table are cut: reported, no fault."""
    rng = np.random.default_rng(4)
    D, page = 128, 32
    c, k, v, _ = _cache(rng, 6, page, 1, D)
    t = np.array([[2, 99, 4], [0, -1, 5], [1, 3, 2 ** 31 - 1]], np.int32)
    lens = [90, 96, 70]
    q, q64 = _queries(rng, 3, 4, D, torch.bfloat16, 1.0)
    assert api.device_status() == 0
    args = (q.cuda(), c, torch.from_numpy(t).cuda())
    out = api.nvfp4_kv_attention(*args, torch.tensor(lens, dtype=torch.int32).cuda())
    assert api.device_status() == api.DEVERR_KV_RANGE
    for b, n in enumerate(lens):
        at = np.arange(n)
        pg = t[b, at // page]
        ok = (pg >= 0) & (pg < 6)
        slots = (pg[ok].astype(np.int64) * page + at[ok] % page)
        _check(out, None, b, q64[b:b + 1], k[slots], v[slots], D ** -0.5, 0)
    t2 = torch.tensor([[0, 1, 2], [3, 4, 5], [5, 1, 0]], dtype=torch.int32).cuda()
    full = api.nvfp4_kv_attention(args[0], c, t2, torch.tensor([96, 96, 96], dtype=torch.int32).cuda())
    assert api.device_status() == 0
    long = api.nvfp4_kv_attention(args[0], c, t2, torch.tensor([97, 96, 2 ** 31 - 1], dtype=torch.int32).cuda())
    assert api.device_status() == api.DEVERR_KV_RANGE
    assert torch.equal(full, long)
    neg = api.nvfp4_kv_attention(args[0], c, t2, torch.tensor([-5, 96, 96], dtype=torch.int32).cuda())
    assert not neg[0].any() and torch.equal(neg[1:], full[1:])
    api.device_status()


def test_row_ranges_outside_the_rows_are_skipped():
    """cu_q beyond the query rows, decreasing or negative: no fault, no write outside, rows of no request untouched."""
    rng = np.random.default_rng(5)
    D, page = 64, 16
    c, k, v, _ = _cache(rng, 6, page, 1, D)
    t = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32).cuda()
    q, _ = _queries(rng, 6, 2, D, torch.bfloat16, 1.0)
    lens = torch.tensor([40, 48], dtype=torch.int32).cuda()
    for cu in ([0, 3, 9], [0, 100, 6], [-4, 2, 6], [5, 2, 1], [0, 2 ** 31 - 1, -2 ** 31], [2, 2, 4]):
        for max_q in (1, 6, 200):
            g = Guarded((6, 2, D), torch.bfloat16)
            api.nvfp4_kv_attention(q.cuda(), c, t, lens, torch.tensor(cu, dtype=torch.int32).cuda(), max_q=max_q, out=g.t)
            g.check("attention out")
            api.device_status()
    g.t.fill_(7.0)
    api.nvfp4_kv_attention(q.cuda(), c, t, lens, torch.tensor([2, 2, 4], dtype=torch.int32).cuda(), out=g.t)
    assert torch.all(g.t[:2] == 7) and torch.all(g.t[4:] == 7) and not torch.any(g.t[2:4] == 7)
    assert api.device_status() == 0


def test_cache_beyond_four_gigabytes():
    D, page, kvh = 128, 64, 8
    n_pages = (1 << 32) // (page * kvh * 144) + 20
    rng = np.random.default_rng(6)
    small, k, v, pages = _cache(rng, 8, page, kvh, D)
    c = api.NVFP4KVCache.empty(n_pages, page, kvh, D, 0.25, 0.05)
    c.pages[-8:].copy_(small.pages)
    t = _table(rng, [333, 100], page, 8)
    q, q64 = _queries(rng, 2, 16, D, torch.bfloat16, 1.0)
    lens = torch.tensor([333, 100], dtype=torch.int32).cuda()
    far = np.where(t >= 0, t + n_pages - 8, -1).astype(np.int32)
    a = api.nvfp4_kv_attention(q.cuda(), small, torch.from_numpy(t).cuda(), lens)
    b = api.nvfp4_kv_attention(q.cuda(), c, torch.from_numpy(far).cuda(), lens)
    assert torch.equal(a, b)


def test_repeat_streams_and_graph():
    """The same bits on every call, on another stream and from a captured graph, with one workspace over calls of
    different shapes."""
    rng = np.random.default_rng(7)
    D, page, kvh, H = 128, 64, 2, 16
    lens = [1500, 10, 800]
    c, k, v, _ = _cache(rng, 40, page, kvh, D)
    t = torch.from_numpy(_table(rng, lens, page, 40)).cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    q, _ = _queries(rng, 3, H, D, torch.bfloat16, 1.0)
    q = q.cuda()
    ws = torch.zeros(api.nvfp4_kv_attention_workspace_bytes(64, 300, 64, kvh, D), dtype=torch.uint8, device="cuda")
    first = api.nvfp4_kv_attention(q, c, t, kv, workspace=ws)
    for i in range(5):
        q2, _ = _queries(rng, 2 + i, 4, D, torch.bfloat16, 1.0)
        api.nvfp4_kv_attention(q2.cuda(), c, t[:1], kv[:1], torch.tensor([0, 2 + i], dtype=torch.int32).cuda(), workspace=ws)
        assert torch.equal(first, api.nvfp4_kv_attention(q, c, t, kv, workspace=ws))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    api.nvfp4_kv_attention(q, c, t, kv, out=out, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(first, out)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.nvfp4_kv_attention(q, c, t, kv, out=out, workspace=ws)
    for n in ([1500, 10, 800], [1, 640, 0], [1500, 10, 800]):
        kv.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        got = out.clone()
        assert torch.equal(got, api.nvfp4_kv_attention(q, c, t, kv))
    assert torch.equal(first, out)
    assert api.device_status() == api.DEVERR_KV_RANGE      # request 1 has no pages for the 640 keys of the second replay


@pytest.mark.parametrize("D", [64, 128])
def test_growing_scores_of_many_rows(D):
    """Scores that rise along the keys by far more than FP16 holds, and fall again, for prompt rows: the maximum that
    the weights refer to has to move again and again, and to stay."""
    rng = np.random.default_rng(8)
    page, n, m, H = 64, 900, 70, 4
    c, k, v, pages = _cache(rng, 15, page, 1, D)
    codes, scales = np.full((n, 1, D), 2, np.uint8), np.zeros((n, 1, D // 16), np.uint8)
    ramp = np.concatenate([np.arange(600), 600 - 2 * np.arange(300)])
    scales[:] = np.clip(8 + ramp // 6, 0, 118)[:, None, None]
    _, _, vc, vs = S.read_slots(pages, np.arange(n), page, D)
    S.write_slots(pages, np.arange(n), page, D, codes, scales, vc, vs)
    c.pages.copy_(torch.from_numpy(pages))
    k[:n] = S.dequantize_rows(codes, scales, 0.25)
    t = torch.arange(15, dtype=torch.int32).cuda()[None]
    q, _ = _queries(rng, m, H, D, torch.bfloat16, 0.02)
    q = q * torch.tensor([1.0, -1.0, 30.0, 0.0], dtype=torch.bfloat16)[None, :, None]
    q[:, :3] = torch.abs(q[:, :3]) * torch.sign(q[:, :3, :1])
    q64 = Q.bf16_bits_to_f32(bits(q)).astype(np.float64)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    cu = torch.tensor([0, m], dtype=torch.int32).cuda()
    for max_q in (1, m):                                # both kernels
        lse = torch.empty((m, H), device="cuda")
        out = api.nvfp4_kv_attention(q.cuda(), c, t, lens, cu, max_q=max_q, lse=lse)
        _check(out, lse, 0, q64, k[:n], v[:n], D ** -0.5, 0)
    assert api.device_status() == 0


def test_many_rows_few_tiles_are_cut_and_merged():
    """Prompt rows of few tiles over many keys (pieces merged by a second launch), with a window, rows of the second
    half missing, and lse; the same bits on repeat calls."""
    for seed, lens, rows, heads, kvh, D, window in ((31, [3000], [40], 8, 2, 128, 0), (32, [2500, 1900], [33, 70], 4, 2, 64, 0),
                                                   (33, [4000], [300], 2, 1, 64, 1500), (34, [1700], [90], 3, 1, 128, 700)):
        _run(seed, lens, rows, heads, kvh, D, 64, window=window, max_q=1000)
    rng = np.random.default_rng(35)
    c, k, v, _ = _cache(rng, 50, 64, 2, 128)
    t = torch.from_numpy(_table(rng, [3100], 64, 50)).cuda()
    q, _ = _queries(rng, 64, 8, 128, torch.bfloat16, 1.0)
    args = (q.cuda(), c, t, torch.tensor([3100], dtype=torch.int32).cuda(), torch.tensor([0, 64], dtype=torch.int32).cuda())
    a = api.nvfp4_kv_attention(*args, max_q=64)
    for _ in range(3):
        assert torch.equal(a, api.nvfp4_kv_attention(*args, max_q=64))


@pytest.mark.parametrize("batch", [33, 200])
def test_prompt_rows_of_many_requests(batch):
    """More requests than a warp counts at once, prompt chunks among single rows and empty requests."""
    rows = [0 if i % 7 == 3 else 70 if i % 11 == 0 else 1 for i in range(batch)]
    _run(batch, [max(r, (37 * i) % 200) for i, r in enumerate(rows)], rows, 4, 1, 64, 16, max_q=70)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 700])
def test_many_rows_of_unequal_lengths(D, window):
    """Requests whose tiles are cut into different numbers of pieces, tiles in one half, in both, and of each with an
    odd number of steps."""
    _run(90 + window, [4100, 90, 0, 2500, 1300, 129], [8, 9, 20, 40, 7, 16], 16, 2, D, 64, window=window)


def test_many_rows_of_more_requests_than_a_warp_has_lanes():
    """Pieces are found across groups of 32 requests, some of them empty."""
    lens = [(i * 531) % 3001 for i in range(45)]
    _run(93, lens, [min(7 + i % 3, n) if i % 7 else 0 for i, n in enumerate(lens)], 8, 1, 128, 32)
