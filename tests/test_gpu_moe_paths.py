"""The experts' kernels where a CTA has several items and its ring of stages goes round, with K split over clusters of every
size, with y in several slabs, and at the sizes of a model: columns of every row tile against FP64.

Tolerances as in test_gpu_moe_experts.py.  The kernels' tiles: 64 places with rows copied by loader warps, 256 with rows laid
out by place (128 places an accumulator).  On 152 SMs; on others the sizes reach some of these paths only.
"""
import numpy as np
import pytest
import torch

from oracle import moe as O
from oracle import nvfp4 as Q
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import bits, to_np

pytestmark = pytest.mark.gpu


def _nvfp4(g, *shape):
    """Random codes and scales (2^-3 .. 3.75) of rows of shape[-1] elements."""
    codes = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(0x20, 0x48, shape[:-1] + (shape[-1] // 16,), generator=g, dtype=torch.uint8, device="cuda")
    return codes, scales


def _plan(counts, k, seed, none=0):
    """ids [T, k] with so many pairs of each expert (and `none` of no expert), shuffled; weights; plan."""
    rng = np.random.default_rng(seed)
    flat = np.concatenate([np.repeat(np.arange(len(counts)), counts), np.full(none, -1)])
    ids = rng.permutation(flat).reshape(-1, k).astype(np.int32)
    weights = rng.random(ids.shape).astype(np.float32)
    r = api.nvfp4_moe_plan(torch.from_numpy(ids).cuda(), len(counts), torch.from_numpy(weights).cuda())
    offsets, pairs, places = O.plan(ids, len(counts))
    assert np.array_equal(to_np(r.offsets), offsets) and np.array_equal(to_np(r.places), places)
    return r, weights, offsets, pairs, places


def _some(n, step, rng):
    """A column of every `step` of n, and the last."""
    return np.unique(np.append(np.minimum(np.arange(0, n, step) + rng.integers(0, step, -(-n // step)), n - 1), n - 1))


def _check_up(r, plan, K, inter, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    E, k = r.experts, r.top_k
    _, offsets, pairs, _ = plan
    xc, xs = _nvfp4(g, r.tokens, K)
    wc, ws = _nvfp4(g, E, 2 * inter, K)
    xg, wg = 1.0 / 3, ((1 + np.arange(E) % 3) / K ** 0.5 / 16).astype(np.float32)
    w = api.nvfp4_moe_pack_weights(wc, ws, torch.from_numpy(wg).cuda(), True)
    x = api.NVFP4Tensor(xc, xs, torch.tensor([xg], device="cuda"))
    h = api.nvfp4_moe_gate_up(x, w, r)
    again = api.nvfp4_moe_gate_up(x, w, r)
    got = Q.bf16_bits_to_f32(bits(h)).astype(np.float64)
    assert torch.equal(h, again) and not got[offsets[-1]:].any()
    at = _some(inter, 64, np.random.default_rng(seed))
    rows = torch.from_numpy(np.concatenate([at, inter + at])).cuda()
    xv = O.values(to_np(xc), to_np(xs), xg)
    c = (K / 64 + 12) * 2.0 ** -23
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        wv = O.values(to_np(wc[e, rows]), to_np(ws[e, rows]), wg[e])
        xe = xv[pairs[a:b] // k]
        gu, B = xe @ wv.T, np.abs(xe) @ np.abs(wv).T
        n = len(at)
        G, U, Bg, Bu = gu[:, :n], gu[:, n:], B[:, :n], B[:, n:]
        silu = G / (1.0 + np.exp(-G))
        tol = (1.1 * c * Bg * (np.abs(U) + c * Bu) + (np.abs(silu) + 1.1 * c * Bg) * c * Bu
               + np.abs(silu * U) * (2.0 ** -8 + 2.0 ** -15))
        assert np.all(np.abs(got[a:b][:, at] - silu * U) <= tol + 1e-37), e
    assert api.device_status() == 0


def _check_down(r, plan, K, N, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    E = r.experts
    weights, offsets, _, places = plan
    hc, hs = _nvfp4(g, r.tokens * r.top_k, K)
    wc, ws = _nvfp4(g, E, N, K)
    hg, wg = 0.7, ((1 + np.arange(E) % 5) / K ** 0.5 / 16).astype(np.float32)
    w = api.nvfp4_moe_pack_weights(wc, ws, torch.from_numpy(wg).cuda(), False)
    h = api.NVFP4Tensor(hc, hs, torch.tensor([hg], device="cuda"))
    y = api.nvfp4_moe_down(h, w, r)
    again = api.nvfp4_moe_down(h, w, r)
    assert torch.equal(y, again)
    at = _some(N, 128, np.random.default_rng(seed))
    rows = torch.from_numpy(at).cuda()
    hv = O.values(to_np(hc), to_np(hs), hg)
    part, size = np.zeros((2, hv.shape[0] + 1, len(at)))          # the last: pairs without a place
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            wv = O.values(to_np(wc[e, rows]), to_np(ws[e, rows]), wg[e])
            part[a:b], size[a:b] = hv[a:b] @ wv.T, np.abs(hv[a:b]) @ np.abs(wv).T
    want, B = np.zeros((2, r.tokens, len(at)))
    for j in range(r.top_k):
        f = weights[:, j, None].astype(np.float64)
        want += f * part[places[:, j]]
        B += f * size[places[:, j]]
    tol = (K / 64 + 12 + r.top_k + 8) * 2.0 ** -23 * B
    got = to_np(y[:, rows]).astype(np.float64)
    assert np.all(np.abs(got - want) <= tol + 1e-37), (np.abs(got - want) / (tol + 1e-37)).max()
    assert api.device_status() == 0


# More items than SMs, four to a CTA; experts of several tiles (the last of them of one accumulator, of two, of 192 columns),
# of 129 to 256 and of up to 128 places, some without any; 7 chunks of K, the last of 64.
COUNTS = [0, 600, 100, 300, 1, 200, 150, 0, 429, 20]


def test_gate_up_many_items_of_a_cta():
    r, *plan = _plan(COUNTS, 2, 1, none=6)
    _check_up(r, plan, 1600, 4352)


def test_down_many_items_of_a_cta():
    r, *plan = _plan(COUNTS, 2, 2, none=6)
    _check_down(r, plan, 1600, 8700)


# few places: no cluster, four items of 7 chunks a CTA; one item of 16; K split over 8 CTAs
@pytest.mark.parametrize("counts,k,K,inter", [([3] * 40, 2, 1600, 1024), ([12, 30, 2, 64, 100], 4, 4096, 1024),
                                              ([1, 2, 1], 2, 2048, 64), ([1, 3], 1, 2112, 64)])
def test_gate_up_few_places(counts, k, K, inter):
    r, *plan = _plan(counts, k, 3)
    _check_up(r, plan, K, inter)


# 7, 6, 5, 4, 3, 2 CTAs a tile of y's columns, and one
@pytest.mark.parametrize("N", [2600, 3200, 3500, 4864, 5001, 7000, 10000])
@pytest.mark.parametrize("T", [1, 9, 64])
def test_sums_shared_by_any_number_of_ctas(N, T):
    counts = np.bincount(np.random.default_rng(T).integers(0, 7, 2 * T), minlength=7)
    r, *plan = _plan(counts, 2, 4)
    _check_down(r, plan, 320, N)


def test_down_in_slabs():
    """22400 pairs: 46 tiles of y's columns fill 512 MB of products, so that 104 take three slabs, the last one short."""
    r, *plan = _plan([560] * 40, 32, 5)
    _check_down(r, plan, 64, 13300)


def test_sizes_of_a_model():
    rng = np.random.default_rng(6)
    counts = rng.multinomial(2048 * 8, rng.dirichlet(np.full(128, 3.0)))
    r, *plan = _plan(counts, 8, 6)
    _check_up(r, plan, 4096, 768)
    _check_down(r, plan, 768, 4096)
