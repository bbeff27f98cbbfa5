"""Routing to experts and the plan of the pairs, against the 64-bit oracle: choices and plans are equal, ties to the lowest.

Weights: expf is off by 2 ulp (2^-22), its argument x - m by 2^-24 |x - m|, a score's sum of up to 512 terms by 21 half ulps
(2^-19.6) and of up to 32 chosen ones by 5, quotient and scale by a half each: 2^-18.5 + 2^-24 |x - m| of the weight, and
what FP32 has no numbers for (2^-126 times the scale).
"""
import numpy as np
import pytest
import torch

from oracle import moe as O
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, to_np

pytestmark = pytest.mark.gpu


def _check(x, r, **kw):
    """x: the logits as FP32 numpy; kw: the oracle's arguments."""
    top_k = r.top_k
    ids, w, bad = O.route(x, top_k, **kw)
    assert np.array_equal(to_np(r.ids), ids)
    got = to_np(r.weights).astype(np.float64)
    z = np.where(np.isfinite(x), x.astype(np.float64), 0.0)
    spread = (z.max(1) - z.min(1))[:, None] if x.shape[0] else 0.0
    tol = np.abs(w) * (2.0 ** -18.5 + 2.0 ** -24 * spread) + 2.0 ** -126 * abs(kw.get("scale", 1.0))
    assert np.all(np.abs(got - w) <= tol), np.abs(got - w).max()
    offsets, pairs, places = O.plan(ids, x.shape[1])
    assert np.array_equal(to_np(r.offsets), offsets)
    assert np.array_equal(to_np(r.pairs), pairs) and np.array_equal(to_np(r.places), places)
    return bad


def _call(x, top_k, bias=None, rows=None, **kw):
    r = api.nvfp4_moe_route(x, top_k, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                            rows=None if rows is None else torch.from_numpy(rows).cuda(), **kw)
    return _check(x.float().cpu().numpy(), r, bias=bias, rows=rows, **kw), r


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 2, 2), (3, 31, 5), (64, 32, 32), (65, 33, 1), (5, 64, 6),
                                   (200, 100, 8), (1000, 128, 8), (1, 257, 32), (700, 512, 10), (2500, 256, 8)])
@pytest.mark.parametrize("score,biased,renormalize", [("softmax", False, True), ("sigmoid", True, True),
                                                      ("softmax", True, False), ("sigmoid", False, False)])
def test_sizes(T, E, k, score, biased, renormalize):
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = (2.0 * torch.randn((T, E), generator=g)).cuda()
    bias = (0.1 * torch.randn(E, generator=g)).numpy() if biased else None
    bad, _ = _call(x, k, bias=bias, score=score, renormalize=renormalize, scale=2.5)
    assert bad == 0 and api.device_status() == 0


@pytest.mark.parametrize("T", [7, 300])
@pytest.mark.parametrize("E,groups,top_groups,best", [(64, 8, 3, 1), (64, 8, 3, 2), (60, 12, 5, 2), (256, 8, 4, 2),
                                                      (32, 32, 9, 2), (6, 2, 1, 2), (384, 16, 15, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(T, E, groups, top_groups, best, biased):
    g = torch.Generator().manual_seed(E + groups)
    x = torch.randn((T, E), generator=g).to(torch.bfloat16).cuda()
    bias = (0.2 * torch.randn(E, generator=g)).numpy() if biased else None
    for score in ("softmax", "sigmoid"):
        _call(x, min(3, E // groups * top_groups), bias=bias, score=score, groups=groups, top_groups=top_groups,
              group_best=best)


def test_ties_go_to_the_lowest():
    x = torch.zeros((3, 96), device="cuda")
    x[1, 40:] = -0.0
    x[2, ::3] = 1.0
    for score in ("softmax", "sigmoid"):
        _, r = _call(x, 5, score=score)
        assert to_np(r.ids).tolist() == [[0, 1, 2, 3, 4]] * 2 + [[0, 3, 6, 9, 12]]
        _, r = _call(x, 5, bias=np.zeros(96, np.float32), score=score, groups=8, top_groups=2, group_best=2)
        assert to_np(r.ids)[0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_only_64_bits_tell_apart(score):
    """Logits one FP32 step from one another, shuffled, under equal biases: the scores differ by less than FP32 resolves
    beside the bias."""
    rng = np.random.default_rng(5)
    for first, step in ((2.0, 1), (-1.0, 3), (0.125, 40)):
        v = [np.float32(first)]
        for _ in range(63):
            for _ in range(step):
                v.append(np.nextafter(v.pop() if len(v) > 63 else v[-1], np.float32(9)))
                if len(v) > 64:
                    v.pop(-2)
        row = np.array(v[:64], np.float32)
        x = np.stack([rng.permutation(row) for _ in range(40)])
        _call(torch.from_numpy(x).cuda(), 8, bias=np.full(64, 1.0, np.float32), score=score)
        _call(torch.from_numpy(x).cuda(), 8, bias=np.full(64, 1.0, np.float32), score=score, groups=8, top_groups=3,
              group_best=2)
        _call(torch.from_numpy(x).cuda(), 8, score=score, groups=8, top_groups=3, group_best=2)


def test_infinities_and_nan():
    inf = float("inf")
    x = torch.zeros((8, 40), device="cuda")
    x[0, 3] = float("nan")
    x[1, 5] = inf
    x[2] = -inf
    x[3, 1:] = -inf                                             # one expert left: the others have score 0
    x[4] = 100.0
    x[5] = -200.0                                               # sigmoids underflow, their shares do not
    x[6, ::2] = -inf
    x[7, 0], x[7, 1] = -300.0, 300.0
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            bad, _ = _call(x, 4, score=score, renormalize=renormalize)
            assert bad == (3 if score == "softmax" else 1)
            assert api.device_status() == api.DEVERR_NO_EXPERT
            _call(x, 4, bias=np.linspace(-1, 1, 40, dtype=np.float32), score=score, renormalize=renormalize)
            assert api.device_status() == api.DEVERR_NO_EXPERT
    bias = np.zeros(40, np.float32)
    bias[2] = np.nan
    assert _call(x[4:], 4, bias=bias, score="sigmoid")[0] == 4
    bias[2] = np.inf
    assert _call(x[4:], 4, bias=bias, score="sigmoid")[0] == 0
    api.device_status()


@pytest.mark.parametrize("T", [6, 333])
def test_rows_without_a_request(T):
    x = torch.randn((T, 24), device="cuda")
    rows = (np.arange(T) % 3 != 1).astype(np.uint8)
    x[1] = float("nan")                                         # not read
    _, r = _call(x, 4, rows=rows)
    assert to_np(r.ids)[1].tolist() == [-1] * 4 and to_np(r.weights)[1].tolist() == [0.0] * 4
    assert api.device_status() == 0
    again = api.nvfp4_moe_route(x, 4, rows=torch.from_numpy(rows.astype(bool)).cuda())
    assert torch.equal(again.ids, r.ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [9, 500])
def test_strided_logits_and_guarded_outputs(dtype, T):
    E, k = 48, 6
    wide = torch.randn((T, 101), device="cuda").to(dtype)
    x = wide[:, 7:7 + E]
    i32 = torch.int32
    out = [Guarded((T, k), i32), Guarded((T, k), torch.float32), Guarded((E + 1,), i32), Guarded((T * k,), i32),
           Guarded((T, k), i32)]
    r = api.nvfp4_moe_route(x, k, out=api.MoERouting(*[g.t for g in out]))
    _check(x.float().cpu().numpy(), r)
    for g, n in zip(out, ("ids", "weights", "offsets", "pairs", "places")):
        g.check(n)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 3, 4), (64, 32, 7), (65, 2, 300), (3000, 8, 128), (9000, 4, 512)])
def test_plan_of_given_choices(T, k, E):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    ids[rng.random(T) < 0.3] = E // 2                          # the same expert several times
    r = api.nvfp4_moe_plan(torch.from_numpy(ids).cuda(), E)
    offsets, pairs, places = O.plan(ids, E)
    assert np.array_equal(to_np(r.offsets), offsets) and np.array_equal(to_np(r.pairs), pairs)
    assert np.array_equal(to_np(r.places), places) and api.device_status() == 0
    ids[0, 0], ids[-1, -1] = E, -7                              # no experts: no pairs, and reported
    r = api.nvfp4_moe_plan(torch.from_numpy(ids).cuda(), E)
    offsets, pairs, places = O.plan(ids, E)
    assert np.array_equal(to_np(r.offsets), offsets) and np.array_equal(to_np(r.places), places)
    assert api.device_status() == api.DEVERR_MOE_RANGE


@pytest.mark.parametrize("T", [4, 2000])
def test_replayed_and_on_two_streams(T):
    x = [torch.randn((T, 64), device="cuda") for _ in range(2)]
    want = [api.nvfp4_moe_route(v, 8) for v in x]
    buf = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    api.nvfp4_moe_route(buf, 8)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = api.nvfp4_moe_route(buf, 8)
    for i in (0, 1, 0):
        buf.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        for name in ("ids", "weights", "offsets", "pairs", "places"):
            assert torch.equal(getattr(got, name), getattr(want[i], name)), name
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    runs = [[api.nvfp4_moe_route(x[i], 8, stream=sides[i]) for i in (0, 1)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in runs:
        for i in (0, 1):
            assert torch.equal(pair[i].pairs, want[i].pairs) and torch.equal(pair[i].weights, want[i].weights)
