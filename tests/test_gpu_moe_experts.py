"""The chosen experts' products against FP64.

A product is summed in FP32 by the tensor core, a rounding (or a cut: 2^-23) per 64 elements and a few more in what is
joined: |g - exact| <= (K/64 + 12) 2^-23 B, B the magnitudes summed up.  Of h = g / (1 + exp(-g)) u: the derivative of
SiLU is at most 1.1; exp and the quotient are off by 2^-16 at most (exp by 2 + 1.173 |g| ulp, where it counts |g| < 88), and
BF16 rounds by 2^-8 (half a step of 2^-7).  y adds up the products in FP32: (K/64 + 12 + pieces) 2^-23 of its magnitudes,
pieces the experts of a token and the CTAs that share its sum (at most 8).
"""
import numpy as np
import pytest
import torch

from oracle import moe as O
from oracle import nvfp4 as Q
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, bits, to_np

pytestmark = pytest.mark.gpu


def _nvfp4(x):
    """FP32 [.., K] -> codes, scales, global of all of it (numpy), and their FP64 values."""
    x = Q.bf16_bits_to_f32(Q.f32_to_bf16_bits(x.astype(np.float32)))
    flat = x.reshape(-1, x.shape[-1])
    c, s, g = Q.quantize_f32(flat)
    return (c.reshape(x.shape[:-1] + (-1,)), s.reshape(x.shape[:-1] + (-1,)), g), O.values(c, s, g).reshape(x.shape)


def _tensor(n, shape=None):
    c, s, g = n
    return api.NVFP4Tensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), torch.tensor([float(g)], device="cuda"))


class Case:
    def __init__(self, ids, E, hidden, inter, seed=0):
        rng = np.random.default_rng(seed)
        self.ids = np.asarray(ids, np.int32)
        (self.T, self.k), self.E, self.hidden, self.inter = self.ids.shape, E, hidden, inter
        self.x, self.xv = _nvfp4(rng.standard_normal((self.T, hidden)))
        self.h, self.hv = _nvfp4(rng.standard_normal((self.T * self.k, inter)) * 0.3)
        ups = [_nvfp4(rng.standard_normal((2 * inter, hidden)) * 0.05 * (1 + e % 3)) for e in range(E)]
        downs = [_nvfp4(rng.standard_normal((hidden, inter)) * 0.02 * (1 + e % 5)) for e in range(E)]
        self.upv, self.downv = (np.stack([v for _, v in m]) for m in (ups, downs))
        stack = lambda m, i: torch.from_numpy(np.stack([n[i] for n, _ in m])).cuda()
        glob = lambda m: torch.tensor([float(n[2]) for n, _ in m], device="cuda")
        self.up_rows = (stack(ups, 0), stack(ups, 1))
        self.up = api.nvfp4_moe_pack_weights(*self.up_rows, glob(ups), gated=True)
        self.down_rows = (stack(downs, 0), stack(downs, 1))
        self.down = api.nvfp4_moe_pack_weights(*self.down_rows, glob(downs), gated=False)
        self.weights = rng.random((self.T, self.k)).astype(np.float32)
        self.plan = O.plan(self.ids, E)
        self.routing = api.nvfp4_moe_plan(torch.from_numpy(self.ids).cuda(), E, torch.from_numpy(self.weights).cuda())

    def check_up(self, h):
        offsets, pairs, _ = self.plan
        want, Bg, Bu, g, u = O.gate_up(self.xv, self.upv, offsets, pairs, self.k)
        c = (self.hidden / 64 + 12) * 2.0 ** -23
        silu = np.abs(g / (1.0 + np.exp(-g)))
        tol = 1.1 * c * Bg * (np.abs(u) + c * Bu) + (silu + 1.1 * c * Bg) * c * Bu + np.abs(want) * (2.0 ** -8 + 2.0 ** -15)
        got = Q.bf16_bits_to_f32(bits(h)).astype(np.float64)
        assert np.all(np.abs(got - want) <= tol + 1e-37), (np.abs(got - want) / (tol + 1e-37)).max()
        assert not got[offsets[-1]:].any()

    def check_down(self, y):
        offsets, _, places = self.plan
        want, B = O.down(self.hv, self.downv, self.weights, places, offsets)
        got = to_np(y).astype(np.float64)
        tol = (self.inter / 64 + 12 + self.k + 8) * 2.0 ** -23 * B
        assert np.all(np.abs(got - want) <= tol + 1e-37), (np.abs(got - want) / (tol + 1e-37)).max()

    def run(self):
        self.check_up(api.nvfp4_moe_gate_up(_tensor(self.x), self.up, self.routing))
        self.check_down(api.nvfp4_moe_down(_tensor(self.h), self.down, self.routing))
        assert api.device_status() == 0


def _ids(rng, T, k, E):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)])


@pytest.mark.parametrize("E,N,K,gated", [(1, 1, 64, False), (3, 129, 320, False), (2, 128, 256, True), (5, 384, 576, True)])
def test_packed_weights(E, N, K, gated):
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    scales = rng.integers(0, 256, (E, N, K // 16)).astype(np.uint8)
    out = Guarded((api.nvfp4_moe_packed_weight_bytes(E, N, K, gated),), torch.uint8)
    api.nvfp4_moe_pack_weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.ones(E, device="cuda"),
                               gated, out=out.t)
    assert np.array_equal(to_np(out.t), O.pack(codes, scales, gated))
    out.check("packed")


# one token to hundreds, tiles of 16, 64, 128 and 256 places, tails of K and of rows, more row tiles than experts
@pytest.mark.parametrize("T,k,E,hidden,inter", [
    (1, 1, 1, 64, 64), (1, 2, 4, 256, 64), (1, 8, 16, 1024, 128), (2, 2, 3, 320, 192), (8, 8, 16, 704, 192),
    (16, 2, 2, 128, 64), (17, 2, 2, 128, 64), (33, 2, 3, 576, 320), (64, 4, 5, 192, 128), (65, 1, 2, 256, 64),
    (70, 3, 4, 320, 128), (129, 2, 2, 64, 64), (130, 1, 1, 448, 64), (200, 4, 40, 128, 64), (300, 2, 3, 256, 192),
    (600, 1, 1, 64, 64)])
def test_sizes(T, k, E, hidden, inter):
    Case(_ids(np.random.default_rng(T + E), T, k, E), E, hidden, inter, seed=T).run()


@pytest.mark.parametrize("T", [3, 40, 150])
def test_pairs_without_an_expert(T):
    """Tokens that have fewer experts, or none; experts that have no tokens."""
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, 3, 9)
    ids[ids == 4] = -1
    ids[1] = -1
    ids[2, :2] = -1
    Case(ids, 9, 192, 64, seed=1).run()


def test_no_pairs_at_all():
    c = Case(np.full((5, 2), -1), 3, 128, 64)
    h = torch.full((10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    assert not to_np(api.nvfp4_moe_gate_up(_tensor(c.x), c.up, c.routing, out=h).float()).any()
    y = torch.full((5, 128), 7.0, device="cuda")
    assert not to_np(api.nvfp4_moe_down(_tensor(c.h), c.down, c.routing, y=y)).any()
    big = Case(np.full((90, 2), -1), 3, 128, 64)
    big.run()


@pytest.mark.parametrize("T", [4, 30, 100, 400])
def test_one_expert_takes_everything(T):
    """All tokens in one expert, some of them twice."""
    ids = np.full((T, 2), 3)
    ids[::2, 1] = 0
    Case(ids, 5, 128, 128, seed=2).run()


@pytest.mark.parametrize("T", [2, 100])
def test_many_experts(T):
    rng = np.random.default_rng(T)
    Case(_ids(rng, T, 8, 300), 300, 64, 64, seed=3).run()


@pytest.mark.parametrize("T", [6, 80])
def test_outputs_are_all_that_is_written(T):
    c = Case(_ids(np.random.default_rng(4), T, 2, 4), 4, 320, 192, seed=5)
    h, y = Guarded((T * 2, 192), torch.bfloat16), Guarded((T, 320), torch.float32)
    need = [max(16, n) for n in (api.nvfp4_moe_gate_up_workspace_bytes(T, 2, 4, 320),
                                 api.nvfp4_moe_down_workspace_bytes(T, 2, 4, 320, 192))]
    ws = [Guarded((n,), torch.uint8) for n in need]
    c.check_up(api.nvfp4_moe_gate_up(_tensor(c.x), c.up, c.routing, out=h.t, workspace=ws[0].t))
    c.check_down(api.nvfp4_moe_down(_tensor(c.h), c.down, c.routing, y=y.t, workspace=ws[1].t))
    for g, n in ((h, "h"), (y, "y"), (ws[0], "workspace of h"), (ws[1], "workspace of y")):
        g.check(n)


@pytest.mark.parametrize("N", [1, 130, 1001])
@pytest.mark.parametrize("T", [3, 70])
def test_odd_columns_of_y(N, T):
    rng = np.random.default_rng(N)
    c = Case(_ids(rng, T, 2, 3), 3, 64, 128)
    n, v = zip(*[_nvfp4(rng.standard_normal((N, 128))) for _ in range(3)])
    c.downv = np.stack(v)
    w = api.nvfp4_moe_pack_weights(*(torch.from_numpy(np.stack([m[i] for m in n])).cuda() for i in (0, 1)),
                                   torch.tensor([float(m[2]) for m in n], device="cuda"), gated=False)
    out = Guarded((T, N), torch.float32)
    c.check_down(api.nvfp4_moe_down(_tensor(c.h), w, c.routing, y=out.t))
    out.check("y")


def test_broken_plans_are_reported():
    """Offsets, pairs and places outside their tables: taken into them or skipped, nothing beyond the outputs written."""
    for T in (4, 100):
        c = Case(_ids(np.random.default_rng(6), T, 2, 4), 4, 128, 64)
        P = 2 * T
        for name, index, value in (("offsets", 4, P + 50), ("offsets", 2, -9), ("offsets", 1, P), ("pairs", 0, P),
                                   ("pairs", 3, -5), ("places", (0, 1), P + 3)):
            r = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), 4, torch.from_numpy(c.weights).cuda())
            getattr(r, name)[index] = value
            h, y = Guarded((P, 64), torch.bfloat16), Guarded((T, 128), torch.float32)
            if name != "places":
                api.nvfp4_moe_gate_up(_tensor(c.x), c.up, r, out=h.t)
                assert api.device_status() == api.DEVERR_MOE_RANGE, (name, index)
            if name != "places" or T > 64:
                api.nvfp4_moe_down(_tensor(c.h), c.down, r, y=y.t)
                assert api.device_status() == (0 if name == "pairs" and T > 64 else api.DEVERR_MOE_RANGE), (name, index)
            h.check("h")
            y.check("y")
        c.run()


@pytest.mark.parametrize("T", [5, 90, 200])
def test_same_bits_again_replayed_and_on_two_streams(T):
    c = Case(_ids(np.random.default_rng(7), T, 4, 12), 12, 512, 256)
    x, h = _tensor(c.x), _tensor(c.h)
    call = lambda s=None: (api.nvfp4_moe_gate_up(x, c.up, c.routing, stream=s),
                           api.nvfp4_moe_down(h, c.down, c.routing, stream=s))
    want = [t.clone() for t in call()]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    runs = [call(s) for _ in range(5) for s in sides]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for run in runs for a, b in zip(run, want))


@pytest.mark.parametrize("T", [1, 8, 100])
def test_a_layer_with_experts(T):
    """Route, gate and up, quantize, down, as a layer runs them: each step against the oracle on its own inputs."""
    E, k, hidden, inter = 16, 4, 256, 128
    rng = np.random.default_rng(T)
    c = Case(np.zeros((T, k), np.int32), E, hidden, inter, seed=8)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    r = api.nvfp4_moe_route(logits, k)
    c.ids, c.weights = to_np(r.ids), to_np(r.weights)
    ids, w, _ = O.route(to_np(logits), k)
    assert np.array_equal(c.ids, ids) and np.allclose(c.weights, w, rtol=1e-5)
    c.plan, c.routing = O.plan(ids, E), r
    h = api.nvfp4_moe_gate_up(_tensor(c.x), c.up, r)
    c.check_up(h)
    hq = api.nvfp4_quantize_act(h)
    codes, scales, g = Q.quantize_bf16(bits(h))
    assert np.array_equal(to_np(hq.codes), codes) and np.array_equal(to_np(hq.scales), scales)
    c.hv = O.values(codes, scales, g)
    c.check_down(api.nvfp4_moe_down(hq, c.down, r))
    assert api.device_status() == 0


def test_bindings_refuse_what_does_not_fit():
    c = Case(_ids(np.random.default_rng(9), 4, 2, 3), 3, 128, 64)
    x, h = _tensor(c.x), _tensor(c.h)
    bare = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), 3)
    other = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), 4)
    for call in (lambda: api.nvfp4_moe_gate_up(x, c.down, c.routing), lambda: api.nvfp4_moe_down(h, c.up, c.routing),
                 lambda: api.nvfp4_moe_gate_up(h, c.up, c.routing), lambda: api.nvfp4_moe_down(x, c.down, c.routing),
                 lambda: api.nvfp4_moe_down(h, c.down, bare), lambda: api.nvfp4_moe_gate_up(x, c.up, other),
                 lambda: api.nvfp4_moe_gate_up(x, c.up, c.routing, out=torch.empty((8, 128), device="cuda")),
                 lambda: api.nvfp4_moe_down(h, c.down, c.routing, y=torch.empty((4, 64), device="cuda")),
                 lambda: api.nvfp4_moe_pack_weights(c.up_rows[0], c.down_rows[1], torch.ones(3, device="cuda"), True),
                 lambda: api.MoERouting(bare.ids, None, bare.offsets, bare.pairs[:3], bare.places)):
        with pytest.raises(ValueError):
            call()


# either side of 32 pairs an expert, where rows of x are laid out first
@pytest.mark.parametrize("T,k,E", [(96, 3, 9), (97, 3, 9), (128, 8, 32), (129, 8, 32), (2000, 2, 500)])
def test_few_and_many_places(T, k, E):
    Case(_ids(np.random.default_rng(T), T, k, E), E, 192, 64, seed=T).run()


@pytest.mark.parametrize("T,E", [(4, 4), (60, 300), (100, 4), (130, 512), (1000, 16)])
def test_offsets_that_fall_are_a_plan_without_pairs(T, E):
    """Ranges that overlap would have more tiles between them than any plan of the pairs."""
    c = Case(_ids(np.random.default_rng(T), T, 2, E), E, 128, 64)
    r = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), E, torch.from_numpy(c.weights).cuda())
    r.offsets[::2], r.offsets[1::2] = 0, 2 * T
    h, y = Guarded((2 * T, 64), torch.bfloat16), Guarded((T, 128), torch.float32)
    h.t.fill_(7.0)
    api.nvfp4_moe_gate_up(_tensor(c.x), c.up, r, out=h.t)
    assert api.device_status() == api.DEVERR_MOE_RANGE
    assert not to_np(h.t.float()).any()
    api.nvfp4_moe_down(_tensor(c.h), c.down, r, y=y.t)
    assert api.device_status() == api.DEVERR_MOE_RANGE
    assert T > 64 or not to_np(y.t).any()
    h.check("h")
    y.check("y")
    c.run()
