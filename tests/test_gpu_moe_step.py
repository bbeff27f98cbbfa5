"""The serving step with positions and experts: q and K rotated on the way into the cache, the layer's MLP by routed
experts; each part against the oracle on the step's own inputs, at the bounds of the parts' own tests."""
import numpy as np
import pytest
import torch

from oracle import decode as OD
from oracle import moe as O
from oracle import nvfp4 as Q
from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from nvfp4_w4a4_decode_gemv_gb300.serving_step import ServingStep
from tests.gpu_util import bits, to_np
from tests.test_gpu_kv_attention import _check
from tests.test_gpu_serving_step import _feed, _slots

pytestmark = pytest.mark.gpu

E, TOP, INTER = 12, 3, 128
SHAPES = [("qkv", 512, 1024), ("o", 512, 512), ("gate_up", 512, 2 * INTER), ("down", INTER, 512)]
HEADS, KVH, D, PAGE, M, VOCAB = 4, 2, 128, 16, 3, 1000
BF = lambda x: Q.bf16_bits_to_f32(Q.f32_to_bf16_bits(x))


def _step(layers=1, **kw):
    return ServingStep(M, layers, HEADS, KVH, D, PAGE, 40, max_len=200, k_global=0.5, v_global=0.25, shapes=SHAPES,
                       vocab=VOCAB, seed=3, rotary=1e4, rotated=64, experts=E,
                       router={"top_k": TOP, "score": "sigmoid", "scale": 1.5}, keep_rowmajor=True, **kw)


def _start(st, rng, lens):
    prompts = {r: torch.from_numpy(rng.integers(0, VOCAB, n).astype(np.int32)).cuda() for r, n in lens.items()}
    total = sum(lens.values())
    rows = [[torch.from_numpy(rng.standard_normal((total, KVH, D)).astype(np.float32)).to(torch.bfloat16).cuda()
             for _ in range(st.layers)] for _ in range(2)]
    return st.start(prompts, *rows), rows


def _cached(st, row, n):
    return S.read_slots(to_np(st.caches[0].pages), _slots(st, row, n), PAGE, D)


@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_step_against_the_oracle(style):
    rng = np.random.default_rng(1)
    st = _step(rope_style=style)
    st.route_bias[0] = torch.linspace(-0.2, 0.2, E, device="cuda")
    lens = {0: 33, 2: 5}                                          # row 1 has no request
    _, (keys, _) = _start(st, rng, lens)
    table = to_np(st.rope)
    at = 0
    for row, n in lens.items():                                   # the prompts' keys stand turned in the cache
        k = Q.bf16_bits_to_f32(bits(keys[0][at:at + n]))
        want = S.quantize_rows(BF(O.rotate(k, np.arange(n), table, style)), 0.5)
        got = _cached(st, row, n)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        at += n
    for step in range(2):
        _feed(st, rng)
        held = to_np(st.lens).copy()
        real, r = st._mlp, []

        def spy(layer, stream, trace):
            real(layer, stream, trace)
            r.append(st.r.clone())
        st._mlp = spy
        st.run()
        st._mlp = real
        y = to_np(st.y_qkv)
        cut = HEADS * D
        q = BF(O.rotate(y[:, :cut].reshape(M, HEADS, D), held, table, style))
        k = BF(O.rotate(y[:, cut:cut + KVH * D].reshape(M, KVH, D), held, table, style))
        for row in lens:
            n = int(held[row]) + 1
            assert np.array_equal(Q.bf16_bits_to_f32(bits(st.q_turned[row])), q[row])
            kc, ks, vc, vs = _cached(st, row, n)
            want = S.quantize_rows(k[row:row + 1], 0.5)
            assert np.array_equal(kc[-1:], want[0]) and np.array_equal(ks[-1:], want[1])
            _check(st.attn[row:row + 1], None, 0, q[row:row + 1].astype(np.float64), S.dequantize_rows(kc, ks, 0.5),
                   S.dequantize_rows(vc, vs, 0.25), D ** -0.5, 0)
        # router logits, choice, products, quantizer, sum
        ref, size = OD.bf16_gemv(bits(r[0]), bits(st.routers[0]))
        logits = to_np(st.route_logits)
        assert np.all(np.abs(logits - ref) <= 1e-4 * size + 1e-6)
        live = np.array([r in lens for r in range(M)])
        ids, w, _ = O.route(logits, TOP, "sigmoid", bias=to_np(st.route_bias[0]), scale=1.5, rows=live)
        assert np.array_equal(to_np(st.routing.ids), ids) and np.allclose(to_np(st.routing.weights), w, rtol=1e-5, atol=0)
        offsets, pairs, places = O.plan(ids, E)
        val = lambda t: O.values(to_np(t.codes), to_np(t.scales), to_np(t.global_scale)[0])
        rows = st.rowmajor[0]
        want, Bg, Bu, g, u = O.gate_up(val(st.xq_gu), np.stack([val(t) for t in rows["gate_up"]]), offsets, pairs, TOP)
        got = Q.bf16_bits_to_f32(bits(st.h_mid)).astype(np.float64)
        c = (512 / 64 + 12) * 2.0 ** -23
        tol = 1.1 * c * Bg * (np.abs(u) + c * Bu) + (np.abs(want) / np.maximum(np.abs(u), 1e-30) + 1.1 * c * Bg) * c * Bu
        assert np.all(np.abs(got - want) <= tol + np.abs(want) * (2.0 ** -8 + 2.0 ** -15) + 1e-37)
        codes, scales, glob = Q.quantize_bf16(bits(st.h_mid))
        assert np.array_equal(to_np(st.xq_d.codes), codes) and np.array_equal(to_np(st.xq_d.scales), scales)
        want, B = O.down(O.values(codes, scales, glob), np.stack([val(t) for t in rows["down"]]), to_np(st.routing.weights),
                         places, offsets)
        got = to_np(st.h)
        assert np.all(np.abs(got - want) <= (INTER / 64 + 12 + TOP + 8) * 2.0 ** -23 * B + 1e-37)
        assert not got[1].any() and to_np(st.routing.ids)[1].tolist() == [-1] * TOP
    assert api.device_status() == 0


def test_captured_step_follows_requests():
    """One graph over steps in which requests end and others start: the tokens of eager steps."""
    def play(captured):
        rng = np.random.default_rng(2)
        st = _step(layers=2)
        _start(st, rng, {0: 20, 1: 7})
        _feed(st, rng)
        if captured:
            lens = [t.clone() for t in (st.lens, st.n_tokens, st.tokens, st.table, st.free_count, st.sampler.state)]
            st.run()                                              # every kernel's attributes are set
            for t, v in zip((st.lens, st.n_tokens, st.tokens, st.table, st.free_count, st.sampler.state), lens):
                t.copy_(v)
            torch.cuda.synchronize()
            st.capture()
        out = []
        for i in range(6):
            if i == 3:
                st.end(torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda"))
                _start(st, rng, {0: 11, 2: 3})
            _feed(st, rng)
            st.graph.replay() if captured else st.run()
            out.append((to_np(st.sampler.token).copy(), to_np(st.h).copy()))
        return out
    for (a, ha), (b, hb) in zip(play(False), play(True)):
        assert np.array_equal(a, b) and np.array_equal(ha, hb)
    assert api.device_status() == 0


def test_steps_share_experts():
    st = _step()
    other = ServingStep(1, 1, HEADS, KVH, D, PAGE, 40, max_len=200, shapes=SHAPES, vocab=VOCAB, rotary=1e4, experts=E,
                        router={"top_k": TOP}, share_weights=st)
    assert other.weights[0]["down"] is st.weights[0]["down"] and other.routers[0] is st.routers[0]
