"""The serving step: page plan, cache append, attention and logit rules inside the decode step.

The cache is compared byte for byte with the recipe on the step's own K and V columns; the attention with FP64 over
what the cache holds, at the bounds of tests/test_gpu_kv_attention.py; the rules with FP64 on the step's own logits;
the sampled token with the sampler on those.  A captured step follows requests that come and go.
"""
import numpy as np
import pytest
import torch

from oracle import nvfp4 as Q
from oracle import reset as R
from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from nvfp4_w4a4_decode_gemv_gb300.serving_step import ServingStep
from tests.gpu_util import bits, to_np
from tests.test_gpu_kv_attention import _check

pytestmark = pytest.mark.gpu

SHAPES = [("qkv", 512, 1024), ("o", 512, 512), ("gate_up", 512, 1024), ("down", 512, 512)]
HEADS, KVH, D, PAGE, M, LAYERS, VOCAB = 4, 2, 128, 16, 3, 2, 1000


def _step(num_pages=40):
    st = ServingStep(M, LAYERS, HEADS, KVH, D, PAGE, num_pages, max_len=200, k_global=0.5, v_global=0.25, shapes=SHAPES,
                     vocab=VOCAB, seed=3)
    st.presence.fill_(0.5)
    st.frequency.fill_(0.25)
    st.repetition.fill_(1.25)
    return st


def _start(st, rng, lens):
    prompts = {r: torch.from_numpy(rng.integers(0, VOCAB, n).astype(np.int32)).cuda() for r, n in lens.items()}
    total = sum(lens.values())
    rows = [[torch.from_numpy(rng.standard_normal((total, KVH, D)).astype(np.float32)).to(torch.bfloat16).cuda()
             for _ in range(LAYERS)] for _ in range(2)]
    return st.start(prompts, *rows)


def _feed(st, rng):
    st.h_in.copy_(torch.from_numpy(rng.standard_normal((M, st.hidden)).astype(np.float32)))
    st.u.copy_(torch.from_numpy(rng.random(M).astype(np.float32)))


def _slots(st, row, n):
    t = to_np(st.table)[row]
    at = np.arange(n)
    return t[at // PAGE].astype(np.int64) * PAGE + at % PAGE


def test_step_against_the_oracle():
    rng = np.random.default_rng(1)
    st = _step()
    _start(st, rng, {0: 33, 1: 16, 2: 1})
    for _ in range(3):
        _feed(st, rng)
        lens, tokens, n_tokens, n_prompt = (to_np(x).copy() for x in (st.lens, st.tokens, st.n_tokens, st.n_prompt))
        y = []
        attn = []
        real = st._attend

        def spy(layer, stream):
            y.append(st.y_qkv.clone())
            real(layer, stream)
            attn.append(st.attn.clone())
        st._attend = spy
        raw = []
        real_sample = st._sample

        def spy_sample(stream):
            raw.append(st.logits.clone())
            return real_sample(stream)
        st._sample = spy_sample
        st.run()
        st._attend, st._sample = real, real_sample
        assert np.array_equal(to_np(st.lens), lens + 1) and to_np(st.plan.info).tolist() == [0, M]
        for layer in range(LAYERS):
            pages = to_np(st.caches[layer].pages)
            yq = Q.bf16_bits_to_f32(Q.f32_to_bf16_bits(to_np(y[layer])))
            for r in range(M):
                n = int(lens[r]) + 1
                slots = _slots(st, r, n)
                kc, ks, vc, vs = S.read_slots(pages, slots, PAGE, D)
                cut = HEADS * D
                want_k = S.quantize_rows(yq[r, cut:cut + KVH * D].reshape(1, KVH, D), 0.5)
                want_v = S.quantize_rows(yq[r, cut + KVH * D:].reshape(1, KVH, D), 0.25)
                assert np.array_equal(kc[-1:], want_k[0]) and np.array_equal(ks[-1:], want_k[1])
                assert np.array_equal(vc[-1:], want_v[0]) and np.array_equal(vs[-1:], want_v[1])
                k, v = S.dequantize_rows(kc, ks, 0.5), S.dequantize_rows(vc, vs, 0.25)
                q = yq[r, :cut].reshape(1, HEADS, D).astype(np.float64)
                _check(attn[layer][r:r + 1], None, 0, q, k, v, D ** -0.5, 0)
        ref, size = S.process_logits(to_np(raw[0]), tokens, n_tokens, n_prompt, np.full(M, 1.25), np.full(M, 0.5),
                                     np.full(M, 0.25))
        got = to_np(st.logits).astype(np.float64)
        assert np.all(np.abs(got - ref) <= 6 * 2.0 ** -24 * size)
        tok, T, u = to_np(st.sampler.token), to_np(st.sampler.T), to_np(st.u)
        for r in range(M):
            lo, hi = R.acceptable_tokens(to_np(st.logits)[r], float(T[r]), float(u[r]), 4e-6)
            assert lo <= tok[r] <= hi
            assert to_np(st.tokens)[r, n_tokens[r]] == tok[r] and to_np(st.n_tokens)[r] == n_tokens[r] + 1
    assert api.device_status() == 0


def test_captured_step_follows_requests():
    """One graph over steps in which requests end, others start in their rows on their pages: the same tokens as
    eager steps."""
    def play(captured):
        rng = np.random.default_rng(2)
        st = _step(num_pages=16)
        _start(st, rng, {0: 40, 1: 15, 2: 3})
        _feed(st, rng)
        if captured:
            # kernels' attributes are set outside the capture: one step on a copy of the state
            other = _step(num_pages=16)
            _start(other, np.random.default_rng(2), {0: 40, 1: 15, 2: 3})
            other.run()
            torch.cuda.synchronize()
            graph = st.capture()
        out = []
        for i in range(12):
            if i == 5:
                st.end(torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda"))
                _start(st, rng, {0: 90})
            _feed(st, rng)
            graph.replay() if captured else st.run()
            out.append((to_np(st.sampler.token).copy(), to_np(st.lens).copy(), to_np(st.logits).copy()))
        return out, int(st.free_count), api.device_status()
    a, fa, sa = play(False)
    b, fb, sb = play(True)
    assert sa == sb == 0 and fa == fb
    for x, y in zip(a, b):
        for u, v in zip(x, y):
            assert np.array_equal(u, v)
    assert a[-1][1].tolist() == [97, 27, 15]


def test_full_pool_refuses_and_other_requests_go_on():
    rng = np.random.default_rng(3)
    st = _step(num_pages=4)
    _start(st, rng, {0: 16, 1: 16, 2: 20})            # all 4 pages: 1 + 1 + 2
    _feed(st, rng)
    st.run()                                          # rows 0 and 1 need a fifth and sixth page
    assert to_np(st.plan.info).tolist() == [2, M] and to_np(st.lens).tolist() == [16, 16, 21]
    assert to_np(st.plan.slots)[:2].tolist() == [-1, -1]
    assert api.device_status() == 0


def test_rows_without_a_request_stay_empty():
    """An ended row takes no page and no token until a request starts in it, and the others' rows stay their own."""
    rng = np.random.default_rng(4)
    st = _step()
    _start(st, rng, {0: 20, 1: 31, 2: 5})
    st.end(torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda"))
    free = int(st.free_count)
    for i in range(2):
        _feed(st, rng)
        y = []
        real = st._attend

        def spy(layer, stream):
            y.append(st.y_qkv.clone())
            real(layer, stream)
        st._attend = spy
        st.run()
        st._attend = real
        assert to_np(st.lens).tolist() == [0, 32 + i, 6 + i] and to_np(st.n_tokens).tolist() == [0, 32 + i, 6 + i]
        assert to_np(st.slots)[0] == -1 and to_np(st.plan.info).tolist() == [0, 2]
        cut = HEADS * D
        for layer in range(LAYERS):
            yq = Q.bf16_bits_to_f32(Q.f32_to_bf16_bits(to_np(y[layer])))
            for r in (1, 2):
                slot = _slots(st, r, int(st.lens[r]))[-1:]
                kc, ks, _, _ = S.read_slots(to_np(st.caches[layer].pages), slot, PAGE, D)
                want = S.quantize_rows(yq[r, cut:cut + KVH * D].reshape(1, KVH, D), 0.5)
                assert np.array_equal(kc, want[0]) and np.array_equal(ks, want[1])
    assert int(st.free_count) == free - 1                     # row 1's third page
    _start(st, rng, {0: 18})
    _feed(st, rng)
    st.run()
    assert to_np(st.lens).tolist() == [19, 34, 8] and api.device_status() == 0
