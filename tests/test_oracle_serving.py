"""Pins of oracle/serving.py: closed forms, hand-worked tables and round trips (no GPU)."""
import numpy as np
import pytest

from oracle import nvfp4 as Q
from oracle import serving as S


def test_plan_by_hand():
    table = np.full((3, 3), -1)
    table[0, 0], table[1, :2] = 7, (4, 5)
    stack = np.array([10, 11, 12, 13])
    # request 0 holds 15 of 16 and gets 2 (one new page), 1 holds 32 = two full pages and gets 1, 2 is new with 17
    t, slots, pos, cu, kv, left, info = S.kv_plan([15, 32, 0], [2, 1, 17], table, stack, 4, 16, 22)
    assert t.tolist() == [[7, 13, -1], [4, 5, 12], [11, 10, -1]]
    assert slots[:3].tolist() == [7 * 16 + 15, 13 * 16, 12 * 16]
    assert slots[3:20].tolist() == list(range(11 * 16, 12 * 16)) + [160]
    assert slots[20:].tolist() == [-1, -1] and pos[:4].tolist() == [15, 16, 32, 0]
    assert cu.tolist() == [0, 2, 3, 20] and kv.tolist() == [17, 33, 17] and left == 0 and info == (0, 20)


def test_plan_refuses_in_order():
    table = np.full((3, 4), -1)
    table[1, 0] = 3
    t, slots, _, cu, kv, left, info = S.kv_plan([0, 4, 0], [40, 3, 16], table, np.array([8, 9]), 2, 16, 59)
    # request 0 needs 3 pages of 2; request 1 needs none; request 2's need comes after request 0's
    assert info == (2, 59) and left == 2 and kv.tolist() == [0, 7, 0]
    assert (slots[:40] == -1).all() and slots[40:43].tolist() == [52, 53, 54] and (slots[43:] == -1).all()


def test_release_order():
    table = np.arange(12).reshape(3, 4)
    stack, n = S.kv_release([17, 64, 33], [1, 0, 1], table, np.full(9, -5), 2, 16)
    assert n == 7 and stack.tolist() == [-5, -5, 0, 1, 8, 9, 10, -5, -5]


@pytest.mark.parametrize("D", [64, 128])
def test_group_layout_is_a_partition(D):
    """Every code nibble and scale byte of a group has a place of its own."""
    o = S.GroupOffsets(D)
    for codes in (o.k_codes, o.v_codes):
        key = codes * 2 + o.nibble // 4
        assert len(np.unique(key)) == 16 * D
    parts = [np.unique(x) for x in (o.k_codes, o.k_scales, o.v_codes, o.v_scales)]
    assert [len(p) for p in parts] == [8 * D, D, 8 * D, D]
    assert np.array_equal(np.concatenate(parts), np.arange(18 * D))


@pytest.mark.parametrize("D", [64, 128])
def test_cache_round_trip(D):
    rng = np.random.default_rng(D)
    pages = np.zeros((3, 2, 2, 18 * D), np.uint8)
    slots = rng.permutation(96)[:50]
    put = [rng.integers(0, n, (50, 2, w)).astype(np.uint8) for n, w in ((16, D), (120, D // 16)) * 2]
    S.write_slots(pages, slots, 32, D, *put)
    for a, b in zip(put, S.read_slots(pages, slots, 32, D)):
        assert np.array_equal(a, b)


def test_quantize_rows_is_the_quantizers_recipe():
    x = (np.random.default_rng(1).standard_normal((5, 64)) * 3).astype(np.float32)
    bits = Q.f32_to_bf16_bits(x)
    codes, scales, g = Q.quantize_bf16(bits)
    c, s = S.quantize_rows(Q.bf16_bits_to_f32(bits), g)
    assert np.array_equal(c, Q.unpack_codes(codes)) and np.array_equal(s, scales)


def test_attention_closed_forms():
    D = 4
    k, v = np.zeros((3, 1, D)), np.arange(3.0)[:, None, None] * np.ones((3, 1, D))
    out, lse, *_ = S.attention(np.ones((2, 2, D)), k, v, 0.5)
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 1.0)      # means of the first 2 and all 3 keys
    assert np.allclose(lse[:, 0], np.log([2, 3]))
    out, lse, *_ = S.attention(np.ones((1, 1, D)), k, v, 0.5, window=2)
    assert np.allclose(out, 1.5)
    out, lse, *_ = S.attention(np.ones((5, 1, D)), k, v, 0.5)         # the first two rows see nothing
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.allclose(out[2], 0)


def test_process_logits_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.0, 5.0]])
    y, _ = S.process_logits(x, np.array([[0, 1, 1, 9]]), [4], [1], [2.0], [0.5], [0.25], np.array([[2, 2, -1]]),
                            np.array([[7.0, 3.0, 9.0]]), np.array([[0b10111]], np.uint32))
    assert y.tolist() == [[1.0, -4.0 - 0.5 - 0.5, 4.0, -np.inf, 5.0]]
