"""Pins of oracle/moe.py: hand-worked choices, round trips and closed forms (no GPU)."""
import numpy as np
import pytest

from oracle import moe as O


def test_route_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 3.0]]))
    ids, w, bad = O.route(x, 2)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, [[4 / 7, 3 / 7]]) and bad == 0
    ids, w, _ = O.route(x, 3, renormalize=False, scale=10.0)
    assert ids.tolist() == [[2, 3, 1]] and np.allclose(w, [[4, 3, 2]])
    ids, w, _ = O.route(x, 2, bias=np.array([0.5, 0.0, 0.0, 0.0]))        # 0.6, 0.2, 0.4, 0.3; weights by score alone
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[1 / 5, 4 / 5]])


def test_route_groups_ties_and_missing():
    x = np.array([[0.0, 3.0, 2.0, 2.0, 1.0, 1.0]])
    # groups of two: sums of sigmoids; maxima 3, 2, 1 and the second group has the largest sum
    assert O.route(x, 1, "sigmoid", groups=3, top_groups=1, group_best=1)[0].tolist() == [[1]]
    assert O.route(x, 2, "sigmoid", groups=3, top_groups=1, group_best=2)[0].tolist() == [[2, 3]]
    assert O.route(np.zeros((1, 5)), 3)[0].tolist() == [[0, 1, 2]]        # ties: the lowest
    ids, w, bad = O.route(np.array([[0.0, np.nan], [np.inf, 0.0], [-np.inf, -np.inf], [-np.inf, 0.0]]), 2)
    assert bad == 3 and ids.tolist() == [[-1, -1]] * 3 + [[1, 0]] and w[3].tolist() == [1.0, 0.0]
    ids, w, bad = O.route(np.full((1, 3), -1e4), 2, "sigmoid")            # no underflow of the sum
    assert bad == 0 and w.tolist() == [[0.5, 0.5]]
    assert O.route(np.zeros((2, 3)), 1, rows=[0, 1])[0].tolist() == [[-1], [0]]


def test_plan_is_a_stable_sort():
    offsets, pairs, places = O.plan(np.array([[2, 0], [-1, 2], [0, 9]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4] and pairs.tolist() == [1, 4, 0, 3, -1, -1]
    assert places.tolist() == [[2, 0], [-1, 3], [1, -1]]


@pytest.mark.parametrize("N,K,gated", [(128, 256, False), (130, 320, False), (256, 576, True)])
def test_packed_image_holds_every_byte_once(N, K, gated):
    rng = np.random.default_rng(N)
    codes = rng.integers(1, 256, (2, N, K // 2)).astype(np.uint8)
    scales = rng.integers(1, 256, (2, N, K // 16)).astype(np.uint8)
    image = O.pack(codes, scales, gated)
    assert np.array_equal(np.sort(image[image > 0]), np.sort(np.concatenate([codes.ravel(), scales.ravel()])))
    blocks = image.reshape(2, -(-N // 128), -(-K // 256), O.BLOCK)
    row = N // 2 + 1 if gated else 3                                      # packed row 3: up row 1
    assert np.array_equal(blocks[1, 0, 0, 3 * 128 + ((1 ^ 3) * 16):][:16], codes[1, row, 16:32])
    assert np.array_equal(blocks[1, 0, 0, 16384 + 512 + 3 * 16:][:4], scales[1, row, 4:8])


def test_products_against_a_loop():
    rng = np.random.default_rng(0)
    T, k, E, K, I = 5, 2, 3, 8, 4
    ids = np.array([[0, 2], [2, 0], [-1, 1], [1, -1], [-1, -1]])
    offsets, pairs, places = O.plan(ids, E)
    x, w = rng.standard_normal((T, K)), rng.standard_normal((E, 2 * I, K))
    h = O.gate_up(x, w, offsets, pairs, k)[0]
    weights, wd = rng.random((T, k)), rng.standard_normal((E, 6, I))
    y, _ = O.down(h, wd, weights, places, offsets)
    for t in range(T):
        want = np.zeros(6)
        for j in range(k):
            if ids[t, j] >= 0:
                gu = w[ids[t, j]] @ x[t]
                want += weights[t, j] * (wd[ids[t, j]] @ (gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]))
        assert np.allclose(y[t], want)


@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_rotation_is_a_complex_product(style):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    pos = np.array([0, 1, 500, 31999])
    y = O.rotate(x, pos, O.rope_table(32000, 32), style)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0], x[0])
    first = np.arange(16) if style == "halves" else 2 * np.arange(16)
    second = first + (16 if style == "halves" else 1)
    angle = pos[:, None, None] * 10000.0 ** (-np.arange(16) / 16)
    z = (x[..., first] + 1j * x[..., second]) * np.exp(1j * angle)
    assert np.allclose(y[..., first], z.real, atol=1e-6) and np.allclose(y[..., second], z.imag, atol=1e-6)
