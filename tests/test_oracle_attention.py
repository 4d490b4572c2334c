"""The float64 definition of norm, rotation and attention against hand-computed cases and
properties the formulas fix."""

import numpy as np

from oracle import attention as oa


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0]]])                      # mean square 12.5
    y = oa.norm(x, [2.0, 1.0], eps=0.0)
    assert np.allclose(y, [[[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]]], rtol=1e-15)
    assert np.array_equal(oa.norm(x), x)
    assert np.all(oa.norm(np.zeros((1, 1, 4)), np.ones(4)) == 0)


def test_rotation_by_hand_in_both_layouts():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    quarter = [0.25, 0.5]                             # a quarter turn, a half turn
    y, mag = oa.rotate(x, [1], quarter)               # pairs (1, 3), (2, 4); 5, 6 pass
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6], atol=1e-15)
    assert np.allclose(mag[0, 0], [4, 6, 4, 6, 5, 6])
    y, _ = oa.rotate(x, [1], quarter, interleaved=True)   # pairs (1, 2), (3, 4)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6], atol=1e-15)
    y, _ = oa.rotate(x, [-1], quarter, amplitude=2.0)
    assert np.allclose(y[0, 0], [6, -4, -2, -8, 5, 6], atol=1e-14)


def test_rotated_products_depend_on_the_distance_only():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 8))
    turns = 10000.0 ** (-np.arange(4) / 4) / (2 * np.pi)
    dots = [np.sum(oa.rotate(q, [p + 7], turns)[0] * oa.rotate(k, [p], turns)[0]) for p in (0, 3, 100000)]
    assert np.allclose(dots, dots[0], rtol=1e-9)


def test_attention_by_hand():
    q, k = np.array([[1.0, 0.0]]), np.array([[0.0, 1.0], [np.log(3.0), 0.0]])
    v = np.array([[4.0, -4.0], [8.0, 0.0]])
    out, spread, reach = oa.attend(q, k, v, 1.0)      # weights 1/4, 3/4
    assert np.allclose(out, [[7.0, -1.0]]) and np.allclose(spread, [[7.0, 1.0]]) and np.isclose(reach, np.log(3.0))
    assert np.allclose(oa.attend(q, k, v, 1.0, [1])[0], [[4.0, -4.0]])
    assert np.all(oa.attend(q, k, v, 1.0, [0])[0] == 0)
    assert oa.attend(q, k[:0], v[:0], 1.0)[0].shape == (1, 2)


def test_prompt_masks_and_groups():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((7, 4, 8)), rng.standard_normal((6, 2, 8)), rng.standard_normal((6, 2, 8))
    out, _, _ = oa.prompt(q, k, v, [0, 3, 5], [0, 2, 6], 0.3)
    assert np.all(out[0] == 0)                        # 3 rows, 2 keys: the first row sees none
    assert np.allclose(out[1, 3], v[0, 1])            # the second sees the first key only
    assert np.all(np.isnan(out[5:]))                  # rows of no sequence
    s = 0.3 * k[2:5, 0] @ q[3, 1]                     # row 0 of 2, 4 keys: sees three
    p = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[3, 1], p @ v[2:5, 0])


def test_decode_equals_prompt_of_one_row():
    rng = np.random.default_rng(2)
    kc, vc = rng.standard_normal((2, 5, 4, 2, 8))     # 5 pages of 4 rows
    table = np.array([[3, 1, 0], [2, 4, 4]])
    q = rng.standard_normal((2, 4, 8))
    out, _, _ = oa.decode(q, kc, vc, table, [9, 0], 0.5)
    k = np.concatenate([kc[3], kc[1], kc[0]])[:9]
    v = np.concatenate([vc[3], vc[1], vc[0]])[:9]
    assert np.allclose(out[0], oa.prompt(q[:1], k, v, [0, 1], [0, 9], 0.5)[0][0])
    assert np.all(out[1] == 0)


def test_append_by_hand():
    cache = np.zeros((2, 3, 1, 1))
    out = oa.append(cache, np.arange(1.0, 4.0).reshape(3, 1, 1), [4, -1, 0])
    assert out.ravel().tolist() == [3, 0, 0, 0, 1, 0] and np.all(cache == 0)
