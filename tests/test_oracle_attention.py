"""Pins of the attention and norm oracle: hand cases, and the properties that its definitions have."""
import numpy as np
import pytest

from oracle import attention as A


def test_visible_by_hand():
    assert A.visible(-1, 5, 0, 0).tolist() == []
    assert A.visible(0, 5, 0, 0).tolist() == [0]
    assert A.visible(3, 3, 0, 0).tolist() == [0, 1, 2]
    assert A.visible(9, 10, 3, 0).tolist() == [7, 8, 9]
    assert A.visible(9, 10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert A.visible(2, 10, 3, 2).tolist() == [0, 1, 2]           # the window covers the first tokens
    assert A.visible(3, 10, 3, 9).tolist() == [0, 1, 2, 3]        # more first tokens than there are
    assert A.visible(4, 10, 1, 0).tolist() == [4]


def test_one_key_gives_its_value_and_none_gives_zero():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    out, mag = A.attend(q, k, v, -2, 0.3)
    assert not out[0].any() and not out[1].any()
    assert np.allclose(out[2], v[0], rtol=1e-15) and np.allclose(mag[2], np.abs(v[0]))


def test_equal_scores_average_and_unseen_values_do_not_matter():
    k, v = np.zeros((6, 4)), np.arange(24.0).reshape(6, 4)
    out, _ = A.attend(np.ones((2, 4)), k, v, 3, 1.0)
    assert np.allclose(out[0], v[:4].mean(0)) and np.allclose(out[1], v[:5].mean(0))
    poisoned = v.copy()
    poisoned[5] = np.nan
    assert np.array_equal(A.attend(np.ones((2, 4)), k, poisoned, 3, 1.0)[0], out)


def test_weights_are_the_softmax():
    q, k, v = np.array([[1.0, 0]]), np.array([[0.0, 5], [np.log(3.0), 1]]), np.array([[1.0, 0], [0, 1]])
    assert np.allclose(A.attend(q, k, v, 1, 1.0)[0], [[0.25, 0.75]])


def test_heads_of_a_group_share_keys():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, _ = A.attend_heads(q, k, v, 3, 0.5)
    for h in range(4):
        assert np.array_equal(out[:, h], A.attend(q[:, h], k[:, h // 2], v[:, h // 2], 3, 0.5)[0])


def test_norm_by_hand():
    h, y = A.add_rmsnorm([[3.0, 4.0]], [[0.0, 0.0]], [1.0, 2.0], 0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]) and np.array_equal(h, [[3.0, 4.0]])
    assert np.array_equal(A.add_rmsnorm(np.zeros((1, 4)), None, np.ones(4), 1e-6)[1], np.zeros((1, 4)))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_blocks_that_are_not_finite_have_the_nan_scale(bad):
    x = np.ones((2, 64), dtype=np.float32)
    x[1, 40] = bad
    q, s = A.quant_block_mxfp8(x)
    assert s[1, 1] == 255 and not q[1, 32:].any() and (s[[0, 0, 1], [0, 1, 0]] != 255).all()
