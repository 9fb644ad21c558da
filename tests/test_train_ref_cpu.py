"""The plain implementations of tests/train_ref.py against published values, closed
forms, differences, and one another."""

import numpy as np
import pytest

import train_ref as ref


@pytest.mark.parametrize("counter,key,words", [
    # Random123's known answers for philox4x32 of 10 rounds
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox(counter, key, words):
    assert tuple(ref.philox(counter, key)) == words


def test_a_mask_is_its_formula():
    m = ref.kept(3, 11, 0.25, (5, -1))
    words = ref.philox((1, 2, 0xffffffff, 0xffffffff), (5, 0))
    assert m[2, 8] == (words[0] & 0xffff >= 16384) and m[2, 9] == (words[0] >> 16 >= 16384)
    assert m[2, 10] == (words[1] & 0xffff >= 16384)
    many = ref.kept(400, 64, 0.25, (1, 2))
    assert abs(many.mean() - 0.75) < 5 * (0.25 * 0.75 / many.size) ** 0.5  # five standard deviations


def test_an_even_route_has_the_loss_scale():
    keys = np.arange(12)[:, None] * 2 % 8 + np.arange(2)[None]  # each of 8 keys 3 times
    (loss, counts, mean, coef), _ = ref.balance(np.zeros((12, 8)), keys, scale=0.5)
    assert loss == pytest.approx(0.5) and (counts == 3).all() and np.allclose(mean, 1 / 8)
    assert coef[0] == pytest.approx(0.5 * 8 / (2 * 12 ** 2))
    # all on one key, whose share is 1: keys / k times as much
    x = np.full((12, 8), -np.inf)
    x[:, 3] = 0
    (loss, *_), _ = ref.balance(x, np.full((12, 1), 3), scale=0.5)
    assert loss == pytest.approx(0.5 * 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("per_chunk", [False, True])
def test_the_gradient_is_the_losses_difference(score, per_chunk):
    rng = np.random.default_rng(1)
    x, keys = rng.normal(size=(12, 7)), rng.integers(-1, 8, size=(12, 3))
    kw = dict(score=score, chunk=4, chunk_valid=np.array([4, 0, 3]), per_chunk=per_chunk)
    (loss, counts, mean, coef), _ = ref.balance(x, keys, scale=3.0, **kw)
    d, _ = ref.balance_backward(x, counts, coef, dloss=2.0, **kw)
    for t in range(12):
        for i in range(7):
            y = x.copy()
            y[t, i] += 1e-6
            up = ref.balance(y, keys, scale=3.0, **kw)[0][0]
            y[t, i] -= 2e-6
            down = ref.balance(y, keys, scale=3.0, **kw)[0][0]
            # central differences: h^2 of the third derivative, and the losses' own rounding over h
            assert d[t, i] == pytest.approx(2 * (up - down) / 2e-6, abs=1e-8)
    assert not d[4:8].any() and not d[11].any()


def test_shares_of_deep_and_masked_rows():
    x = np.array([-1e30, -1e30, -np.inf])
    assert np.allclose(ref.shares(x, "sigmoid")[0], [0.5, 0.5, 0])
    x = np.array([-70.0, -71.0, -200.0])
    s = 1 / (1 + np.exp(-x))
    assert np.allclose(ref.shares(x, "sigmoid")[0], s / s.sum(), rtol=1e-12, atol=0)
    assert not ref.shares(np.full(4, -np.inf), "softmax")[0].any()


def test_bank_grad_by_hand():
    out, size, count = ref.bank_grad(3, np.array([2, -1, 0, 2, 3]), lambda e: np.array([[1.0], [0], [5], [-4], [9]])[e], 1)
    assert out.ravel().tolist() == [5, 0, -3] and size.ravel().tolist() == [5, 0, 5] and count.tolist() == [1, 0, 2]
    assert ref.factor(1.0, 0.5) == 2 and ref.threshold(0.1) == 6554
