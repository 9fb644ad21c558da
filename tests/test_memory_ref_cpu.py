"""The plain implementations of tests/memory_ref.py against hand-worked values,
differences and torch, so that they can be held against the kernels."""

import numpy as np
import pytest
import torch

import memory_ref as ref


def test_route_by_hand():
    x = np.log(np.array([[1.0, 4.0, 3.0, 2.0]]))
    keys, w = ref.route(x, 2)
    assert keys.tolist() == [[1, 2]] and np.allclose(w, [[0.4, 0.3]])
    keys, w = ref.route(x, 2, normalise=True, scale=7)
    assert keys.tolist() == [[1, 2]] and np.allclose(w, [[4, 3]])
    # the bias steers the choice and leaves the weights
    keys, w = ref.route(x, 2, bias=[0.5, 0, 0, 0])
    assert keys.tolist() == [[0, 1]] and np.allclose(w, [[0.1, 0.4]])
    # ties to the lowest key; masked keys last, with weight 0
    keys, w = ref.route([[1.0, -np.inf, 1.0, np.nan]], 4, score="sigmoid")
    assert keys.tolist() == [[0, 2, 1, 3]] and w[0, 2] == 0 and w[0, 3] == 0
    # two groups: 0.1 + 0.4 against 0.3 + 0.2 is a tie; by the largest alone the first group wins too
    keys, _ = ref.route(x, 2, groups=2, kept=1, top=1)
    assert keys.tolist() == [[1, 0]]
    keys, _ = ref.route(np.log([[1.0, 4.0, 3.0, 2.5]]), 2, groups=2, kept=1, top=2)
    assert keys.tolist() == [[2, 3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [False, True])
def test_route_backward_against_differences(score, normalise):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 9))
    x[1, 4] = -np.inf
    keys, _ = ref.route(x, 4, score=score)
    dw = rng.standard_normal((3, 4))

    def loss(y):
        total = 0.0
        for t in range(3):
            s = ref.scores(y[t], score)[keys[t]]
            total += (2.5 * (s / s.sum() if normalise else s) * dw[t]).sum()
        return total

    got, _ = ref.route_backward(x, keys, dw, score=score, normalise=normalise, scale=2.5)
    for t in range(3):
        for i in range(9):
            if x[t, i] == -np.inf:
                assert got[t, i] == 0
                continue
            up, down = x.copy(), x.copy()
            up[t, i] += 1e-6
            down[t, i] -= 1e-6
            # central differences: 1e-12 of curvature, 1e-16 / 1e-6 of rounding, sizes near 1
            assert abs((loss(up) - loss(down)) / 2e-6 - got[t, i]) < 1e-8


def test_pack_by_hand():
    codes, scales = ref.pack(np.array([[448.0, -1.0, 0.0, -0.0, 27.0]], np.float32), "mx8")
    # scale 1: 448 = 0x7e; -1 = 0xb8; 27 lies between 26 and 28 and takes the even 28 (1.75 2^4)
    assert scales.tolist() == [[127, 0, 0, 0]]
    assert codes[0, :5].tolist() == [0x7e, 0xb8, 0, 0x80, 0x5e] and not codes[0, 5:].any()
    codes, scales = ref.pack(np.array([[6.0, -0.25, 0.75, -5.0, 2.5]], np.float32), "mx4")
    assert scales.tolist() == [[127, 0, 0, 0]]
    assert codes[0, :3].tolist() == [0x87, 0xe2, 0x04]
    codes, scales = ref.pack(np.array([[6.5, 1.0]], np.float32), "mx4")
    assert scales[0, 0] == 128 and codes[0, 0] == 0x15  # 3.25 -> 3, 0.5


def test_pack8_agrees_with_torch_at_scale_one():
    x = np.concatenate([[448.0], np.random.default_rng(1).uniform(-448, 448, 31 * 400)])[:32 * 300]
    x = x.reshape(300, 32).astype(np.float32)
    x[:, 0] = 448.0
    codes, scales = ref.pack(x, "mx8")
    assert (scales[:, 0] == 127).all()
    assert np.array_equal(codes[:, :32], torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("kind", ["mx8", "mx4"])
@pytest.mark.parametrize("hd", [1, 31, 33, 100, 128])
def test_pack_round_trip(kind, hd):
    rng = np.random.default_rng(hd)
    x = (rng.standard_normal((40, hd)) * np.exp2(rng.integers(-140, 120, (40, 1)))).astype(np.float32)
    codes, scales = ref.pack(x, kind)
    assert codes.shape == (40, ref.row_bytes(hd, kind)) and scales.shape == (40, ref.scale_bytes(hd))
    y = ref.unpack(codes, scales, hd, kind)
    again = ref.pack(y.astype(np.float32), kind)
    assert np.array_equal(y, y.astype(np.float32).astype(np.float64))  # float32 holds every value
    assert np.array_equal(ref.unpack(*again, hd, kind), y)
    # half a step: of the value (4 or 2 significant bits), or of the smallest code
    step, least = (2.0 ** -4, 2.0 ** -10) if kind == "mx8" else (2.0 ** -2, 2.0 ** -2)
    scale = np.exp2(scales[:, np.arange(hd) // 32].astype(np.float64) - 127)
    assert (np.abs(y - x) <= np.maximum(step * np.abs(x), least * scale)).all()
