"""What pins the oracle of the norm, rotation and 8-bit rows (CPU)."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from oracle import rows_oracle as R

FREQ = 10000.0 ** (-np.arange(4) / 4.0)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_relative_and_keeps_norms(inter):
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal(16), rng.standard_normal(16)

    def rot(x, pos):
        return R.norm_rope_row(x, pos, None, 0, 8, FREQ, 0.0, inter)

    assert np.allclose(rot(a, 0), a)
    for p in (1, 17, 131071):
        assert np.isclose(np.linalg.norm(rot(a, p)), np.linalg.norm(a))
        assert np.allclose(rot(a, p)[:8], a[:8])
        # the product of two rotated rows depends on the distance alone
        assert np.isclose(rot(a, p) @ rot(b, p + 5), rot(a, 0) @ rot(b, 5))
    # the pairs: position pi/2 / freq_0 turns the first pair's (1, 0) into (0, 1)
    e = np.zeros(16)
    e[8] = 1.0
    y = R.norm_rope_row(e, 1, None, 0, 8, np.array([np.pi / 2, 0, 0, 0]), 0.0, inter)
    assert np.isclose(y[9 if inter else 12], 1.0) and np.isclose(y[8], 0.0, atol=1e-15)


def test_norm_closed_forms():
    y = R.norm_rope_row(np.full(8, 3.0), 5, np.arange(1, 9.0), 8, 0, None, 0.0, False)
    assert np.allclose(y, np.arange(1, 9.0))                       # x / rms = 1
    y = R.norm_rope_row(np.array([3.0, 4, 7, 9]), 0, None, 2, 0, None, 0.0, False)
    assert np.allclose(y, [3 / np.sqrt(12.5), 4 / np.sqrt(12.5), 7, 9])


@pytest.mark.parametrize("norm,rope,inter", [(16, 8, False), (16, 8, True), (8, 8, False), (0, 8, True), (16, 16, False),
                                             (16, 0, False)])
def test_gradients_by_differences(norm, rope, inter):
    rng = np.random.default_rng(norm + rope)
    x, dy, w = rng.standard_normal(16), rng.standard_normal(16), rng.standard_normal(norm)
    f = 10000.0 ** (-np.arange(rope // 2) / max(1, rope // 2))
    args = dict(norm=norm, rope=rope, inv_freq=f, eps=1e-3, interleaved=inter)
    dx, dw = R.norm_rope_grad_row(x, dy, 37, w, **args)
    h = 1e-6
    for c in range(16):
        e = np.eye(16)[c] * h
        num = (dy @ R.norm_rope_row(x + e, 37, w, **args) - dy @ R.norm_rope_row(x - e, 37, w, **args)) / (2 * h)
        assert abs(num - dx[c]) <= 1e-8 * max(1, abs(num)) * 100
    for c in range(norm):
        e = np.eye(norm)[c] * h
        num = (dy @ R.norm_rope_row(x, 37, w + e, **args) - dy @ R.norm_rope_row(x, 37, w - e, **args)) / (2 * h)
        assert abs(num - dw[c]) <= 1e-6


def test_e4m3_encode_against_torch_and_its_inverse():
    for b in range(256):
        if b & 0x7F == 0x7F:
            continue
        assert int(R.e4m3_encode(O.e4m3_decode(np.uint8(b)))) == b
    rng = np.random.default_rng(3)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.05, 0.05, 4000),
                        (O.e4m3_decode(np.arange(126, dtype=np.uint8)) + O.e4m3_decode(np.arange(1, 127, dtype=np.uint8))) / 2])
    y = y.astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_encode(y), want)


def test_row_scale_is_the_smallest_power_of_two():
    for amax, e in ((448.0, 0), (449.0, 1), (1.0, -8), (0.875, -9), (0.876, -8), (0.0, -48), (2.0 ** -60, -48),
                    (3.3e38, 120)):
        b, s = R.quantise_row([amax, 0.0])
        assert s == 2.0 ** e, (amax, s)
        assert abs(float(O.e4m3_decode(b)[0]) * s - amax) <= (2.0 ** -4 * amax if e > -48 else 2.0 ** -58)
    b, s = R.quantise_row([3.3e38, -np.inf, 1.0])          # stays finite in FP32
    assert np.array_equal(O.e4m3_decode(b) * s, [240 * 2.0 ** 120, -240 * 2.0 ** 120, 0.0])


def test_attention_row_bounds_and_empty():
    rng = np.random.default_rng(4)
    q, kv = rng.standard_normal((3, 8)), rng.standard_normal((10, 8))
    out, lse, A, pm = R.attention_row(q, kv, np.array([1, -1, 5, 5]), 6, 0.5)
    o2, l2 = O.sparse_attention_row(q, kv, np.array([1, 5, 5]), 6, 0.5)
    assert np.allclose(out, o2) and np.allclose(lse, l2)
    assert (A >= np.abs(out) - 1e-15).all() and (pm <= 1).all() and (pm > 1 / 4).all()
    out, lse, _, _ = R.attention_row(q, kv, np.array([-1, -1]), 6, 0.5)
    assert (out == 0).all() and np.isneginf(lse).all()
