"""FP64 CPU oracle for the operators around the path: the norm and rotation of
head rows, the 8-bit cache rows, and attention over them.

TEST INFRASTRUCTURE ONLY, like dsa_oracle.py: only tests import it, and it
shares no code with the product.  Plain NumPy in float64, one row at a time.
"""
from __future__ import annotations

import numpy as np

from oracle import dsa_oracle as O

E4M3_MAX = 448.0
MIN_EXP = -48


# ---------------------------------------------------------------- norm and rotation

def _pairs(D: int, rope: int, interleaved: bool):
    """Column pairs (a, b) of the rotated columns D - rope .. D."""
    i = np.arange(rope // 2)
    if interleaved:
        return D - rope + 2 * i, D - rope + 2 * i + 1
    return D - rope + i, D - rope + rope // 2 + i


def norm_rope_row(x, pos: int, weight, norm: int, rope: int, inv_freq, eps: float, interleaved: bool):
    """One head row x [D]: the first `norm` columns divided by their root mean
    square and weighted, then the last `rope` columns rotated by pos * inv_freq."""
    z = np.asarray(x, np.float64).copy()
    if norm:
        w = np.ones(norm) if weight is None else np.asarray(weight, np.float64)
        z[:norm] = w * z[:norm] / np.sqrt(np.mean(z[:norm] ** 2) + eps)
    if rope:
        a, b = _pairs(z.shape[0], rope, interleaved)
        ang = pos * np.asarray(inv_freq, np.float64)
        za, zb = z[a], z[b]
        z[a], z[b] = za * np.cos(ang) - zb * np.sin(ang), za * np.sin(ang) + zb * np.cos(ang)
    return z


def norm_rope_grad_row(x, dy, pos: int, weight, norm: int, rope: int, inv_freq, eps: float, interleaved: bool):
    """Gradients (dx [D], dweight [norm]) of sum(dy * norm_rope_row(x))."""
    x = np.asarray(x, np.float64)
    g = np.asarray(dy, np.float64).copy()
    if rope:
        a, b = _pairs(x.shape[0], rope, interleaved)
        ang = pos * np.asarray(inv_freq, np.float64)
        ga, gb = g[a], g[b]
        g[a], g[b] = ga * np.cos(ang) + gb * np.sin(ang), -ga * np.sin(ang) + gb * np.cos(ang)
    if not norm:
        return g, np.zeros(0)
    w = np.ones(norm) if weight is None else np.asarray(weight, np.float64)
    rho = 1.0 / np.sqrt(np.mean(x[:norm] ** 2) + eps)
    dw = g[:norm] * x[:norm] * rho
    wg = w * g[:norm]
    dx = g
    dx[:norm] = rho * wg - x[:norm] * rho ** 3 * np.mean(wg * x[:norm])
    return dx, dw


# ---------------------------------------------------------------- e4m3 rows

_E4M3 = O.e4m3_decode(np.arange(127, dtype=np.uint8))     # the finite non-negative values, ascending


def e4m3_encode(y) -> np.ndarray:
    """Bytes of the nearest e4m3 numbers, ties to the even byte (|y| <= 448)."""
    y = np.asarray(y, np.float64)
    a = np.abs(y)
    hi = np.searchsorted(_E4M3, a).clip(0, 126)             # first value >= a
    lo = np.maximum(hi - 1, 0)
    dh, dl = _E4M3[hi] - a, a - _E4M3[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    byte = np.where(up, hi, lo).astype(np.uint8)
    return byte | (np.signbit(y).astype(np.uint8) << 7)


def quantise_row(x):
    """(bytes, scale) of a row: scale 2^e with the smallest e >= -48 that has
    max|x| <= 448 * 2^e; what lies past 240 * 2^120 (whose byte would stand for
    2^128, no FP32 number) is taken as that."""
    x = np.clip(np.asarray(x, np.float64), -240 * 2.0 ** 120, 240 * 2.0 ** 120)
    e = MIN_EXP
    while np.abs(x).max() > E4M3_MAX * 2.0 ** e:
        e += 1
    return e4m3_encode(x / 2.0 ** e), 2.0 ** e


def dequantise(b, scale):
    """float64 rows of bytes b [..., D] with scales [...]."""
    return O.e4m3_decode(b) * np.asarray(scale, np.float64)[..., None]


# ---------------------------------------------------------------- attention over them

def attention_row(q_t, kv, sel, d_v: int, tau: float):
    """(out [H, d_v], lse [H], A [H, d_v], pmax [H]) over rows `sel` (-1 skipped)
    of the dequantised cache kv: dsa_oracle's attention, with what its error
    bounds need: A = sum_k w_k |V_k| and the largest softmax weight.  No key:
    out 0, lse -inf."""
    sel = np.asarray(sel)
    sel = sel[sel >= 0]
    H = q_t.shape[0]
    if sel.size == 0:
        return np.zeros((H, d_v)), np.full(H, -np.inf), np.zeros((H, d_v)), np.zeros(H)
    out, lse = O.sparse_attention_row(q_t, kv, sel, d_v, tau)
    w = np.exp(tau * (np.asarray(q_t, np.float64) @ kv[sel].T) - lse[:, None])
    return out, lse, w @ np.abs(kv[sel][:, :d_v]), w.max(axis=1)
