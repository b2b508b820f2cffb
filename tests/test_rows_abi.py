"""Refusals of the norm, cache and 8-bit attention entry points: answered on
the host before anything touches a device (CPU)."""
import ctypes

import pytest
import torch

from long_context_05_b200 import dsa

INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p(1 << 20)          # never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned


@pytest.fixture(scope="module")
def L():
    from long_context_05_b200 import build
    build.build()
    return dsa.lib()


def shape(**kw):
    f = dict(B=2, T=3, S=64, H_I=4, D_I=32, H=8, d_k=80, d_v=64, k=16, q_block=3)
    return dsa.make_shape(None, **{**f, **kw})


def desc(**kw):
    f = dict(Hq=2, Hk=1, D=80, norm_cols=64, rope_cols=16, interleaved=0, eps=1e-6, q_weight=None, k_weight=None,
             inv_freq=1 << 20)
    return dsa.NormRope(**{**f, **kw})


BAD_SHAPES = [(dict(T=65), INVALID), (dict(D_I=48), UNSUPPORTED), (dict(d_k=576, d_v=64), UNSUPPORTED),
              (dict(H=12), UNSUPPORTED), (dict(k=2049), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
              (dict(page_size=16), INVALID), (dict(B=0), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_bad_shapes(L, kw, code):
    s = ctypes.byref(shape(**kw))
    d = ctypes.byref(desc())
    assert L.dsa_norm_rope(s, d, P, P, P, P, None) == code
    assert L.dsa_norm_rope_workspace_size(s, d) == 0
    assert L.dsa_norm_rope_backward(s, d, P, P, P, P, P, P, None, None, None, 0, None) == code
    assert L.dsa_cache_write(s, *[P] * 9, None) == code
    assert L.dsa_cache_read(s, 0, 1, *[P] * 6, None) == code
    assert L.dsa_workspace8_size(s) == 0
    assert L.dsa_sparse_attn8(s, P, P, P, P, P, None, P, 1 << 40, None) == code
    assert L.dsa_dense_attn8(s, P, P, P, P, None, P, 1 << 40, None) == code
    ins = dsa.Inputs8(*[1 << 20] * 8)
    assert L.dsa_forward8(s, ctypes.byref(ins), P, None, P, P, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(D=0), INVALID), (dict(Hq=-1), INVALID), (dict(Hq=0, Hk=0), INVALID), (dict(norm_cols=88), INVALID),
    (dict(rope_cols=96), INVALID), (dict(inv_freq=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(q_weight=(1 << 20) + 4), INVALID), (dict(D=84), UNSUPPORTED),
    (dict(D=1032), UNSUPPORTED), (dict(norm_cols=60), UNSUPPORTED), (dict(rope_cols=24), UNSUPPORTED),
    (dict(D=1024, rope_cols=272), UNSUPPORTED), (dict(Hq=1025), UNSUPPORTED)])
def test_bad_descriptions(L, kw, code):
    s, d = ctypes.byref(shape()), ctypes.byref(desc(**kw))
    assert L.dsa_norm_rope(s, d, P, P, P, P, None) == code
    assert L.dsa_norm_rope_backward(s, d, P, P, P, P, P, P, None, None, None, 0, None) == code
    assert L.dsa_norm_rope_workspace_size(s, d) == 0


def test_rows_that_do_not_fit_an_int(L):
    s = ctypes.byref(shape(B=1 << 12, T=1 << 14, S=1 << 14))
    assert L.dsa_norm_rope(s, ctypes.byref(desc(Hq=128)), P, P, P, P, None) == UNSUPPORTED
    assert L.dsa_cache_write(ctypes.byref(shape(B=1 << 12, T=1 << 14, S=1 << 14, H_I=64)), *[P] * 9, None) == UNSUPPORTED
    big = ctypes.byref(shape(B=1 << 12, T=1 << 12, S=1 << 12, H=128))
    assert L.dsa_sparse_attn8(big, *[P] * 6, P, 1 << 40, None) == UNSUPPORTED
    assert L.dsa_dense_attn8(big, *[P] * 5, P, 1 << 40, None) == UNSUPPORTED
    assert L.dsa_workspace8_size(big) == 0
    assert L.dsa_cache_read(ctypes.byref(shape(B=1 << 12, T=1, S=1 << 20)), 0, 1 << 20, *[P] * 6, None) == UNSUPPORTED


def test_pointers_of_the_norm(L):
    s, d = ctypes.byref(shape()), ctypes.byref(desc())
    ok = [P, P, P, P]
    for i in range(4):
        for bad in (None, ODD):
            a = list(ok)
            a[i] = bad
            assert L.dsa_norm_rope(s, d, *a, None) == INVALID
    ok = [P] * 6
    for i in range(6):
        for bad in (None, ODD):
            a = list(ok)
            a[i] = bad
            assert L.dsa_norm_rope_backward(s, d, *a, None, None, None, 0, None) == INVALID
    assert L.dsa_norm_rope(None, d, *[P] * 4, None) == INVALID
    assert L.dsa_norm_rope(s, None, *[P] * 4, None) == INVALID


def test_parts_of_the_cache_are_whole(L):
    s = ctypes.byref(shape())
    assert L.dsa_cache_write(s, *[None] * 10) == INVALID                     # nothing to do
    for part in range(3):
        for miss in range(3):
            a = [P] * 9
            a[3 * part + miss] = None
            assert L.dsa_cache_write(s, *a, None) == INVALID
        for odd in range(2):                                                 # rows and bytes are vectors
            a = [P] * 9
            a[3 * part + odd] = ODD
            assert L.dsa_cache_write(s, *a, None) == INVALID
    assert L.dsa_cache_read(s, 0, 1, *[None] * 7) == INVALID
    for miss in range(6):
        a = [P] * 6
        a[miss] = None
        assert L.dsa_cache_read(s, 0, 1, *a, None) == INVALID
    for begin, count in ((-1, 1), (0, -1), (0, 65), (64, 1), (2**31 - 1, 2**31 - 1)):
        assert L.dsa_cache_read(s, begin, count, *[P] * 6, None) == INVALID


def test_pointers_of_the_attention(L):
    s = ctypes.byref(shape())
    for i in range(5):                       # q, kv8, kv_scale, idx, out
        a = [P] * 5
        a[i] = None
        assert L.dsa_sparse_attn8(s, *a, None, P, 1 << 40, None) == INVALID
    for i in (0, 1, 4):
        a = [P] * 5
        a[i] = ODD
        assert L.dsa_sparse_attn8(s, *a, None, P, 1 << 40, None) == INVALID
    assert L.dsa_sparse_attn8(s, *[P] * 5, None, ODD, 1 << 40, None) == INVALID
    for i in range(4):
        a = [P] * 4
        a[i] = None
        assert L.dsa_dense_attn8(s, *a, None, P, 1 << 40, None) == INVALID
    for name in dsa.INPUT8_NAMES:
        ins = dsa.Inputs8(*[None if n == name else 1 << 20 for n in dsa.INPUT8_NAMES])
        assert L.dsa_forward8(s, ctypes.byref(ins), P, None, P, P, 1 << 40, None) == INVALID
    ins = dsa.Inputs8(*[1 << 20] * 8)
    assert L.dsa_forward8(s, None, P, None, P, P, 1 << 40, None) == INVALID
    assert L.dsa_forward8(s, ctypes.byref(ins), P, None, None, P, 1 << 40, None) == INVALID
    dec = shape(mode=dsa.DSA_DECODE)         # T = 3
    assert L.dsa_forward8(ctypes.byref(dec), ctypes.byref(ins), P, None, P, P, 1 << 40, None) == INVALID


def test_workspace_covers_the_path(L):
    for kw in (dict(), dict(mode=dsa.DSA_DECODE, T=1), dict(B=1, T=1, S=131072, k=2048, d_k=576, d_v=512, H=128)):
        s = shape(**kw)
        assert dsa.workspace8_size(s) >= dsa.workspace_size(s) > 0
    assert L.dsa_launch_count() == 0


def test_binding_refuses_what_it_is_not_given():
    s = shape()
    cpu = torch.zeros(2 * 3 * 80, dtype=torch.bfloat16)
    u8 = torch.zeros(2 * 64 * 80, dtype=torch.uint8)
    sc = torch.zeros(2 * 64)
    with pytest.raises(ValueError):
        dsa.cache_write(s, kv=cpu, kv8=u8, kv_scale=sc)                       # CPU tensors
    with pytest.raises(ValueError):
        dsa.cache_write(s, kv=cpu.float(), kv8=u8, kv_scale=sc)
    with pytest.raises(ValueError):
        dsa.norm_rope(s, desc(), cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError):
        dsa.dense_attn8(s, cpu, u8, sc, cpu, None, None)
    with pytest.raises(ValueError):
        dsa.make_norm_rope(Hq=1, Hk=0, D=32, norm_cols=32, rope_cols=0, q_weight=torch.ones(32))
