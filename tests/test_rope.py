"""Host checks of the rotary positions (CPU): the oracle's pins, what the C calls and the binding refuse before any device
work, and the fixed-point angles."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_79_gb300 as fa
from oracle import rope as orope

FAKE = ctypes.c_void_p(1 << 20)      # never dereferenced
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(fa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fa.load()


def freqs(n):
    return [1e4 ** (-i / n) for i in range(n)]


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 5, 24))
    f, axis = freqs(8), [0, 0, 1, 1, 1, 2, 2, 0]
    pos = rng.integers(-50, 5000, (3, 5))
    y = orope.rotate(x, f, axis, pos, interleaved)
    for i in range(8):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * f[i] * pos[axis[i]])
        assert np.allclose(y[..., a], z.real, atol=1e-11) and np.allclose(y[..., b], z.imag, atol=1e-11)
    assert (y[..., 16:] == x[..., 16:]).all()
    assert np.allclose(orope.rotate(y, f, axis, pos, interleaved, inverse=True), x, atol=1e-12)


def test_oracle_products_depend_on_distances_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    f = freqs(8)
    dots = [float((orope.rotate(q, f, [0] * 8, [[p + 7]]) * orope.rotate(k, f, [0] * 8, [[p]])).sum()) for p in (0, 3, 10 ** 6, 2 ** 30)]
    assert np.allclose(dots, dots[0], atol=1e-8)


def test_turns_are_exact_at_far_positions():
    """position * turns mod 2^64 is the angle: the upper 32 bits of it against a computation in rationals."""
    from fractions import Fraction
    f = freqs(64) + [math.pi, 6.0, 1e-12]
    plan = fa.new_rope(f[:64], device="cpu")
    assert plan.turns.dtype == torch.int64 and plan.axis is None and plan.interleaved is False
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)
    for i in (0, 1, 31, 63):
        for pos in (1, -1, 12345, 2 ** 31 - 1, -2 ** 31):
            got = (int(plan.turns[i]) * pos) % 2 ** 64 / 2 ** 64
            want = float(Fraction(f[i]) * pos / (2 * pi) % 1)
            off = abs(got - want)
            assert min(off, 1 - off) <= abs(pos) * 2.0 ** -65 + 2.0 ** -52, (i, pos)
    assert fa.new_rope([0.0, -1.0, 2 * math.pi, 7.0], device="cpu").turns[0] == 0


def call_rope(lib, q=FAKE, qs=(12800, 64, 128), qo=FAKE, qos=(12800, 64, 128), Hq=2, k=FAKE, ks=(12800, 64, 128), ko=FAKE,
              kos=(12800, 64, 128), Hkv=2, B=1, T=100, d=64, elt=2, pairs=32, axes=1, turns=1 << 20, plan=True, pos=FAKE, sa=100, sb=0):
    r = fa._Rope(turns, None, pairs, axes, 0)
    return lib.fa_rope(q, *qs, qo, *qos, Hq, k, *ks, ko, *kos, Hkv, B, T, d, elt, ctypes.byref(r) if plan else None, pos, sa, sb, 0, NULL)


def test_rope_c_refusals(lib):
    off = ctypes.c_void_p((1 << 20) + 8)
    for bad in (dict(q=NULL), dict(qo=NULL), dict(k=NULL), dict(ko=NULL), dict(pos=NULL), dict(plan=False), dict(turns=0), dict(q=off),
                dict(ko=off), dict(Hq=0), dict(Hkv=-1), dict(B=0), dict(T=0), dict(d=60), dict(d=264), dict(elt=1), dict(elt=8),
                dict(pairs=0), dict(pairs=36), dict(axes=0), dict(qs=(12800, 64, 132)), dict(qs=(12800, -64, 128)),
                dict(qos=(12800, 64, 0)), dict(kos=(12800, 0, 128)), dict(B=2, qos=(0, 64, 128)), dict(sa=-1), dict(sb=-1)):
        assert call_rope(lib, **bad) == 1, bad
    assert call_rope(lib, pairs=30) == 2
    assert call_rope(lib, B=1 << 16, T=1 << 16, qos=(1 << 30, 64, 128), kos=(1 << 30, 64, 128)) == 2


def test_append_rope_c_refusals(lib):
    c = fa._Cache8(1 << 20, 1 << 20, 1 << 20, 1 << 20, None, 10, 2, 64)

    def call(pairs=32, axes=1, turns=1 << 20, plan=True, sa=0, cache=True, k=FAKE):
        r = fa._Rope(turns, None, pairs, axes, 0)
        return lib.fa_cache8_append_rope(k, 64, 128, FAKE, 64, 128, FAKE, FAKE, 1, 5, ctypes.byref(c) if cache else None, FAKE, 4,
                                         ctypes.byref(r) if plan else None, NULL, sa, NULL)
    for bad in (dict(pairs=0), dict(pairs=36), dict(axes=0), dict(turns=0), dict(plan=False), dict(sa=-1), dict(cache=False), dict(k=NULL)):
        assert call(**bad) == 1, bad
    assert call(pairs=6) == 2


def test_binding_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(4, 10, 64, dtype=bf), torch.zeros(2, 10, 64, dtype=bf)
    r = fa.new_rope(freqs(32), device="cpu")
    pos = torch.zeros(1, 10, dtype=i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.rope(q, k, r, pos)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.rope(q, None, r, pos)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        fa.rope(q.half(), k, r, pos)
    with pytest.raises(ValueError, match=r"\[H, T, d\]"):
        fa.rope(q[0], k, r, pos)
    with pytest.raises(ValueError, match="^k:"):
        fa.rope(q, k[:, :9], r, pos)
    with pytest.raises(ValueError, match="^k:"):
        fa.rope(q, k.float(), r, pos)
    with pytest.raises(ValueError, match="as many dimensions"):
        fa.rope(q, k[None], r, pos)
    with pytest.raises(ValueError, match="k_out without k"):
        fa.rope(q, None, r, pos, k_out=k)
    with pytest.raises(ValueError, match="^q_out:"):
        fa.rope(q, k, r, pos, q_out=k)
    with pytest.raises(ValueError, match="^k_out:"):
        fa.rope(q, k, r, pos, k_out=q)
    with pytest.raises(ValueError, match="multiples of 8"):
        fa.rope(torch.zeros(4, 10, 68, dtype=bf)[..., :64], k, r, pos)
    with pytest.raises(ValueError, match="contiguous"):
        fa.rope(torch.zeros(4, 64, 10, dtype=bf).transpose(1, 2), k, r, pos)
    for bad in (pos.long(), pos[:, :9], pos[None], torch.zeros(10, 2, dtype=i32).t()[:1], torch.zeros(1, 10, 2, dtype=i32)[..., 0]):
        with pytest.raises(ValueError, match="positions"):
            fa.rope(q, k, r, bad)
    with pytest.raises(ValueError, match="positions"):
        fa.rope(q[None], k[None], r, torch.zeros(1, 3, 10, dtype=i32))
    with pytest.raises(ValueError, match="rope.axis"):
        fa.rope(q, k, r._replace(axis=torch.zeros(31, dtype=i32)), pos)
    with pytest.raises(ValueError, match="rope.turns"):
        fa.rope(q, k, r._replace(turns=torch.zeros(32)), pos)
    c = fa.new_cache8(4, 2, 64, device="cpu")
    cu, table, start = torch.tensor([0, 10], dtype=i32), torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError, match="positions without rope"):
        fa.cache8_append(c, k, k, cu, table, start, positions=pos)
    with pytest.raises(ValueError, match="positions must"):
        fa.cache8_append(c, k, k, cu, table, start, rope=r, positions=pos[:, :9])
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.cache8_append(c, k, k, cu, table, start, rope=r, positions=pos)
