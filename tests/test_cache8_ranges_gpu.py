"""Attention over the 8-bit cache at the ends of what bf16 queries and the cache's scales can be, on the GPU against 64 bits.

The bounds are those of test_cache8_chunk_gpu.check and test_cache8_gpu.check_attention, which are relative to the row's own
values but for 1e-30. O is linear in V's scales, so results near that are compared times a power of two, taken in 64 bits:
V's scales and O both, which changes no relative bound. A bf16 below 2^-126 is off by at most 2^-134; with V scales of 2^-126
the bound is 2^-11 sum p |code| 2^-126, which is more as soon as the mean magnitude of the codes is 2^3, and here it is about 38.
"""
import numpy as np
import pytest
import torch

from test_cache8_chunk_gpu import check, run
from test_cache8_gpu import DEV, bf16, check_attention, ints, make, to_gpu

pytestmark = pytest.mark.gpu

# new tokens and cached ones before them, Hq, Hkv, d: an item of one row tile, whole and over many CTAs; of two row tiles; wide
CASES = [
    ([20], [200], 4, 2, 128),
    ([300, 3], [70, 9000], 4, 2, 128),
    ([130, 3], [100, 3000], 2, 2, 256),
]


def spread_rows(x, exponents):
    """x, row after row (tokens; the dimension before the last) times 2 to one of the exponents, as bf16."""
    e = torch.tensor([exponents[i % len(exponents)] for i in range(x.shape[-2])], dtype=torch.float64)
    return (x.double() * torch.exp2(e)[:, None]).to(torch.bfloat16)


# exponents of the rows' values and of K's scales: logits of up to some tens in the rows that count most
ENDS = [(list(range(100, 126)), -126), (list(range(-117, -103)), 104), (list(range(-133, -113)), 115)]


@pytest.mark.parametrize("rows,k_scale", ENDS)
@pytest.mark.parametrize("news,past,Hq,Hkv,d", CASES)
def test_queries_of_any_size(fa, news, past, Hq, Hkv, d, rows, k_scale):
    """Rows of the largest finite values down to subnormal ones, against K scales that make moderate logits of them."""
    lens = [a + b for a, b in zip(news, past)]
    c, table = make(d + k_scale % 97, lens, Hkv, d)
    c["k_scale"][:] = 2.0 ** k_scale
    q = spread_rows(bf16(np.random.default_rng(7), Hq, sum(news), d), rows)
    assert torch.isfinite(q).all()
    q = q.to(DEV)
    o, lse = run(fa, c, q, table, news, lens, scale=0.01)
    check(c, q, table, news, lens, True, 0.01, o, lse, rows=30)


def scaled(c, o, power):
    """The cache with V's scales, and O, times 2^power, in 64 bits."""
    return dict(c, v_scale=c["v_scale"].astype(np.float64) * 2.0 ** power), o.double() * 2.0 ** power


V_ENDS = [(-126, -117, 100), (-126, -60, 80), (108, 117, -100)]


@pytest.mark.parametrize("low,high,power", V_ENDS)
@pytest.mark.parametrize("news,past,Hq,Hkv,d", CASES)
def test_values_of_any_size(fa, news, past, Hq, Hkv, d, low, high, power):
    lens = [a + b for a, b in zip(news, past)]
    c, table = make(d + low % 97, lens, Hkv, d)
    rng = np.random.default_rng(3)
    c["v_scale"] = np.exp2(rng.integers(low, high + 1, c["v_scale"].shape)).astype(np.float32)
    q = bf16(np.random.default_rng(8), Hq, sum(news), d).to(DEV)
    o, lse = run(fa, c, q, table, news, lens)
    c, o = scaled(c, o, power)
    check(c, q, table, news, lens, True, d ** -0.5, o, lse, rows=30)


# lengths, Hq, Hkv, Nq, d of the single tokens' call: row groups that stay whole, that are split and joined, wide heads
SINGLE = [([300, 40], 8, 2, 1, 128), ([9000], 16, 2, 2, 64), ([5000, 700], 4, 4, 4, 256)]


@pytest.mark.parametrize("rows,k_scale", ENDS)
@pytest.mark.parametrize("lens,Hq,Hkv,Nq,d", SINGLE)
def test_single_tokens_queries_of_any_size(fa, lens, Hq, Hkv, Nq, d, rows, k_scale):
    c, table = make(d + k_scale % 97, lens, Hkv, d)
    c["k_scale"][:] = 2.0 ** k_scale
    x = bf16(np.random.default_rng(7), len(lens) * Hq * Nq, d)
    q = spread_rows(x, rows).view(len(lens), Hq, Nq, d)
    assert torch.isfinite(q).all()
    q = q.to(DEV)
    o, lse = fa.fwd_cache8(q, to_gpu(fa, c), ints(table), ints(lens), scale=0.01)
    fa.check_device_status()
    check_attention(c, q, table, lens, True, 0.01, o, lse, None)


@pytest.mark.parametrize("low,high,power", V_ENDS)
@pytest.mark.parametrize("lens,Hq,Hkv,Nq,d", SINGLE)
def test_single_tokens_values_of_any_size(fa, lens, Hq, Hkv, Nq, d, low, high, power):
    c, table = make(d + low % 97, lens, Hkv, d)
    rng = np.random.default_rng(3)
    c["v_scale"] = np.exp2(rng.integers(low, high + 1, c["v_scale"].shape)).astype(np.float32)
    q = bf16(np.random.default_rng(8), len(lens), Hq, Nq, d).to(DEV)
    o, lse = fa.fwd_cache8(q, to_gpu(fa, c), ints(table), ints(lens))
    fa.check_device_status()
    c, o = scaled(c, o, power)
    check_attention(c, q, table, lens, True, d ** -0.5, o, lse, None)
