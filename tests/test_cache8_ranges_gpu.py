"""Attention over the 8-bit cache at the ends of what bf16 queries and the cache's scales can be, on the GPU against 64 bits.

The bounds are those of test_cache8_chunk_gpu.check and test_cache8_gpu.check_attention, which are relative to the row's own
values but for 1e-30. O is linear in V's scales, so results near that are compared times a power of two, taken in 64 bits:
V's scales and O both, which changes no relative bound. A bf16 below 2^-126 is off by at most 2^-134; with V scales of 2^-126
the bound is 2^-11 sum p |code| 2^-126, which is more as soon as the mean magnitude of the codes is 2^3, and here it is about 38.
"""
import numpy as np
import pytest
import torch

from oracle import cache8 as oc
from test_cache8_chunk_gpu import check, run
from test_cache8_gpu import DEV, bf16, check_attention, f64, ints, make, to_gpu

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


@pytest.mark.parametrize("d", [64, 256])
def test_small_columns_beside_a_large_one(fa, d):
    """A row's columns of 2^-6 to 2^-13 of its largest count to the bit, smaller ones to 2^-21 of it. K is 0 where Q is large, so
    that the logits are the small columns' alone: off by (2 d + 8) 2^-23 of sum |q k| over those (two terms of d products
    added in fp32) and by 2^-21 of the row's largest times sum |k| over the ones below 2^-13. (A second
    term that is off by 2^-17 of the largest in each column, as in e4m3, fails at d 64.)"""
    n, scale = 7, d ** -0.5
    c, table = make(d, [n], 1, d)
    c["k"][table[0, 0], :, :n, 0] = 0
    e = np.concatenate([[0], -(6.0 + 12.0 * np.arange(d - 1) / d)])
    rng = np.random.default_rng(5)
    for low in (-13, -18):
        x = np.exp2(np.maximum(e, low)) * rng.uniform(1, 2, (2, n, d)) * rng.choice([-1, 1], (2, n, d))
        x[..., 0] = 1.5
        q = torch.from_numpy(x * 1024).to(torch.bfloat16).to(DEV)
        o, lse = run(fa, c, q, table, [n], [n], causal=False, scale=scale)
        K, V, _ = oc.gather(c, table[0], 0, n)
        qd = f64(q)
        for j in range(2):
            for r in range(n):
                y, top = qd[j, r], np.abs(qd[j, r]).max()
                s = scale * (K @ y)
                rl = s.max() + np.log(np.exp(s - s.max()).sum())
                p = np.exp(s - rl)
                ds = (2 * d + 8) * 2.0 ** -23 * scale * (np.abs(K) @ np.abs(y)).max() + \
                    2.0 ** -21 * top * scale * np.abs(K)[:, np.abs(y) < 2.0 ** -13 * top].sum(1).max()
                assert abs(f64(lse)[j, r] - rl) <= ds + 2.0 ** -20 + n * 2.0 ** -23 + abs(rl) * 2.0 ** -22
                rel = 2.0 ** -11 + 2.0 ** -20 + 2 * ds + 2 * n * 2.0 ** -23
                tol = 2.0 ** -8 * np.abs(p @ V) + rel * (p @ np.abs(V)) + 2.0 ** -31 * np.abs(V).max(0)
                assert (np.abs(f64(o)[j, r] - p @ V) <= tol).all()
