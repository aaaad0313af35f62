"""Rotary positions on the GPU against the double-precision oracle (oracle/rope.py), and the cache's append with the
rotation on the way.

Bound of a rotated value a cos t - b sin t in fp32: the angle is within 2^-32 of a turn, 2^-24 of itself (its conversion to
fp32), 2^-24 (a product) and 2^-25 (2 pi / 2^32), each times at most pi / 4: 2^-23 in all. The sums of sine and cosine end
below 2^-27 and round four times, below 2^-24 each step with the last alone at full weight: 2^-23. With the products' and the sum's
roundings (2^-24 (|a| + |b|) and 2^-24 of the result) that is at most 2^-21 (|a| + |b|). bf16 results: 2^-8 of the value on top.
"""
import numpy as np
import pytest
import torch

from oracle import cache8 as oc
from oracle import rope as orope
from oracle.fp8 import e4m3_decode

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FP32 = 2.0 ** -21


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def freqs(n):
    return [1e4 ** (-i / n) for i in range(n)]


def magnitude(x, n, interleaved):
    """|a| + |b| of the pair that each column belongs to."""
    m = np.abs(np.asarray(x, np.float64)).copy()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    s = m[..., a] + m[..., b]
    m[..., a], m[..., b] = s, s
    return m


def check(got, x, f, axis, pos, interleaved, inverse, dtype):
    want = orope.rotate(f64(x), f, axis, pos, interleaved, inverse)
    tol = FP32 * magnitude(f64(x), len(f), interleaved) + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), float((err / (tol + 1e-300)).max())
    assert (f64(got)[..., 2 * len(f):] == f64(x)[..., 2 * len(f):]).all()


# B (0: no batch dimension), T, Hq, Hkv, d, pairs, axes, interleaved, dtype
CASES = [
    (0, 1, 1, 0, 8, 4, 1, False, torch.bfloat16),
    (0, 1, 64, 8, 128, 64, 1, False, torch.bfloat16),
    (0, 5, 3, 1, 72, 36, 2, False, torch.bfloat16),                # pairs no multiple of 8
    (0, 5, 3, 1, 72, 36, 2, True, torch.bfloat16),
    (0, 33, 7, 7, 64, 32, 3, True, torch.bfloat16),
    (2, 130, 4, 2, 256, 128, 1, False, torch.bfloat16),
    (3, 17, 5, 2, 96, 20, 3, False, torch.bfloat16),               # less than half of the columns
    (3, 17, 5, 2, 96, 20, 3, True, torch.float32),
    (2, 700, 4, 4, 80, 40, 2, False, torch.float32),
    (0, 2500, 12, 4, 128, 64, 3, True, torch.bfloat16),            # several tokens per CTA
    (0, 2500, 2, 1, 16, 4, 1, False, torch.float32),
    (1, 2048, 16, 0, 64, 32, 1, False, torch.bfloat16),            # no K
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,pairs,axes,interleaved,dtype", CASES)
def test_rope(fa, B, T, Hq, Hkv, d, pairs, axes, interleaved, dtype, inverse):
    rng = np.random.default_rng(T + d + Hq)
    gen = torch.Generator().manual_seed(T + d)
    f, axis = freqs(pairs), [int(a) for a in rng.integers(0, axes, pairs)]
    batch = (B,) if B else ()
    pos = rng.integers(-(1 << 31), 1 << 31, (axes, *batch, T)) if T % 2 else rng.integers(0, 1 << 20, (axes, *batch, T))
    plan = fa.new_rope(f, axis, interleaved)
    # a projection's layout: [B, T, H, d] in memory
    q = torch.randn(*batch, T, Hq, d, generator=gen).to(dtype).to(DEV).transpose(-3, -2)
    k = torch.randn(*batch, T, Hkv, d, generator=gen).to(dtype).to(DEV).transpose(-3, -2) if Hkv else None
    gq, gk = fa.rope(q, k, plan, ints(pos), inverse=inverse)
    fa.check_device_status()
    check(gq, q, f, axis, pos, interleaved, inverse, dtype)
    assert gq.stride() == q.stride() or T == 1 or Hq == 1
    if Hkv:
        check(gk, k, f, axis, pos, interleaved, inverse, dtype)
    # to [B, H, T, d], and in place: the same bits
    dense = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    oq, ok = fa.rope(q, None, plan, ints(pos), inverse=inverse, q_out=dense)
    assert oq is dense and ok is None and torch.equal(dense, gq)
    mine = q.clone()
    fa.rope(mine, None, plan, ints(pos), inverse=inverse, q_out=mine)
    assert torch.equal(mine, gq)


def test_positions_layouts(fa):
    """[T], [axes, T] and [axes, B, T] say the same where they can; strided positions and heads cut out of a wider
    projection; axis numbers outside the positions are taken within."""
    gen = torch.Generator().manual_seed(3)
    q = torch.randn(2, 4, 50, 64, generator=gen).to(torch.bfloat16).to(DEV)
    plan = fa.new_rope(freqs(32))
    pos = torch.arange(50, dtype=torch.int32, device=DEV) * 3 + 1000
    a, _ = fa.rope(q, None, plan, pos)
    for other in (pos[None], pos[None].expand(2, 50), pos[None, None].expand(1, 2, 50),
                  torch.stack([pos, pos + 1], 0)[:1], torch.stack([pos, pos, pos], 0).repeat(1, 2)[:, :50][1:2]):
        assert torch.equal(fa.rope(q, None, plan, other)[0], a)
    two = torch.stack([pos, pos + 9])                                # [B, T], one axis
    b, _ = fa.rope(q, None, plan, two)
    assert torch.equal(b[0], a[0]) and torch.equal(b[1], fa.rope(q[1], None, plan, pos + 9)[0])
    wide = torch.randn(50, 12, 64, generator=gen).to(torch.bfloat16).to(DEV)       # [T, q, k, v heads, d]
    x, y = wide[:, :8].transpose(0, 1), wide[:, 8:10].transpose(0, 1)
    gx, gy = fa.rope(x, y, plan, pos)
    check(gx, x, freqs(32), [0] * 32, pos[None].cpu().numpy(), False, False, torch.bfloat16)
    check(gy, y, freqs(32), [0] * 32, pos[None].cpu().numpy(), False, False, torch.bfloat16)
    odd = plan._replace(axis=ints([-5, 99] * 16))
    lo_hi = torch.stack([pos, pos + 5])
    c, _ = fa.rope(q, None, odd, lo_hi)
    assert torch.equal(c, fa.rope(q, None, plan._replace(axis=ints([0, 1] * 16)), lo_hi)[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(fa, interleaved):
    """<d y, R x> has the gradient R^T d y, against differences of the forward (linear, so exact but for rounding)."""
    gen = torch.Generator().manual_seed(5)
    T, H, d = 6, 2, 24
    plan = fa.new_rope(freqs(8), [0, 1] * 4, interleaved)
    pos = ints([[5, -3, 100, 7, 0, 2 ** 30], [1, 2, 3, 4, 5, 6]])
    x, dy = (torch.randn(H, T, d, generator=gen).to(DEV) for _ in range(2))
    dx, _ = fa.rope(dy, None, plan, pos, inverse=True)
    for i in range(0, H * T * d, 7):
        e = torch.zeros(H * T * d, device=DEV)
        e[i] = 1.0
        up, _ = fa.rope(e.view(H, T, d), None, plan, pos)
        assert abs(float((up.double() * dy.double()).sum() - dx.flatten()[i].double())) <= 2 * FP32 * 2 * float(dy.abs().max())
    back, _ = fa.rope(fa.rope(x, None, plan, pos)[0], None, plan, pos, inverse=True)
    assert float((back - x).abs().max()) <= 4 * FP32 * 2 * float(x.abs().max())


def test_infinities_and_nan_stay_in_their_pairs(fa):
    q = torch.ones(1, 3, 32, device=DEV)
    q[0, 1, 3], q[0, 2, 30] = float("inf"), float("nan")
    plan = fa.new_rope(freqs(8))
    y, _ = fa.rope(q, None, plan, ints([[1, 2, 3]]))
    bad = ~torch.isfinite(y)
    assert bad[0, 1].nonzero().flatten().tolist() == [3, 11] and bad[0, 2].nonzero().flatten().tolist() == [30]
    assert not bad[0, 0].any()


def test_streams_and_graph(fa):
    gen = torch.Generator().manual_seed(9)
    q = torch.randn(64, 8, 128, generator=gen).to(torch.bfloat16).to(DEV).transpose(0, 1)
    plan, pos = fa.new_rope(freqs(64)), torch.arange(64, dtype=torch.int32, device=DEV)
    want, _ = fa.rope(q, None, plan, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q)
    with torch.cuda.stream(s):
        fa.rope(q, None, plan, pos, q_out=out)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        fa.rope(q, None, plan, pos, q_out=out)
    pos += 100
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fa.rope(q, None, plan, pos)[0])


# ------------------------------------------------------------------ the append
def empty_cache(fa, rng, P, Hkv, d):
    """A pool whose slots hold NaN codes and whose scales are powers of two."""
    c = {x: np.full((P, Hkv, 64, d), 0x7F, np.uint8) for x in ("k", "v")}
    c.update({x: np.exp2(rng.integers(-9, -5, (P, Hkv))).astype(np.float32) for x in ("k_scale", "v_scale")})
    c["weight"] = np.full((P, Hkv, 64), 3.0, np.float32)
    return c


def check_append(c, got, k, v, f, axis, pos, interleaved, cu, start, table):
    """V, weights and untouched slots to the bit. K: each code a nearest one to the rotated value, but for values within
    their bound of the middle between two codes, and the scale the smallest that fits, but for an amax within its bound
    of a power's limit."""
    rk = orope.rotate(f64(k), f, axis, pos, interleaved)
    err = FP32 * magnitude(f64(k), len(f), interleaved)
    want = oc.append(c, rk, f64(v), cu, start, table)
    for name in ("v", "v_scale", "weight"):
        assert (f64(getattr(got, name)) == want[name].astype(np.float64)).all() if name != "v" else \
            (got.v.cpu().numpy() == want["v"]).all(), name
    gk, gs = got.k.cpu().numpy(), got.k_scale.cpu().numpy()
    same = gk == want["k"]
    assert (gs == want["k_scale"]).all(), np.abs(gs / want["k_scale"]).max()
    new = np.zeros(gk.shape, bool)
    flips = 0
    for b in range(len(start)):
        for i, tok in enumerate(range(cu[b], cu[b + 1])):
            at = start[b] + i
            if at >= table.shape[1] * 64 or not 0 <= table[b, at // 64] < gk.shape[0]:
                continue
            page, slot = table[b, at // 64], at % 64
            new[page, :, slot] = True
            if same[page, :, slot].all():
                continue
            s = gs[page].astype(np.float64)[:, None]
            off = np.abs(e4m3_decode(gk[page, :, slot]) * s - rk[:, tok])
            best = np.abs(e4m3_decode(want["k"][page, :, slot]) * s - rk[:, tok])
            assert (off <= best + 2 * err[:, tok]).all()
            flips += int((~same[page, :, slot]).sum())
    assert (same | new).all()
    return flips


# (held, new) per sequence, Hkv, d, pairs, axes, interleaved, own positions
APPENDS = [
    ([(0, 1)], 1, 16, 8, 1, False, False),
    ([(5, 1), (64, 1), (0, 1), (127, 1)], 2, 128, 64, 1, False, True),
    ([(0, 200), (63, 2), (10, 54), (10, 55)], 3, 64, 32, 3, True, True),
    ([(30, 300)], 5, 80, 20, 2, False, True),                       # pairs no multiple of 8, columns that stay
    ([(30, 300), (0, 0), (1, 64)], 2, 112, 56, 1, False, False),
    ([(7, 129)], 2, 256, 128, 3, False, True),
    ([(7, 129), (60, 9)], 9, 192, 96, 1, True, False),              # more heads than one CTA takes
    ([(3, 4000), (100, 2000)], 8, 48, 24, 1, False, True),          # several heads per CTA
]


@pytest.mark.parametrize("seqs,Hkv,d,pairs,axes,interleaved,own_positions", APPENDS)
def test_append(fa, seqs, Hkv, d, pairs, axes, interleaved, own_positions):
    rng = np.random.default_rng(sum(n for _, n in seqs) + d)
    gen = torch.Generator().manual_seed(d)
    width = max(-(-(a + n) // 64) for a, n in seqs) + 1
    P = len(seqs) * width + 2
    table = rng.permutation(P)[: len(seqs) * width].reshape(len(seqs), width).astype(np.int32)
    c = empty_cache(fa, rng, P, Hkv, d)
    for b, (held, _) in enumerate(seqs):
        for at in range(held):
            for x in ("k", "v"):
                c[x][table[b, at // 64], :, at % 64] = (torch.randn(Hkv, d, generator=gen) * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])])
    T = int(cu[-1])
    start = np.array([a for a, _ in seqs])
    k, v = (torch.randn(T, Hkv, d, generator=gen).mul(3).to(torch.bfloat16).to(DEV).transpose(0, 1) for _ in range(2))
    f, axis = freqs(pairs), [int(a) for a in rng.integers(0, axes, pairs)]
    own = np.concatenate([np.arange(a, a + n) for a, n in seqs])
    pos = rng.integers(-1000, 1 << 20, (axes, T)) if own_positions else np.broadcast_to(own, (axes, T))
    g = fa.Cache8(**{n: torch.from_numpy(x.copy()).to(DEV) for n, x in c.items()})
    plan = fa.new_rope(f, axis, interleaved)
    fa.cache8_append(g, k, v, ints(cu), ints(table), ints(start), rope=plan, positions=ints(pos) if own_positions else None)
    fa.check_device_status()
    flips = check_append(c, g, k, v, f, axis, pos, interleaved, cu, start, table)
    assert flips <= 2 + 1e-5 * T * Hkv * d
    # the same call again gives the same bits, and a growing scale re-encodes what is there
    if min(a for a, _ in seqs) > 0:
        fa.cache8_append(g, k * 64, v, ints(cu), ints(table), ints(start), rope=plan, positions=ints(pos) if own_positions else None)
        c2 = oc.append(c, orope.rotate(f64(k), f, axis, pos, interleaved), f64(v), cu, start, table)
        check_append(c2, g, k * 64, v, f, axis, pos, interleaved, cu, start, table)


def test_append_infinities_nan_and_absent_blocks(fa):
    """An infinity is held at 448 s and takes no part in s, a NaN stays; pages outside the pool and positions behind the
    table are not written; scales that are no powers of two are divided by."""
    rng = np.random.default_rng(2)
    c = empty_cache(fa, rng, 4, 1, 32)
    c["k_scale"][:] = 0.75
    for p in range(4):
        c["k"][p, :, :5] = 0x38                                      # 1.0
    table = np.array([[0, 9, 2], [-1, 1, 3]], np.int32)
    k = torch.randn(1, 300, 32, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    k[0, 3, 1], k[0, 4, 30] = float("inf"), float("nan")
    k = k.to(DEV)
    cu, start = np.array([0, 150, 300]), np.array([5, 70])
    pos = np.zeros((1, 300), int)                                    # angle 0: the values as they are
    g = fa.Cache8(**{n: torch.from_numpy(x.copy()).to(DEV) for n, x in c.items()})
    plan = fa.new_rope(freqs(8))
    fa.cache8_append(g, k, k, ints(cu), ints(table), ints(start), rope=plan, positions=ints(pos))
    plain = fa.Cache8(**{n: torch.from_numpy(x.copy()).to(DEV) for n, x in c.items()})
    fa.cache8_append(plain, k, k, ints(cu), ints(table), ints(start))
    fa.check_device_status()
    # (inf cos 0 - y sin 0 is inf, inf sin 0 is NaN: the infinity's pair is compared apart)
    a, b = g.k.cpu(), plain.k.cpu()
    a[0, 0, 8, 9] = b[0, 0, 8, 9]
    a[0, 0, 8, 1] = b[0, 0, 8, 1]
    assert torch.equal(a, b) and torch.equal(g.k_scale, plain.k_scale) and torch.equal(g.v, plain.v)
    assert g.k[0, 0, 8, 1].item() == 0x7E and (g.k[0, 0, 8, 9].item() & 0x7F) == 0x7F and (g.k[0, 0, 9, 30].item() & 0x7F) == 0x7F


def test_append_without_positions_in_a_graph(fa):
    """None: each token's own position, from `start` as it is at the replay."""
    plan = fa.new_rope(freqs(32))
    gen = torch.Generator().manual_seed(4)
    k = torch.randn(2, 3, 64, generator=gen).to(torch.bfloat16).to(DEV)
    cu, table = ints([0, 1, 2, 3]), ints([[0, 1], [2, 3], [4, 5]])
    start = ints([0, 0, 0])
    a, b = fa.new_cache8(6, 2, 64), fa.new_cache8(6, 2, 64)
    fa.cache8_append(a, k, k, cu, table, start, rope=plan)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.cache8_append(a, k, k, cu, table, start, rope=plan)
    start.copy_(ints([5, 64, 70]))
    g.replay()
    fa.cache8_append(b, k, k, cu, table, ints([0, 0, 0]), rope=plan)
    fa.cache8_append(b, k, k, cu, table, start, rope=plan, positions=start)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))
