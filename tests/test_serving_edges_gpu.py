"""The serving operators at the ends of what their documentation allows, against the double-precision oracle."""
import numpy as np
import pytest
import torch

from oracle import cache8 as oc
from oracle.fp8 import e4m3_decode
from test_cache8_gpu import DEV, bf16, f64, ints, make, to_gpu
from test_packed_gpu import inputs

pytestmark = pytest.mark.gpu


def same_cache(g, want):
    for n, x in want.items():
        assert np.array_equal(getattr(g, n).cpu().numpy(), x, equal_nan=x.dtype == np.float32), n


def test_evict_writes_no_block_past_those_it_needs(fa):
    """A table of destinations of more than 2^26 entries, where 64 times an entry's number is no int: all but the first two
    name a block that holds something else."""
    lens, keep, recent = [300], 100, 10
    c, table = make(61, lens, 2, 16, spare=3)
    to, table = table[:, -3:].copy(), table[:, :-3].copy()
    g = to_gpu(fa, c)
    wide = torch.full((1, 2 ** 26 + 70), int(to[0, 2]), dtype=torch.int32, device=DEV)
    wide[0, :2] = ints(to[0, :2])
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), keep, recent, wide)
    fa.check_device_status()
    want, wn, wk = oc.evict(c, table, lens, keep, recent, to)
    assert np.array_equal(new.cpu().numpy(), wn) and np.array_equal(kept.cpu().numpy(), wk)
    same_cache(g, want)


def test_evict_with_the_largest_keep(fa):
    """keep = 2^31 - 1: everything stays and -1 fills the rest of the positions."""
    lens, keep = [70], 2 ** 31 - 1
    free, _ = torch.cuda.mem_get_info()
    assert free > 20 << 30
    c, table = make(62, lens, 1, 16, spare=2)
    to, table = table[:, -2:].copy(), table[:, :-2].copy()
    g = to_gpu(fa, c)
    wide = torch.full((1, 2 ** 25), -1, dtype=torch.int32, device=DEV)
    wide[0, :2] = ints(to[0])
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), keep, 0, wide)
    fa.check_device_status()
    want, wn, _ = oc.evict(c, table, lens, 128, 0, to)
    assert np.array_equal(new.cpu().numpy(), wn)
    assert torch.equal(kept[0, 0, :70].cpu(), torch.arange(70, dtype=torch.int32)) and bool((kept[0, 0, 70:] == -1).all())
    same_cache(g, want)


@pytest.mark.parametrize("width", [2, 12])             # one CTA per row group; groups cut between CTAs
def test_a_row_that_sees_no_key_is_zero_whatever_v_holds(fa, width):
    """More queries than keys, over a NaN among V and one among K."""
    lens, Nq, d = [100], 128, 64
    c, table = make(63, lens, 1, d, spare=width - 2)
    c["v"][table[0, 1], 0, 35, 3] = c["k"][table[0, 0], 0, 7, 5] = 0x7F
    q = bf16(np.random.default_rng(64), 1, 1, Nq, d).to(DEV)
    o, lse = fa.fwd_cache8(q, to_gpu(fa, c), ints(table), ints(lens))
    fa.check_device_status()
    blind = Nq - lens[0]                                # row i sees the keys up to i - 28
    assert bool((o[0, 0, :blind] == 0).all()) and bool(torch.isneginf(lse[0, 0, :blind]).all())
    assert bool(torch.isnan(o[0, 0, -1]).all())


@pytest.mark.parametrize("width", [2, 12])
def test_a_nan_under_a_scale_of_zero_is_a_nan(fa, width):
    c, table = make(67, [100], 1, 64, spare=width - 2)
    c["v_scale"][table[0, :2]] = 0.0
    c["v"][table[0, 1], 0, 20, 3] = 0x7F
    q = bf16(np.random.default_rng(68), 1, 2, 1, 64).to(DEV)
    o, lse = fa.fwd_cache8(q, to_gpu(fa, c), ints(table), ints([100]))
    assert bool(torch.isnan(o[..., 3]).all()) and bool((o[..., :3] == 0).all()) and bool((o[..., 4:] == 0).all())
    assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("new,past,Hkv,d", [([70, 1, 5, 64], [30, 63, 0, 10], 2, 64), ([40, 3], [0, 100], 3, 256)])
def test_append_under_scales_of_any_value(fa, new, past, Hkv, d):
    c, table = make(sum(new) + d, [a + b for a, b in zip(new, past)], Hkv, d, spread=2, po2=False)
    rng = np.random.default_rng(d)
    k, v = (torch.from_numpy((rng.standard_normal((Hkv, sum(new), d)) * np.exp2(rng.integers(-6, 6, (Hkv, sum(new), 1)))).astype(np.float32))
            .to(torch.bfloat16) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(new)])
    g = to_gpu(fa, c)
    fa.cache8_append(g, k.to(DEV), v.to(DEV), ints(cu), ints(table), ints(past))
    fa.check_device_status()
    same_cache(g, oc.append(c, f64(k), f64(v), cu, past, table))


def test_append_divides_by_a_held_scale(fa):
    """Quotients next to the border of two codes, where x times the rounded 1 / s falls on the other side; and scales so
    small that 1 / s is infinite."""
    pairs = [("0x1.733332p+0", 145), ("0x1.77bdf0p+0", 182), ("0x1.5b6db6p+0", 228), ("0x1.d642cap+0", 169),
             ("0x1.dffffep+0", 255), ("0x1.696968p+0", 192), ("0x1.ba6f4ep+0", 159), ("0x1.0p-140", 0), ("0x1.6p-130", 0)]
    B, d = len(pairs), 16
    c, table = make(65, [2] * B, 1, d, spare=0)
    k = torch.zeros(1, B, d, dtype=torch.bfloat16)
    for b, (s, x) in enumerate(pairs):
        c["k_scale"][table[b, 0], 0] = c["v_scale"][table[b, 0], 0] = float.fromhex(s)
        c["k"][table[b, 0], 0, :2], c["v"][table[b, 0], 0, :2] = 0x38, 0xB8
        k[0, b, :9] = x
    g = to_gpu(fa, c)
    fa.cache8_append(g, k.to(DEV), -k.to(DEV), ints(np.arange(B + 1)), ints(table), ints([1] * B))
    fa.check_device_status()
    want = oc.append(c, f64(k), -f64(k), np.arange(B + 1), [1] * B, table)
    for n in ("k_scale", "v_scale", "weight"):
        assert np.array_equal(getattr(g, n).cpu().numpy(), want[n], equal_nan=True), n
    for n in ("k", "v"):                                # (the sign of a zero says nothing)
        got, ref = (e4m3_decode(x[n] if isinstance(x, dict) else getattr(x, n).cpu().numpy()) for x in (g, want))
        assert np.array_equal(got, ref, equal_nan=True), n


@pytest.mark.parametrize("lens,keep,recent,Hkv,d", [([517, 192], 130, 32, 3, 64), ([400], 200, 0, 1, 256)])
def test_evict_from_blocks_with_scales_of_any_value(fa, lens, keep, recent, Hkv, d):
    room = -(-keep // 64)
    c, table = make(sum(lens) + keep, lens, Hkv, d, spare=room, po2=False)
    to, table = table[:, -room:].copy(), table[:, :-room].copy()
    g = to_gpu(fa, c)
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), keep, recent, ints(to))
    fa.check_device_status()
    want, wn, wk = oc.evict(c, table, lens, keep, recent, to)
    assert np.array_equal(new.cpu().numpy(), wn) and np.array_equal(kept.cpu().numpy(), wk)
    same_cache(g, want)


def border_scales():
    """(code, scale) whose exact product is above 448 and rounds to 448."""
    for code in range(1, 0x7F):
        x = float(e4m3_decode(np.uint8(code)))
        s = np.float32(448.0 / x)
        if x * float(s) > 448.0 and np.float32(x * float(s)) == np.float32(448.0):
            yield code, s


def test_evict_takes_the_largest_value_as_it_is(fa):
    """The scale is the smallest power of two with max|x| <= 448 s for x = code * scale, not for x rounded; and values of
    scales below 2^-126 are not rounded to that grid first."""
    cases = list(border_scales())
    assert len(cases) >= 8
    # the largest value has a scale of 2^-126 of its own; every code under a subnormal scale beside it
    cases += [(0x7E, np.float32(float.fromhex("0x1.8p-127"))), (0x7E, np.float32(float.fromhex("0x1.2345678p-128")))]
    B, d = len(cases), 128
    lens = [3] * B
    c, table = make(66, lens, 1, d, spare=1)
    to, table = table[:, -1:].copy(), table[:, :-1].copy()
    for b, (code, s) in enumerate(cases):
        c["k_scale"][table[b, 0], 0] = c["v_scale"][table[b, 0], 0] = s
        few = np.arange(min(code, d - 1) + 1, dtype=np.uint8)
        for x in ("k", "v"):
            c[x][table[b, 0], 0, :3] = 0
            c[x][table[b, 0], 0, 1, : len(few)] = few[::-1]
    g = to_gpu(fa, c)
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), 2, 0, ints(to))
    fa.check_device_status()
    c2 = {n: x.copy() for n, x in c.items()}
    want, wn, wk = oc.evict(c2, table, lens, 2, 0, to)
    assert np.array_equal(kept.cpu().numpy(), wk)
    same_cache(g, want)


def test_evict_of_zeros_under_a_huge_scale(fa):
    """The ratio of the scales is past all floats, and the codes it multiplies are 0."""
    lens, d = [66], 32
    c, table = make(69, lens, 1, d, spare=1)
    to, table = table[:, -1:].copy(), table[:, :-1].copy()
    for x in ("k", "v"):
        c[x][table[0, 0]] = 0
        c[x + "_scale"][table[0]] = np.array([[1.5 * 2.0 ** 126], [1.25 * 2.0 ** -126]], np.float32)
    c["weight"][table[0, 0]] = 1.0
    g = to_gpu(fa, c)
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), 40, 2, ints(to))
    want, wn, wk = oc.evict(c, table, lens, 40, 2, to)
    assert np.array_equal(kept.cpu().numpy(), wk)
    same_cache(g, want)


def test_packed_rows_of_nan(fa):
    """A NaN in a row of Q, or in a key that a row sees, is that row's O and LSE, and no other row's."""
    q, k, v, cu = inputs(7, [200, 150], 4, 2, 64)
    cu_d = ints(cu)
    g = [x.to(DEV) for x in (q, k, v)]
    want, wl = fa.fwd_packed(*g, cu_d)
    g[0][1, 40, 3] = float("nan")
    g[1][1, 320, 5] = float("nan")                      # the second sequence's row 120, of heads 2 and 3
    got, gl = fa.fwd_packed(*g, cu_d)
    fa.check_device_status()
    hit = torch.zeros(4, 350, dtype=torch.bool, device=DEV)
    hit[1, 40] = True
    hit[2:, 320:] = True
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(gl[~hit], wl[~hit])
    assert bool(torch.isnan(got[hit]).all()) and bool(torch.isnan(gl[hit]).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_packed_values_that_are_no_numbers_reach_their_128_rows_at_most(fa, bad):
    """V of row 150: rows that see it, and O of those before it in the same 128 rows of its sequence, whose P is 0; no LSE."""
    lens, at = [70, 300], 150
    q, k, v, cu = inputs(8, lens, 4, 2, 128)
    g = [x.to(DEV) for x in (q, k, v)]
    want, wl = fa.fwd_packed(*g, ints(cu))
    g[2][1, 70 + at, 9] = bad
    got, gl = fa.fwd_packed(*g, ints(cu))
    fa.check_device_status()
    assert torch.equal(gl, wl)
    assert torch.equal(got[:2], want[:2]) and torch.equal(got[2:, : 70 + 128], want[2:, : 70 + 128])
    other = torch.arange(128, device=DEV) != 9
    assert torch.equal(got[..., other], want[..., other])
    assert not torch.isfinite(got[2:, 70 + at:, 9]).any()


def test_packed_hundreds_of_thousands_of_sequences(fa):
    """2^18 sequences of one row, of three, or of none: O is V where a row sees itself alone. The look for an item goes on
    where the one before ended: a time that grows with the square of the sequences would be ten times what is allowed here."""
    S, Hq, d = 2 ** 18, 4, 64
    lens = np.array([1, 3, 0, 1])[np.random.default_rng(70).integers(0, 4, S)]
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    T = int(lens.sum())
    gen = torch.Generator(device=DEV).manual_seed(71)
    q, k, v = (torch.randn(H, T, d, device=DEV, generator=gen).to(torch.bfloat16) for H in (Hq, 2, 2))
    fa.fwd_packed(q[:, :9], k[:, :9], v[:, :9], ints([0, 9]))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    o, lse = fa.fwd_packed(q, k, v, cu)
    end.record()
    torch.cuda.synchronize()
    fa.check_device_status()
    assert start.elapsed_time(end) < 1500
    first = torch.from_numpy(np.cumsum(lens) - lens).to(DEV)[torch.from_numpy(lens > 0).to(DEV)]
    assert torch.equal(o[:, first], v.repeat_interleave(2, 0)[:, first])
    three = (torch.from_numpy(np.cumsum(lens) - lens).to(DEV)[torch.from_numpy(lens == 3).to(DEV)])[:10000, None] + torch.arange(3, device=DEV)
    qs, ks, vs = (x.double()[:, three] for x in (q, k.repeat_interleave(2, 0), v.repeat_interleave(2, 0)))       # [Hq, n, 3, d]
    s = (qs[..., :, None, :] * ks[..., None, :, :]).sum(-1) * d ** -0.5
    s = s.masked_fill(torch.ones(3, 3, device=DEV, dtype=torch.bool).triu(1), float("-inf"))
    p = s.softmax(-1)
    want, size = ((p[..., None] * x[..., None, :, :]).sum(-2) for x in (vs, vs.abs()))
    # logits (d + 8) 2^-23 A, P 2^-8 and 2^-20, sums 3 2^-23 twice, O 2^-8
    A = (qs[..., :, None, :] * ks[..., None, :, :]).abs().sum(-1).amax(-1, keepdim=True) * d ** -0.5
    rel = 2.0 ** -8 + 2.0 ** -20 + 2 * (d + 8) * 2.0 ** -23 * A + 6 * 2.0 ** -23
    assert bool(((o.double()[:, three] - want).abs() <= 2.0 ** -8 * want.abs() + rel * size + 1e-30).all())
    ltol = (d + 8) * 2.0 ** -23 * A[..., 0] + 2.0 ** -20 + 3 * 2.0 ** -23 + s.logsumexp(-1).abs() * 2.0 ** -22
    assert bool(((lse.double()[:, three] - s.logsumexp(-1)).abs() <= ltol).all())
