"""Attention over packed sequences on the GPU against the double-precision oracle, every element.

Bound, with A = scale max_j sum_c |q_c k_jc| of the row over its n keys: logits (d + 8) 2^-23 A (d exact products
added in fp32 by the tensor core, scale); P 2^-8 (bf16) and 2^-20 (ex2 and its argument's sum), as a ratio to l twice
the logits' error; sums n 2^-23 each for O and l; result 2^-8 |O|. P is taken relative to a reference that trails the
maximum by at most 2^8, and keeps bf16's 8 bits wherever it is."""
import numpy as np
import pytest
import torch

from oracle import cache8 as oc
from oracle import forward

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def inputs(seed, lens, Hq, Hkv, d, before=0, behind=0):
    rng = np.random.default_rng(seed)
    T = before + sum(lens) + behind
    q, k, v = (torch.from_numpy(rng.standard_normal((H, T, d)).astype(np.float32)).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    cu = before + np.concatenate([[0], np.cumsum(lens)])
    return q, k, v, cu


def gpu(x, layout):
    if layout == "token":                                       # [T, H, d] in memory
        return x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    if layout == "fused":                                       # heads of a wider projection, 8 values between rows
        w = torch.zeros(x.shape[1], x.shape[0], x.shape[2] + 8, dtype=x.dtype, device=DEV)
        w[..., : x.shape[2]] = x.transpose(0, 1).to(DEV)
        return w[..., : x.shape[2]].transpose(0, 1)
    return x.to(DEV)


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def check(q, k, v, cu, causal, o, lse):
    q, k, v, o, lse = (f64(x) for x in (q, k, v, o, lse))
    d, G = q.shape[2], q.shape[0] // k.shape[0]
    scale = d ** -0.5
    for a, e in zip(cu[:-1], cu[1:]):
        n = e - a
        if n == 0:
            continue
        ro, rl = (x[0] for x in forward(q[None, :, a:e], k[None, :, a:e], v[None, :, a:e], causal, scale))
        seen = np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)
        for h in range(q.shape[0]):
            kk, vv = k[h // G, a:e], v[h // G, a:e]
            p = np.where(seen, np.exp(scale * q[h, a:e] @ kk.T - rl[h][:, None]), 0)
            A = scale * np.where(seen, np.abs(q[h, a:e]) @ np.abs(kk).T, 0).max(1, keepdims=True)
            ds = (d + 8) * 2.0 ** -23 * A
            rel = 2.0 ** -8 + 2.0 ** -20 + 2 * ds + 2 * n * 2.0 ** -23
            tol = 2.0 ** -8 * np.abs(ro[h]) + rel * (p @ np.abs(vv)) + 1e-30
            err = np.abs(o[h, a:e] - ro[h])
            assert (err <= tol).all(), (a, h, float((err / tol).max()))
            ltol = ds[:, 0] + 2.0 ** -20 + n * 2.0 ** -23 + np.abs(rl[h]) * 2.0 ** -22
            assert (np.abs(lse[h, a:e] - rl[h]) <= ltol).all(), (a, h)


CASES = [
    # lens, Hq, Hkv, d, causal, layout
    ([1], 1, 1, 64, True, "head"),
    ([1, 2, 0, 127, 128, 129, 255, 256, 257], 2, 1, 128, True, "token"),
    ([300, 1000, 5], 4, 2, 128, False, "token"),
    ([0, 700, 0, 0, 513], 3, 3, 64, True, "head"),
    ([640, 130], 2, 2, 96, True, "fused"),
    ([200, 77], 4, 1, 8, True, "token"),
    ([200, 77], 4, 1, 112, False, "fused"),
    ([3] * 70 + [260], 2, 1, 64, True, "token"),                # more sequences than a warp has lanes
    ([1500, 1400, 300], 1, 1, 128, True, "head"),
    ([2] * 300 + [130, 0, 700] + [1, 0] * 100 + [290], 2, 1, 64, True, "token"),    # more than the look-up keeps in registers
    ([5, 0, 1] * 120 + [385], 3, 3, 128, False, "head"),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,causal,layout", CASES)
def test_every_row_and_nothing_else(fa, lens, Hq, Hkv, d, causal, layout):
    """Rows before the first and behind the last sequence hold NaN and infinities and are left as they were in o and lse."""
    q, k, v, cu = inputs(sum(lens) + d, lens, Hq, Hkv, d, before=3, behind=5)
    for x in (q, k, v):
        x[:, :3], x[:, -5:] = float("nan"), float("inf")
    o = gpu(torch.full_like(q, 7.0), layout)
    lse = torch.full((Hq, q.shape[1]), 7.0, device=DEV)
    got = fa.fwd_packed(*(gpu(x, layout) for x in (q, k, v)), torch.as_tensor(cu, dtype=torch.int32, device=DEV),
                        causal=causal, out=o, lse=lse)
    fa.check_device_status()
    assert got[0] is o and got[1] is lse
    assert (o[:, :3] == 7).all() and (o[:, -5:] == 7).all() and (lse[:, :3] == 7).all() and (lse[:, -5:] == 7).all()
    if layout == "fused":
        assert (o.transpose(0, 1).as_strided((o.shape[1], Hq, d + 8), (Hq * (d + 8), d + 8, 1))[..., d:] == 0).all()
    check(q, k, v, cu, causal, o, lse)


def test_a_neighbours_nan_and_infinities_do_not_reach_a_sequence(fa):
    lens = [100, 30, 200, 129]
    q, k, v, cu = inputs(1, lens, 4, 2, 128)
    put = [x.to(DEV) for x in (q, k, v)]
    cu_d = torch.as_tensor(cu, dtype=torch.int32, device=DEV)
    want, wl = fa.fwd_packed(*put, cu_d)
    for x in put:
        x[:, 100:130] = float("nan")
        x[:, 330:] = float("inf")
    got, gl = fa.fwd_packed(*put, cu_d)
    for a, e in ((0, 100), (130, 330)):
        assert torch.equal(got[:, a:e], want[:, a:e]) and torch.equal(gl[:, a:e], wl[:, a:e])


def test_one_sequence_gives_the_bits_of_fwd(fa):
    for n, d, causal in ((1000, 128, True), (1024, 64, False)):
        q, k, v, cu = inputs(2, [n], 4, 2, d)
        q, k, v = (x.to(DEV) for x in (q, k, v))
        o, lse = fa.fwd_packed(q, k, v, torch.as_tensor(cu, dtype=torch.int32, device=DEV), causal=causal)
        o2, l2 = fa.fwd(q[None], k[None], v[None], causal=causal)
        assert torch.equal(o, o2[0]) and torch.equal(lse, l2[0])


def test_lengths_outside_the_rules_stay_in_bounds(fa):
    """cu_seqlens past T and below 0 are taken within the rows there are; a sequence in order is right."""
    q, k, v, _ = inputs(3, [300], 2, 1, 64)
    g = [x.to(DEV) for x in (q, k, v)]
    o, lse = fa.fwd_packed(*g, torch.tensor([-50, 120, 10 ** 9], dtype=torch.int32, device=DEV))
    fa.check_device_status()
    check(q, k, v, [0, 120, 300], True, o, lse)


def test_no_tokens_no_sequences(fa):
    q = torch.zeros(4, 0, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = fa.fwd_packed(q, q, q, torch.zeros(3, dtype=torch.int32, device=DEV))
    assert o.shape == (4, 0, 64) and lse.shape == (4, 0)
    q = torch.ones(4, 10, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3)
    fa.fwd_packed(q, q, q, torch.zeros(1, dtype=torch.int32, device=DEV), out=out)
    fa.fwd_packed(q, q, q, torch.full((4,), 10, dtype=torch.int32, device=DEV), out=out)
    assert (out == 3).all()


def test_captured_call_follows_new_lengths(fa):
    q, k, v, cu = inputs(4, [200, 100, 84], 4, 2, 128)
    g = [x.to(DEV) for x in (q, k, v)]
    cu_d = torch.as_tensor(cu, dtype=torch.int32, device=DEV)
    fa.fwd_packed(*g, cu_d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.fwd_packed(*g, cu_d)
    for lens in ([200, 100, 84], [1, 382, 1], [0, 0, 384]):
        cu_d.copy_(torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = fa.fwd_packed(*g, cu_d)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_a_stalled_call_reports_and_the_next_one_works(fa, monkeypatch):
    q, k, v, cu = inputs(5, [130, 64], 1, 1, 64)
    g = [x.to(DEV) for x in (q, k, v)]
    cu_d = torch.as_tensor(cu, dtype=torch.int32, device=DEV)
    want = fa.fwd_packed(*g, cu_d)
    monkeypatch.setenv("FA_TEST_STALL", "1")
    fa.fwd_packed(*g, cu_d)
    with pytest.raises(fa.FAError) as e:
        fa.check_device_status()
    assert e.value.code == 5
    monkeypatch.delenv("FA_TEST_STALL")
    got = fa.fwd_packed(*g, cu_d)
    fa.check_device_status()
    assert torch.equal(got[0], want[0])


def test_prompts_into_the_cache_and_on(fa):
    """Packed prompts attended to, their K and V appended to a cache, and the next token's attention over it against
    the oracle on the cache's values; and the last prompt rows against the packed call's, within what e4m3 allows."""
    lens, Hq, Hkv, d = [150, 40, 65], 4, 2, 64
    q, k, v, cu = inputs(6, lens, Hq, Hkv, d)
    g = [gpu(x, "token") for x in (q, k, v)]
    cu_d = torch.as_tensor(cu, dtype=torch.int32, device=DEV)
    o, _ = fa.fwd_packed(*g, cu_d)
    check(q, k, v, cu, True, o, fa.fwd_packed(*g, cu_d)[1])
    cache = fa.new_cache8(9, Hkv, d)
    table = torch.tensor([[8, 1, 4], [0, 7, 2], [3, 6, 5]], dtype=torch.int32, device=DEV)
    fa.cache8_append(cache, g[1], g[2], cu_d, table, torch.zeros(3, dtype=torch.int32, device=DEV))
    last = q[:, cu[1:] - 1].transpose(0, 1)[:, :, None].contiguous()      # [3, Hq, 1, d]
    o2, l2 = fa.fwd_cache8(last.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    fa.check_device_status()
    c = {n: getattr(cache, n).cpu().numpy() for n in ("k", "v", "k_scale", "v_scale")}
    ro, rl, _ = oc.attend(c, f64(last), table.cpu().numpy(), lens, True, d ** -0.5)
    # P 2^-11, result 2^-8, of values whose weighted magnitudes are below max|V|
    assert np.abs(f64(o2) - ro).max() <= 2.0 ** -8 * np.abs(ro).max() + 2.0 ** -9 * f64(v).__abs__().max()
    assert np.abs(f64(l2) - rl).max() <= 1e-4
    # codes are off by at most 2^-4 of each value: O moves by 2^-4 of V and by the logits' 2^-4 A on both sides of the softmax
    qd, kd, vd = f64(q), f64(k), f64(v)
    for s, n in enumerate(lens):
        for h in range(Hq):
            i, a = cu[s + 1] - 1, cu[s]
            A = d ** -0.5 * (np.abs(qd[h, i]) @ np.abs(kd[h // 2, a:i + 1]).T).max() * 2.0 ** -4
            p = np.exp(d ** -0.5 * kd[h // 2, a:i + 1] @ qd[h, i])
            p /= p.sum()
            bound = (2.0 ** -4 + 2.0 ** -7 + np.expm1(2 * A)) * (p @ np.abs(vd[h // 2, a:i + 1])) + 2.0 ** -7
            assert (np.abs(f64(o2)[s, h, 0] - f64(o)[h, i]) <= bound).all()
