"""What stands behind the cache's attention sees its results and may overwrite its cache: calls whose row groups are all
whole although their block table is wide (nothing is left for the second kernel), with a copy or an append directly behind
them, on a stream and in a graph, against the same calls with a synchronisation in between."""
import numpy as np
import pytest
import torch

from test_cache8_gpu import DEV, bf16, ints, make, to_gpu

pytestmark = pytest.mark.gpu

CASES = [
    # lens, Hq, Hkv, Nq, d, width of the table
    ([60], 32, 8, 1, 128, 16),               # eight row groups of one block each: as many parts
    ([60, 1, 64, 33], 8, 2, 1, 64, 40),
    ([64 * 12] * 38, 64, 8, 1, 128, 24),     # 304 row groups of equal length on 304 parts
    ([50, 3], 4, 2, 4, 256, 12),
]


@pytest.mark.parametrize("lens,Hq,Hkv,Nq,d,width", CASES)
@pytest.mark.parametrize("graph", [False, True])
def test_the_next_call_waits_for_the_attention(fa, lens, Hq, Hkv, Nq, d, width, graph):
    B = len(lens)
    c, table = make(sum(lens) + d, lens, Hkv, d, spare=width - max(-(-n // 64) for n in lens))
    rng = np.random.default_rng(d)
    q = bf16(rng, B, Hq, Nq, d).to(DEV)
    # the last token of each sequence again, so large that its block's scale grows and its codes are rounded anew
    x = (bf16(rng, Hkv, B, d) * 2.0 ** 14).to(DEV)
    tb, n, at, cu = ints(table), ints(lens), ints([m - 1 for m in lens]), ints(np.arange(B + 1))

    def run(g, between=lambda: None):
        o, lse = fa.fwd_cache8(q, g, tb, n)
        between()
        copies = o.clone(), lse.clone()
        between()
        o2, l2 = fa.fwd_cache8(q, g, tb, n)
        between()
        fa.cache8_append(g, x, x, cu, tb, at)
        between()
        return [o, lse, *copies, o2, l2, *fa.fwd_cache8(q, g, tb, n)]

    want_g = to_gpu(fa, c)
    want = run(want_g, torch.cuda.synchronize)
    torch.cuda.synchronize()
    fresh, g = to_gpu(fa, c), to_gpu(fa, c)
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = run(g)
    for _ in range(5):
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(g, name).copy_(getattr(fresh, name))
        if graph:
            for t in got:
                t.zero_()
            captured.replay()
        else:
            got = run(g)
        torch.cuda.synchronize()
        fa.check_device_status()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(g.k, want_g.k) and torch.equal(g.v, want_g.v)
    assert not torch.equal(want[4], want[6])            # the append did change what is there
