"""Host checks of the packed forward (CPU): what the C call and the binding refuse before any device work, and the
order in which its CTAs take the query-tile pairs."""
import ctypes

import pytest
import torch

import exact_attention_79_gb300 as fa

FAKE = ctypes.c_void_p(1 << 20)      # never dereferenced
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(fa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fa.load()


def call(lib, q=FAKE, sh=64 * 100, st=64, o_sh=64, o_st=64 * 4, lse=FAKE, cu=FAKE, S=2, T=100, Hq=4, Hkv=2, d=64, scale=0.1):
    return lib.fa_fwd_packed(q, sh, st, FAKE, sh, st, FAKE, sh, st, FAKE, o_sh, o_st, lse, cu, S, T, Hq, Hkv, d, 1, scale, NULL)


def test_c_refusals(lib):
    for bad in (dict(q=NULL), dict(lse=NULL), dict(cu=NULL), dict(q=ctypes.c_void_p((1 << 20) + 8)), dict(S=0), dict(T=0),
                dict(Hkv=3), dict(d=60), dict(d=264), dict(scale=0.0), dict(st=0), dict(st=68), dict(o_sh=56), dict(o_st=-64),
                dict(sh=1 << 39)):
        assert call(lib, **bad) == 1, bad
    assert call(lib, d=136, st=136, sh=13600, o_sh=136, o_st=544) == 2


def test_binding_refusals(lib):
    bf = torch.bfloat16
    q, k = torch.zeros(4, 10, 64, dtype=bf), torch.zeros(2, 10, 64, dtype=bf)
    cu = torch.tensor([0, 4, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.fwd_packed(q, k, k, cu)
    with pytest.raises(ValueError, match="^v:"):
        fa.fwd_packed(q, k, k[:, :9], cu)
    with pytest.raises(ValueError, match="^q:"):
        fa.fwd_packed(q.float(), k, k, cu)
    with pytest.raises(ValueError, match="contiguous"):
        fa.fwd_packed(torch.zeros(4, 64, 10, dtype=bf).transpose(1, 2), k, k, cu)
    with pytest.raises(ValueError, match="multiples of 8"):
        fa.fwd_packed(torch.zeros(4, 10, 68, dtype=bf)[..., :64], k, k, cu)
    with pytest.raises(ValueError, match="^lse:"):
        fa.fwd_packed(q, k, k, cu, lse=torch.zeros(4, 9))
    with pytest.raises(ValueError, match="^cu_seqlens:"):
        fa.fwd_packed(q, k, k, cu.long())
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        fa.fwd_packed(q, k, k, cu[:0])
    with pytest.raises(ValueError, match="^out:"):
        fa.fwd_packed(q, k, k, cu, out=k)


def item(r, pairs):
    """The kernel's look-up (packed_item), step by step: the r-th (pair, sequence), or None."""
    count = lambda w: sum(max(0, n - w) for n in pairs)          # noqa: E731
    if count(0) <= r:
        return None
    lo, hi = 0, max(pairs)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if count(mid) > r:
            lo = mid
        else:
            hi = mid
    k = r - count(lo + 1)
    return lo, [s for s, n in enumerate(pairs) if n > lo][k]


@pytest.mark.parametrize("lens", [[1], [256], [257, 1, 0, 900], [0, 0, 5], [2000, 2000, 2000], [256 * 7, 3, 512, 511, 513]])
def test_every_pair_is_taken_once_largest_first(lens):
    pairs = [(n + 255) // 256 for n in lens]
    total = sum(pairs)
    got = [item(r, pairs) for r in range(total)]
    assert sorted(got) == sorted((w, s) for s, n in enumerate(pairs) for w in range(n))
    assert [w for w, _ in got] == sorted((w for w, _ in got), reverse=True)
    assert item(total, pairs) is None and total <= (sum(lens) + 255 * len(lens)) // 256


def test_more_sequences_than_can_be_looked_up_in_time(lib):
    assert call(lib, S=(1 << 24) + 1) == 2
