"""The 8-bit cache's host checks: what the C calls and the binding refuse before any device work (CPU)."""
import ctypes

import pytest
import torch

import exact_attention_79_gb300 as fa


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(fa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fa.load()


P = ctypes.c_void_p
FAKE = P(1 << 20)       # never dereferenced: validation fails first
OTHER = P(2 << 20)
NULL = P(0)


def cache(**kw):
    f = dict(k=1 << 20, v=1 << 20, k_scale=1 << 20, v_scale=1 << 20, weight=1 << 20, num_blocks=4, Hkv=2, d=64)
    f.update(kw)
    return ctypes.byref(fa._Cache8(*(f[n] for n, _ in fa._Cache8._fields_)))


def append(lib, c=None, k=FAKE, sh=64, st=64, B=1, T=1, cu=FAKE, start=FAKE, table=FAKE, mb=4):
    return lib.fa_cache8_append(k, sh, st, FAKE, 64, 64, cu, start, B, T, c if c is not None else cache(), table, mb, NULL)


def fwd(lib, c=None, q=FAKE, table=FAKE, mb=4, lengths=FAKE, o=OTHER, lse=FAKE, ws=FAKE, nws=1 << 30, B=1, Hq=4, Nq=1,
        scale=0.1, add=0, decay=1.0):
    return lib.fa_fwd_cache8(q, c if c is not None else cache(), table, mb, lengths, o, lse, ws, nws, B, Hq, Nq, 1, scale,
                             add, decay, NULL)


def evict(lib, c=None, B=1, keep=10, recent=2, to=FAKE, tb=1, kept=FAKE, new=OTHER, lengths=FAKE, mb=4):
    return lib.fa_cache8_evict(c if c is not None else cache(), FAKE, mb, lengths, B, keep, recent, to, tb, kept, new, NULL)


@pytest.mark.parametrize("call", [append, fwd, evict])
def test_cache_rules(lib, call):
    for bad in (dict(k=0), dict(v=0), dict(k_scale=0), dict(v_scale=0), dict(k=(1 << 20) + 8), dict(weight=(1 << 20) + 4),
                dict(num_blocks=0), dict(Hkv=0), dict(Hkv=70000), dict(d=0)):
        assert call(lib, c=cache(**bad)) == 1, bad
    for d in (8, 24, 100, 272):
        assert call(lib, c=cache(d=d)) == 2, d
    assert call(lib, c=NULL) == 1
    assert call(lib, B=0) == 1 and call(lib, B=70000) == 1
    assert call(lib, mb=0) == 1 and call(lib, mb=(1 << 24) + 1) == 1


def test_append_rules(lib):
    for bad in (dict(k=NULL), dict(k=P((1 << 20) + 8)), dict(sh=-8), dict(sh=12), dict(st=4), dict(T=0), dict(cu=NULL),
                dict(start=NULL), dict(table=NULL)):
        assert append(lib, **bad) == 1, bad


def test_fwd_rules(lib):
    for bad in (dict(q=NULL), dict(o=NULL), dict(lse=NULL), dict(lengths=NULL), dict(table=NULL), dict(Hq=3), dict(Nq=0),
                dict(scale=0.0), dict(scale=float("nan")), dict(add=1, decay=-1.0), dict(add=1, decay=float("inf")),
                dict(add=1, c=cache(weight=0)), dict(q=P((1 << 20) + 8)), dict(o=FAKE)):
        assert fwd(lib, **bad) == 1, bad
    assert fwd(lib, Hq=4, Nq=65) == 2                      # 2 heads per KV head x 65 rows
    need = lib.fa_fwd_cache8_workspace_bytes(1, 4, 2, 1, 64, 9, 0)
    more = lib.fa_fwd_cache8_workspace_bytes(1, 4, 2, 1, 64, 9, 1)
    assert 256 < need < more and fwd(lib, mb=9, add=1, nws=more - 1) == 6
    assert fwd(lib, mb=4, add=1, ws=NULL) == 6 and fwd(lib, mb=4, ws=NULL, nws=0) not in (1, 6)      # none is needed
    assert fwd(lib, B=65535, Hq=64, c=cache(Hkv=16), mb=1 << 24) == 2      # more than 2^31 units of work
    assert fwd(lib, mb=9, nws=need - 1) == 6 and fwd(lib, mb=9, ws=NULL) == 6 and fwd(lib, mb=9, ws=P((1 << 20) + 128)) == 6


def test_workspace_bytes(lib):
    # at most 304 parts (152 at d > 128 with more than 8 rows, 456 at d <= 64 with up to 4) of two partial results each, as many as units where fewer:
    # [columns][D] and [columns][3] floats; none where row groups have 8 blocks or fewer each (16 where there are more than 152 of
    # them). With weights the scores of every unit: 64 tokens x rows
    ws = lib.fa_fwd_cache8_workspace_bytes
    assert ws(1, 4, 2, 1, 64, 9, 0) == 2 * 18 * 4 * 128 * 4 + -(-2 * 18 * 4 * 3 * 4 // 256) * 256     # D = 128 up to d = 128
    assert ws(1, 4, 2, 1, 64, 9, 1) == ws(1, 4, 2, 1, 64, 9, 0) + 18 * 64 * 4 * 4         # 2 rows, kept as 4
    assert ws(1, 4, 2, 1, 64, 8, 0) == 256 and ws(1, 4, 2, 1, 64, 4, 1) == 8 * 64 * 4 * 4
    assert ws(80, 4, 2, 1, 64, 16, 0) == 256 and ws(76, 4, 2, 1, 64, 16, 0) > 256
    assert ws(64, 64, 8, 1, 128, 1000, 0) == 2 * 304 * 8 * (128 + 3) * 4
    assert ws(64, 32, 8, 1, 64, 1000, 0) == 2 * 456 * 4 * (128 + 3) * 4
    assert ws(1, 32, 1, 1, 128, 10, 1) == 2 * 20 * 16 * (128 + 3) * 4 + 20 * 64 * 16 * 4      # two chunks of 16 rows
    assert ws(1, 40, 1, 1, 128, 10, 1) == 2 * 50 * 8 * 128 * 4 + -(-2 * 50 * 8 * 3 * 4 // 256) * 256 + 50 * 64 * 8 * 4     # five of 8
    for bad in ((0, 4, 2, 1, 64, 4), (1, 3, 2, 1, 64, 4), (1, 4, 2, 0, 64, 4), (1, 4, 2, 1, 100, 4), (1, 4, 2, 1, 64, 0),
                (1, 4, 2, 65, 64, 4), (65535, 64, 16, 1, 64, 1 << 24)):
        assert ws(*bad, 0) == 0, bad


def test_evict_rules(lib):
    for bad in (dict(keep=0), dict(recent=-1), dict(recent=11), dict(tb=0), dict(keep=65, tb=1), dict(to=NULL), dict(kept=NULL),
                dict(new=NULL), dict(lengths=NULL), dict(new=FAKE, lengths=FAKE), dict(c=cache(weight=0))):
        assert evict(lib, **bad) == 1, bad


def test_evict_counts_the_blocks_it_fills_not_the_tables(lib):
    wide = evict(lib, B=65535, keep=64, tb=1 << 24)        # one block a sequence: no refusal (here it finds no device)
    assert wide not in (1, 2)
    assert evict(lib, B=65535, keep=1 << 22, tb=1 << 16) == 2      # 65535 * 65536 of them


def test_binding_refuses_before_any_launch(lib):
    c = fa.new_cache8(4, 2, 64, device="cpu", weight=True)
    i32 = torch.int32
    table, lens = torch.zeros(1, 3, dtype=i32), torch.ones(1, dtype=i32)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    kv = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 5], dtype=i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.fwd_cache8(q, c, table, lens)
    with pytest.raises(ValueError, match="^lengths:"):
        fa.fwd_cache8(q, c, table, lens.long())
    with pytest.raises(ValueError, match="^block_table:"):
        fa.fwd_cache8(q, c, table.long(), lens)
    with pytest.raises(ValueError, match="block_table must be"):
        fa.fwd_cache8(q, c, table[0], lens)
    with pytest.raises(ValueError, match="^q:"):
        fa.fwd_cache8(q[..., :32], c, table, lens)
    with pytest.raises(ValueError, match="^out:"):
        fa.fwd_cache8(q, c, table, lens, out=torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="weights"):
        fa.fwd_cache8(q, c._replace(weight=None), table, lens, weight_decay=1.0)
    with pytest.raises(ValueError, match="^cache.v_scale:"):
        fa.fwd_cache8(q, c._replace(v_scale=c.v_scale[:3]), table, lens)
    with pytest.raises(ValueError, match="^k:"):
        fa.cache8_append(c, kv[:1], kv, cu, table, lens)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.cache8_append(c, kv, kv, cu, table, lens)
    with pytest.raises(ValueError, match="^cu_seqlens:"):
        fa.cache8_append(c, kv, kv, cu[:1], table, lens)
    with pytest.raises(ValueError, match="contiguous"):
        fa._heads_strides(torch.zeros(2, 64, 5, dtype=torch.bfloat16).transpose(1, 2), "k", 2, 5, 64)
    with pytest.raises(ValueError, match="weights"):
        fa.cache8_evict(c._replace(weight=None), table, lens, 10, 2, table)
    with pytest.raises(ValueError, match="^to_table:"):
        fa.cache8_evict(c, table, lens, 10, 2, table.long())
    with pytest.raises(ValueError, match="^kept:"):
        fa.cache8_evict(c, table, lens, 10, 2, table, kept=torch.zeros(1, 2, 9, dtype=i32))
