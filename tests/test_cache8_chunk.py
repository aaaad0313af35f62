"""Host checks of the chunks' attention over the 8-bit cache (CPU): what the C call and the binding refuse before any
device work, and the workspace's size."""
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


def call_packed(lib, q=FAKE, qs=(64 * 100, 64), o=ctypes.c_void_p(1 << 30), os_=(64, 64 * 8), lse=FAKE, cu=FAKE, lengths=FAKE, ws=FAKE, nbytes=1 << 40,
                B=2, T=100, Hq=8, Hkv=2, d=64, mb=8, scale=0.1, table=FAKE):
    c = fa._Cache8(1 << 20, 1 << 20, 1 << 20, 1 << 20, None, 10, Hkv, d)
    return lib.fa_fwd_cache8_packed(q, *qs, ctypes.byref(c), table, mb, cu, lengths, o, *os_, lse, ws, nbytes, B, T, Hq, 1, scale, NULL)


def test_c_refusals(lib):
    off = ctypes.c_void_p((1 << 20) + 8)
    for bad in (dict(q=NULL), dict(o=NULL), dict(lse=NULL), dict(cu=NULL), dict(lengths=NULL), dict(table=NULL), dict(q=off), dict(o=off),
                dict(B=0), dict(B=65536), dict(T=0), dict(Hq=0), dict(Hq=7), dict(mb=0), dict(scale=0.0), dict(scale=float("inf")),
                dict(qs=(6400, 60)), dict(qs=(0, 64)), dict(os_=(64, 68)), dict(os_=(64, 0)), dict(os_=(-64, 512)),
                dict(o=FAKE)):
        assert call_packed(lib, **bad) == 1, bad
    assert call_packed(lib, Hq=258, Hkv=2) == 2
    assert call_packed(lib, d=72, qs=(7200, 72), os_=(72, 576)) == 2
    assert call_packed(lib, T=(1 << 30) + 1) == 2
    assert call_packed(lib, ws=NULL) == 6 and call_packed(lib, ws=ctypes.c_void_p((1 << 20) + 128)) == 6
    assert call_packed(lib, nbytes=1000) == 6


def test_workspace_bytes(lib):
    f = lib.fa_fwd_cache8_packed_workspace_bytes
    # two partial results per CTA (152): rows of an item x D floats, three statistics per row, and eight ints per CTA
    assert f(2, 100, 8, 2, 64, 8) == 2 * 152 * 256 * (128 + 3) * 4 + 152 * 8 * 4
    assert f(2, 100, 8, 2, 256, 8) == 2 * 152 * 128 * (256 + 3) * 4 + 152 * 8 * 4
    assert f(2, 100, 8, 2, 64, 2) == 256
    for bad in ((0, 100, 8, 2, 64, 8), (2, 0, 8, 2, 64, 8), (2, 100, 7, 2, 64, 8), (2, 100, 8, 2, 72, 8), (2, 100, 258, 2, 64, 8), (2, 100, 8, 2, 64, 0)):
        assert f(*bad) == 0, bad


def test_binding_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    c = fa.new_cache8(6, 2, 64, device="cpu")
    q, table = torch.zeros(4, 10, 64, dtype=bf), torch.zeros(2, 3, dtype=i32)
    cu, lens = torch.tensor([0, 4, 10], dtype=i32), torch.tensor([4, 6], dtype=i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.fwd_cache8_packed(q, c, cu, table, lens)
    with pytest.raises(ValueError, match=r"\[Hq, T, d\]"):
        fa.fwd_cache8_packed(q[None], c, cu, table, lens)
    with pytest.raises(ValueError, match="^q:"):
        fa.fwd_cache8_packed(q.float(), c, cu, table, lens)
    with pytest.raises(ValueError, match="^q:"):
        fa.fwd_cache8_packed(q[..., :32], c, cu, table, lens)
    with pytest.raises(ValueError, match="multiples of 8"):
        fa.fwd_cache8_packed(torch.zeros(4, 10, 68, dtype=bf)[..., :64], c, cu, table, lens)
    with pytest.raises(ValueError, match="^cu_seqlens:"):
        fa.fwd_cache8_packed(q, c, cu[:2], table, lens)
    with pytest.raises(ValueError, match="^lengths:"):
        fa.fwd_cache8_packed(q, c, cu, table, lens.long())
    with pytest.raises(ValueError, match="block_table must"):
        fa.fwd_cache8_packed(q, c, cu, table[None], lens)
    with pytest.raises(ValueError, match="^out:"):
        fa.fwd_cache8_packed(q, c, cu, table, lens, out=q[:2])
    with pytest.raises(ValueError, match="^lse:"):
        fa.fwd_cache8_packed(q, c, cu, table, lens, lse=torch.zeros(4, 9))
    with pytest.raises(ValueError, match="^workspace:"):
        fa.fwd_cache8_packed(q, c, cu, table, lens, workspace=torch.zeros(9))
