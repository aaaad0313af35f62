"""Tensors whose offsets pass 2^31 elements, and 2^32 bytes, on the GPU: the rotation, the append and the chunks' attention give
the same bits on them as on dense ones (which other tests hold against 64 bits).

Memory is taken as needed and not filled: 4 to 19 GB at a time.
"""
import numpy as np
import pytest
import torch

from test_cache8_gpu import DEV, bf16, ints
from test_rope_gpu import freqs

pytestmark = pytest.mark.gpu
FAR = 1 << 31                # elements between heads, batches or tokens


def spread(x, far):
    """x in memory where its dimension number 0 is `far` elements apart; the others dense."""
    inner = x[0].numel()
    mem = torch.empty((x.shape[0] - 1) * far + inner, dtype=x.dtype, device=DEV)
    strides = [far]
    for n in x.shape[1:]:
        inner //= n
        strides.append(inner)
    y = mem.as_strided(x.shape, strides)
    y.copy_(x)
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(fa, dtype):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 70, 64, generator=gen).to(dtype).to(DEV)               # [far, 3, T, d]
    plan, pos = fa.new_rope(freqs(32)), torch.arange(70, dtype=torch.int32, device=DEV) + (1 << 30)
    want, _ = fa.rope(x, None, plan, pos)
    out = spread(torch.zeros_like(x), FAR + 8)
    got, _ = fa.rope(spread(x, FAR + 64), None, plan, pos, q_out=out)            # batches far apart
    assert got is out and torch.equal(got, want)
    del out, got
    one = x[:, :1].contiguous()                                                  # [2 heads] far apart, in place
    y = spread(one[:, 0], FAR)
    fa.rope(y, None, plan, pos, q_out=y)
    assert torch.equal(y, want[:, 0])
    del y
    z = spread(x[0].transpose(0, 1).contiguous()[:2], FAR)                       # two tokens far apart: [T, H, d]
    got, _ = fa.rope(z.transpose(0, 1), None, plan, pos[:2])
    assert torch.equal(got, want[0, :, :2])
    fa.check_device_status()


@pytest.mark.parametrize("d", [128, 256])
def test_append_and_chunks(fa, d):
    """K, V, Q and O with heads far apart, and a pool of more than 2^32 bytes of codes whose last blocks are used."""
    Hq, Hkv, T, past = 4, 2, 150, 300
    rng = np.random.default_rng(d)
    plan = fa.new_rope(freqs(d // 2))
    k, v = (bf16(rng, Hkv, past + T, d).to(DEV) for _ in range(2))
    q = bf16(rng, Hq, T, d).to(DEV)
    n = past + T
    cu, start, lens = ints([0, n]), ints([0]), ints([n])
    results = []
    for far in (False, True):
        blocks = (1 << 32) // (Hkv * 64 * d) + 9 if far else 9
        cache = fa.new_cache8(9, Hkv, d)
        if far:                                          # (a pool of torch.empty: new_cache8's is filled)
            cache = fa.Cache8(*(torch.empty(blocks, Hkv, 64, d, dtype=torch.uint8, device=DEV) for _ in range(2)),
                              *(torch.ones(blocks, Hkv, device=DEV) for _ in range(2)))
            assert cache.k.numel() > 1 << 32
        table = torch.arange(blocks - 8, blocks, dtype=torch.int32, device=DEV)[None]
        fa.cache8_append(cache, spread(k, FAR) if far else k, spread(v, FAR) if far else v, cu, table, start, rope=plan)
        out = spread(torch.zeros_like(q), FAR) if far else None
        o, lse = fa.fwd_cache8_packed(spread(q, FAR) if far else q, cache, ints([0, T]), table, lens, out=out)
        fa.check_device_status()
        results.append((cache.k[-8:].clone(), cache.v[-8:].clone(), cache.k_scale[-8:].clone(), cache.v_scale[-8:].clone(), o.contiguous(), lse))
        del cache, out, o
    (k0, v0, *a), (k1, v1, *b) = results
    used = torch.zeros(8, 1, 64, 1, dtype=torch.bool, device=DEV)
    used.view(-1)[:n] = True                             # slots behind the last token hold anything
    assert torch.equal(k0 * used, k1 * used) and torch.equal(v0 * used, v1 * used)
    whole = -(-n // 64)
    assert torch.equal(a[0][:whole], b[0][:whole]) and torch.equal(a[1][:whole], b[1][:whole])
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
