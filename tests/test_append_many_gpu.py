"""The rotating append over many blocks, on the GPU: more blocks times KV heads than go to the kernel that takes K and V of a
head together, so that V is written by the plain kernel and K by one with up to four heads to a CTA. (The cases of
test_rope_gpu.py, of 776 at most, all go to the former.) Against 64 bits, and to the bit against the same tokens appended in
calls of few blocks.
"""
import numpy as np
import pytest
import torch

from test_rope_gpu import DEV, check_append, empty_cache, freqs, ints

pytestmark = pytest.mark.gpu
FEW = 1216               # blocks times heads up to which K and V of a head go together


def blocks(T, B):
    """Blocks that T new tokens of B sequences may touch, as the launch counts them."""
    return min(T, (T + 126 * B) // 64)


# (held, new) per sequence, Hkv, d, pairs, axes, interleaved, own positions
CASES = [
    ([(30, 8600)], 9, 128, 64, 1, False, True),                     # heads in CTAs of 4, 4 and 1
    ([(5, 8000), (0, 900), (63, 1)], 9, 128, 32, 3, True, True),    # half of the columns stay
    ([(7, 6300)], 13, 80, 20, 2, False, False),
    ([(30, 15700)], 5, 256, 128, 1, False, True),
    ([(1, 5000), (64, 4000)], 10, 192, 96, 3, True, True),
    ([(11, 26000)], 3, 64, 32, 1, True, False),                     # fewer heads than a CTA takes
]


def prepare(fa, seqs, Hkv, d, pairs, axes, own_positions, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    width = max(-(-(a + n) // 64) for a, n in seqs) + 1
    P = len(seqs) * width + 2
    table = rng.permutation(P)[: len(seqs) * width].reshape(len(seqs), width).astype(np.int32)
    c = empty_cache(fa, rng, P, Hkv, d)
    for b, (held, _) in enumerate(seqs):
        for at in range(held):
            for x in ("k", "v"):
                c[x][table[b, at // 64], :, at % 64] = (torch.randn(Hkv, d, generator=gen) * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])])
    start = np.array([a for a, _ in seqs])
    T = int(cu[-1])
    # magnitudes that differ from head to head and along the tokens: each head's scales are its own, and some grow
    size = torch.exp2(torch.arange(Hkv) % 5 - 2.0)[None, :, None] * torch.exp2(torch.arange(T) // 40 % 4)[:, None, None]
    k, v = ((torch.randn(T, Hkv, d, generator=gen) * size).to(torch.bfloat16).to(DEV).transpose(0, 1) for _ in range(2))
    f, axis = freqs(pairs), [int(a) for a in rng.integers(0, axes, pairs)]
    own = np.concatenate([np.arange(a, a + n) for a, n in seqs])
    pos = rng.integers(-1000, 1 << 20, (axes, T)) if own_positions else np.broadcast_to(own, (axes, T))
    return c, table, cu, start, k, v, f, axis, pos


def on_gpu(fa, c):
    return fa.Cache8(**{n: torch.from_numpy(x.copy()).to(DEV) for n, x in c.items()})


@pytest.mark.parametrize("seqs,Hkv,d,pairs,axes,interleaved,own_positions", CASES)
def test_many_blocks(fa, seqs, Hkv, d, pairs, axes, interleaved, own_positions):
    T = sum(n for _, n in seqs)
    assert blocks(T, len(seqs)) * Hkv > FEW
    c, table, cu, start, k, v, f, axis, pos = prepare(fa, seqs, Hkv, d, pairs, axes, own_positions, T + d)
    plan = fa.new_rope(f, axis, interleaved)
    positions = ints(pos) if own_positions else None
    g = on_gpu(fa, c)
    fa.cache8_append(g, k, v, ints(cu), ints(table), ints(start), rope=plan, positions=positions)
    # the same call on another copy: the same bits
    again = on_gpu(fa, c)
    fa.cache8_append(again, k, v, ints(cu), ints(table), ints(start), rope=plan, positions=positions)
    # piece by piece, each within few blocks and up to a block's end, so that every block is written once
    few = on_gpu(fa, c)
    for b, (held, new) in enumerate(seqs):
        at = 0
        while at < new:
            n = min(new - at, 64 * ((FEW // Hkv - 2) // 2) - (held + at) % 64)
            assert blocks(n, 1) * Hkv <= FEW
            i = int(cu[b]) + at
            fa.cache8_append(few, k[:, i:i + n], v[:, i:i + n], ints([0, n]), ints(table[b:b + 1]), ints([held + at]), rope=plan,
                             positions=None if positions is None else positions[:, i:i + n])
            at += n
    fa.check_device_status()
    for name in ("k", "v", "k_scale", "v_scale", "weight"):
        assert torch.equal(getattr(g, name), getattr(again, name)), name
        assert torch.equal(getattr(g, name), getattr(few, name)), name
    flips = check_append(c, g, k, v, f, axis, pos, interleaved, cu, start, table)
    assert flips <= 2 + 1e-5 * T * Hkv * d


@pytest.mark.parametrize("T", [8577, 8578])
def test_on_both_sides_of_the_border(fa, T):
    """The last size that goes to the kernel for few blocks and the first that does not: both right."""
    Hkv, d = 9, 128
    assert (blocks(T, 1) * Hkv > FEW) == (T == 8578)
    c, table, cu, start, k, v, f, axis, pos = prepare(fa, [(50, T)], Hkv, d, 64, 1, True, 3)
    g = on_gpu(fa, c)
    fa.cache8_append(g, k, v, ints(cu), ints(table), ints(start), rope=fa.new_rope(f, axis), positions=ints(pos))
    fa.check_device_status()
    check_append(c, g, k, v, f, axis, pos, False, cu, start, table)
