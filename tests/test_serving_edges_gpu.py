"""The serving operators at the ends of what their documentation allows, against the double-precision oracle."""
import numpy as np
import pytest
import torch

from oracle import cache8 as oc
from test_cache8_gpu import DEV, bf16, ints, make, to_gpu

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
