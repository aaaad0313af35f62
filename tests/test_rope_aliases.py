"""Host checks of the rotation's outputs (CPU): the C call refuses, before any device work, an output that begins where the
other tensor or the other output does, or where its own input does with other strides."""
import ctypes

import pytest

import exact_attention_79_gb300 as fa

Q, K, QO, KO = (1 << 20, 2 << 20, 3 << 20, 4 << 20)      # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(fa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fa.load()


def call(lib, q=Q, k=K, qo=QO, ko=KO, qs=(12800, 64, 128), qos=(12800, 64, 128), ks=(12800, 64, 128), kos=(12800, 64, 128),
         B=2, T=100, Hq=2, Hkv=2):
    plan = fa._Rope(1 << 20, None, 32, 1, 0)
    return lib.fa_rope(ctypes.c_void_p(q), *qs, ctypes.c_void_p(qo), *qos, Hq, ctypes.c_void_p(k), *ks, ctypes.c_void_p(ko), *kos, Hkv,
                       B, T, 64, 2, ctypes.byref(plan), ctypes.c_void_p(1 << 20), 100, 0, 0, None)


def test_outputs_that_are_other_tensors(lib):
    for bad in (dict(qo=K), dict(ko=Q), dict(qo=K, ko=Q), dict(ko=QO), dict(qo=Q, ko=Q), dict(k=Q, qo=Q)):
        assert call(lib, **bad) == 1, bad


def test_in_place_with_other_strides(lib):
    for bad in (dict(qos=(25600, 64, 128)), dict(qos=(12800, 128, 128)), dict(qos=(12800, 6400, 64))):
        assert call(lib, qo=Q, **bad) == 1, bad
        assert call(lib, ko=K, kos=bad["qos"]) == 1, bad
