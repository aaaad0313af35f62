import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a GB300 (sm_103) GPU and the built CUDA library")


# CPU tests of calls that pass every check, with pointers to nothing: they end at the missing device, so they need one
# to be missing.
NEED_NO_DEVICE = {("test_cache8.py", "test_fwd_rules"),
                  ("test_cache8.py", "test_evict_counts_the_blocks_it_fills_not_the_tables")}


def pytest_collection_modifyitems(items):
    chosen = [i for i in items if (os.path.basename(str(i.fspath)), getattr(i, "originalname", None)) in NEED_NO_DEVICE]
    if chosen:
        import torch
        if torch.cuda.is_available():
            for i in chosen:
                i.add_marker(pytest.mark.skip(reason="the call would go through, and its pointers are none"))


@pytest.fixture(scope="session")
def fa():
    """The CUDA library binding, built in-tree. GPU tests only."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_79_gb300 as fa_mod
    fa_mod.load()          # raises if the compiled library is missing
    return fa_mod
