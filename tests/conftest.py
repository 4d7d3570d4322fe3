import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: full-size workloads")


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle

    oracle.build()
    return oracle


# Calls with addresses that nothing backs, which pass every host check and fail for want of a
# device: on a machine with a GPU a kernel would follow them.
NO_DEVICE_ONLY = {"test_rope_append_accepts_in_place_query", "test_adjacent_buffers_are_not_aliases"}


def pytest_collection_modifyitems(items):
    marked = [i for i in items if getattr(i, "originalname", i.name) in NO_DEVICE_ONLY]
    if not marked:
        return
    import torch

    if torch.cuda.is_available():
        for item in marked:
            item.add_marker(pytest.mark.skip(reason="passes addresses that nothing backs to a launch"))
