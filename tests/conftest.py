import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


# Refusals through the C ABI that are given made-up device addresses: only the refusal keeps the addresses
# from being read, so they run where no GPU could read them.
MADE_UP_ADDRESSES = re.compile(r"(?:[^\[]*/)?(?:test_linear_unit_refusals\.py::\w+_refuses|"
                               r"test_capi_host\.py::test_zero3_step_rejects_bad_arguments_before_launch)")


def pytest_collection_modifyitems(items):
    made_up = [i for i in items if MADE_UP_ADDRESSES.match(i.nodeid)]
    if not made_up:
        return
    import torch
    if torch.cuda.is_available():
        skip = pytest.mark.skip(reason="made-up device addresses: only where there is no GPU")
        for i in made_up:
            i.add_marker(skip)
