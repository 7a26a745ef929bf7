"""Tests that hand the library made-up device addresses are skipped where a GPU could read them. No GPU:
torch is made to say that there is one while the tests are collected and, in their place, nothing runs."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# file, tests of it that are given no addresses
FILES = [("tests/test_linear_unit_refusals.py", ["test_act_backward_workspace", "test_dw_workspace"]),
         ("tests/test_capi_host.py::test_zero3_step_rejects_bad_arguments_before_launch", [])]

# What a pytest run would do with each collected test, by its marks; none is run.
CODE = """
import sys, pytest, torch
torch.cuda.is_available = lambda: {gpu}
class Notes:
    @pytest.hookimpl(tryfirst=True)
    def pytest_runtest_protocol(self, item):
        counts[any(m.name == "skip" for m in item.iter_markers())] += 1
        return True
counts = {{False: 0, True: 0}}
rc = pytest.main(["-q", "-p", "no:cacheprovider", *sys.argv[1:]], plugins=[Notes()])
print("counts", counts[False], counts[True])
"""


def counts(gpu, *names):
    r = subprocess.run([sys.executable, "-c", CODE.format(gpu=gpu), *names], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    line = [s for s in r.stdout.splitlines() if s.startswith("counts")]
    assert line, r.stdout[-2000:] + r.stderr[-2000:]
    return tuple(int(n) for n in line[-1].split()[1:])


@pytest.mark.parametrize("name,others", FILES)
def test_skipped_where_there_is_a_gpu(name, others):
    run, skipped = counts(False, name)
    assert run > 0 and skipped == 0
    assert counts(True, name) == (len(others), run - len(others))
    if others:
        assert counts(True, *[f"{name}::{t}" for t in others]) == (len(others), 0)


def test_others_are_not():
    assert counts(True, __file__) == (3, 0)  # whose parameters name them
    run, skipped = counts(True, "tests/test_capi_host.py", "tests/test_binding_checks.py")
    assert run > 10 and skipped == 1
