"""Kernels launched while the one before still runs (programmatic dependent
launch) read that one's outputs: never through the read-only path, which is for
memory that nobody writes during the kernel's whole life, and whose loads the
compiler may move ahead of the wait."""
import os
import re

import pytest

import int8_weight_only_b200

CSRC = os.path.join(os.path.dirname(int8_weight_only_b200.__file__), "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if "pdl_wait()" in _code(n)))
def test_no_read_only_loads(name):
    code = _code(name)
    assert "__ldg" not in code and "global.nc" not in code
