import os
import pathlib
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


# Tests without the gpu marker that also make calls which pass every check, on made-up addresses:
# without a GPU such a call ends with an error, with one it would run a kernel on them. What
# they check is checked call by call in test_fp8b128_refusals.py.
REACH_THE_DEVICE = {"test_fp8b128_args.py": {"test_bad_flags_and_shapes", "test_backward_arguments"}}


def device_present():
    """Whether this machine has the device node that the HIP runtime opens."""
    return os.path.exists("/dev/kfd")


def pytest_collection_modifyitems(items):
    if not device_present():
        return
    skip = pytest.mark.skip(reason="would run kernels on made-up addresses; see test_fp8b128_refusals.py")
    for item in items:
        if getattr(item, "originalname", None) in REACH_THE_DEVICE.get(item.path.name, ()):
            item.add_marker(skip)


def read_golden(name):
    """Rows of whitespace-separated fields from tests/golden/<name>, comments skipped."""
    rows = []
    with open(os.path.join(GOLDEN, name)) as f:
        for line in f:
            line = line.strip()
            if line and not line.startswith("#"):
                rows.append(line.split())
    return rows


@pytest.fixture
def golden():
    return read_golden
