import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


# Tests that hold a value the definition does not have, and why: they run, and fail at that value.
OUTDATED = {
    "test_rows_under_large_negative_biases":
        "holds gradients of 0 for rows whose o is a mean of v; P adds up to 1 there, so dv = P^T d_o adds up to d_o "
        "(test_gpu_attention_steep.py holds these)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = OUTDATED.get(getattr(item, "originalname", None))
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))


@pytest.fixture(scope="session")
def golden_dir():
    return os.path.join(ROOT, "tests", "golden")
