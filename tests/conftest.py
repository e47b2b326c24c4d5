import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

try:
    import torch  # noqa: F401
    from fp8_block_scaled_amd import _args  # noqa: F401
    CHECKS = "native"
except ImportError:                                        # an extra that needs Python's headers: its own tests need it
    CHECKS, collect_ignore = "Python", ["test_tensor_arguments.py"]


def pytest_report_header(config):
    return f"checks of tensor arguments: {CHECKS}"


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


def pytest_collection_modifyitems(config, items):
    # GPU tests skip (not fail) where no GPU is visible, e.g. in a CPU-only container.
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no GPU visible")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
