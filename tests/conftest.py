import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# Tests with a call that passes every check on made-up addresses: without a GPU it ends at its first
# CUDA call, with one it would launch a kernel on them.
WITHOUT_A_GPU_ONLY = {"test_abi.py::test_compressor_argument_checks"}


def pytest_collection_modifyitems(items):
    import torch

    if torch.cuda.is_available():
        for item in items:
            if f"{item.path.name}::{item.name}" in WITHOUT_A_GPU_ONLY:
                item.add_marker(pytest.mark.skip(reason="a call on made-up addresses is made without a GPU only"))


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
