import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU; calls the HIP path")


# Tests that pass made-up device addresses to calls that are accepted: nothing but the
# missing GPU keeps those from a launch.
MADE_UP_ADDRESSES = {
    "test_abi.py": {"test_null_lora_allowed_without_rank_all_entries", "test_null_lora_allowed_without_rank",
                    "test_quantize_rank_zero_needs_no_lora_pointers"},
    "test_block_refusals.py": {"test_quantize_accepts", "test_few_accepts", "test_rotary_accepts", "test_attention_accepts"},
}


def pytest_collection_modifyitems(config, items):
    # GPU tests are skipped, never silently rerouted, where no GPU is present;
    # tests that would launch on made-up addresses, where one is.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        skip = pytest.mark.skip(reason="made-up device addresses: needs a machine without a GPU")
        for item in items:
            if item.name.split("[")[0] in MADE_UP_ADDRESSES.get(os.path.basename(str(item.fspath)), ()):
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no GPU visible (torch.cuda.is_available() is False)")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
