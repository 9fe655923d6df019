import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) and the built CUDA library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


def pytest_collection_modifyitems(config, items):
    """The host checks of test_abi.py pass made-up device addresses and expect valid
    calls to stop at the missing device: with a GPU those calls would run."""
    import pytest
    import torch
    mine = [i for i in items if os.path.basename(str(i.fspath)) == "test_abi.py"]
    if mine and torch.cuda.is_available():
        for i in mine:
            i.add_marker(pytest.mark.skip(reason="valid calls on made-up addresses: no GPU wanted"))
