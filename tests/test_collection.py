"""What conftest.py keeps away from a GPU."""
import types

import conftest


class Item:
    def __init__(self, path):
        self.fspath, self.marks = path, []

    def add_marker(self, m):
        self.marks.append(m)


def test_host_checks_on_made_up_addresses_are_skipped_where_a_gpu_is_present(monkeypatch):
    import torch
    for gpu in (True, False):
        monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
        items = [Item("/x/tests/test_abi.py"), Item("/x/tests/test_ops_abi.py")]
        conftest.pytest_collection_modifyitems(types.SimpleNamespace(), items)
        assert [bool(i.marks) for i in items] == [gpu, False]
