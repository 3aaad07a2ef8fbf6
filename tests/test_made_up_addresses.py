"""Calls on made-up addresses never run where the driver has a GPU, whatever torch sees, and the recurrence's are
refused wherever they run."""
import pathlib
import types

import conftest


class Item:
    def __init__(self, name):
        self.path = pathlib.Path("tests") / name
        self.marks = []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def test_files_with_made_up_addresses_are_skipped_where_there_is_a_gpu(monkeypatch):
    names = ["test_abi_cpu.py", "test_recurrence_abi_cpu.py", "test_layer_gpu.py"]
    for there in (True, False):
        monkeypatch.setattr(conftest, "driver_has_a_gpu", lambda: there)
        items = [Item(n) for n in names]
        conftest.pytest_collection_modifyitems(items)
        assert [i.marks for i in items] == ([["skip"], ["skip"], []] if there else [[], [], []])


def test_the_driver_is_asked(monkeypatch):
    def driver(init, count):
        def get(at):
            at._obj.value = count
            return 0
        return types.SimpleNamespace(cuInit=lambda flags: init, cuDeviceGetCount=get)

    for init, count, there in ((0, 1, True), (0, 0, False), (100, 1, False)):
        monkeypatch.setattr(conftest.ctypes, "CDLL", lambda name: driver(init, count))
        assert conftest.driver_has_a_gpu() is there

    def none(name):
        raise OSError(name)

    monkeypatch.setattr(conftest.ctypes, "CDLL", none)
    assert conftest.driver_has_a_gpu() is False


def test_the_recurrence_makes_no_call_that_is_accepted():
    """KDA_ERR_CUDA is what an accepted call gives without a GPU: none of that file's expects it."""
    text = (pathlib.Path(__file__).parent / "test_recurrence_abi_cpu.py").read_text()
    assert "== CUDA" not in text and "== 4" not in text
