"""Tests without the gpu marker cannot reach a GPU: a run of them alone sees none, and
the one that gets past the library's argument checks is skipped where there is one."""

import os

import conftest


class Config:
    def __init__(self, markexpr):
        self.option = type("Option", (), {"markexpr": markexpr})()

    def addinivalue_line(self, *args):
        pass


class Item:
    def __init__(self, name):
        self.name, self.markers = name, []

    def add_marker(self, marker):
        self.markers.append(marker)


def test_a_run_of_these_alone_sees_no_gpu(monkeypatch):
    for expr, hidden in (("not gpu", True), ("gpu", False), ("", False)):
        monkeypatch.setenv("CUDA_VISIBLE_DEVICES", "0")
        conftest.pytest_configure(Config(expr))
        assert (os.environ["CUDA_VISIBLE_DEVICES"] == "") is hidden


def test_calls_with_invented_addresses_are_skipped_beside_a_gpu(monkeypatch):
    for visible, driver, skipped in (("0", True, 1), ("", True, 0), ("0", False, 0)):
        monkeypatch.setenv("CUDA_VISIBLE_DEVICES", visible)
        monkeypatch.setattr(conftest.os.path, "exists", lambda p, driver=driver: driver)
        items = [Item("test_x_planes_scratch_is_not_needed"), Item("test_other")]
        conftest.pytest_collection_modifyitems(items)
        assert [len(i.markers) for i in items] == [skipped, 0]
