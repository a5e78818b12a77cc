"""The binding is built again when torch or Python is another one than it was built for."""
import pytest

from mixture_experts_ffn_sort_b200 import build


@pytest.fixture
def built(monkeypatch, tmp_path):
    build.build()
    calls = []
    monkeypatch.setattr(build, "_build_library", lambda *a: calls.append("library"))
    monkeypatch.setattr(build, "_build_binding", lambda *a: calls.append("binding"))
    return calls


def test_nothing_to_do(built):
    build.build()
    assert built == []


def test_another_torch(built, monkeypatch):
    monkeypatch.setattr(build, "_versions", lambda: "torch 9.9, Python 3.99")
    build.build()
    assert built == ["binding"]


def test_no_record(built, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BUILT_FOR", str(tmp_path / "none.txt"), raising=False)
    build.build()
    assert built == ["binding"]


def test_a_torch_without_package_metadata(built, monkeypatch):
    import importlib.metadata

    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(importlib.metadata, "version", none)
    build.build()
    assert built == []
