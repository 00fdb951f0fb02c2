"""The compiled Python calls belong to one torch: with another one they are built again, and refused until then."""
import pytest
import torch

import top_routed_block_b200 as fv
from top_routed_block_b200 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_binding_of_another_torch_is_stale(monkeypatch):
    assert not _build._binding_stale()
    monkeypatch.setattr(torch, "__version__", "0.1.0")
    assert _build._binding_stale()


def test_binding_of_another_torch_is_refused(monkeypatch):
    monkeypatch.setattr(fv, "_native", None)
    assert fv._native_calls().built_for == _build.binding_target()
    monkeypatch.setattr(fv, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.1.0")
    with pytest.raises(fv.FvattnError, match="built for"):
        fv._native_calls()
    assert fv._native is None
