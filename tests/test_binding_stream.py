"""The binding takes the current stream's handle the short way where torch offers it, and through the public call where it
does not."""
import types

import pytest

import int4_routed_expert_02_amd as moe


@pytest.fixture
def fresh(monkeypatch):
    import torch
    monkeypatch.setattr(moe, "_torch", None)
    monkeypatch.setattr(moe, "_current", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=77))
    return torch


@pytest.mark.parametrize("missing", ["_cuda_getDevice", "_cuda_getCurrentRawStream"])
def test_without_torch_internals(fresh, missing, monkeypatch):
    monkeypatch.setattr(fresh._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(fresh._C, "_cuda_getCurrentRawStream", lambda d: 55, raising=False)
    monkeypatch.delattr(fresh._C, missing)
    assert moe._stream(None) == 77


def test_with_them(fresh, monkeypatch):
    monkeypatch.setattr(fresh._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(fresh._C, "_cuda_getCurrentRawStream", lambda d: 50 + d, raising=False)
    assert moe._stream(None) == 53


def test_given_stream(fresh):
    assert moe._stream(types.SimpleNamespace(cuda_stream=9)) == 9
