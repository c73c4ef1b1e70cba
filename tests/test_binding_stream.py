"""The binding's current device and stream, with torch's own lookups and without them (CPU: both
are stand-ins)."""
from types import SimpleNamespace

import pytest
import torch

from mla_latent_kv_46_b200 import _binding


@pytest.fixture(autouse=True)
def lookups(monkeypatch):
    monkeypatch.setattr(_binding, "_cuda", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=100 + device))


@pytest.mark.parametrize("missing", ["_cuda_getDevice", "_cuda_getCurrentRawStream"])
def test_public_lookups_serve_where_torchs_own_are_missing(monkeypatch, missing):
    monkeypatch.delattr(torch._C, missing, raising=False)
    assert _binding._stream(None) == 103
    assert _binding._stream(None) == 103      # and from then on


def test_torchs_own_lookups_serve_where_they_are(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 5, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 200 + device, raising=False)
    assert _binding._stream(None) == 205


def test_a_given_stream_is_taken_as_it_is():
    assert _binding._stream(17) == 17 and _binding._stream(SimpleNamespace(cuda_stream=18)) == 18
    assert _binding._cuda is None
