"""LayerStep without a residual on the CPU: which rows its calls are given."""
from types import SimpleNamespace

import pytest
import torch

from mla_latent_kv_46_b200 import _binding
from mla_latent_kv_46_b200.decoder import LayerStep

T, M, H = 3, 96, 64


class _Step:
    """What a LayerStep needs of a DecodeStep, its calls left out."""

    def __init__(self):
        self.spec = SimpleNamespace(H=H, R=512, Dr=64, Dn=128, Dv=128)
        self.T, self.B, self.q_len, self.fp8, self.device = T, T, 1, False, torch.device("cpu")
        self.max_pages = self.num_pages = 1
        self.dims = self.block_table = self.seq_lens = None

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype)
        self.q_nope, self.q_rope, self.out = empty(T, H, 128), empty(T, H, 64), empty(T, H, 128)
        self.q_lat, self.o_lat = empty(T, H, 512), empty(T, H, 512, dtype=torch.float32)
        self.lse, self.workspace, self.kv = empty(T, H), empty(256), empty(1, 64, 576)

    def run(self, append, stream):
        assert not append


def _layer():
    def empty(*shape):
        return torch.empty(shape, dtype=torch.bfloat16)
    return LayerStep(_Step(), {"gain": empty(M), "W_QN": empty(H * 128, M), "W_QR": empty(H * 64, M),
                               "W_DKV": empty(576, M), "kv_gain": empty(512), "W_O": empty(M, H * 128)})


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("mla_add_rmsnorm", "mla_linear", "mla_cache_write"):
        monkeypatch.setattr(_binding, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def test_x_alone_is_the_stream(calls):
    lay = _layer()
    x = torch.empty(T, M, dtype=torch.bfloat16)
    assert lay.run(x, None) is lay.y
    x_, residual, _, residual_out, out = calls[0][1][:5]
    assert x_ is x and residual is None and residual_out is None and out is lay.hidden
    assert calls[-1][0] == "mla_linear" and calls[-1][1][4] is x and calls[-1][1][5] is lay.y


def test_with_a_residual_the_stored_sum_is_the_stream(calls):
    lay = _layer()
    x, r = torch.empty(T, M, dtype=torch.bfloat16), torch.empty(T, M, dtype=torch.bfloat16)
    lay.run(x, None)
    lay.run(x, r)
    norm = [a for n, a in calls if n == "mla_add_rmsnorm"][1]
    assert norm[1] is r and norm[3] is lay.residual
    assert calls[-1][1][4] is lay.residual


def test_a_buffer_written_before_the_end_is_refused(calls):
    lay = _layer()
    with pytest.raises(ValueError):
        lay.run(lay.hidden, None)
    with pytest.raises(ValueError):
        lay.run(lay.step.q_nope.view(-1)[:T * M].view(T, M), None)
    assert not calls
    lay.run(lay.y, None)
    lay.run(lay.residual, None)
