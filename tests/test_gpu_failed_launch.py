"""A call whose launch the runtime refuses reports it, and the calls after it are not affected."""
import contextlib
import ctypes

import pytest
import torch

import mla_latent_kv_46_b200 as mla

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CAPTURE_RELAXED = 2


@contextlib.contextmanager
def capturing_stream():
    """A stream of the kind that waits for the legacy default stream, being captured: the runtime
    refuses (on the host) every launch into the default stream meanwhile."""
    cu = ctypes.CDLL("libcuda.so.1")
    s, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(s), 0) == 0
    assert cu.cuStreamBeginCapture_v2(s, CAPTURE_RELAXED) == 0
    yield
    cu.cuStreamEndCapture(s, ctypes.byref(graph))      # invalidated by the refused launch
    if graph.value:
        cu.cuGraphDestroy(graph)
    assert cu.cuStreamDestroy_v2(s) == 0


def test_a_refused_launch_is_reported_once():
    T, M, N = 4, 256, 64
    x = torch.ones(T, M, dtype=torch.bfloat16, device=DEV)
    gain, W = x[0].clone(), torch.ones(N, M, dtype=torch.bfloat16, device=DEV)
    y, out = torch.empty_like(x), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.empty(T, M, dtype=torch.uint8, device=DEV), torch.empty(T, dtype=torch.uint8, device=DEV)
    calls = [lambda s: mla.mla_add_rmsnorm(x, None, gain, None, y, T, M, 1e-6, mla.MLA_BF16, stream=s),
             lambda s: mla.mla_linear(x, W, None, None, None, out, T, N, M, mla.MLA_ACT_NONE, stream=s),
             lambda s: mla.mla_quantize_fp8(x, codes, scales, T, M, mla.MLA_BF16, stream=s)]
    other = torch.cuda.Stream()      # does not wait for the default stream
    torch.cuda.synchronize()
    for call in calls:
        with capturing_stream(), pytest.raises(mla.MlaError) as e:
            call(0)      # the default stream
        assert e.value.status == mla._binding.MLA_ERR_CUDA
        for after in calls:
            after(other)
    other.synchronize()
    assert bool((out == M).all()) and bool((y == 1).all())
