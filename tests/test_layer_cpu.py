"""The layer's operators around the attention, on the CPU: pins of their fp64 oracle
(oracle/layer.py) against library routines and closed forms, and the refusals of the C ABI
(every call here must fail validation before any launch, or launches nothing)."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import mla_latent_kv_46_b200 as mla
from mla_latent_kv_46_b200.decoder import LayerStep
from oracle import fp8, layer

INVALID = mla._binding.MLA_ERR_INVALID
UNSUPPORTED = mla._binding.MLA_ERR_UNSUPPORTED


# ----------------------------------------------------------------------------- oracle pins
def test_add_rmsnorm_equals_torch():
    rng = np.random.default_rng(1)
    x, r, g = rng.standard_normal((5, 48)), rng.standard_normal((5, 48)), rng.standard_normal(48)
    s, y = layer.add_rmsnorm(x, r, g, 1e-6)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (48,), torch.from_numpy(g), 1e-6).numpy()
    assert np.abs(s - (x + r)).max() == 0
    assert np.abs(y - want).max() < 1e-13


def test_add_rmsnorm_closed_form():
    """A row of equal values a normalises to gain (eps 0); a zero row with eps to zero."""
    g = np.arange(1.0, 9.0)
    assert np.allclose(layer.add_rmsnorm(np.full((1, 8), -3.0), None, g, 0.0)[1], -g, atol=1e-15)
    assert np.all(layer.add_rmsnorm(np.zeros((1, 8)), None, g, 1e-6)[1] == 0)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu", "gelu"])
def test_linear_equals_torch(act):
    rng = np.random.default_rng(2)
    x, W, b = rng.standard_normal((4, 10)), rng.standard_normal((7, 10)), rng.standard_normal(7)
    m, r = rng.standard_normal((4, 7)), rng.standard_normal((4, 7))
    f = {"none": lambda v: v, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu}[act]
    want = f(torch.nn.functional.linear(*map(torch.from_numpy, (x, W, b)))).numpy() * m + r
    assert np.abs(layer.linear(x, W, b, m, r, act) - want).max() < 1e-12


def test_linear_scalar_loops():
    rng = np.random.default_rng(3)
    x, W = rng.standard_normal((2, 3)), rng.standard_normal((4, 3))
    got = layer.linear(x, W)
    for t in range(2):
        for n in range(4):
            assert abs(got[t, n] - sum(x[t, k] * W[n, k] for k in range(3))) < 1e-14


def test_linear_fp8_is_linear_of_what_the_codes_stand_for():
    rng = np.random.default_rng(4)
    x, W = rng.standard_normal((3, 32)) * 5, rng.standard_normal((6, 32)) * 0.01
    (cx, sx), (cw, sw) = fp8.quantise_rows(x), fp8.quantise_rows(W)
    got = layer.linear_fp8(cx, sx, cw, sw)
    # E4M3 keeps 4 significant bits: every factor is within 2^-4, or half a subnormal step
    # (2^-10 of the row's unit) of its value
    assert np.abs(got - x @ W.T).max() <= ((2 * 2.0 ** -4 + 2.0 ** -8) * np.abs(x) @ np.abs(W).T).max() + 1e-3


def test_activations_at_their_ends():
    v = np.array([-1000.0, 1000.0, 0.0])
    assert np.array_equal(layer.activation(v, "sigmoid"), [0.0, 1.0, 0.5])
    assert np.array_equal(layer.activation(v, "silu"), [0.0, 1000.0, 0.0])
    assert np.array_equal(layer.activation(v, "gelu"), [0.0, 1000.0, 0.0])


# ----------------------------------------------------------------------------- refusals
def norm_args(**over):
    a = dict(x=1 << 20, residual=2 << 20, gain=3 << 20, residual_out=4 << 20, out=5 << 20, T=4, M=64, eps=1e-6,
             dtype=mla.MLA_BF16, stream=0)
    a.update(over)
    return a


def norm8_args(**over):
    a = norm_args(codes=6 << 20, scales=7 << 20)
    a.update(over)
    return a


def lin_args(**over):
    a = dict(x=1 << 20, W=2 << 20, bias=3 << 20, mul=4 << 20, residual=5 << 20, out=6 << 20, T=4, N=16, K=64,
             act=mla.MLA_ACT_SILU, stream=0)
    a.update(over)
    return a


def lin8_args(**over):
    a = dict(x_codes=1 << 20, x_scales=7 << 20, W_codes=2 << 20, W_scales=8 << 20, bias=3 << 20, mul=4 << 20,
             residual=5 << 20, out=6 << 20, T=4, N=16, K=64, act=mla.MLA_ACT_SILU, stream=0)
    a.update(over)
    return a


NORM_BAD = [dict(T=-1), dict(M=0), dict(M=-8), dict(eps=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
            dict(dtype=2), dict(x=None), dict(gain=None), dict(out=None), dict(residual=None),
            dict(residual_out=None), dict(x=(1 << 20) + 1), dict(out=(5 << 20) + 1),
            dict(dtype=mla.MLA_F32, gain=(3 << 20) + 2),
            dict(out=(1 << 20) + 2),            # one element off x: rows would be overwritten before they are read
            dict(residual_out=(2 << 20) + 128), dict(out=4 << 20), dict(out=3 << 20)]
NORM8_BAD = [dict(codes=None), dict(scales=None), dict(codes=1 << 20), dict(scales=(6 << 20) + 10),
             dict(codes=(5 << 20) + 64), dict(scales=3 << 20), dict(x=None)]
LIN_BAD = [dict(T=-1), dict(N=0), dict(K=0), dict(K=-4), dict(act=4), dict(act=-1), dict(x=None), dict(W=None),
           dict(out=None), dict(x=(1 << 20) + 1), dict(bias=(3 << 20) + 1), dict(out=1 << 20), dict(out=2 << 20),
           dict(out=3 << 20), dict(out=(4 << 20) + 2), dict(out=(5 << 20) - 2)]
LIN8_BAD = [dict(x_scales=None), dict(W_scales=None), dict(x_codes=None), dict(out=7 << 20), dict(out=8 << 20),
            dict(K=0), dict(out=1 << 20), dict(residual=(5 << 20) + 1)]


def refused(fn, args, status=INVALID):
    with pytest.raises(mla.MlaError) as e:
        fn(**args)
    assert e.value.status == status
    assert mla.mla_last_error()


@pytest.mark.parametrize("over", NORM_BAD, ids=str)
def test_add_rmsnorm_refuses(over):
    refused(mla.mla_add_rmsnorm, norm_args(**over))


@pytest.mark.parametrize("over", NORM8_BAD, ids=str)
def test_add_rmsnorm_fp8_refuses(over):
    refused(mla.mla_add_rmsnorm_fp8, norm8_args(**over))


@pytest.mark.parametrize("over", LIN_BAD, ids=str)
def test_linear_refuses(over):
    refused(mla.mla_linear, lin_args(**over))


@pytest.mark.parametrize("over", LIN8_BAD, ids=str)
def test_linear_fp8_refuses(over):
    refused(mla.mla_linear_fp8, lin8_args(**over))


@pytest.mark.parametrize("over", [dict(n=-1), dict(width=0), dict(dtype=7), dict(rows=None), dict(codes=None),
                                  dict(scales=None), dict(rows=(1 << 20) + 1), dict(codes=(1 << 20) + 64),
                                  dict(scales=2 << 20)], ids=str)
def test_quantize_fp8_refuses(over):
    a = dict(rows=1 << 20, codes=2 << 20, scales=3 << 20, n=4, width=64, dtype=mla.MLA_BF16, stream=0)
    a.update(over)
    refused(mla.mla_quantize_fp8, a)


def test_no_rows_is_a_launch_free_call():
    mla.mla_add_rmsnorm(**norm_args(T=0))
    mla.mla_add_rmsnorm_fp8(**norm8_args(T=0))
    mla.mla_linear(**lin_args(T=0))
    mla.mla_linear_fp8(**lin8_args(T=0))
    mla.mla_quantize_fp8(None, None, None, 0, 64, mla.MLA_BF16, stream=0)


def test_a_strided_tensor_is_refused_not_misread():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)[:, :64]
    for fn, args in ((mla.mla_add_rmsnorm, norm_args(x=x)), (mla.mla_linear, lin_args(W=x)),
                     (mla.mla_linear_fp8, lin8_args(x_codes=x)), (mla.mla_add_rmsnorm_fp8, norm8_args(out=x))):
        with pytest.raises(mla.MlaError) as e:
            fn(**args)
        assert e.value.status == INVALID


def test_a_host_tensor_is_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for fn, args in ((mla.mla_add_rmsnorm, norm_args(x=x)), (mla.mla_linear, lin_args(W=x)),
                     (mla.mla_quantize_fp8, dict(rows=x, codes=2 << 20, scales=3 << 20, n=4, width=64, dtype=0,
                                                 stream=0))):
        with pytest.raises(mla.MlaError) as e:
            fn(**args)
        assert e.value.status == INVALID


@pytest.mark.parametrize("fn,args", [(mla.mla_linear, lin_args(K=33)), (mla.mla_linear, lin_args(x=(1 << 20) + 2)),
                                     (mla.mla_linear_fp8, lin8_args(K=40)),
                                     (mla.mla_linear_fp8, lin8_args(W_codes=(2 << 20) + 8))],
                         ids=["K", "x", "K8", "W8"])
def test_linear_tensor_core_policy_refuses_what_tma_cannot_move(fn, args):
    mla.mla_set_policy(mla.MLA_POLICY_TCGEN05)
    try:
        refused(fn, args, UNSUPPORTED)
    finally:
        mla.mla_set_policy(mla.MLA_POLICY_AUTO)


# ----------------------------------------------------------------------------- the layer's step
class _Step:
    """What a LayerStep needs of a DecodeStep before it launches anything."""

    def __init__(self, dtype=torch.bfloat16, fp8=False):
        self.spec = SimpleNamespace(H=64, R=512, Dr=64, Dn=128, Dv=128)
        self.T, self.fp8, self.device = 3, fp8, torch.device("cpu")
        self.q_nope = torch.empty(3, 64, 128, dtype=dtype)


def _weights(M=96):
    def empty(*shape):
        return torch.empty(shape, dtype=torch.bfloat16)
    return {"gain": empty(M), "W_QN": empty(64 * 128, M), "W_QR": empty(64 * 64, M), "W_DKV": empty(576, M),
            "kv_gain": empty(512), "W_O": empty(M, 64 * 128), "W_G": empty(64 * 128, M)}


def test_layer_step_takes_its_weights():
    lay = LayerStep(_Step(), _weights())
    assert lay.gated and lay.M == 96 and lay.y.shape == (3, 96)
    assert not LayerStep(_Step(), {**_weights(), "W_G": None}).gated


@pytest.mark.parametrize("name", sorted(_weights()))
@pytest.mark.parametrize("change", ["short", "float32", "transposed"])
def test_layer_step_refuses_a_weight_it_would_misread(name, change):
    w = _weights()
    if change == "short":
        w[name] = w[name][:-1].contiguous()
    elif change == "float32":
        w[name] = w[name].float()
    elif change == "transposed":
        if w[name].dim() == 1:
            w[name] = torch.empty(2 * w[name].numel(), dtype=torch.bfloat16)[::2]
        else:
            w[name] = torch.empty(*reversed(w[name].shape), dtype=torch.bfloat16).T
    with pytest.raises(ValueError):
        LayerStep(_Step(), w)


@pytest.mark.parametrize("name", ["W_QN", "W_QR", "W_DKV", "kv_gain", "W_O"])
def test_layer_step_refuses_a_missing_weight(name):
    w = _weights()
    del w[name]
    with pytest.raises(ValueError):
        LayerStep(_Step(), w)


def test_layer_step_refuses_a_step_in_fp32_or_8_bits():
    for step in (_Step(dtype=torch.float32), _Step(fp8=True)):
        with pytest.raises(ValueError):
            LayerStep(step, _weights())
    with pytest.raises(ValueError):
        LayerStep(_Step(), _weights(), projections="fp4")


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("bad", [torch.empty(2, 96, dtype=torch.bfloat16), torch.empty(3, 96),
                                 torch.empty(96, 3, dtype=torch.bfloat16).T])
def test_layer_step_refuses_rows_it_would_misread(which, bad):
    lay = LayerStep(_Step(), _weights())
    rows = [torch.empty(3, 96, dtype=torch.bfloat16) for _ in range(2)]
    rows[which] = bad
    with pytest.raises(ValueError):
        lay.run(*rows)
