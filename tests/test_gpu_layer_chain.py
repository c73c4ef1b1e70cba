"""LayerStep without a residual: a first layer, and layers chained by their results."""
import pytest
import torch

from inputs import workloads as wl
from mla_latent_kv_46_b200 import decoder as dec

import mla_latent_kv_46_b200 as mla

pytestmark = pytest.mark.gpu


def layer(projections, M=1024, seed=5, lens=(70, 5, 129, 1)):
    spec = wl.WorkloadSpec(name="layer", B=0, H=64, R=512, Dr=64, Dn=128, Dv=128, q_len=1, dtype="bf16", seq_len=None,
                           w_std=1.0 / 512 ** 0.5)
    st = dec.DecodeStep(wl.make(spec, seed=seed, seq_lens=list(lens), new_rows_in_cache=False), sms=8)
    t = {k: dec.to_torch(v, st.device) for k, v in wl.layer_inputs(spec, st.T, M, seed=seed).items()}
    x = t.pop("x")
    t.pop("residual")
    return st, x, dec.LayerStep(st, t, projections=projections)


# A residual of zeros changes no bit of x + residual, so both forms must give the same bits. (Steps may
# be repeated: each writes the same cache rows again.)
@pytest.mark.parametrize("projections", ["bf16", "fp8"])
def test_first_layer_runs_without_a_residual(projections):
    st, x, lay = layer(projections)
    zeros = torch.zeros_like(x)
    want, hidden = lay.run(x, zeros).clone(), lay.hidden.clone()
    assert torch.equal(lay.residual, x)
    before = x.clone()
    got = lay.run(x, None)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(lay.hidden, hidden) and torch.equal(x, before)
    assert not torch.equal(got, x)
    # with a residual again: the rows that Wo adds to are the sum's, not the last x
    assert torch.equal(lay.run(zeros, x), want)
    mla.mla_check_status()


@pytest.mark.parametrize("projections", ["bf16", "fp8"])
def test_layers_chain_by_their_results(projections):
    _, x, first = layer(projections)
    _, _, second = layer(projections, seed=6)
    zeros = torch.zeros_like(x)
    y1 = first.run(x, zeros).clone()
    y2 = second.run(y1, zeros).clone()
    got = second.run(first.run(x, None), None)
    torch.cuda.synchronize()
    assert torch.equal(first.y, y1) and torch.equal(got, y2)
    # the step's own result as its next input: y is read and written in place by the last projection
    want = first.run(y1, zeros).clone()
    first.y.copy_(y1)
    assert torch.equal(first.run(first.y, None), want)
    mla.mla_check_status()


def test_first_layer_replays_from_a_graph():
    _, x, lay = layer("fp8")
    a, b = lay.run(x, None).clone(), lay.run(2 * x, None).clone()
    into = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.run(into, None)
    lay.run(x, torch.ones_like(x))      # what an eager run leaves behind does not reach the graph's replay
    for rows, want in ((x, a), (2 * x, b)):
        into.copy_(rows)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.y, want)


def test_a_buffer_that_the_run_writes_is_refused_as_the_stream():
    st, x, lay = layer("fp8", M=64 * 128)
    lay.hidden.copy_(x)
    for own in (lay.hidden, st.out.view(st.T, -1)):
        with pytest.raises(ValueError):
            lay.run(own, None)
    lay.run(lay.hidden, torch.zeros_like(x))      # with a residual the sum is stored apart
    want = lay.y.clone()
    assert torch.equal(lay.run(x, None), want)
    lay.residual.copy_(x)
    assert torch.equal(lay.run(lay.residual, None), want)
