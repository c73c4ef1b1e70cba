"""LayerStep on a padded batch: sequences with no token, and chunks longer than their sequence."""
import numpy as np
import pytest
import torch

import mla_latent_kv_46_b200 as mla
from inputs import workloads as wl
from mla_latent_kv_46_b200 import decoder as dec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("projections", ["bf16", "fp8"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("q_len,lens", [(1, [64, 0, 5]), (1, [0]), (2, [1, 0, 70])])
def test_a_query_that_sees_nothing_leaves_its_row_of_the_stream(projections, gate, q_len, lens):
    """Such a query's attention is zero, so y is the residual stream there, bit for bit; the others are
    what they are without the padding, and no page of theirs is touched by it."""
    M = 1024
    spec = wl.WorkloadSpec(name="layer", B=0, H=64, R=512, Dr=64, Dn=128, Dv=128, q_len=q_len, dtype="bf16",
                           seq_len=None, w_std=1.0 / np.sqrt(512))
    st = dec.DecodeStep(wl.make(spec, seed=3, seq_lens=lens, new_rows_in_cache=False), sms=8)
    t = {k: dec.to_torch(v, st.device) for k, v in wl.layer_inputs(spec, st.T, M, seed=3, gate=gate).items()}
    x, r = t.pop("x"), t.pop("residual")
    lay = dec.LayerStep(st, t, projections=projections)
    kv = st.kv.clone()
    y = lay.run(x, r)
    torch.cuda.synchronize()
    mla.mla_check_status()
    sees = torch.tensor([max(0, n - q_len + i + 1) > 0 for n in lens for i in range(q_len)])
    assert torch.equal(y[~sees.to(y.device)], lay.residual[~sees.to(y.device)])
    assert bool(torch.isfinite(y).all())
    if bool(sees.any()):
        assert not torch.equal(y[sees.to(y.device)], lay.residual[sees.to(y.device)])
    # one cache row a token that exists
    changed = (st.kv != kv).any(dim=2)
    assert int(changed.sum()) == int(sees.sum())
