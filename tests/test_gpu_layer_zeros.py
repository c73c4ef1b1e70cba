"""A zero keeps its sign through the row operators, at any width and alignment: without a
residual s is x itself, not x + 0."""
import numpy as np
import pytest
import torch

import mla_latent_kv_46_b200 as mla
from oracle import fp8

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


# rows of a warp, a block, shifted; too wide for a block's registers, and (shift) not 16-byte aligned
@pytest.mark.parametrize("M,shift", [(64, 0), (1111, 0), (7168, 0), (20000, 0), (20001, 0), (64, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_the_sign_of_zero(M, shift, dtype):
    T = 3
    rows = torch.zeros(T, M)
    rows[:, 1::3] = -0.0
    rows[1, M - 1], rows[2, 5] = 2.5, -1e-6      # codes of small negative values round to -0 as well
    whole = torch.zeros(T * M + shift, dtype=dtype, device=DEV)
    x = whole[shift:].view(T, M)
    x.copy_(rows)
    name = mla.MLA_BF16 if dtype == torch.bfloat16 else mla.MLA_F32
    codes, scales = torch.empty(T, M, dtype=torch.uint8, device=DEV), torch.empty(T, dtype=torch.uint8, device=DEV)
    mla.mla_quantize_fp8(x, codes, scales, T, M, name)
    want_codes, want_scales = fp8.quantise_rows(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    gain = torch.ones(M, dtype=dtype, device=DEV)
    y = torch.empty(T, M, dtype=dtype, device=DEV)
    mla.mla_add_rmsnorm(x, None, gain, None, y, T, M, 1e-6, name)
    assert torch.equal(torch.signbit(y), torch.signbit(x))
