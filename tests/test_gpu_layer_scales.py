"""The scale byte of the norm's 8-bit rows where a row is not finite: NaNs count towards no scale,
whatever made them."""
import pytest
import torch

import mla_latent_kv_46_b200 as mla

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


# rows of every kernel: a warp's, a block's, shifted, element by element; many rows: streamed
@pytest.mark.parametrize("T,M", [(16, 64), (16, 1111), (16, 4096), (16, 20000), (1300, 2048)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_and_scales_are_the_quantisers_of_the_fp32_rows(T, M, eps, residual):
    """The 8-bit output is the fp32 output's, quantised: codes and scale bytes must equal
    mla_quantize_fp8's of it bit for bit, for rows with infinities and NaNs too (max |s g| times a
    positive number is the maximum of the products, for rounding is monotonic)."""
    g = torch.Generator(device="cpu").manual_seed(M)
    x = torch.randn(T, M, generator=g)
    gain = 1 + 0.3 * torch.randn(M, generator=g)
    x[1, M // 3] = INF                    # the row's other values are 0, this one NaN
    x[2, M - 1] = NAN                     # every value NaN
    x[3] = 0                              # NaN with eps = 0
    x[4] *= 1e25                          # the sum of squares overflows
    x[5] *= 1e-30                         # .. underflows
    x[6, 0], x[6, 1] = INF, -INF
    x[7, 0], x[7, 5] = NAN, INF
    x[8] = -INF
    x[9, ::2] = NAN
    x, gain = x.to(DEV), gain.to(DEV)
    r = torch.zeros_like(x) if residual else None
    ro = torch.empty_like(x) if residual else None
    y = torch.empty_like(x)
    codes, scales = torch.empty(T, M, dtype=torch.uint8, device=DEV), torch.empty(T, dtype=torch.uint8, device=DEV)
    want_codes, want_scales = torch.empty_like(codes), torch.empty_like(scales)
    mla.mla_add_rmsnorm_fp8(x, r, gain, ro, y, codes, scales, T, M, eps, mla.MLA_F32)
    mla.mla_quantize_fp8(y, want_codes, want_scales, T, M, mla.MLA_F32)
    torch.cuda.synchronize()
    assert torch.equal(scales, want_scales)
    nan = torch.isnan(y)
    assert torch.equal(codes[~nan], want_codes[~nan]) and bool(((codes[nan] & 0x7F) == 0x7F).all())
    # rows with no value that counts have the smallest scale
    none = (torch.nan_to_num(y, nan=0.0) == 0).all(dim=1)
    assert bool(none[1]) and bool(none[2]) and bool((scales[none] == 1).all()) and not bool(none[0])


def test_scales_of_bf16_rows_that_are_not_finite():
    x = torch.ones(3, 256, dtype=torch.bfloat16, device=DEV)
    x[0, 7], x[1, 255] = NAN, INF
    gain = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.empty(3, 256, dtype=torch.uint8, device=DEV), torch.empty(3, dtype=torch.uint8, device=DEV)
    mla.mla_add_rmsnorm_fp8(x, None, gain, None, None, codes, scales, 3, 256, 1e-6, mla.MLA_BF16)
    torch.cuda.synchronize()
    # a row of ones: y a little below 1, above 448 2^-9 = 0.875 and not above 448 2^-8
    assert scales.tolist() == [1, 1, 127 - 8]
