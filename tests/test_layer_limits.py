"""Bounds of the layer's operators on the CPU: every call here must fail validation before any
launch (the addresses are made up)."""
import pytest

import mla_latent_kv_46_b200 as mla

INVALID = mla._binding.MLA_ERR_INVALID
LONGEST = 0x7FFFF000      # elements of a row
# rows far enough apart in the address space that they do not overlap
BASE = 1 << 40
P = [BASE * i for i in range(1, 9)]


def refused(fn, *args):
    with pytest.raises(mla.MlaError) as e:
        fn(*args, stream=0)
    assert e.value.status == INVALID and "bad sizes" in mla.mla_last_error()


@pytest.mark.parametrize("n", [LONGEST + 1, 2 ** 31 - 1024, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [mla.MLA_BF16, mla.MLA_F32], ids=["bf16", "f32"])
def test_rows_whose_element_count_would_wrap_are_refused(n, dtype):
    """The kernels' 32-bit counters step past a row's end by up to 1024 elements: a row that ends
    within that of 2^31 would be followed by negative indices."""
    refused(mla.mla_add_rmsnorm, P[0], None, P[1], None, P[2], 1, n, 1e-6, dtype)
    refused(mla.mla_add_rmsnorm, P[0], P[3], P[1], P[4], P[2], 1, n, 1e-6, dtype)
    refused(mla.mla_add_rmsnorm_fp8, P[0], None, P[1], None, None, P[5], P[6], 1, n, 1e-6, dtype)
    refused(mla.mla_quantize_fp8, P[0], P[5], P[6], 1, n, dtype)


@pytest.mark.parametrize("K", [LONGEST + 1, LONGEST + 16, 2 ** 31 - 128, 2 ** 31 - 16, 2 ** 31 - 1])
def test_projections_whose_k_would_wrap_are_refused(K):
    refused(mla.mla_linear, P[0], P[1], None, None, None, P[2], 1, 8, K, mla.MLA_ACT_NONE)
    refused(mla.mla_linear_fp8, P[0], P[3], P[1], P[4], None, None, None, P[2], 1, 8, K, mla.MLA_ACT_NONE)
    # with no rows as well: what is refused does not depend on how many there are
    refused(mla.mla_linear, P[0], P[1], None, None, None, P[2], 0, 8, K, mla.MLA_ACT_NONE)
