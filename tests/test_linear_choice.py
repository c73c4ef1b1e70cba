"""The projections' choice of a kernel, on the CPU: what a device cannot run is not chosen."""
import pytest

import mla_latent_kv_46_b200 as mla

SMS = 148
SIZES = [(T, N, K) for T in (1, 2, 17, 48, 65, 128, 200, 333, 777, 2048, 5000) for N in (8, 130, 1056, 2050, 4098, 7168)
         for K in (16, 576, 2048, 4096, 16384)]


def choices(max_slices, sms=SMS):
    return {(T, N, K, e): mla.mla_debug_linear_choice(T, N, K, e, 1, sms, max_slices) for T, N, K in SIZES for e in (0, 1)}


def test_no_more_slices_than_the_devices_clusters_hold():
    """A cluster is two CTAs a slice, each with an SM's shared memory: on a device whose clusters hold
    fewer than sixteen such CTAs a launch of eight slices is an error, not a slower call."""
    free = choices(8)
    assert any(c[2] == 8 for c in free.values())
    for most in (4, 2, 1):
        held = choices(most)
        assert all(c[2] <= most for c in held.values()) and any(c[2] == most for c in held.values())
        # and what the device can run anyway stays
        assert all(held[k] == c for k, c in free.items() if c[2] <= most)


@pytest.mark.parametrize("sms", [20, 74, 148])
def test_choices_are_launchable(sms):
    for pair, nt, slices, ctas in choices(8, sms).values():
        assert 16 <= nt <= 256 and nt % 16 == 0 and slices in (1, 2, 4, 8) and ctas in (1, 2)
        assert not pair or (slices, ctas) == (1, 1)


@pytest.mark.parametrize("bad", [(0, 8, 16), (1, 0, 16), (1, 8, 0), (1, 8, 2 ** 31 - 1)])
def test_bad_arguments_are_refused(bad):
    for args in ((*bad, 0, 0, SMS, 8), (1, 8, 16, 0, 3, SMS, 8), (1, 8, 16, 0, -1, SMS, 8), (1, 8, 16, 0, 0, SMS, 0),
                 (1, 8, 16, 0, 0, SMS, 16)):
        with pytest.raises(mla.MlaError) as e:
            mla.mla_debug_linear_choice(*args)
        assert e.value.status == mla._binding.MLA_ERR_INVALID
