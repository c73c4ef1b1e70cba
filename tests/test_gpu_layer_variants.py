"""Every variant of the few-token projection that its choice picks, and forms of the streaming norm,
against the fp64 oracle; offsets past 32 bits; the layer step's output projection."""
import numpy as np
import pytest
import torch

import mla_latent_kv_46_b200 as mla
from inputs import workloads as wl
from mla_latent_kv_46_b200 import decoder as dec
from oracle import fp8, layer
from oracle import mla_oracle as orc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 64
STAT = 2.0 ** -18      # the norm's fp32 statistics: a tree of sums, halved by the root, five roundings


def host(t):
    return t.double().cpu().numpy()


def bf16(a):
    return None if a is None else torch.from_numpy(a).to(torch.bfloat16).to(DEV)


# (T, N, K, 8 bits) -> tokens a tile, K slices, CTAs an SM. Tokens that end inside a chunk of 16,
# features that end inside a pair's 256, rows of whole 16-byte pieces (N % 8 == 0) and others; more
# chunks than pairs, so that a pair finishes several, and as many or fewer.
SPLIT = {
    (82, 9749, 16, 0): (32, 1, 2), (148, 9849, 16, 0): (64, 1, 2), (155, 9568, 16, 0): (64, 1, 2),
    (1, 3652, 3216, 0): (16, 2, 1), (17, 9723, 14064, 0): (32, 2, 2), (97, 3852, 2864, 0): (64, 2, 1),
    (17, 4098, 4096, 0): (32, 2, 1), (100, 4098, 4096, 0): (64, 2, 1), (49, 7376, 3888, 0): (64, 2, 1),
    (941, 1090, 3280, 0): (128, 2, 2), (230, 3624, 3952, 0): (80, 2, 2),
    (1, 1878, 2000, 0): (16, 4, 1), (1, 4992, 2672, 0): (16, 4, 2), (65, 2050, 2048, 0): (80, 4, 1),
    (1615, 8, 2240, 0): (208, 4, 1), (128, 2050, 2048, 0): (48, 4, 2), (200, 2050, 2048, 0): (80, 4, 2),
    (257, 1048, 1728, 0): (80, 4, 2), (128, 7168, 16384, 0): (128, 4, 2),
    (1, 9, 1536, 0): (16, 8, 1), (923, 9, 1264, 0): (160, 8, 1), (833, 8, 1312, 0): (144, 8, 1),
    (91, 9822, 16, 1): (32, 1, 2), (145, 9877, 16, 1): (64, 1, 2), (162, 9488, 16, 1): (64, 1, 2),
    (1, 3727, 5888, 1): (16, 2, 1), (100, 4022, 6544, 1): (64, 2, 1), (103, 4088, 5632, 1): (64, 2, 1),
    (197, 4833, 6288, 1): (112, 2, 2), (199, 4920, 6976, 1): (112, 2, 2),
    (1, 1850, 3888, 1): (16, 4, 1), (1, 4680, 4896, 1): (16, 4, 2), (1576, 9, 4928, 1): (208, 4, 1),
    (1665, 8, 4576, 1): (224, 4, 1), (262, 1066, 3312, 1): (80, 4, 2), (522, 544, 3328, 1): (80, 4, 2),
    (128, 7168, 16384, 1): (128, 4, 2),
    (1, 9, 3088, 1): (16, 8, 1), (824, 10, 2480, 1): (144, 8, 1), (789, 8, 2512, 1): (144, 8, 1),
}


@pytest.mark.parametrize("T,N,K,eight", sorted(SPLIT))
def test_few_token_variants_are_exact_on_integers(T, N, K, eight):
    """Sums of integers below 12 K < 2^18, and what the epilogue makes of them, have fewer than 24
    significant bits: exact in fp32 in any order, and the output is their one rounding."""
    for operands in (0, 2):
        assert mla.mla_debug_linear_choice(T, N, K, eight, operands) == (False, *SPLIT[T, N, K, eight])
    rng = np.random.default_rng(T + 31 * N + K)

    def ints(hi, *shape):
        return rng.integers(-hi, hi + 1, size=shape).astype(np.float64)
    x, W, bias, mul, res = ints(4, T, K), ints(3, N, K), ints(9, N), ints(3, T, N), ints(99, T, N)
    tb, tm, tr = bf16(bias), bf16(mul), bf16(res)
    if eight:
        kx, kw = rng.integers(-3, 4, size=T), rng.integers(-3, 4, size=N)
        tx, tw = (torch.from_numpy(fp8.e4m3_encode(a)).to(DEV) for a in (x, W))
        sx, sw = (torch.from_numpy((k + 127).astype(np.uint8)).to(DEV) for k in (kx, kw))
        x, W = np.ldexp(x, kx[:, None]), np.ldexp(W, kw[:, None])
    else:
        tx, tw = bf16(x), bf16(W)

    def run(bias, mul, res, out):
        if eight:
            mla.mla_linear_fp8(tx, sx, tw, sw, bias, mul, res, out, T, N, K, mla.MLA_ACT_NONE)
        else:
            mla.mla_linear(tx, tw, bias, mul, res, out, T, N, K, mla.MLA_ACT_NONE)
        torch.cuda.synchronize()
        mla.mla_check_status()
    whole = torch.full((T * N + 2 * GUARD,), 77, dtype=torch.bfloat16, device=DEV)
    out = whole[GUARD:-GUARD].view(T, N)
    sums = x @ W.T
    for b, m, r in ((None, None, None), (tb, tm, tr)):
        run(b, m, r, out)
        want = sums if b is None else res + mul * (sums + bias)
        want = orc.round_bf16(want)
        assert np.array_equal(host(out), want), f"{np.sum(host(out) != want)} of {want.size} differ"
        assert bool((whole[:GUARD] == 77).all()) and bool((whole[-GUARD:] == 77).all())
    for into in (tm, tr):      # out is mul's or the residual's own buffer
        own = into.clone()
        run(tb, own if into is tm else tm, own if into is tr else tr, own)
        assert np.array_equal(host(own), want)


def test_every_listed_kind_of_few_token_variant_is_reached():
    kinds = {(e, N % 8 == 0, nt > 48, slices, ctas) for (T, N, K, e), (nt, slices, ctas) in SPLIT.items()}
    assert len({k[0:1] + k[3:] for k in kinds}) >= 11 and {k[1:3] for k in kinds} == {(a, b) for a in (0, 1) for b in (0, 1)}


# ----------------------------------------------------------------------------- the streaming norm's other forms
@pytest.mark.parametrize("M", [1024, 7168])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual,outputs", [(False, "y"), (False, "both"), (False, "codes"), (True, "codes")])
def test_many_rows_without_a_residual_or_with_codes_alone(M, dtype, residual, outputs):
    T = 3000
    dt, name = (torch.bfloat16, mla.MLA_BF16) if dtype == "bf16" else (torch.float32, mla.MLA_F32)
    g = torch.Generator(device="cpu").manual_seed(M)
    x = torch.randn(T, M, generator=g).to(dt).to(DEV)
    r = torch.randn(T, M, generator=g).to(dt).to(DEV) if residual else None
    gain = (1 + 0.3 * torch.randn(M, generator=g)).to(dt).to(DEV)
    ro = torch.empty_like(x) if residual else None
    y = torch.empty_like(x) if outputs != "codes" else None
    codes = torch.empty(T, M, dtype=torch.uint8, device=DEV) if outputs != "y" else None
    scales = torch.empty(T, dtype=torch.uint8, device=DEV) if outputs != "y" else None
    if codes is None:
        mla.mla_add_rmsnorm(x, r, gain, ro, y, T, M, 1e-6, name)
    else:
        mla.mla_add_rmsnorm_fp8(x, r, gain, ro, y, codes, scales, T, M, 1e-6, name)
    torch.cuda.synchronize()
    mla.mla_check_status()
    s, ref = layer.add_rmsnorm(host(x), None if r is None else host(r), host(gain), 1e-6)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    if residual:
        assert np.all(np.abs(host(ro) - s) <= half * np.abs(s))
    if y is not None:
        assert np.all(np.abs(host(y) - ref) <= (half + STAT) * np.abs(ref) + 1e-30)
    if codes is not None:
        k = scales.cpu().numpy().astype(np.int64) - 127
        top = np.abs(ref).max(axis=1)
        assert np.all(top * (1 - STAT) <= np.ldexp(448.0, k)) and np.all(top * (1 + STAT) > np.ldexp(448.0, k - 1))
        got = fp8.dequantise_rows(codes.cpu().numpy(), scales.cpu().numpy())
        bound = np.maximum((2.0 ** -4 + STAT) * np.abs(ref), np.ldexp(1.0, k - 10)[:, None]) * (1 + STAT)
        assert np.all(np.abs(got - ref) <= bound)


# ----------------------------------------------------------------------------- offsets past 32 bits
def test_norm_rows_past_two_billion_elements():
    M, T = 7168, 300_007      # 2.15e9 elements
    x = torch.zeros(T, M, dtype=torch.bfloat16, device=DEV)
    y, codes = torch.empty_like(x), torch.empty(T, M, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, dtype=torch.uint8, device=DEV)
    rows = [0, 1, T // 2, T - 2, T - 1]
    x[rows] = torch.randn(len(rows), M, generator=torch.Generator(device="cpu").manual_seed(1)).to(torch.bfloat16).to(DEV)
    gain = torch.ones(M, dtype=torch.bfloat16, device=DEV)
    mla.mla_add_rmsnorm_fp8(x, None, gain, None, y, codes, scales, T, M, 1e-6, mla.MLA_BF16)
    torch.cuda.synchronize()
    ref = layer.add_rmsnorm(host(x[rows]), None, host(gain), 1e-6)[1]
    assert np.all(np.abs(host(y[rows]) - ref) <= (2.0 ** -8 + STAT) * np.abs(ref))
    got = fp8.dequantise_rows(codes[rows].cpu().numpy(), scales[rows].cpu().numpy())
    step = np.ldexp(1.0, scales[rows].cpu().numpy().astype(np.int64) - 127 - 10)[:, None]
    assert np.all(np.abs(got - ref) <= np.maximum((2.0 ** -4 + STAT) * np.abs(ref), step) * (1 + STAT))
    y[rows] = 0
    assert not bool(y.any())      # the rows of zeros


@pytest.mark.parametrize("N", [16384, 16390])
def test_projection_outputs_past_two_billion_elements(N):
    T, K = 140_003, 64
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(N)
    W, rows = rng.integers(-3, 4, size=(N, K)).astype(np.float64), [0, 777, T // 2, T - 20, T - 1]
    xr = rng.integers(-4, 5, size=(len(rows), K)).astype(np.float64)
    x[rows] = bf16(xr)
    out = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    mla.mla_linear(x, bf16(W), None, None, None, out, T, N, K, mla.MLA_ACT_NONE)
    torch.cuda.synchronize()
    mla.mla_check_status()
    assert np.array_equal(host(out[rows]), orc.round_bf16(xr @ W.T))
    out[rows] = 0
    assert not bool(out.any())


# ----------------------------------------------------------------------------- the layer step's output projection
@pytest.mark.parametrize("H,M,lens", [(64, 1024, [70, 64, 333]), (128, 7168, [40])])
@pytest.mark.parametrize("projections", ["bf16", "fp8"])
def test_layer_step_adds_its_output_projection(projections, H, M, lens):
    """y on what the run stored before it, element by element: K additions err by at most 2^-23 of the
    products' magnitudes each, the store by half a step. The residual alone must not pass."""
    spec = wl.WorkloadSpec(name="layer", B=0, H=H, R=512, Dr=64, Dn=128, Dv=128, q_len=1, dtype="bf16", seq_len=None,
                           w_std=1.0 / np.sqrt(512))
    st = dec.DecodeStep(wl.make(spec, seed=31, seq_lens=lens, new_rows_in_cache=False), sms=8)
    t = {k: dec.to_torch(v, st.device) for k, v in wl.layer_inputs(spec, st.T, M, seed=31, gate=False).items()}
    lay = dec.LayerStep(st, {k: v for k, v in t.items() if k not in ("x", "residual")}, projections=projections)
    lay.run(t["x"], t["residual"])
    torch.cuda.synchronize()
    mla.mla_check_status()
    o, W, r = host(st.out).reshape(st.T, -1), host(t["W_O"]), host(lay.residual)
    if projections == "fp8":
        codes, scales = fp8.quantise_rows(o)
        assert np.array_equal(lay.out_codes.cpu().numpy(), codes) and np.array_equal(lay.out_scales.cpu().numpy(), scales)
        o, W = fp8.dequantise_rows(codes, scales), fp8.dequantise_rows(*fp8.quantise_rows(W))
    ref = r + o @ W.T
    bound = (H * 128 + 2) * 2.0 ** -23 * (np.abs(o) @ np.abs(W).T) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * np.abs(r)
    err = np.abs(host(lay.y) - ref)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3f} of the bound"
    assert np.mean(np.abs(orc.round_bf16(r) - ref) > bound) > 0.5


# ----------------------------------------------------------------------------- activations of very negative sums
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_activations_vanish_where_their_exponential_does(act):
    """From 1 + e^-v = 2^126 on, v = -87.3, the quotient may be 0: sigmoid is below 1.2e-38 there and
    silu below 1.1e-36; above it both are within the store's half step and 2^-18."""
    v = wl.bf16_bits_to_f32(np.arange(0xC2A0, 0xC2DD, dtype=np.uint16)).astype(np.float64)      # -80 .. -110
    assert v[0] == -80 and v[-1] == -110
    x, W = np.zeros((len(v), 16)), np.zeros((8, 16))
    x[:, 2], W[:, 2] = v, 1
    out = torch.empty(len(v), 8, dtype=torch.bfloat16, device=DEV)
    code = {"sigmoid": mla.MLA_ACT_SIGMOID, "silu": mla.MLA_ACT_SILU}[act]
    mla.mla_linear(bf16(x), bf16(W), None, None, None, out, len(v), 8, 16, code)
    ref = layer.activation(v, act)[:, None]
    assert np.all(np.abs(host(out) - ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref) + {"sigmoid": 1.2e-38, "silu": 1.1e-36}[act])
