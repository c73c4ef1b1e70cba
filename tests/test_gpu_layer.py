"""GPU parity of the layer's operators around the attention with their fp64 oracle.

Tolerances, from the arithmetic. A store rounds by at most half a step: 2^-8 of the value in
bf16, 2^-24 in fp32, 2^-4 in E4M3 (or half its subnormal step, 2^-10 of the row's scale).
The norm's fp32 statistics: a sum of M squares in a tree of at most 16 terms a thread and 10
levels, halved by the square root, and five further roundings: below 2^-18 relative.
Projections: on integers whose sums stay below 2^24 every fp32 step is exact and the output
must equal the rounded exact value bit for bit; on random values K additions err by at most
2^-23 of sum |x w| each, an activation passes an error on by at most 1.13 times and adds
2^-20 of its value.
"""
import numpy as np
import pytest
import torch

import mla_latent_kv_46_b200 as mla
from mla_latent_kv_46_b200 import decoder as dec
from inputs import workloads as wl
from oracle import fp8, layer
from oracle import mla_oracle as orc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 64      # elements on either side of an output that must keep their value
STAT = 2.0 ** -18
ACT = {"none": mla.MLA_ACT_NONE, "sigmoid": mla.MLA_ACT_SIGMOID, "silu": mla.MLA_ACT_SILU, "gelu": mla.MLA_ACT_GELU}
POLICIES = {"auto": mla.MLA_POLICY_AUTO, "simt": mla.MLA_POLICY_SIMT}


@pytest.fixture(autouse=True)
def _reset():
    yield
    mla.mla_set_policy(mla.MLA_POLICY_AUTO)
    mla.mla_check_status()


def host(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A contiguous output tensor with guard elements before and after it. `shift`: the
    tensor starts that many elements past an aligned address."""

    def __init__(self, shape, dtype, shift=0):
        n = int(np.prod(shape))
        self.n, self.at = n, GUARD + shift
        self.whole = torch.full((n + 2 * GUARD + shift,), 77, dtype=dtype, device=DEV)
        self.t = self.whole[self.at:self.at + n].view(*shape)

    def check(self):
        assert bool((self.whole[:self.at] == 77).all()) and bool((self.whole[self.at + self.n:] == 77).all())


def shifted(t, shift):
    """t's values in a contiguous tensor that starts `shift` elements past an aligned address."""
    if shift == 0:
        return t
    whole = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    whole[shift:] = t.reshape(-1)
    return whole[shift:].view(t.shape)


# ----------------------------------------------------------------------------- residual add + RMS norm
def norm_inputs(T, M, dtype, seed=0, residual=True):
    g = torch.Generator(device="cpu").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.randn(T, M, generator=g).to(dt).to(DEV)
    loud = 1 + 20 * (torch.rand(M, generator=g) < 0.02)
    r = (torch.randn(T, M, generator=g) * loud).to(dt).to(DEV) if residual else None
    gain = (1 + 0.3 * torch.randn(M, generator=g)).to(dt).to(DEV)
    return x, r, gain


def check_rounded(got, ref, half, what):
    err = np.abs(got - ref)
    bound = (half + STAT) * np.abs(ref) + 1e-30
    assert np.all(err <= bound), f"{what}: worst {np.max(err / bound):.3f} of the bound"


def check_codes(codes, scales, y, what=""):
    """The scale is the smallest power of two the row fits (up to the statistics' error) and
    every code is the nearest to its value (within it)."""
    c, k = codes.cpu().numpy(), scales.cpu().numpy().astype(np.int64) - 127
    amax = np.abs(y).max(axis=1)
    assert np.all((amax * (1 - STAT) <= np.ldexp(448.0, k)) | (k == 7)), what
    assert np.all((amax * (1 + STAT) > np.ldexp(448.0, k - 1)) | (k == -126)), what
    val = fp8.dequantise_rows(c, (k + 127).astype(np.uint8))
    top = np.ldexp(448.0, k)[:, None]
    yc = np.clip(y, -top, top)
    bound = (2.0 ** -4 + STAT) * np.abs(yc) * (1 + STAT)
    bound = np.maximum(bound, np.ldexp(1.0, k - 10)[:, None] * (1 + STAT))
    assert np.all(np.abs(val - yc) <= bound), what


def run_norm(x, r, gain, T, M, dtype, codes, with_y=True, shift=0, eps=1e-6):
    dt = x.dtype
    dtype = mla.MLA_BF16 if dtype == "bf16" else mla.MLA_F32
    ro = Guarded((T, M), dt, shift) if r is not None else None
    y = Guarded((T, M), dt, shift) if with_y else None
    c = Guarded((T, M), torch.uint8, shift) if codes else None
    s = Guarded((T,), torch.uint8, shift) if codes else None
    t = lambda v: None if v is None else v.t  # noqa: E731
    if codes:
        mla.mla_add_rmsnorm_fp8(x, r, gain, t(ro), t(y), c.t, s.t, T, M, eps, dtype)
    else:
        mla.mla_add_rmsnorm(x, r, gain, t(ro), y.t, T, M, eps, dtype)
    torch.cuda.synchronize()
    for v in (ro, y, c, s):
        if v is not None:
            v.check()
    return t(ro), t(y), t(c), t(s)


NORM_SHAPES = [(1, 1), (17, 1), (9, 3), (40, 5), (3, 2), (2, 8), (5, 31), (1, 64), (7, 96), (33, 255), (9, 256), (5, 257), (4, 512), (3, 1000),
               (2, 1111), (129, 1536), (2, 4100), (1, 7168), (150, 7168), (2, 8192), (2, 8200), (3, 12290), (1, 16384),
               (2, 16385), (1, 20000), (1, 40001),
               # many rows: the streaming kernel, with rows that are not a multiple of 16 bytes too
               (1200, 7168), (1111, 7161), (8000, 1030), (3001, 2049), (3000, 4100), (500, 16379), (9001, 1024)]


@pytest.mark.parametrize("codes", [False, True], ids=["plain", "codes"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,M", NORM_SHAPES)
def test_add_rmsnorm_matches_oracle(T, M, dtype, codes):
    x, r, gain = norm_inputs(T, M, dtype, seed=T + M)
    ro, y, c, s = run_norm(x, r, gain, T, M, dtype, codes)
    ref_s, ref_y = layer.add_rmsnorm(host(x), host(r), host(gain), 1e-6)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    check_rounded(host(ro), ref_s, half, "residual")
    check_rounded(host(y), ref_y, half, "y")
    if codes:
        check_codes(c, s, ref_y)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_add_rmsnorm_at_any_alignment(dtype, shift):
    T, M = 5, 520
    x, r, gain = norm_inputs(T, M, dtype, seed=shift)
    ro, y, c, s = run_norm(shifted(x, shift), shifted(r, shift), shifted(gain, shift), T, M, dtype, True, shift=shift)
    a_ro, a_y, a_c, a_s = run_norm(x, r, gain, T, M, dtype, True)
    ref_s, ref_y = layer.add_rmsnorm(host(x), host(r), host(gain), 1e-6)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    check_rounded(host(ro), ref_s, half, "residual")
    check_rounded(host(y), ref_y, half, "y")
    check_codes(c, s, ref_y)
    assert torch.equal(ro, a_ro)


@pytest.mark.parametrize("T,M", [(3, 200), (2, 7168), (2, 16400)])
def test_add_rmsnorm_without_residual_and_codes_alone(T, M):
    x, _, gain = norm_inputs(T, M, "bf16", seed=9, residual=False)
    _, y, c, s = run_norm(x, None, gain, T, M, "bf16", True, with_y=False)
    assert y is None
    check_codes(c, s, layer.add_rmsnorm(host(x), None, host(gain), 1e-6)[1])


@pytest.mark.parametrize("M", [96, 1111, 7168, 20000])
def test_add_rmsnorm_in_place(M):
    """residual_out on residual and out on x, and the two swapped: bitwise the same."""
    T = 6
    x, r, gain = norm_inputs(T, M, "bf16", seed=M)
    ro, y, _, _ = run_norm(x, r, gain, T, M, "bf16", False)
    a, b = x.clone(), r.clone()
    mla.mla_add_rmsnorm(a, b, gain, b, a, T, M, 1e-6, mla.MLA_BF16)
    assert torch.equal(a, y) and torch.equal(b, ro)
    a, b = x.clone(), r.clone()
    mla.mla_add_rmsnorm(a, b, gain, a, b, T, M, 1e-6, mla.MLA_BF16)
    assert torch.equal(a, ro) and torch.equal(b, y)


@pytest.mark.parametrize("M", [64, 1111, 7168, 20000])
def test_add_rmsnorm_special_rows(M):
    """Zero rows, tiny and huge rows, and rows with an infinity or a NaN: no other row moves."""
    x, r, gain = norm_inputs(8, M, "f32", seed=4)
    _, base, bc, bs = run_norm(x, r, gain, 8, M, "f32", True)
    x2, r2 = x.clone(), r.clone()
    x2[1], r2[1] = 0, 0
    x2[2, M // 2] = float("inf")
    x2[3, M - 1] = float("nan")
    x2[4], r2[4] = x[4] * 1e-20, 0
    x2[5], r2[5] = x[5] * 1e15, 0
    ro, y, c, s = run_norm(x2, r2, gain, 8, M, "f32", True)
    for row in (0, 6, 7):
        assert torch.equal(y[row], base[row]) and torch.equal(c[row], bc[row]) and s[row] == bs[row]
    assert bool((y[1] == 0).all()) and bool(((c[1] & 0x7F) == 0).all()) and s[1] == 1
    want = torch.zeros(M, device=DEV)
    want[M // 2] = float("nan")        # inf / inf; the others finite / inf
    assert torch.equal(torch.isnan(y[2]), torch.isnan(want)) and bool((y[2][~torch.isnan(want)] == 0).all())
    assert bool(torch.isnan(y[3]).all())
    assert bool(((c[3] & 0x7F) == 0x7F).all())
    ref = layer.add_rmsnorm(host(x2[4:6]), host(r2[4:6]), host(gain), 1e-6)[1]
    check_rounded(host(y[4:6]), ref, 2.0 ** -24, "y")
    check_codes(c[4:6], s[4:6], ref)


@pytest.mark.parametrize("M", [7168, 7163])
def test_add_rmsnorm_many_rows_in_place_and_with_special_rows(M):
    """The streaming kernel: outputs on their inputs' buffers, and rows with a NaN or an infinity
    beside rows that share a 16-byte piece with them."""
    T = 1300
    x, r, gain = norm_inputs(T, M, "bf16", seed=M)
    ro, y, c, s = run_norm(x, r, gain, T, M, "bf16", True)
    a, b = x.clone(), r.clone()
    mla.mla_add_rmsnorm(a, b, gain, b, a, T, M, 1e-6, mla.MLA_BF16)
    assert torch.equal(a, y) and torch.equal(b, ro)
    x2 = x.clone()
    x2[5, 0] = float("nan")
    x2[5, M - 1] = float("inf")
    x2[T - 1, M - 1] = float("inf")
    ro2, y2, c2, s2 = run_norm(x2, r, gain, T, M, "bf16", True)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[5, T - 1]] = False
    assert torch.equal(y2[keep], y[keep]) and torch.equal(c2[keep], c[keep]) and torch.equal(s2[keep.to(DEV)], s[keep.to(DEV)])
    assert bool(torch.isnan(y2[5]).all()) and bool(torch.isnan(y2[T - 1, M - 1])) and bool((y2[T - 1, :M - 1] == 0).all())


def test_add_rmsnorm_zero_row_without_eps_is_nan():
    x, _, gain = norm_inputs(2, 64, "bf16", residual=False)
    x[0] = 0
    _, y, _, _ = run_norm(x, None, gain, 2, 64, "bf16", False, eps=0.0)
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isfinite(y[1]).all())


# ----------------------------------------------------------------------------- the quantiser
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,width", [(1, 1), (3, 17), (9, 576), (5, 1000), (2, 7168), (2, 16383), (1, 33000)])
def test_quantize_fp8_is_bit_exact(n, width, dtype):
    """No arithmetic but the scaling by a power of two comes before the rounding, so codes and
    scale bytes equal the oracle's for every row, tiny, huge and tied values among them."""
    rng = np.random.default_rng(width)
    rows = rng.standard_normal((n, width)) * np.ldexp(1.0, rng.integers(-30, 12, size=(n, 1)))
    rows[:, ::7] = np.ldexp(np.round(np.ldexp(rows[:, ::7], 6)) + 0.5, -6)
    t = torch.from_numpy(rows).to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(DEV)
    c, s = Guarded((n, width), torch.uint8), Guarded((n,), torch.uint8)
    mla.mla_quantize_fp8(t, c.t, s.t, n, width, mla.MLA_BF16 if dtype == "bf16" else mla.MLA_F32)
    torch.cuda.synchronize()
    want_c, want_s = fp8.quantise_rows(host(t))
    assert np.array_equal(s.t.cpu().numpy(), want_s)
    assert np.array_equal(c.t.cpu().numpy(), want_c)
    c.check(), s.check()


def test_quantize_fp8_boundaries_and_special_rows():
    tiny = 2.0 ** -126 * 448
    rows = torch.tensor([[448.0, 1], [448.0 * 1.001, 1], [0.0, -0.0], [tiny, 0], [tiny / 64, 0], [448.0 * 128, 1],
                         [448.0 * 200, 1], [float("inf"), 1.0], [float("nan"), 3.0], [0.875, 0.4375]],
                        dtype=torch.float32, device=DEV)
    n = rows.shape[0]
    c = torch.zeros(n, 2, dtype=torch.uint8, device=DEV)
    s = torch.zeros(n, dtype=torch.uint8, device=DEV)
    mla.mla_quantize_fp8(rows, c, s, n, 2, mla.MLA_F32)
    finite = [0, 1, 2, 3, 4, 5, 6, 9]
    want_c, want_s = fp8.quantise_rows(host(rows)[finite])
    assert np.array_equal(s.cpu().numpy()[finite], want_s)
    assert np.array_equal(c.cpu().numpy()[finite], want_c)
    assert s[7] == 134 and c[7, 0] == 0x7E          # an infinity saturates at the largest scale
    assert (c[8, 0] & 0x7F) == 0x7F and s[8] == fp8.quantise_rows(np.array([[3.0]]))[1][0]


# ----------------------------------------------------------------------------- projections
def ints(rng, lo, hi, *shape):
    return rng.integers(lo, hi + 1, size=shape).astype(np.float64)


def bf16(a):
    return torch.from_numpy(a).to(torch.bfloat16).to(DEV)


def run_linear(x, W, bias, mul, res, T, N, K, act="none", scales=None, shift=0):
    out = Guarded((T, N), torch.bfloat16, shift)
    if scales is None:
        mla.mla_linear(x, W, bias, mul, res, out.t, T, N, K, ACT[act])
    else:
        mla.mla_linear_fp8(x, scales[0], W, scales[1], bias, mul, res, out.t, T, N, K, ACT[act])
    torch.cuda.synchronize()
    mla.mla_check_status()
    out.check()
    return out.t


LIN_SHAPES = [(1, 1, 1), (1, 8, 16), (1, 128, 64), (2, 129, 72), (1, 300, 4096), (3, 1000, 1111), (15, 64, 80),
              (16, 256, 512), (17, 127, 1008), (31, 1111, 328), (33, 130, 2048), (64, 640, 576), (65, 257, 1000),
              (127, 200, 96), (128, 512, 4096), (129, 385, 640), (200, 136, 16), (255, 128, 208), (256, 1024, 1024),
              (257, 1025, 520), (300, 77, 33), (511, 513, 1104), (777, 1111, 1000), (1030, 900, 64), (2500, 300, 264),
              (5001, 1300, 144)]      # the last: more 256 x 256 tiles than pairs of SMs


def exact_case(T, N, K, eight, epilogue, policy, shift=0):
    rng = np.random.default_rng(T * 7919 + N * 31 + K)
    x, W = ints(rng, -4, 4, T, K), ints(rng, -3, 3, N, K)
    bias = ints(rng, -9, 9, N) if epilogue else None
    mul = ints(rng, -3, 3, T, N) if epilogue else None
    res = ints(rng, -99, 99, T, N) if epilogue else None
    dev = lambda a: None if a is None else shifted(bf16(a), shift)  # noqa: E731
    mla.mla_set_policy(POLICIES[policy])
    if eight:
        kx, kw = rng.integers(-3, 4, size=T), rng.integers(-3, 4, size=N)
        code = lambda a: shifted(torch.from_numpy(fp8.e4m3_encode(a)).to(DEV), shift)  # noqa: E731
        byte = lambda k: shifted(torch.from_numpy((k + 127).astype(np.uint8)).to(DEV), shift)  # noqa: E731
        got = run_linear(code(x), code(W), dev(bias), dev(mul), dev(res), T, N, K, scales=(byte(kx), byte(kw)),
                         shift=shift)
        x, W = np.ldexp(x, kx[:, None]), np.ldexp(W, kw[:, None])
    else:
        got = run_linear(dev(x), dev(W), dev(bias), dev(mul), dev(res), T, N, K, shift=shift)
    # the products' sum is an integer below 12 K < 2^16 (times a power of two), and what the
    # epilogue makes of it has fewer than 24 significant bits: exact in fp32
    want = orc.round_bf16(layer.linear(x, W, bias, mul, res))
    assert np.array_equal(host(got), want), f"{np.sum(host(got) != want)} of {want.size} differ"


@pytest.mark.parametrize("epilogue", [False, True], ids=["bare", "epilogue"])
@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,N,K", LIN_SHAPES)
def test_linear_is_exact_on_integers(T, N, K, eight, epilogue):
    exact_case(T, N, K, eight, epilogue, "auto")


@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,N,K", [(1, 128, 64), (65, 257, 1000), (130, 70, 48)])
def test_linear_on_cuda_cores_is_exact_on_integers(T, N, K, eight):
    exact_case(T, N, K, eight, True, "simt")


@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shift", [1, 8])
def test_linear_at_any_alignment(shift, eight):
    exact_case(33, 130, 144, eight, True, "auto", shift=shift)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,N,K", [(1, 300, 512), (37, 129, 1000), (200, 257, 640), (600, 520, 1024)])
def test_linear_matches_oracle_on_random_values(T, N, K, eight, act):
    rng = np.random.default_rng(T + N + K)
    x, W = rng.standard_normal((T, K)), rng.standard_normal((N, K)) * 2 / np.sqrt(K)
    bias, mul, res = bf16(rng.standard_normal(N)), bf16(rng.standard_normal((T, N))), bf16(rng.standard_normal((T, N)))
    if eight:
        (cx, sx), (cw, sw) = fp8.quantise_rows(x), fp8.quantise_rows(W)
        t = [torch.from_numpy(a).to(DEV) for a in (cx, sx, cw, sw)]
        got = run_linear(t[0], t[2], bias, mul, res, T, N, K, act, scales=(t[1], t[3]))
        x, W = fp8.dequantise_rows(cx, sx), fp8.dequantise_rows(cw, sw)
    else:
        xb, Wb = bf16(x), bf16(W)
        got = run_linear(xb, Wb, bias, mul, res, T, N, K, act)
        x, W = host(xb), host(Wb)
    b, m, r = host(bias), host(mul), host(res)
    ref = layer.linear(x, W, b, m, r, act)
    acc = (K + 2) * 2.0 ** -23 * (np.abs(x) @ np.abs(W).T + np.abs(b))
    part = np.abs(m) * (1.13 * acc + 2.0 ** -20 * np.abs(layer.activation(x @ W.T + b, act)))
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (part + 2.0 ** -22 * np.abs(r)) + 1e-30
    err = np.abs(host(got) - ref)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3f} of the bound"


@pytest.mark.parametrize("T,N,K", [(5, 200, 512), (300, 520, 640)])
def test_linear_in_place_on_its_residual_and_on_mul(T, N, K):
    rng = np.random.default_rng(5)
    x, W, m, r = (bf16(rng.standard_normal(s)) for s in ((T, K), (N, K), (T, N), (T, N)))
    want = run_linear(x, W, None, m, r, T, N, K, "sigmoid")
    a = r.clone()
    mla.mla_linear(x, W, None, m, a, a, T, N, K, mla.MLA_ACT_SIGMOID)
    b = m.clone()
    mla.mla_linear(x, W, None, b, r, b, T, N, K, mla.MLA_ACT_SIGMOID)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


# many tokens and rows of whole 16-byte pieces: features that end inside a warp's 32, tokens that end
# inside a piece of 8 and a sweep of 32, tiles for every pair of SMs and more
WIDE_SHAPES = [(2049, 8, 16), (2060, 40, 64), (2500, 304, 272), (3007, 136, 1008), (4101, 2568, 64), (5001, 1304, 144)]


@pytest.mark.parametrize("operands", ["bare", "bias", "mul", "res", "mul res", "bias mul res"])
@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,N,K", WIDE_SHAPES)
def test_linear_of_many_tokens_is_exact_with_any_operands(T, N, K, eight, operands):
    rng = np.random.default_rng(T + 31 * N + K)
    x, W = ints(rng, -4, 4, T, K), ints(rng, -3, 3, N, K)
    bias = ints(rng, -9, 9, N) if "bias" in operands else None
    mul = ints(rng, -3, 3, T, N) if "mul" in operands else None
    res = ints(rng, -99, 99, T, N) if "res" in operands else None
    dev = lambda a: None if a is None else bf16(a)  # noqa: E731
    scales = None
    tx, tw = bf16(x), bf16(W)
    if eight:
        kx, kw = rng.integers(-3, 4, size=T), rng.integers(-3, 4, size=N)
        tx, tw = (torch.from_numpy(fp8.e4m3_encode(a)).to(DEV) for a in (x, W))
        scales = tuple(torch.from_numpy((k + 127).astype(np.uint8)).to(DEV) for k in (kx, kw))
        x, W = np.ldexp(x, kx[:, None]), np.ldexp(W, kw[:, None])
    want = orc.round_bf16(layer.linear(x, W, bias, mul, res))      # exact in fp32, as above
    got = run_linear(tx, tw, dev(bias), dev(mul), dev(res), T, N, K, scales=scales)
    assert np.array_equal(host(got), want), f"{np.sum(host(got) != want)} of {want.size} differ"
    for into in ("mul", "res"):      # out is the operand's own buffer
        if into in operands:
            m, r = dev(mul), dev(res)
            out = m if into == "mul" else r
            if eight:
                mla.mla_linear_fp8(tx, scales[0], tw, scales[1], dev(bias), m, r, out, T, N, K, mla.MLA_ACT_NONE)
            else:
                mla.mla_linear(tx, tw, dev(bias), m, r, out, T, N, K, mla.MLA_ACT_NONE)
            torch.cuda.synchronize()
            assert np.array_equal(host(out), want), into


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("N", [264, 259])
def test_linear_of_many_tokens_applies_the_activation_to_the_sum(N, act):
    """The same sums by themselves and in front of mul and residual, with 16-byte rows and without."""
    rng = np.random.default_rng(N)
    T, K = 2077, 64
    x, W = rng.standard_normal((T, K)), rng.standard_normal((N, K)) / 4
    xb, Wb = bf16(x), bf16(W)
    bias, mul, res = bf16(rng.standard_normal(N)), bf16(rng.standard_normal((T, N))), bf16(rng.standard_normal((T, N)))
    b, m, r = host(bias), host(mul), host(res)
    x, W = host(xb), host(Wb)
    got = run_linear(xb, Wb, bias, mul, res, T, N, K, act)
    ref = layer.linear(x, W, b, m, r, act)
    acc = (K + 2) * 2.0 ** -23 * (np.abs(x) @ np.abs(W).T + np.abs(b))
    part = np.abs(m) * (1.13 * acc + 2.0 ** -20 * np.abs(layer.activation(x @ W.T + b, act)))
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (part + 2.0 ** -22 * np.abs(r)) + 1e-30
    assert np.all(np.abs(host(got) - ref) <= bound)


@pytest.mark.parametrize("T,N,K", [(3, 140, 256), (260, 140, 256)])
def test_linear_keeps_a_rows_nan_and_infinity_in_that_row(T, N, K):
    rng = np.random.default_rng(6)
    x, W = bf16(rng.standard_normal((T, K))), bf16(rng.standard_normal((N, K)))
    want = run_linear(x, W, None, None, None, T, N, K)
    y = x.clone()
    y[1, 3] = float("nan")
    y[2, K - 1] = float("inf")
    got = run_linear(y, W, None, None, None, T, N, K)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[2]).any())


@pytest.mark.parametrize("act,lo,hi", [("sigmoid", 0.0, 1.0), ("silu", 0.0, 3e4), ("gelu", 0.0, 3e4)])
def test_linear_activations_at_their_ends(act, lo, hi):
    """Sums of -30000 and +30000: no overflow, no NaN."""
    x = bf16(np.array([[-3e4], [3e4]] * 1).repeat(16, axis=1) / 16)
    W = bf16(np.ones((8, 16)))
    got = host(run_linear(x, W, None, None, None, 2, 8, 16, act))
    v = float(bf16(np.array([3e4 / 16]))[0]) * 16
    assert np.all(got[0] == lo) and np.all(np.abs(got[1] - (1.0 if act == "sigmoid" else v)) <= 2.0 ** -8 * v)


@pytest.mark.parametrize("T", [100, 0], ids=["few", "all"])
@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
def test_linear_activations_over_their_range(act, T):
    """Every bf16 value of magnitude 2^-10 .. 20 as a sum by itself: the activation's own error. The
    exponential's argument is off by at most 2^-24 of its size (20), its approximation and the
    quotient's by 2^-22: below 2^-18 together, on top of the store's half step."""
    bits = np.arange(0x3A80, 0x41A1, dtype=np.uint16)
    v = wl.bf16_bits_to_f32(np.concatenate([bits, bits | 0x8000])).astype(np.float64)
    v = v[::len(v) // T][:T] if T else v
    x = np.zeros((len(v), 16))
    x[:, 3] = v
    W = np.zeros((8, 16))
    W[:, 3] = 1
    got = host(run_linear(bf16(x), bf16(W), None, None, None, len(v), 8, 16, act))
    ref = layer.activation(v, act)[:, None]
    # half a step of the binade the value lies in
    half = np.ldexp(1.0, np.frexp(np.abs(ref))[1] - 9)
    assert np.all(np.abs(got - ref) <= half * (1 + 2.0 ** -8) + 2.0 ** -18 * np.abs(ref) + 1e-38)


def test_two_runs_are_bitwise_equal():
    rng = np.random.default_rng(8)
    for T, N, K in ((1, 7168, 2048), (37, 2000, 4096), (700, 1111, 1000)):
        x, W = bf16(rng.standard_normal((T, K))), bf16(rng.standard_normal((N, K)))
        a = run_linear(x, W, None, None, None, T, N, K)
        assert torch.equal(a, run_linear(x, W, None, None, None, T, N, K))


# ----------------------------------------------------------------------------- a layer's step, all of it
def layer_case(H, q_len, lens, M, projections, gate, seed=21):
    spec = wl.WorkloadSpec(name="layer", B=0, H=H, R=512, Dr=64, Dn=128, Dv=128, q_len=q_len, dtype="bf16",
                           seq_len=None, w_std=1.0 / np.sqrt(512))
    w = wl.make(spec, seed=seed, seq_lens=lens, new_rows_in_cache=False)
    st = dec.DecodeStep(w, sms=8)
    pin = wl.layer_inputs(spec, st.T, M, seed=seed, gate=gate)
    t = {k: dec.to_torch(v, st.device) for k, v in pin.items()}
    lay = dec.LayerStep(st, {k: v for k, v in t.items() if k not in ("x", "residual")}, projections=projections)
    return spec, w, st, t, lay


def near(got, ref, terms, what):
    """bf16 output of an fp32 sum of `terms` products whose operands are exact: half a step,
    and 2^-23 of the sum of magnitudes per addition (bounded by terms times the largest output)."""
    bound = 2.0 ** -8 * np.abs(ref) + terms * 2.0 ** -23 * max(1.0, np.abs(ref).max()) * np.sqrt(terms)
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{what}: worst {np.max(err / bound):.3f} of the bound"


@pytest.mark.parametrize("projections,gate,H,q_len,lens,M", [
    ("bf16", True, 64, 1, [70, 5, 129, 1], 1024), ("fp8", True, 64, 1, [70, 64, 333], 1024),
    ("bf16", False, 128, 2, [130, 2, 65], 576), ("fp8", False, 128, 1, [40], 7168)])
def test_layer_step_matches_the_oracle_stage_by_stage(projections, gate, H, q_len, lens, M):
    """The run as a layer uses it: norm, query projections, cache write, attention, gate, Wo.
    Every stage against the oracle on the values that the stage before it stored."""
    spec, w, st, t, lay = layer_case(H, q_len, lens, M, projections, gate)
    lay.norm_and_queries(t["x"], t["residual"])
    ref_s, ref_h = layer.add_rmsnorm(host(t["x"]), host(t["residual"]), host(t["gain"]), 1e-6)
    check_rounded(host(lay.residual), ref_s, 2.0 ** -8, "residual")
    check_rounded(host(lay.hidden), ref_h, 2.0 ** -8, "hidden")

    def weight(name):
        if projections == "bf16":
            return host(t[name])
        c, s = (v.cpu().numpy() for v in lay.w8[name])
        want_c, want_s = fp8.quantise_rows(host(t[name]))
        assert np.array_equal(c, want_c) and np.array_equal(s, want_s)
        return fp8.dequantise_rows(c, s)
    if projections == "fp8":
        check_codes(lay.codes, lay.scales, ref_h)
        hid = fp8.dequantise_rows(lay.codes.cpu().numpy(), lay.scales.cpu().numpy())
    else:
        hid = host(lay.hidden)
    T = st.T
    near(host(st.q_nope).reshape(T, -1), layer.linear(hid, weight("W_QN")), M, "q_nope")
    near(host(st.q_rope).reshape(T, -1), layer.linear(hid, weight("W_QR")), M, "q_rope")
    q_rope = host(st.q_rope)
    lay.cache_write()
    pos = orc.token_positions(lens, q_len)
    rows = orc.cache_write_rows(host(lay.hidden), host(t["W_DKV"]), host(t["kv_gain"]), pos, spec.R, eps=1e-6)
    kv = host(st.kv)
    for i, p in enumerate(pos):
        row = kv[int(w["block_table"][i // q_len][p // 64]), p % 64]
        assert np.all(np.abs(row - rows[i]) <= 2e-3 + 1e-2 * np.abs(rows[i]))
    turned = orc.rope(q_rope, pos[:, None])
    assert np.all(np.abs(host(st.q_rope) - turned) <= 2e-3 + 1e-2 * np.abs(turned))
    st.run(append=False)
    ref = orc.decode_absorbed(host(st.q_nope), host(st.q_rope), kv, w["block_table"], np.asarray(lens), host(st.W_UK),
                              host(st.W_UV), spec.scale, q_len=q_len, intermediates="q_lat")["out"]
    att = host(st.out)
    assert np.all(np.abs(att - ref.reshape(att.shape)) <= 2e-3 + 1e-2 * np.abs(ref.reshape(att.shape)))
    lay.gate_and_output()
    mla.mla_check_status()
    if gate:
        want = layer.linear(hid, weight("W_G"), mul=att.reshape(T, -1), act="sigmoid")
        near(host(st.out).reshape(T, -1), want, M, "gate")
    o = host(st.out).reshape(T, -1)
    if projections == "fp8":
        want_c, want_s = fp8.quantise_rows(o)
        assert np.array_equal(lay.out_codes.cpu().numpy(), want_c)
        o = fp8.dequantise_rows(want_c, want_s)
    near(host(lay.y), layer.linear(o, weight("W_O"), residual=host(lay.residual)), H * 128, "y")


@pytest.mark.parametrize("projections", ["bf16", "fp8"])
def test_layer_step_replays_from_a_graph(projections):
    """One captured step replayed twice equals the eager one bitwise, with new inputs in the same
    buffers the second time."""
    spec, w, st, t, lay = layer_case(64, 1, [70, 5, 129, 1], 1024, projections, True)
    x, res = t["x"].clone(), t["residual"].clone()
    kv0 = st.kv.clone()

    def eager(a, b):
        st.kv.copy_(kv0)
        return lay.run(a, b).clone(), st.kv.clone()
    want1 = eager(t["x"], t["residual"])
    want2 = eager(t["residual"], t["x"] * 2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.run(x, res)
    for a, b, want in ((t["x"], t["residual"], want1), (t["residual"], t["x"] * 2, want2)):
        x.copy_(a)
        res.copy_(b)
        st.kv.copy_(kv0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.y, want[0]) and torch.equal(st.kv, want[1])


def test_layer_step_refuses_the_8_bit_cache():
    spec = wl.WorkloadSpec(name="layer8", B=0, H=64, R=512, Dr=64, Dn=128, Dv=128, q_len=1, dtype="bf16", seq_len=None,
                           w_std=1.0 / np.sqrt(512))
    st = dec.DecodeStep(wl.make(spec, seed=1, seq_lens=[5]), cache="fp8")
    with pytest.raises(ValueError):
        dec.LayerStep(st, {"gain": torch.ones(64, device=DEV)})


def test_layer_step_runs_on_a_stream_other_than_its_constructors():
    """The 8-bit weights are whole when the constructor returns, though its stream had work queued."""
    spec, w, st, t, lay = layer_case(64, 1, [70, 5, 129, 1], 1024, "fp8", True)
    kv0 = st.kv.clone()
    want = lay.run(t["x"], t["residual"]).clone()
    st.kv.copy_(kv0)
    weights = {k: v for k, v in t.items() if k not in ("x", "residual")}
    busy = bf16(np.ones((8192, 8192)))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(busy, busy)
    again = dec.LayerStep(st, weights, projections="fp8")
    with torch.cuda.stream(other):
        got = again.run(t["x"], t["residual"], stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ----------------------------------------------------------------------------- streams
def test_calls_on_two_streams_at_once():
    """No workspace and no state is shared: calls that overlap on the GPU give what they give alone."""
    rng = np.random.default_rng(12)
    jobs = []
    for T, N, K in ((5, 2000, 4096), (900, 1111, 1000), (130, 4096, 2048), (2000, 700, 512)):
        x, W, r = (bf16(rng.standard_normal(s)) for s in ((T, K), (N, K), (T, N)))
        jobs.append((x, W, r, T, N, K, run_linear(x, W, None, None, r, T, N, K, "silu")))
    xs, rs, gain = norm_inputs(1500, 7168, "bf16", seed=3)
    want_ro, want_y, _, _ = run_norm(xs, rs, gain, 1500, 7168, "bf16", False)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for i, (x, W, r, T, N, K, _) in enumerate(jobs):
            o = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
            outs.append(o)
            mla.mla_linear(x, W, None, None, r, o, T, N, K, mla.MLA_ACT_SILU, stream=streams[i % 2])
        ro, y = torch.empty_like(xs), torch.empty_like(xs)
        mla.mla_add_rmsnorm(xs, rs, gain, ro, y, 1500, 7168, 1e-6, mla.MLA_BF16, stream=streams[2])
        torch.cuda.synchronize()
        for o, j in zip(outs, jobs):
            assert torch.equal(o, j[6])
        assert torch.equal(ro, want_ro) and torch.equal(y, want_y)


def test_dependent_calls_in_a_row():
    """Back-to-back calls where each reads what the one before it wrote (their launches overlap:
    the second kernel may start before the first has ended), and overwrites what it read."""
    rng = np.random.default_rng(13)
    T, M = 64, 1024
    x, r = bf16(rng.standard_normal((T, M))), bf16(rng.standard_normal((T, M)))
    gain, W = bf16(1 + 0.1 * rng.standard_normal(M)), bf16(rng.standard_normal((M, M)) / 32)

    def chain(sync):
        a, b = x.clone(), r.clone()
        h, y = torch.empty_like(x), torch.empty_like(x)
        for _ in range(40):
            mla.mla_add_rmsnorm(a, b, gain, b, h, T, M, 1e-6, mla.MLA_BF16)
            if sync:
                torch.cuda.synchronize()
            mla.mla_linear(h, W, None, None, None, y, T, M, M, mla.MLA_ACT_SILU)
            if sync:
                torch.cuda.synchronize()
            mla.mla_linear(y, W, None, None, h, a, T, M, M, mla.MLA_ACT_NONE)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return a, b
    want = chain(True)
    for _ in range(5):
        got = chain(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
