"""Timed cases of the layer's operators around the latent attention: the residual stream's
RMS norm (bf16, fp32 or 8-bit output) and the projections with their fused epilogue.

    s = x + r,  y = s g / sqrt(mean(s^2) + eps)          mla_add_rmsnorm, mla_add_rmsnorm_fp8
    out = residual + mul * act(x W^T + bias)              mla_linear, mla_linear_fp8

An 8-bit row is E4M3 codes and one power-of-two scale 2^k, stored as the byte k + 127, with k
the smallest integer in [-126, 7] for which max |y| <= 448 2^k.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
WIDTH = 7168            # hidden width of the benchmark's cache-write prologue
PREFILL = 4 * 4096      # tokens of the benchmark's prefill batch
Q128, Q64 = 128 * 128, 64 * 128   # query content widths at 128 and 64 heads
LARGEST_NORM = PREFILL * WIDTH
LARGEST_LINEAR = PREFILL * Q64 * WIDTH
ACTS = ("none", "sigmoid", "silu", "gelu")


def norm(name, T, M, dtype="bf16", out="bf16", residual=True):
    return {"name": name, "op": "norm", "T": T, "M": M, "dtype": dtype, "out": out, "residual": residual}


def linear(name, T, N, K, dtype="bf16", act="none", bias=False, mul=False, residual=False):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias, "mul": mul,
            "residual": residual}


def listed():
    return [
        # one new token of one sequence: what counts is the call's latency
        norm("norm_token", 1, WIDTH),
        # a decode batch whose query projections run in 8 bits while the cache write takes bf16
        norm("norm_batch_both", 128, WIDTH, out="both"),
        # a prefill's rows, in and out in bf16 / out in 8 bits only
        norm("norm_prefill", PREFILL, WIDTH),
        norm("norm_prefill_fp8", PREFILL, WIDTH, out="fp8"),
        # an odd width in fp32 without a residual (no row but the first is aligned)
        norm("norm_odd_f32", 4097, 1111, dtype="f32", out="f32", residual=False),
        # the content queries of one token: 128 heads' weights streamed for one row
        linear("query_token", 1, Q128, WIDTH),
        linear("query_token_fp8", 1, Q128, WIDTH, dtype="fp8"),
        # the output projection of a decode batch, added to the residual stream
        linear("out_batch", 128, WIDTH, Q128, residual=True),
        # the output gate of a ragged batch: sigmoid(x Wg^T) times the attention's output
        linear("gate_ragged", 131, Q128, WIDTH, act="sigmoid", mul=True),
        # every epilogue input at odd sizes (nothing divides a tile)
        linear("odd_full_epilogue", 777, 1111, 1000, act="silu", bias=True, mul=True, residual=True),
        # a prefill's query projection at 64 heads
        linear("query_prefill", PREFILL, Q64, WIDTH, bias=True),
        linear("query_prefill_fp8", PREFILL, Q64, WIDTH, dtype="fp8", bias=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(step, min(hi, int(v)) // step * step)


def draw(rng):
    if rng.random() < 0.4:
        T, M = _log_int(rng, 1, PREFILL), _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            M = max(8, M // 8 * 8)
        T = max(1, min(T, LARGEST_NORM // M // 2))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        out = rng.choice((dtype, "fp8", "both"))
        return norm("", T, M, dtype=dtype, out=out, residual=rng.random() < 0.7) | {"name": "norm"}
    T, N = _log_int(rng, 1, PREFILL), _log_int(rng, 64, 16384)
    K = _log_int(rng, 64, 16384, 16)
    T = max(1, min(T, LARGEST_LINEAR // (N * K)))
    return linear("linear", T, N, K, dtype=rng.choice(("bf16", "fp8")), act=rng.choice(ACTS), bias=rng.random() < 0.5,
                  mul=rng.random() < 0.4, residual=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _pow2(k):
    """2^k in fp32, exactly, for integers k in [-126, 127]."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(y):
    """Codes and scale bytes of the rows of y (fp32)."""
    amax = y.abs().amax(dim=1)
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 7)
    k = torch.where(amax > 0, k, torch.full_like(k, -126)).to(torch.int32)
    codes = (y * _pow2(-k)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8)


def _make(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEVICE).mul_(std)

    T = case["T"]
    s = {"case": case}
    if case["op"] == "norm":
        M = case["M"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # the residual stream holds a few channels far larger than the others
        loud = 1.0 + 15.0 * (torch.rand(M, generator=g, device=DEVICE) < 0.01)
        s["x"] = randn(T, M).to(dt)
        s["r"] = (randn(T, M) * loud).to(dt) if case["residual"] else None
        s["gain"] = (1.0 + randn(M, std=0.2)).to(dt)
        return s
    N, K = case["N"], case["K"]
    x, W = randn(T, K), randn(N, K, std=1.0 / math.sqrt(K))
    if case["dtype"] == "fp8":
        s["x"], s["xs"] = _quantise(x.bfloat16().float())
        s["W"], s["Ws"] = _quantise(W.bfloat16().float())
    else:
        s["x"], s["W"] = x.bfloat16(), W.bfloat16()
    s["bias"] = randn(N, std=0.5).bfloat16() if case["bias"] else None
    s["mul"] = randn(T, N).bfloat16() if case["mul"] else None
    s["res"] = randn(T, N).bfloat16() if case["residual"] else None
    return s


def prepare(case, seed):
    s = _make(case, seed)
    T = case["T"]
    if case["op"] == "norm":
        x = s["x"]
        s["r_out"] = torch.empty_like(x) if case["residual"] else None
        s["y"] = torch.empty_like(x) if case["out"] != "fp8" else None
        eight = case["out"] in ("fp8", "both")
        s["codes"] = torch.empty(x.shape, dtype=torch.uint8, device=DEVICE) if eight else None
        s["scales"] = torch.empty(T, dtype=torch.uint8, device=DEVICE) if eight else None
    else:
        s["out"] = torch.empty(T, case["N"], dtype=torch.bfloat16, device=DEVICE)
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _library(s)
    return _plain_norm(s) if s["case"]["op"] == "norm" else _plain_linear(s)


def _plain_norm(s):
    case, x = s["case"], s["x"]
    v = x.float()
    if s["r"] is not None:
        v = v + s["r"].float()
    y = v * s["gain"].float() * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
    codes = scales = None
    if s["codes"] is not None:
        codes, scales = _quantise(y)
        scales = scales.view(torch.float8_e8m0fnu)
    return {"residual": v.to(x.dtype) if s["r"] is not None else None, "y": y.to(x.dtype) if s["y"] is not None else None,
            "codes": codes, "scales": scales}


def _plain_linear(s):
    case, x, W = s["case"], s["x"].float(), s["W"].float()
    if case["dtype"] == "fp8":
        x = x * _pow2(s["xs"].int() - 127)[:, None]
        W = W * _pow2(s["Ws"].int() - 127)[:, None]
    v = x @ W.t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    act = case["act"]
    if act == "sigmoid":
        v = 1.0 / (1.0 + torch.exp(-v))
    elif act == "silu":
        v = v / (1.0 + torch.exp(-v))
    elif act == "gelu":
        v = 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(torch.bfloat16)


def _library(s):
    import mla_latent_kv_46_b200 as mla
    case = s["case"]
    if case["op"] == "norm":
        dtype = mla.MLA_BF16 if case["dtype"] == "bf16" else mla.MLA_F32
        if s["codes"] is None:
            mla.mla_add_rmsnorm(s["x"], s["r"], s["gain"], s["r_out"], s["y"], case["T"], case["M"], EPS, dtype)
            return {"residual": s["r_out"], "y": s["y"], "codes": None, "scales": None}
        mla.mla_add_rmsnorm_fp8(s["x"], s["r"], s["gain"], s["r_out"], s["y"], s["codes"], s["scales"], case["T"],
                                case["M"], EPS, dtype)
        return {"residual": s["r_out"], "y": s["y"], "codes": s["codes"].view(torch.float8_e4m3fn),
                "scales": s["scales"].view(torch.float8_e8m0fnu)}
    act = {"none": mla.MLA_ACT_NONE, "sigmoid": mla.MLA_ACT_SIGMOID, "silu": mla.MLA_ACT_SILU,
           "gelu": mla.MLA_ACT_GELU}[case["act"]]
    if case["dtype"] == "fp8":
        mla.mla_linear_fp8(s["x"], s["xs"], s["W"], s["Ws"], s["bias"], s["mul"], s["res"], s["out"], case["T"],
                           case["N"], case["K"], act)
    else:
        mla.mla_linear(s["x"], s["W"], s["bias"], s["mul"], s["res"], s["out"], case["T"], case["N"], case["K"], act)
    return s["out"]


# ------------------------------------------------------------------------------ floors and the definition
def work(case):
    T = case["T"]
    if case["op"] == "norm":
        M = case["M"]
        e = 2 if case["dtype"] == "bf16" else 4
        nbytes = T * M * e + M * e
        if case["residual"]:
            nbytes += 2 * T * M * e
        if case["out"] != "fp8":
            nbytes += T * M * e
        if case["out"] in ("fp8", "both"):
            nbytes += T * M + T
        return {"bytes": nbytes, "flops": 6 * T * M}
    N, K = case["N"], case["K"]
    e = 1 if case["dtype"] == "fp8" else 2
    nbytes = (T + N) * (K * e + (1 if e == 1 else 0)) + 2 * T * N
    nbytes += (2 * N if case["bias"] else 0) + (2 * T * N if case["mul"] else 0) + (2 * T * N if case["residual"] else 0)
    return {"bytes": nbytes, "flops": 2 * T * N * K}


def exact(case, seed):
    s = _make(case, seed)
    if case["op"] == "norm":
        total = s["x"].double() if s["r"] is None else s["x"].double().add_(s["r"].double())
        root = torch.sqrt((total * total).sum(1) / case["M"] + EPS)
        y = total / root[:, None] * s["gain"].double()
        codes = scales = None
        if case["out"] in ("fp8", "both"):
            top = y.abs().max(dim=1).values / 448.0
            k = torch.ceil(torch.log2(top.clamp_min(2.0 ** -126))).clamp(-126, 7)
            k = torch.where(torch.pow(2.0, k - 1) >= top, (k - 1).clamp_min(-126), k)
            scales = torch.pow(2.0, k)
            codes = (y / scales[:, None]).clamp(-448, 448)
        return {"residual": total if case["residual"] else None, "y": y if case["out"] != "fp8" else None,
                "codes": codes, "scales": scales}
    x, W = s["x"].double(), s["W"].double()
    if case["dtype"] == "fp8":
        x *= torch.pow(2.0, s["xs"].double() - 127)[:, None]
        W *= torch.pow(2.0, s["Ws"].double() - 127)[:, None]
    out = torch.mm(x, W.T)
    if s["bias"] is not None:
        out += s["bias"].double()
    if case["act"] == "sigmoid":
        out = torch.special.expit(out)
    elif case["act"] == "silu":
        out = out * torch.special.expit(out)
    elif case["act"] == "gelu":
        out = out * torch.special.ndtr(out)
    if s["mul"] is not None:
        out *= s["mul"].double()
    if s["res"] is not None:
        out += s["res"].double()
    return out
