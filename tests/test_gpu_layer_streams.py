"""The layer's operators where what they read comes from another stream: their early launch (the set-up
runs under the kernel before them) must not reach past an event."""
import pytest
import torch

import mla_latent_kv_46_b200 as mla

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T, M, N = 96, 1024, 512


def operands(seed):
    g = torch.Generator(device="cpu").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).to(DEV)
    return randn(T, M), randn(M), randn(N, M)


def chain(x, gain, W, h, out, stream=None):
    mla.mla_add_rmsnorm(x, None, gain, None, h, T, M, 1e-6, mla.MLA_BF16, stream=stream)
    mla.mla_linear(h, W, None, None, None, out, T, N, M, mla.MLA_ACT_SILU, stream=stream)


def test_a_call_behind_an_event_waits_for_what_the_other_stream_writes():
    rows, gain, W = operands(1)
    h, want, out, other = (torch.empty(T, n, dtype=torch.bfloat16, device=DEV) for n in (M, N, N, N))
    chain(rows, gain, W, h, want)
    x = torch.zeros_like(rows)
    busy = torch.ones(4096, 4096, dtype=torch.bfloat16, device=DEV)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(a):
            x.zero_()
        b.wait_stream(a)
        with torch.cuda.stream(a):
            for _ in range(4):
                torch.mm(busy, busy)
            x.copy_(rows)
            done = torch.cuda.Event()
            done.record(a)
        # kernels of b's own before the wait: those behind it may start under their tails
        mla.mla_linear(rows, W, None, None, None, other, T, N, M, mla.MLA_ACT_NONE, stream=b)
        b.wait_event(done)
        chain(x, gain, W, h, out, stream=b)
        a.wait_stream(b)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_captured_branches_join_before_the_call_that_reads_both():
    """In a captured graph a call's two predecessors, on two streams, both of them calls whose
    successors may start early."""
    rows, gain, W = operands(2)
    x = rows.clone()
    h, mul, out = (torch.empty(T, n, dtype=torch.bfloat16, device=DEV) for n in (M, N, N))

    def step(main, side):
        side.wait_stream(main)
        for _ in range(8):      # the longer branch
            mla.mla_add_rmsnorm(x, None, gain, None, h, T, M, 1e-6, mla.MLA_BF16, stream=side)
        mla.mla_linear(x, W, None, None, None, mul, T, N, M, mla.MLA_ACT_SIGMOID, stream=main)
        main.wait_stream(side)
        mla.mla_linear(h, W, None, mul, None, out, T, N, M, mla.MLA_ACT_NONE, stream=main)
    side = torch.cuda.Stream()
    wants = []
    for r in (rows, -2 * rows):
        x.copy_(r)
        step(torch.cuda.current_stream(), side)
        torch.cuda.synchronize()
        wants.append(out.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(torch.cuda.current_stream(), side)
    for k in range(20):
        x.copy_((rows, -2 * rows)[k % 2])
        h.fill_(float("nan")), mul.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wants[k % 2])
    mla.mla_check_status()
