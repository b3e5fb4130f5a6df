"""The layer operators' functions as programs call them: in captured graphs, under checkpointing, on streams of their
own, on nothing at all."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from layertest import DT
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
B, N, H, Hk, D = 2, 190, 4, 2, 64


def parameters(seed, dtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).to(DEV)  # noqa: E731
    p = dict(x=r(B, N, H * D), w=r(H * D), b=r(H * D), k=r(B, N, Hk, D), v=r(B, N, Hk, D), lam=r(H), dy=r(B, N, H, D))
    return {n: t.requires_grad_(n != "dy") for n, t in p.items()}


def step(p, plan, pos):
    q = lh.layer_norm(p["x"], p["w"], p["b"]).view(B, N, H, D)
    q, k = lh.rotary(q, p["k"], pos, plan, maps=2)
    return lh.differential_attention(q, k, p["v"], p["lam"])


def gradients(p, plan, pos):
    o = step(p, plan, pos)
    leaves = [t for n, t in p.items() if n != "dy"]
    return [o.detach(), *torch.autograd.grad(o, leaves, p["dy"])]


def tables():
    return lh.RopePlan(D // 2, device=DEV), torch.arange(N, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_captured_with_its_gradients(dtype):
    """Forward and backward in one graph, replayed on other inputs: the bits of the eager step."""
    p, (plan, pos) = parameters(1, dtype), tables()
    gradients(p, plan, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients(p, plan, pos)
    other = parameters(2, dtype)
    with torch.no_grad():
        for n, t in p.items():
            t.copy_(other[n])
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, gradients(other, plan, pos)))
    assert lh.get_device_error() == (0, 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_recomputed_under_checkpointing(dtype):
    p, (plan, pos) = parameters(3, dtype), tables()
    leaves = [t for n, t in p.items() if n != "dy"]
    want = gradients(p, plan, pos)[1:]
    o = checkpoint(lambda: step(p, plan, pos), use_reentrant=False)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(o, leaves, p["dy"]), want))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_two_steps_on_two_streams(dtype):
    (plan, pos), ps = tables(), [parameters(s, dtype) for s in (4, 5)]
    want = [gradients(p, plan, pos) for p in ps]
    streams, got = [torch.cuda.Stream() for _ in ps], []
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for p, st in zip(ps, streams):
            with torch.cuda.stream(st):
                got.append(gradients(p, plan, pos))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nothing_to_do(dtype):
    e = lambda *s: torch.zeros(*s, dtype=DT[dtype], device=DEV, requires_grad=True)  # noqa: E731
    plan = lh.RopePlan(D, device=DEV)
    x, w = e(2, 0, D), e(D)
    y = lh.layer_norm(x, w)
    y.backward(torch.zeros_like(y))
    assert y.shape == x.shape and not w.grad.any()
    q, k = lh.rotary(e(2, 0, H, D), e(2, 0, Hk, D), torch.zeros(0, dtype=torch.int32, device=DEV), plan)
    assert q.shape == (2, 0, H, D) and k.shape == (2, 0, Hk, D)
    q, k = lh.rotary(e(2, 3, H, D), e(2, 3, 0, D), torch.arange(3, dtype=torch.int32, device=DEV), plan)
    assert k.numel() == 0
    lam = e(H)
    o = lh.differential_attention(e(2, 0, H, D), e(2, 0, Hk, D), e(2, 0, Hk, D), lam)
    o.backward(torch.zeros_like(o))
    assert o.shape == (2, 0, H, D) and not lam.grad.any()
    lam2 = e(H)
    o = lh.differential_attention(e(5, H, D), e(5, Hk, D), e(5, Hk, D), lam2, cu=torch.zeros(3, dtype=torch.int32, device=DEV))
    o.backward(torch.ones_like(o))
    assert not o.any() and not lam2.grad.any()
    torch.cuda.synchronize()
    assert lh.get_device_error() == (0, 0)


def test_a_frozen_input_and_an_unused_output():
    p, (plan, pos) = parameters(6, "bf16"), tables()
    q = p["x"].detach().view(B, N, H, D)
    k = p["k"]
    kr = lh.rotary(q, k, pos, plan, maps=2)[1]           # q's result is not used: its gradient is zeros
    dk = p["dy"][:, :, :Hk].contiguous()
    (gk,) = torch.autograd.grad(kr, k, dk)
    assert torch.equal(gk, lh.rotary(q, dk, -pos, plan, maps=2)[1])
    o = lh.differential_attention(q, k.detach(), p["v"].detach(), p["lam"])
    (g,) = torch.autograd.grad(o, p["lam"], p["dy"])
    full = [t.detach().clone().requires_grad_() for t in (q, k, p["v"], p["lam"])]
    assert torch.equal(g, torch.autograd.grad(lh.differential_attention(*full), full[3], p["dy"])[0])
