"""The layer operators together, as a layer runs them: in front of the Lighthouse path (fused.qkv_project_pool
with norm and positions), and one differential attention layer, forward and backward."""

import math

import pytest
import torch

from long_context_symmetric_b200 import fused, lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def rand(g, *shape, mul=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * mul).to(torch.bfloat16)


@pytest.mark.parametrize("B,H,N,D,p,L,chunk,sections,pairs,pos_type", [
    (2, 2, 4096, 64, 4, 3, 512, [8, 12, 12], "half", torch.int32),
    (1, 4, 8192, 128, 8, 3, 2048, None, "next", torch.int64),
    (2, 1, 516, 64, 2, 2, 6, [20, 12], "half", torch.int32),        # 2-token blocks: chunks that start at odd pairs of tokens
])
def test_chunked_front_equals_the_whole_calls(B, H, N, D, p, L, chunk, sections, pairs, pos_type):
    """Norm, projections, rotation and pool chunk by chunk: the same bits as one call after the other, and again as a
    replayed graph."""
    if N % chunk:
        chunk = fused.chunk_tokens(lh.make_config(B, H, N, D, p, L, 16), chunk)
    g = torch.Generator(device=DEV).manual_seed(5)
    dm = H * D
    x, w = rand(g, B, N, dm), [rand(g, dm, dm, mul=dm ** -0.5) for _ in range(3)]
    nw, nb = 1 + rand(g, dm, mul=0.1), rand(g, dm, mul=0.1)
    plan = lh.RopePlan(D, sections, device=DEV)
    pos = torch.randint(0, 1 << 20, (plan.axes, B, N), generator=g, device=DEV).to(pos_type)
    cfg = lh.make_config(B, H, N, D, p, L, 16, "bf16")
    ws, ref = (lh.Workspace(cfg, DEV, backward=False) for _ in range(2))
    q, k, v = (torch.empty(B, N, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    norm = fused.InputNorm(nw, nb, torch.empty_like(x), *(torch.empty(B, N, device=DEV) for _ in range(2)))
    run = lambda: fused.qkv_project_pool(cfg, ws, x, *w, q, k, v, chunk=chunk, norm=norm, rope=fused.Positions(pos, plan, pairs))  # noqa: E731
    run()
    # one after the other (the GEMMs cut alike: a library GEMM may add in another order at another size)
    ncfg = lh.make_norm_config(B * N, dm)
    xn, mean, rstd = torch.empty_like(x), torch.empty(B, N, device=DEV), torch.empty(B, N, device=DEV)
    lh.norm_fwd(ncfg, x, nw, nb, xn, mean, rstd)
    qr, kr, vr = (torch.empty_like(q) for _ in range(3))
    for t0 in range(0, N, chunk):
        for b in range(B):
            for wt, out in zip(w, (qr, kr, vr)):
                torch.matmul(xn[b, t0:t0 + chunk], wt, out=out[b, t0:t0 + chunk].view(chunk, dm))
    rc = lh.make_rope_config(B, N, H, H, D, axes=plan.axes, pairs=pairs, pos64=pos_type == torch.int64)
    lh.rope(rc, qr, kr, pos, plan.freq, plan.axis, qr, kr)
    lh.pool(cfg, qr, kr, vr, ref.pyr_q, ref.pyr_k, ref.pyr_v, ref.sq, ref.scale)
    torch.cuda.synchronize()

    def same():
        assert lh.get_device_error() == (0, 0)
        pairs_ = [(norm.xn, xn), (norm.mean, mean), (norm.rstd, rstd), (q, qr), (k, kr), (v, vr), (ws.pyr_q, ref.pyr_q),
                  (ws.pyr_k, ref.pyr_k), (ws.pyr_v, ref.pyr_v), (ws.sq, ref.sq)]
        assert all(torch.equal(a, b) for a, b in pairs_)

    same()
    if N // chunk <= 16:
        graph = fused.Graphed(run)
        for t in (norm.xn, q, k, v, ws.sq):
            t.zero_()
        graph()
        torch.cuda.synchronize()
        same()


def test_front_refuses_positions_of_another_shape():
    cfg = lh.make_config(1, 2, 256, 64, 4, 2, 16, "bf16")
    t = torch.empty(1, 256, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.empty(1, 256, 2, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.empty(128, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(2, 1, 256, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="positions"):
        fused.qkv_project_pool(cfg, lh.Workspace(cfg, DEV, backward=False), t, w, w, w, q, q, q,
                               rope=fused.Positions(pos, lh.RopePlan(64, device=DEV)))


def layer64(x, p, pos, plan, H, Hk, D):
    """The layer in 64-bit torch operations (its gradients by autograd)."""
    B, N, _ = x.shape

    def ln(t, w, b):
        m = t.mean(-1, keepdim=True)
        return (t - m) / ((t - m).square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def turn(t):
        ang = (pos.double()[plan.axis.long()].movedim(0, -1) * plan.freq)[:, :, None]
        a, b = t.chunk(2, -1)
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    xn = ln(x, p["w1"], p["b1"])
    q = turn((xn @ p["wq"]).view(B, N, H, D))
    k, v = turn((xn @ p["wk"]).view(B, N, Hk, D)), (xn @ p["wv"]).view(B, N, Hk, D)
    k, v = (t.repeat_interleave(H // Hk, 2) for t in (k, v))
    late = torch.ones(N, N, dtype=torch.bool, device=x.device).triu(1)
    a = [torch.einsum("bihd,bjhd->bhij", q[..., s], k[..., s]).div(math.sqrt(D / 2)).masked_fill(late, -math.inf).softmax(-1)
         for s in (slice(0, D // 2), slice(D // 2, D))]
    o = torch.einsum("bhij,bjhd->bihd", a[0] - p["lam"].view(1, H, 1, 1) * a[1], v)
    return ln(o, p["w2"], p["b2"]).reshape(B, N, H * D) @ p["wo"]


def layer(x, p, pos, plan, H, Hk, D):
    B, N, _ = x.shape
    xn = lh.layer_norm(x, p["w1"], p["b1"])
    q, k = lh.rotary((xn @ p["wq"]).view(B, N, H, D), (xn @ p["wk"]).view(B, N, Hk, D), pos, plan)
    o = lh.differential_attention(q, k, (xn @ p["wv"]).view(B, N, Hk, D), p["lam"])
    return lh.layer_norm(o, p["w2"], p["b2"]).reshape(B, N, H * D) @ p["wo"]


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-5), (torch.bfloat16, 4e-2)])
def test_differential_layer(dtype, tol):
    """Output and every gradient of a layer against its 64-bit form, in the 2-norm. A layer in this type rounds at
    about ten places on the way forward and back (norm, projection, rotation, attention, head norm, projection, and
    the gradients of each), every time by at most eps / 2 of the value, and the head norm divides by a deviation that
    the difference of the maps makes a few times smaller than what it is formed from: ten roundings of 2^-8 are 4e-2;
    fp32's matrix products add sqrt(256) roundings each: 10 * 16 * 2^-24 = 1e-5, twice for the maps' exponents."""
    B, N, H, Hk, D, dm = 2, 173, 4, 2, 64, 256
    g = torch.Generator(device=DEV).manual_seed(8)
    r = lambda *s, mul=1.0: torch.randn(*s, generator=g, device=DEV) * mul  # noqa: E731
    p = dict(w1=1 + r(dm, mul=0.1), b1=r(dm, mul=0.1), wq=r(dm, H * D, mul=dm ** -0.5), wk=r(dm, Hk * D, mul=dm ** -0.5),
             wv=r(dm, Hk * D, mul=dm ** -0.5), lam=0.2 + 0.3 * torch.rand(H, generator=g, device=DEV), w2=1 + r(D, mul=0.1),
             b2=r(D, mul=0.1), wo=r(H * D, dm, mul=(H * D) ** -0.5))
    p = {n: t.to(dtype) for n, t in p.items()}
    x, dy = r(B, N, dm).to(dtype), r(B, N, dm).to(dtype)
    plan = lh.RopePlan(D, [16, 8, 8], device=DEV)
    pos = torch.randint(0, 4096, (3, B, N), generator=g, device=DEV, dtype=torch.int32)
    own = {n: t.clone().requires_grad_() for n, t in dict(p, x=x).items()}
    ref = {n: t.double().requires_grad_() for n, t in dict(p, x=x).items()}
    y = layer(own["x"], own, pos, plan, H, Hk, D)
    y.backward(dy)
    z = layer64(ref["x"], ref, pos, plan, H, Hk, D)
    z.backward(dy.double())
    assert lh.get_device_error() == (0, 0)
    off = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert off(y.detach(), z.detach()) < tol
    for n in own:
        assert off(own[n].grad, ref[n].grad) < tol, n
