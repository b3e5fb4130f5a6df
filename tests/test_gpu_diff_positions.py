"""Rotary positions in front of differential attention: each of a head's two maps is rotated by itself, so that its
scores depend on the distance between a query's and a key's positions and on nothing else."""

import math

import pytest
import torch

from layertest import DT, HALF, U, assert_within
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def inputs(B, N, H, Hk, D, dtype):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).to(DEV)  # noqa: E731
    q, k, v, do = r(B, N, H, D), r(B, N, Hk, D), r(B, N, Hk, D), r(B, N, H, D)
    return q, k, v, (0.2 + 0.6 * torch.rand(H, generator=g)).to(DT[dtype]).to(DEV), do


def scores_by_distance(q, k, pos, plan, pairs):
    """[maps][B, H, N, N] of 64-bit scores: for every pair of tokens the query's map turned by the distance of their
    positions; and the sums of the magnitudes that a rotation mixes."""
    B, N, H, D = q.shape
    h = D // 2
    far = pos.double()[plan.axis.long()]                                      # [R, B, N]
    ang = (far[:, :, :, None] - far[:, :, None, :]).permute(1, 2, 3, 0) * plan.freq     # [B, N, N, R]
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    out, mag = [], []
    for m in (0, 1):
        a, b = q[..., m * h:m * h + h].transpose(1, 2), k[..., m * h:m * h + h].transpose(1, 2)
        two = (lambda t: t.chunk(2, -1)) if pairs == "half" else (lambda t: (t[..., ::2], t[..., 1::2]))
        (a0, a1), (b0, b1) = two(a), two(b)
        a0, a1, b0, b1 = a0[:, :, :, None], a1[:, :, :, None], b0[:, :, None], b1[:, :, None]
        # <turn(p_i) a, turn(p_j) b> = <turn(p_i - p_j) a, b>
        out.append((((a0 * c - a1 * s) * b0 + (a1 * c + a0 * s) * b1).sum(-1)) / math.sqrt(h))
        mag.append(((a0.abs() + a1.abs()) * (b0.abs() + b1.abs())).sum(-1) / math.sqrt(h))
    return out, mag


def reference(q, k, v, lam, pos, plan, pairs):
    H, Hk, N = q.shape[2], k.shape[2], q.shape[1]
    k, v = (t.repeat_interleave(H // Hk, 2) for t in (k, v))
    late = torch.ones(N, N, dtype=torch.bool, device=DEV).triu(1)
    s, mag = scores_by_distance(q, k, pos, plan, pairs)
    A = [x.masked_fill(late, -math.inf).softmax(-1) for x in s]
    o = torch.einsum("bhij,bjhd->bihd", A[0] - lam.view(1, H, 1, 1) * A[1], v)
    return o, A, [x.masked_fill(late, 0) for x in mag], v


@pytest.mark.parametrize("pairs", ["half", "next"])
@pytest.mark.parametrize("H,Hk,D,sections", [(2, 2, 64, None), (4, 2, 128, [12, 10, 10])])
@pytest.mark.parametrize("shift", [0, 1, 1 << 17])
def test_scores_depend_on_the_distance_alone(H, Hk, D, sections, pairs, shift):
    """fp32: outputs within the rounding of the rotations and of the attention from the form that only knows
    distances; gradients in the 2-norm."""
    B, N, h = 2, 85, D // 2
    q, k, v, lam, do = inputs(B, N, H, Hk, D, "fp32")
    plan = lh.RopePlan(h, sections, device=DEV)
    pos = torch.randint(0, 512, (plan.axes, B, N), generator=torch.Generator().manual_seed(6)).to(torch.int32).to(DEV)
    own = [t.clone().requires_grad_() for t in (q, k, v, lam)]
    qr, kr = lh.rotary(own[0], own[1], pos + shift, plan, pairs, maps=2)
    o = lh.differential_attention(qr, kr, own[2], own[3])
    o.backward(do)
    ref = [t.double().requires_grad_() for t in (q, k, v, lam)]
    want, A, mag, vv = reference(*ref, pos, plan, pairs)
    want.backward(do.double())
    # a rotated element is off by (7 + 2^-27 of its angle) U of |a| + |b| (fp32 cosine, sine, products and sum; the angle
    # in 64 bits), on both sides of a score; the score's own sum and exponent (h + 4) U; the row's maximum and
    # denominator double it; then as in layertest.diff_ref
    R = [2 * (h + 4 + 2 * (7 + 2.0 ** -27 * (shift + 512))) * U * m.amax(-1, keepdim=True) + 2.0 ** -21 + (N / 64 + 96) * U for m in mag]
    tol = torch.einsum("bhij,bjhd->bihd", A[0] * R[0] + lam.view(1, H, 1, 1) * A[1] * R[1] + (N / 8 + 96) * U * (A[0] + A[1]), vv.abs())
    assert_within(o, want.detach(), (tol + U * want.abs()).detach(), "o")
    # gradients: the same roundings once more on the way back, each at most 2^-24 of sums of at most 2 * 64 terms
    for a, b, n in zip(own, ref, ("dq", "dk", "dv", "dlam")):
        assert float((a.grad.double() - b.grad).norm() / b.grad.norm()) < 2e-5, n
    if shift == 1 << 17 and pairs == "half":
        # what this guards against: rows rotated as a whole give another output at another place
        whole = lh.RopePlan(D, device=DEV)
        one = pos[:1]
        a, b = (lh.differential_attention(*lh.rotary(q, k, p, whole), v, lam) for p in (one, one + shift))
        assert float((a - b).norm() / a.norm()) > 1e-2


def test_bf16_rows_and_the_same_call_as_twice_the_heads():
    B, N, H, Hk, D = 1, 130, 4, 2, 128
    q, k, v, lam, do = inputs(B, N, H, Hk, D, "bf16")
    plan, pos = lh.RopePlan(D // 2, device=DEV), torch.arange(N, dtype=torch.int32, device=DEV)
    qr, kr = lh.rotary(q, k, pos, plan, maps=2)
    q2, k2 = lh.rotary(q.view(B, N, 2 * H, D // 2), k.view(B, N, 2 * Hk, D // 2), pos, plan)
    assert torch.equal(qr, q2.view_as(q)) and torch.equal(kr, k2.view_as(k))
    # strided inputs, as slices of one projection
    wide = torch.cat([q, k, v], 2)
    qs, ks = lh.rotary(wide[:, :, :H], wide[:, :, H:H + Hk], pos, plan, maps=2)
    assert torch.equal(qs, qr) and torch.equal(ks, kr)
    o = lh.differential_attention(qr, kr, v, lam)
    want, A, _, vv = reference(*(t.double() for t in (q, k, v, lam)), pos.view(1, 1, N), plan, "half")
    # bf16 rounds the rotated rows, 2^-9 of each element: scores of 64 products are off by 2 * 2^-9 sqrt(64) / 8 times an
    # element's size (4 at the most here) at random, so the maps by 2^-8 * 4 * 2 of themselves; the output once more
    off = float((o.double() - want).norm() / torch.einsum("bhij,bjhd->bihd", A[0] + A[1], vv.abs()).norm())
    assert off < 2.0 ** -5 + HALF["bf16"]
