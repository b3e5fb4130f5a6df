"""Rotary positions over one and several axes against their 64-bit form."""

import pytest
import torch

from layertest import DT, HALF, assert_within, rope_ref
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def rand(seed, *shape, dtype="fp32"):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).to(DEV)


def positions(seed, axes, B, N, top=1 << 20, dtype=torch.int32):
    return torch.randint(-top, top, (axes, B, N), generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def check(got, x, pos, plan, pairs, dtype, inverse=False):
    ref, err = rope_ref(x, pos, plan.freq, plan.axis, pairs, plan.rot, inverse)
    u = HALF[dtype]
    tol = u * ref.abs() + (1 + u) * err
    tol[..., plan.rot:] = 0          # copied
    assert_within(got, ref, tol, "rotated")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pairs", ["half", "next"])
@pytest.mark.parametrize("B,N,H,Hk,D,rot,sections", [
    (1, 1, 1, 1, 2, 2, None), (2, 7, 3, 1, 64, 64, None), (1, 130, 16, 16, 128, 128, [16, 24, 24]), (3, 5, 4, 2, 72, 40, [7, 13]),
    (1, 33, 2, 0, 6, 4, [1, 1]), (2, 9, 5, 5, 10, 6, None), (1, 17, 8, 2, 64, 48, [8, 8, 8]), (1, 3, 1, 1, 1024, 1022, [500, 11]),
    (2, 4, 2, 1, 256, 16, [2, 2, 2, 2])])
def test_against_64_bits(dtype, pairs, B, N, H, Hk, D, rot, sections):
    plan = lh.RopePlan(rot, sections, device=DEV)
    q, k = rand(1, B, N, H, D, dtype=dtype), rand(2, B, N, max(Hk, 1), D, dtype=dtype)
    pos = positions(3, plan.axes, B, N)
    cfg = lh.make_rope_config(B, N, H, Hk, D, rot, plan.axes, dtype, pairs)
    for inverse in (False, True):
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        lh.rope(cfg, q, k if Hk else None, pos, plan.freq, plan.axis, qo, ko if Hk else None, inverse=inverse)
        torch.cuda.synchronize()
        check(qo, q, pos, plan, pairs, dtype, inverse)
        if Hk:
            check(ko, k, pos, plan, pairs, dtype, inverse)
        # in place, and back again: within the two roundings of the way there and back
        q2, k2 = q.clone(), k.clone()
        lh.rope(cfg, q2, k2 if Hk else None, pos, plan.freq, plan.axis, q2, k2 if Hk else None, inverse=inverse)
        torch.cuda.synchronize()
        assert torch.equal(q2, qo) and (not Hk or torch.equal(k2, ko))
    assert lh.get_device_error() == (0, 0)


@pytest.mark.parametrize("dtype,top", [(torch.int32, (1 << 31) - 1), (torch.int64, 1 << 31), (torch.int64, 5)])
def test_position_types_and_far_positions(dtype, top):
    plan = lh.RopePlan(64, device=DEV)
    q, k = rand(1, 2, 50, 2, 64), rand(2, 2, 50, 1, 64)
    pos = positions(4, 1, 2, 50, top, dtype)
    cfg = lh.make_rope_config(2, 50, 2, 1, 64, pos64=dtype == torch.int64, dtype="fp32")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    lh.rope(cfg, q, k, pos, plan.freq, plan.axis, qo, ko)
    torch.cuda.synchronize()
    check(qo, q, pos, plan, "half", "fp32")
    check(ko, k, pos, plan, "half", "fp32")


def test_quarter_turns_are_exact():
    """Frequencies of a quarter turn: the pairs are exchanged and negated without a rounding."""
    plan = lh.RopePlan(8, device=DEV, freq=[torch.pi / 2] * 4)
    q = rand(1, 1, 9, 1, 8)
    pos = torch.arange(-4, 5, dtype=torch.int32, device=DEV).view(1, 1, 9)
    out = torch.empty_like(q)
    lh.rope(lh.make_rope_config(1, 9, 1, 0, 8, dtype="fp32"), q, None, pos, plan.freq, plan.axis, out, None)
    torch.cuda.synchronize()
    a, b = q[0, :, 0, :4], q[0, :, 0, 4:]
    for t in range(9):
        want = [(a[t], b[t]), (-b[t], a[t]), (-a[t], -b[t]), (b[t], -a[t])][(t - 4) % 4]
        assert torch.equal(out[0, t, 0], torch.cat(want)), t


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_views_of_a_fused_projection(dtype):
    """q and k rotated in place inside one [B, N, (H + 2 Hk) D] buffer; v between the rows stays."""
    B, N, H, Hk, D = 2, 37, 4, 2, 64
    qkv = rand(1, B, N, (H + 2 * Hk) * D, dtype=dtype)
    was = qkv.clone()
    ld = qkv.shape[-1]
    q, k = qkv[..., :H * D], qkv[..., H * D:(H + Hk) * D]
    plan = lh.RopePlan(D, [16, 8, 8], device=DEV)
    pos = positions(3, 3, B, N, 4096)
    cfg = lh.make_rope_config(B, N, H, Hk, D, axes=3, dtype=dtype, q_ld=ld, k_ld=ld, qo_ld=ld, ko_ld=ld)
    lh.rope(cfg, q, k, pos, plan.freq, plan.axis, q, k)
    torch.cuda.synchronize()
    check(q.reshape(B, N, H, D), was[..., :H * D].reshape(B, N, H, D), pos, plan, "half", dtype)
    check(k.reshape(B, N, Hk, D), was[..., H * D:(H + Hk) * D].reshape(B, N, Hk, D), pos, plan, "half", dtype)
    assert torch.equal(qkv[..., (H + Hk) * D:], was[..., (H + Hk) * D:])


def test_odd_strides_and_shared_positions():
    B, N, D = 2, 11, 16
    buf, out = rand(1, B * N * 37 + 64, dtype="bf16"), rand(2, B * N * 41 + 64, dtype="bf16")
    was = out.clone()
    plan = lh.RopePlan(D, device=DEV)
    pos = positions(3, 1, 1, N, 1000)
    cfg = lh.make_rope_config(B, N, 2, 0, D, shared_pos=True, q_ld=37, q_bs=37 * N + 5, qo_ld=41, qo_bs=41 * N + 3)
    lh.rope(cfg, buf, None, pos, plan.freq, plan.axis, out, None)
    torch.cuda.synchronize()
    src = buf.as_strided((B, N, 2, D), (37 * N + 5, 37, D, 1))
    got = out.as_strided((B, N, 2, D), (41 * N + 3, 41, D, 1))
    check(got, src, pos.expand(1, B, N), plan, "half", "bf16")
    got.copy_(was.as_strided((B, N, 2, D), (41 * N + 3, 41, D, 1)))
    assert torch.equal(out, was)


def test_axis_out_of_range_is_reported():
    plan = lh.RopePlan(8, device=DEV)
    q = rand(1, 1, 3, 1, 8)
    pos = torch.zeros(1, 1, 3, dtype=torch.int32, device=DEV)
    axis = torch.tensor([0, 7, 0, -1], dtype=torch.int32, device=DEV)
    lh.rope(lh.make_rope_config(1, 3, 1, 0, 8, dtype="fp32"), q, None, pos, plan.freq, axis, torch.empty_like(q), None)
    assert lh.get_device_error() == (9, 401)
    assert lh.get_device_error() == (0, 0)


@pytest.mark.parametrize("pairs", ["half", "next"])
def test_autograd_turns_back(pairs):
    plan = lh.RopePlan(48, [8, 8, 8], device=DEV, order="cycle", ladder="own")
    q, k = rand(1, 2, 21, 4, 64).requires_grad_(), rand(2, 2, 21, 2, 64).requires_grad_()
    pos = positions(3, 3, 2, 21, 5000, torch.int64)
    qo, ko = lh.rotary(q, k, pos, plan, pairs)
    gq, gk = rand(5, 2, 21, 4, 64), rand(6, 2, 21, 2, 64)
    torch.autograd.backward([qo, ko], [gq, gk])
    check(qo, q.detach(), pos, plan, pairs, "fp32")
    check(q.grad, gq, pos, plan, pairs, "fp32", inverse=True)
    check(k.grad, gk, pos, plan, pairs, "fp32", inverse=True)
    # differences: the map is linear, so a step of 1 along one element is the gradient
    ref = lambda x: float((rope_ref(x, pos, plan.freq, plan.axis, pairs, 48, False)[0] * gq.double().cpu()).sum())  # noqa: E731
    x = q.detach().double().cpu()
    y = x.clone()
    y[1, 3, 2, 5] += 1
    assert abs(ref(y) - ref(x) - float(q.grad[1, 3, 2, 5])) < 1e-5


def test_graph_and_another_stream():
    plan = lh.RopePlan(128, [16, 24, 24], device=DEV)
    q, k = rand(1, 1, 3001, 8, 128, dtype="bf16"), rand(2, 1, 3001, 8, 128, dtype="bf16")
    pos = positions(3, 3, 1, 3001, 100000)
    cfg = lh.make_rope_config(1, 3001, 8, 8, 128, axes=3)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    lh.rope(cfg, q, k, pos, plan.freq, plan.axis, qo, ko)
    torch.cuda.synchronize()
    rq, rk = qo.clone(), ko.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lh.rope(cfg, q, k, pos, plan.freq, plan.axis, qo, ko)
    qo.zero_()
    ko.zero_()
    g.replay()
    st = torch.cuda.Stream()
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    st.wait_stream(torch.cuda.current_stream())
    lh.rope(cfg, q, k, pos, plan.freq, plan.axis, q2, k2, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(qo, rq) and torch.equal(ko, rk) and torch.equal(q2, rq) and torch.equal(k2, rk)


def test_offsets_past_32_bits():
    """Token rows 2^25 elements apart, in place: the last ones start beyond element 2^31."""
    N, D, ld = 70, 64, 1 << 25
    q = rand(1, 1, N, 1, D, dtype="bf16")
    plan, pos = lh.RopePlan(D, device=DEV), positions(3, 1, 1, N)
    want = torch.empty_like(q)
    lh.rope(lh.make_rope_config(1, N, 1, 0, D), q, None, pos, plan.freq, plan.axis, want, None)
    far = torch.empty((N - 1) * ld + D, dtype=torch.bfloat16, device=DEV).as_strided((N, D), (ld, 1))
    far.copy_(q[0, :, 0])
    lh.rope(lh.make_rope_config(1, N, 1, 0, D, q_ld=ld, qo_ld=ld), far, None, pos, plan.freq, plan.axis, far, None)
    torch.cuda.synchronize()
    assert torch.equal(far, want[0, :, 0])
