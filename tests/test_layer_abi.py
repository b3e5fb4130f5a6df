"""Refusals of the layer operators (layer norm, rotary positions, differential
attention): bad sizes, types, modes and pointers return a status before any
CUDA call, and the binding refuses tensors that do not fit a call."""

import ctypes
import math
import types

import pytest
import torch

from long_context_symmetric_b200 import lh

NULL, SHAPE, ALIGN, DTYPE, MODE, WORKSPACE = 1, 2, 3, 4, 5, 6
A = 1 << 20          # an aligned address that nothing here dereferences


def norm(**kw):
    c = lh.make_norm_config(64, 256)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(M=(1 << 40) + 1), SHAPE), (dict(d=0), SHAPE), (dict(d=16385), SHAPE), (dict(ldx=255), SHAPE),
    (dict(ldy=8), SHAPE), (dict(eps=-1e-5), SHAPE), (dict(eps=math.inf), SHAPE), (dict(eps=math.nan), SHAPE),
    (dict(dtype=2), DTYPE), (dict(wdtype=7), DTYPE)])
def test_norm_refuses(kw, want):
    c, f = norm(**kw), lh.lib()
    n = ctypes.c_size_t()
    assert f.lh_norm_plan(ctypes.byref(c), ctypes.byref(n)) == want
    assert f.lh_norm_fwd(ctypes.byref(c), A, A, A, A, A, A, None) == want
    assert f.lh_norm_bwd(ctypes.byref(c), A, A, A, A, A, A, A, A, A, 1 << 30, None) == want


def test_norm_refuses_pointers():
    f, c = lh.lib(), norm()
    r, before = ctypes.byref(c), lh.launch_count()
    assert f.lh_norm_plan(None, None) == NULL
    assert f.lh_norm_fwd(None, A, A, A, A, A, A, None) == NULL
    assert f.lh_norm_fwd(r, None, A, A, A, A, A, None) == NULL
    assert f.lh_norm_fwd(r, A, A, A, None, A, A, None) == NULL
    assert f.lh_norm_fwd(r, A + 8, A, A, A, A, A, None) == ALIGN
    assert f.lh_norm_fwd(r, A, A + 2, A, A, A, A, None) == ALIGN
    assert f.lh_norm_fwd(r, A, A, A, A, A + 2, A, None) == ALIGN
    assert f.lh_norm_bwd(r, A, A, A, None, A, A, A, A, A, 1 << 30, None) == NULL
    assert f.lh_norm_bwd(r, A, A, A, A, A, A, A, A, None, 0, None) == NULL
    need = lh.norm_ws_bytes(c)
    assert need > 0 and f.lh_norm_bwd(r, A, A, A, A, A, A, A, None, A, need - 1, None) == WORKSPACE
    assert lh.norm_ws_bytes(norm(M=0)) == 0
    assert f.lh_norm_fwd(ctypes.byref(norm(M=0)), None, None, None, None, None, None, None) == 0   # no rows: no work
    assert lh.launch_count() == before


def rope(**kw):
    c = lh.make_rope_config(2, 16, 4, 2, 64, axes=3)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(N=-1), SHAPE), (dict(B=1 << 16, N=1 << 16), SHAPE), (dict(H=0), SHAPE), (dict(Hk=-1), SHAPE),
    (dict(D=1), SHAPE), (dict(D=1026), SHAPE), (dict(rot=0), SHAPE), (dict(rot=3), SHAPE), (dict(rot=66), SHAPE),
    (dict(axes=0), SHAPE), (dict(axes=9), SHAPE), (dict(q_ld=255), SHAPE), (dict(ko_ld=127), SHAPE), (dict(q_bs=-1), SHAPE),
    (dict(pos_as=-1), SHAPE), (dict(dtype=5), DTYPE), (dict(pairs=2), MODE), (dict(pos64=2), MODE)])
def test_rope_refuses(kw, want):
    assert lh.lib().lh_rope(ctypes.byref(rope(**kw)), A, A, A, A, A, 0, A, A, None) == want


def test_rope_refuses_pointers():
    f, r, before = lh.lib(), ctypes.byref(rope()), lh.launch_count()
    assert f.lh_rope(None, A, A, A, A, A, 0, A, A, None) == NULL
    for at in (0, 1, 2, 3, 4, 6, 7):
        args = [A, A, A, A, A, 0, A, A]
        args[at] = None
        assert f.lh_rope(r, *args, None) == NULL
        args[at] = A + (2 if at == 2 else 8)          # positions: their own alignment suffices
        assert f.lh_rope(r, *args, None) == ALIGN
    assert f.lh_rope(ctypes.byref(rope(N=0)), None, None, None, None, None, 0, None, None, None) == 0
    assert lh.launch_count() == before


def diff(**kw):
    c = lh.make_diff_config(2, 64, 4, 64, Hk=2)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), SHAPE), (dict(T=-2), SHAPE), (dict(T=1 << 30), SHAPE), (dict(T=129), SHAPE), (dict(H=0), SHAPE), (dict(Hk=3), SHAPE),
    (dict(Hk=0), SHAPE), (dict(D=96), SHAPE), (dict(D=256), SHAPE), (dict(ldq=255), SHAPE), (dict(ldq=260), SHAPE),
    (dict(ldk=120), SHAPE), (dict(ldo=8), SHAPE), (dict(dtype=4), DTYPE), (dict(packed=2), MODE), (dict(train=3), MODE)])
def test_diff_refuses(kw, want):
    c, f = diff(**kw), lh.lib()
    assert f.lh_diff_plan(ctypes.byref(c), ctypes.byref(lh.DiffPlan())) == want
    assert f.lh_diff_attn_fwd(ctypes.byref(c), A, A, A, A, None, A, A, 1 << 40, None) == want
    assert f.lh_diff_attn_bwd(ctypes.byref(c), A, A, A, A, A, None, A, 1 << 40, A, 1 << 40, A, A, A, A, None) == want


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_diff_refuses_pointers(dtype):
    f, c = lh.lib(), lh.make_diff_config(2, 64, 4, 64, dtype, Hk=2)
    r, before, pl = ctypes.byref(c), lh.launch_count(), lh.diff_plan(c)
    assert f.lh_diff_plan(r, None) == NULL
    for at in (0, 1, 2, 3, 5, 6):
        args = [A, A, A, A, None, A, A]
        args[at] = None
        assert f.lh_diff_attn_fwd(r, *args, 1 << 40, None) == NULL
        args[at] = A + 8
        assert f.lh_diff_attn_fwd(r, *args, 1 << 40, None) == ALIGN
    assert f.lh_diff_attn_fwd(r, A, A, A, A, None, A, A, pl.saved_bytes - 1, None) == WORKSPACE
    assert f.lh_diff_attn_fwd(r, A, A, A, A, A, A, A, 1 << 40, None) == MODE           # cu without packed
    for at in (0, 1, 2, 3, 4, 6, 8, 10, 11, 12, 13):
        args = [A, A, A, A, A, None, A, 1 << 40, A, 1 << 40, A, A, A, A]
        args[at] = None
        assert f.lh_diff_attn_bwd(r, *args, None) == NULL, at
    assert f.lh_diff_attn_bwd(r, A, A, A, A, A, None, A, 1 << 40, A, pl.ws_bytes - 1, A, A, A, A, None) == WORKSPACE
    packed = lh.make_diff_config(3, 0, 4, 64, dtype, Hk=2, rows=100)
    assert f.lh_diff_attn_fwd(ctypes.byref(packed), A, A, A, A, None, A, A, 1 << 40, None) == NULL   # packed without cu
    infer = lh.make_diff_config(2, 64, 4, 64, dtype, Hk=2, train=False)
    assert lh.diff_plan(infer).saved_bytes < pl.saved_bytes and lh.diff_plan(infer).ws_bytes == 0
    assert f.lh_diff_attn_bwd(ctypes.byref(infer), A, A, A, A, A, None, A, 1 << 40, A, 1 << 40, A, A, A, A, None) == MODE
    empty = lh.make_diff_config(2, 0, 4, 64, dtype)
    assert f.lh_diff_attn_fwd(ctypes.byref(empty), None, None, None, None, None, None, None, 0, None) == 0
    assert lh.launch_count() == before


def test_binding_refuses_tensors_that_do_not_fit():
    """Wrong types, devices and sizes raise in the binding, before the library is asked."""
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    f32 = torch.zeros(8)
    cfg = lh.make_norm_config(8, 64)
    with pytest.raises(ValueError, match="type"):
        lh.norm_fwd(cfg, x.float(), None, None, x)
    with pytest.raises(ValueError, match="ends before"):
        lh.norm_fwd(cfg, x[:7].clone(), None, None, x)
    with pytest.raises(ValueError, match="contiguous"):
        lh.norm_fwd(cfg, x, x[0, :63], None, x)
    with pytest.raises(ValueError, match="on meta"):
        lh.norm_fwd(cfg, x, None, None, x, mean=f32.to("meta"))
    with pytest.raises(ValueError, match="contiguous"):
        lh.norm_fwd(cfg, x, torch.zeros(128, dtype=torch.bfloat16)[::2], None, x)
    rc = lh.make_rope_config(1, 8, 2, 1, 32)
    q, k = torch.zeros(1, 8, 2, 32, dtype=torch.bfloat16), torch.zeros(1, 8, 1, 32, dtype=torch.bfloat16)
    pos, plan = torch.arange(8, dtype=torch.int32), lh.RopePlan(32, device="cpu")
    with pytest.raises(ValueError, match="pos has type"):
        lh.rope(rc, q, k, pos.long(), plan.freq, plan.axis, q, k)
    with pytest.raises(ValueError, match="freq"):
        lh.rope(rc, q, k, pos, plan.freq[:15], plan.axis, q, k)
    with pytest.raises(ValueError, match="ko ends"):
        lh.rope(rc, q, k, pos, plan.freq, plan.axis, q, k[:, :7].clone())
    dc = lh.make_diff_config(1, 8, 2, 64)
    t = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    ws = lh.DiffWorkspace(dc, "cpu")
    with pytest.raises(ValueError, match="lam"):
        lh.diff_attn_fwd(dc, t, t, t, torch.zeros(2), t, ws)
    with pytest.raises(ValueError, match="v ends"):
        lh.diff_attn_fwd(dc, t, t, t[:, :7].clone(), t[0, 0, :, 0], t, ws)
    pc = lh.make_diff_config(2, 0, 2, 64, rows=8)
    with pytest.raises(ValueError, match="cu"):
        lh.diff_attn_fwd(pc, t, t, t, t[0, 0, 0], t, ws)
    with pytest.raises(ValueError, match="cu"):
        lh.diff_attn_fwd(pc, t, t, t, t[0, 0, 0], t, ws, cu=torch.zeros(2, dtype=torch.int32))


def test_functions_refuse_shapes_that_do_not_belong_together():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lh.layer_norm(x, torch.ones(63, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        lh.layer_norm(x, torch.ones(64), torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        lh.layer_norm(x.half())
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    plan = lh.RopePlan(64, device="cpu")
    with pytest.raises(ValueError):
        lh.rotary(q, q[:, :3], torch.arange(4), plan)
    with pytest.raises(ValueError):
        lh.rotary(q, q, torch.arange(4.0), plan)
    with pytest.raises(ValueError):
        lh.rotary(q, q, torch.arange(5), plan)
    with pytest.raises(ValueError):
        lh.differential_attention(q, q, q[:, :3], q[0, 0, :, 0])
    with pytest.raises(ValueError):
        lh.differential_attention(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        lh.differential_attention(q, q, q, q[0, 0, :, 0], cu=torch.zeros(2, dtype=torch.int32))
    for bad in (dict(sections=[1, 2]), dict(sections=[33, -1]), dict(order="other"), dict(ladder="none"), dict(freq=[1.0] * 31)):
        with pytest.raises(ValueError):
            lh.RopePlan(64, device="cpu", **bad)


def test_rope_plan_tables():
    p = lh.RopePlan(16, [4, 2, 2], device="cpu")
    assert p.axis.tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert torch.allclose(p.freq, torch.tensor([10000.0 ** (-i / 8) for i in range(8)], dtype=torch.float64), rtol=1e-15)
    p = lh.RopePlan(16, [4, 2, 2], device="cpu", order="cycle", ladder="own")
    assert p.axis.tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    own = [10000.0 ** (-i / 4) for i in range(4)], [10000.0 ** (-i / 2) for i in range(2)]
    assert torch.allclose(p.freq, torch.tensor([own[0][0], own[1][0], own[1][0], own[0][1], own[1][1], own[1][1], own[0][2], own[0][3]],
                                               dtype=torch.float64), rtol=1e-15)


@pytest.mark.parametrize("kw", [
    dict(B=65537, T=65537), dict(T=1 << 29, H=1 << 12), dict(H=1 << 15, Hk=1 << 14)])
def test_diff_refuses_what_no_grid_holds(kw):
    test_diff_refuses(kw, SHAPE)


def test_in_place_needs_equal_strides():
    f, before = lh.lib(), lh.launch_count()
    c = ctypes.byref(lh.make_norm_config(4, 64, ldx=128))
    assert f.lh_norm_fwd(c, A, A, None, A, None, None, None) == SHAPE
    assert f.lh_norm_bwd(c, A, A + 4096, None, A, A, A, None, None, None, 0, None) == SHAPE
    for kw in (dict(q_ld=512), dict(ko_ld=512), dict(q_bs=1 << 16), dict(ko_bs=1 << 16)):
        assert f.lh_rope(ctypes.byref(rope(**kw)), A, A + 4096, A, A, A, 0, A, A + 4096, None) == SHAPE
    assert lh.launch_count() == before


def test_binding_refuses_strides_that_are_not_the_calls():
    """A view that steps otherwise than the configuration says is refused; one that steps so reaches the library
    (which refuses these calls for other reasons, before any CUDA call)."""
    bf, legacy = torch.bfloat16, types.SimpleNamespace(cuda_stream=None)
    wide = torch.zeros(4, 9, 80, dtype=bf)[:, :5, :64]
    y = torch.empty(20, 64, dtype=bf)
    for x, kw in ((wide, {}), (wide, dict(ldx=80)), (torch.zeros(64, 20, dtype=bf).t(), {}),
                  (torch.zeros(64, dtype=bf).expand(20, 64), {})):
        with pytest.raises(ValueError, match="x has strides"):
            lh.norm_fwd(lh.make_norm_config(20, 64, **kw), x, None, None, y)
    with pytest.raises(lh.LHError, match="status 2"):
        lh.norm_fwd(lh.make_norm_config(20, 64, eps=-1.0, ldx=80), torch.zeros(4, 5, 80, dtype=bf)[..., :64], None, None, y,
                    stream=legacy)
    plan, pos = lh.RopePlan(64, device="cpu"), torch.zeros(1, 2, 8, dtype=torch.int32)
    q, k = torch.zeros(2, 8, 2, 64, dtype=bf), torch.zeros(2, 8, 1, 64, dtype=bf)
    heads_first = torch.zeros(2, 2, 8, 64, dtype=bf).transpose(1, 2)
    for bad in (heads_first, torch.zeros(2, 16, 2, 64, dtype=bf)[:, ::2], torch.zeros(2, 9, 2, 64, dtype=bf)[:, :8]):
        with pytest.raises(ValueError, match="q has strides"):
            lh.rope(lh.make_rope_config(2, 8, 2, 1, 64), bad, k, pos, plan.freq, plan.axis, q, k)
    with pytest.raises(ValueError, match="pos has strides"):
        lh.rope(lh.make_rope_config(2, 8, 2, 1, 64), q, k, torch.zeros(8, 2, dtype=torch.int32).t(), plan.freq, plan.axis, q, k)
    part = torch.zeros(2, 9, 2, 64, dtype=bf)[:, :8]
    rc = lh.make_rope_config(2, 8, 2, 1, 64, q_bs=9 * 128)
    rc.pairs = 5
    with pytest.raises(lh.LHError, match="status 5"):
        lh.rope(rc, part, k, pos, plan.freq, plan.axis, q, k, stream=legacy)
    dc = lh.make_diff_config(2, 8, 2, 64)
    with pytest.raises(ValueError, match="k has strides"):
        lh.diff_attn_fwd(dc, q, heads_first, q, q[0, 0, :, 0].contiguous(), q, lh.DiffWorkspace(dc, "cpu"))
