"""Causal differential attention, forward and backward, against its 64-bit form."""

import os

import pytest
import torch

from layertest import DT, HALF, assert_within, diff_ref
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
OP = {"fp32": 0.0, "bf16": torch.finfo(torch.float16).eps / 2}


def rand(seed, *shape, dtype="fp32", mul=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * mul).to(DT[dtype]).to(DEV)


def inputs(seed, T, H, Hk, D, dtype, mul=1.0):
    q, do = rand(seed, T, H, D, dtype=dtype, mul=mul), rand(seed + 1, T, H, D, dtype=dtype)
    k, v = rand(seed + 2, T, Hk, D, dtype=dtype), rand(seed + 3, T, Hk, D, dtype=dtype)
    lam = (0.2 + 0.6 * torch.rand(H, generator=torch.Generator().manual_seed(seed + 4))).to(DT[dtype]).to(DEV)
    return q, k, v, lam, do


def run(cfg, q, k, v, lam, do, cu=None, fill=7.0):
    ws = lh.DiffWorkspace(cfg, DEV)
    ws.saved.fill_(255)          # NaN wherever a value is read that no kernel wrote
    ws.ws.fill_(255)
    o, dq, dk, dv, dlam = (torch.full_like(t, fill) for t in (q, q, k, v, lam))
    lh.diff_attn_fwd(cfg, q, k, v, lam, o, ws, cu=cu)
    lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, dq, dk, dv, dlam, cu=cu)
    torch.cuda.synchronize()
    assert lh.get_device_error() == (0, 0)
    return dict(o=o, dq=dq, dk=dk, dv=dv, dlam=dlam)


def check(got, q, k, v, lam, do, spans, dtype):
    ref, err = diff_ref(q, k, v, lam, spans, do, OP[dtype])
    u = HALF[dtype]
    for n in ref:
        x = got[n].reshape(ref[n].shape)
        if n != "dlam":
            seen = torch.zeros(ref[n].shape[0], dtype=torch.bool)
            for lo, hi in spans:
                seen[lo:hi] = True
            assert (x.cpu()[~seen] == 7).all(), f"{n}: rows outside the sequences were written"
            x, r, e = x.cpu()[seen], ref[n][seen], err[n][seen]
        else:
            r, e = ref[n], err[n]
        assert_within(x, r, u * r.abs() + (1 + u) * e, n)


def spans_of(B, N):
    return [(b * N, b * N + N) for b in range(B)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,N,H,Hk,D", [
    (1, 1, 1, 1, 64), (3, 1, 2, 1, 128), (1, 2, 1, 1, 128), (2, 3, 2, 2, 64), (1, 31, 1, 1, 64), (1, 63, 2, 1, 128), (2, 64, 1, 1, 64),
    (1, 65, 3, 3, 128), (1, 127, 1, 1, 128), (2, 128, 2, 1, 64), (1, 129, 1, 1, 128), (1, 200, 6, 2, 64), (1, 257, 2, 2, 128),
    (2, 300, 4, 1, 128), (1, 511, 1, 1, 64), (1, 640, 2, 1, 128), (1, 1000, 1, 1, 128)])
def test_against_64_bits(B, N, H, Hk, D, dtype):
    q, k, v, lam, do = inputs(11, B * N, H, Hk, D, dtype)
    shape = lambda t: t.view(B, N, *t.shape[1:])  # noqa: E731
    cfg = lh.make_diff_config(B, N, H, D, dtype, Hk)
    got = run(cfg, shape(q), shape(k), shape(v), lam, shape(do))
    check(got, q, k, v, lam, do, spans_of(B, N), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D,H,Hk", [(64, 4, 2), (128, 2, 2)])
@pytest.mark.parametrize("ends,T", [
    ([0, 100, 100, 101, 300, 428], 428),            # an empty sequence, one of one token, a whole number of tiles
    ([0, 0, 0, 5], 9),                              # empty ones first, rows behind the last sequence
    ([17, 80, 209, 337], 400),                      # rows before the first sequence too
    ([0, 0], 12), ([6, 6, 6], 12),                  # nothing at all
    ([0, 1, 2, 3, 4, 5, 6, 7, 8], 8)])              # eight tokens on their own
def test_packed_sequences(ends, T, D, H, Hk, dtype):
    q, k, v, lam, do = inputs(21, T, H, Hk, D, dtype)
    cu = torch.tensor(ends, dtype=torch.int32, device=DEV)
    cfg = lh.make_diff_config(len(ends) - 1, 0, H, D, dtype, Hk, rows=T)
    got = run(cfg, q, k, v, lam, do, cu=cu)
    check(got, q, k, v, lam, do, list(zip(ends, ends[1:])), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_of_others_do_not_leak(dtype):
    """NaN and infinities in the rows around a sequence change no bit of its results."""
    T, H, Hk, D = 420, 2, 1, 128
    q, k, v, lam, do = inputs(31, T, H, Hk, D, dtype)
    cu = torch.tensor([40, 170, 333], dtype=torch.int32, device=DEV)
    cfg = lh.make_diff_config(2, 0, H, D, dtype, Hk, rows=T)
    ref = run(cfg, q, k, v, lam, do, cu=cu)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(DT[dtype]).min):
        dirty = [t.clone() for t in (q, k, v, do)]
        for t in dirty:
            t[:40], t[333:] = bad, bad
        got = run(cfg, *dirty[:3], lam, dirty[3], cu=cu)
        assert all(torch.equal(got[n], ref[n]) for n in ref), bad
    # one sequence's data does not reach the other
    other = [t.clone() for t in (q, k, v, do)]
    for t in other:
        t[170:333] *= 2
    got = run(cfg, *other[:3], lam, other[3], cu=cu)
    assert all(torch.equal(got[n][:170], ref[n][:170]) for n in ("o", "dq", "dk", "dv"))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_fused_projection_strides(dtype):
    """q, k, v as slices of one [T, (H + 2 Hk) D] buffer, gradients into a buffer of the same layout."""
    B, N, H, Hk, D = 2, 150, 4, 2, 64
    W = (H + 2 * Hk) * D
    buf, grad = rand(41, B * N, W, dtype=dtype), torch.full((B * N, W), 7.0, dtype=DT[dtype], device=DEV)
    cut = lambda t: (t[:, :H * D], t[:, H * D:(H + Hk) * D], t[:, (H + Hk) * D:])  # noqa: E731
    _, _, _, lam, _ = inputs(42, 1, H, Hk, D, dtype)
    do, o = rand(43, B * N, H * D + 8, dtype=dtype), torch.full((B * N, H * D + 8), 7.0, dtype=DT[dtype], device=DEV)
    cfg = lh.make_diff_config(B, N, H, D, dtype, Hk, ldq=W, ldk=W, ldv=W, ldo=H * D + 8)
    ws = lh.DiffWorkspace(cfg, DEV)
    dlam = torch.empty_like(lam)
    lh.diff_attn_fwd(cfg, *cut(buf), lam, o, ws)
    lh.diff_attn_bwd(cfg, do, *cut(buf), lam, ws, *cut(grad), dlam)
    torch.cuda.synchronize()
    assert (o[:, H * D:] == 7).all()
    heads = lambda t: t.reshape(B * N, -1, D)  # noqa: E731
    got = dict(zip(("o", "dq", "dk", "dv"), map(heads, (o[:, :H * D], *cut(grad)))), dlam=dlam)
    check(got, *map(heads, cut(buf)), lam, heads(do[:, :H * D]), spans_of(B, N), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("la", [0.0, 1.0, -0.75, 40.0])
def test_lambda_values(la, dtype):
    q, k, v, lam, do = inputs(51, 190, 2, 1, 64, dtype)
    lam = torch.full_like(lam, la)
    cfg = lh.make_diff_config(1, 190, 2, 64, dtype, 1)
    check(run(cfg, q, k, v, lam, do), q, k, v, lam, do, [(0, 190)], dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mq,mk,mv,mo", [(30.0, 1.0, 1.0, 1.0), (2.0 ** 20, 2.0 ** -20, 2.0 ** 18, 2.0 ** -14), (1e-3, 1e-3, 1e-6, 1e-4)])
def test_magnitudes(mq, mk, mv, mo, dtype):
    """Sharp maps (one key takes all), and values far outside the range of fp16."""
    q, k, v, lam, do = inputs(61, 260, 2, 2, 128, dtype)
    q, k, v, do = q * mq, k * mk, v * mv, do * mo
    cfg = lh.make_diff_config(1, 260, 2, 128, dtype, 2)
    check(run(cfg, q, k, v, lam, do), q, k, v, lam, do, [(0, 260)], dtype)


def test_bad_offsets_are_reported():
    q, k, v, lam, do = inputs(71, 64, 1, 1, 64, "fp32")
    cfg = lh.make_diff_config(3, 0, 1, 64, "fp32", rows=64)
    for ends in ([0, 40, 20, 64], [0, 10, 20, 65], [-3, 10, 20, 64], [0, 64, 0, 64]):
        ws, o = lh.DiffWorkspace(cfg, DEV), torch.zeros_like(q)
        lh.diff_attn_fwd(cfg, q, k, v, lam, o, ws, cu=torch.tensor(ends, dtype=torch.int32, device=DEV))
        assert lh.get_device_error() == (9, 402), ends
    assert lh.get_device_error() == (0, 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_inference_equals_training(dtype):
    q, k, v, lam, do = inputs(81, 333, 4, 2, 128, dtype)
    tr, inf = (lh.make_diff_config(1, 333, 4, 128, dtype, 2, train=t) for t in (True, False))
    a, b = torch.empty_like(q), torch.empty_like(q)
    lh.diff_attn_fwd(tr, q, k, v, lam, a, lh.DiffWorkspace(tr, DEV))
    lh.diff_attn_fwd(inf, q, k, v, lam, b, lh.DiffWorkspace(inf, DEV))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_same_bits_every_run_in_graphs_and_on_two_streams(dtype):
    args = [inputs(s, 700, 4, 2, 64, dtype) for s in (91, 191)]
    cu = torch.tensor([0, 130, 131, 500, 700], dtype=torch.int32, device=DEV)
    cfg = lh.make_diff_config(4, 0, 4, 64, dtype, 2, rows=700)
    refs = [run(cfg, *a, cu=cu) for a in args]
    for a, r in zip(args, refs):
        again = run(cfg, *a, cu=cu)
        assert all(torch.equal(again[n], r[n]) for n in r)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in args]
    for a in args:
        q, k, v, lam, do = a
        ws, t = lh.DiffWorkspace(cfg, DEV), [torch.empty_like(x) for x in (q, q, k, v, lam)]

        def step(q=q, k=k, v=v, lam=lam, do=do, ws=ws, t=t):
            lh.diff_attn_fwd(cfg, q, k, v, lam, t[0], ws, cu=cu)
            lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, *t[1:], cu=cu)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
        outs.append(t)
    for t in outs:
        for x in t:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for t, r in zip(outs, refs):
        assert all(torch.equal(x, r[n]) for x, n in zip(t, ("o", "dq", "dk", "dv", "dlam")))


def test_autograd_and_differences():
    """The autograd function (dense and packed) against the formula's gradients, and against central differences."""
    B, N, H, Hk, D = 2, 70, 2, 1, 64
    q, k, v, lam, do = inputs(101, B * N, H, Hk, D, "fp32")
    leaves = [t.view(B, N, *t.shape[1:]).clone().requires_grad_() for t in (q, k, v)] + [lam.clone().requires_grad_()]
    o = lh.differential_attention(*leaves)
    o.backward(do.view(B, N, H, D))
    check(dict(o=o, dq=leaves[0].grad, dk=leaves[1].grad, dv=leaves[2].grad, dlam=leaves[3].grad), q, k, v, lam, do, spans_of(B, N), "fp32")
    f = lambda *a: float((diff_ref(*a, spans_of(B, N))[0]["o"] * do.double().cpu()).sum())  # noqa: E731
    h = 2.0 ** -12
    for n, at in ((0, (75, 1, 40)), (1, (3, 0, 9)), (2, (100, 0, 63)), (3, (1,))):
        a = [t.double().cpu().clone() for t in (q, k, v, lam)]
        a[n][at] += h
        up = f(*a)
        a[n][at] -= 2 * h
        got = float(leaves[n].grad.reshape(a[n].shape)[at])
        # h^2 / 6 of a third derivative of order 10, and the kernel's own error
        assert abs((up - f(*a)) / (2 * h) - got) < 2e-4 * max(1.0, abs(got))
    cu = torch.tensor([0, N, 2 * N], dtype=torch.int32, device=DEV)
    packed = [t.clone().requires_grad_() for t in (q, k, v, lam)]
    o2 = lh.differential_attention(*packed, cu=cu)
    o2.backward(do)
    assert torch.equal(o2.view_as(o), o)
    for a, b in zip(leaves, packed):
        assert torch.equal(a.grad.view_as(b.grad), b.grad)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_dlam_of_a_sum_that_cancels(dtype):
    """dlam is a sum over all rows that can be small beside its terms. Its terms are A2 dP, kept in fp32, so its error
    counts fp32 roundings of the sum of the magnitudes (of which a thread adds n/2 and the rest goes by trees), and a
    single rounding of the result."""
    N, D = 3000, 128
    q, k, v, lam, do = inputs(111, N, 1, 1, D, dtype)
    Q, K, V, G = (t[:, 0].double() for t in (q, k, v, do))
    late = torch.ones(N, N, dtype=torch.bool, device=DEV).triu(1)
    a2 = (Q[:, 64:] @ K[:, 64:].T / 8).masked_fill(late, -torch.inf).softmax(-1)
    terms = a2 * (G @ V.T)
    mag = a2 * (G.abs() @ V.abs().T)
    # the part of do along a2 v that makes the sum nearly vanish is taken out
    o2 = a2 @ V
    do2 = (G - (terms.sum() / (o2 * o2).sum()) * o2).to(DT[dtype]).view(N, 1, D)
    want = -(do2[:, 0].double() * o2).sum()
    cfg = lh.make_diff_config(1, N, 1, D, dtype)
    got = run(cfg, q, k, v, lam, do2)["dlam"].double()
    U = 2.0 ** -24
    # scores of 64 products, scale and exponent: 2 (64 + 4) U |s| <= 2 * 68 * 16 U relative, the exponential 2^-21, the
    # products and sums of dP 136 U, the sum over columns (N / 2 + 64) U; statistically independent, so their root mean
    # square over the terms carries into the sum: sqrt(sum of squares) times 8 covers it
    rel = (2 * 68 * 16 + 136 + 64 + 2 ** 3) * U + 2.0 ** -21
    tol = 8 * rel * float(mag.square().sum().sqrt()) + (N / 2 + 64) * U * float(terms.abs().sum()) / N ** 0.5
    assert abs(float(got - want)) <= tol + HALF[dtype] * abs(float(want)), (float(got), float(want), tol)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_saved_buffer_of_another_problem_is_not_followed(dtype):
    q, k, v, lam, do = inputs(121, 300, 2, 1, 64, dtype)
    cfg = lh.make_diff_config(1, 300, 2, 64, dtype, 1)
    other = lh.make_diff_config(2, 150, 2, 64, dtype, 1)      # the same rows, cut otherwise
    ws, o = lh.DiffWorkspace(other, DEV), torch.empty_like(q)   # as large as either needs
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    dlam = torch.empty_like(lam)
    ws.saved.fill_(255)                               # never written
    lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, *grads, dlam)
    assert lh.get_device_error() == (9, 404)
    lh.diff_attn_fwd(other, q, k, v, lam, o, ws)
    lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, *grads, dlam)
    assert lh.get_device_error() == (9, 404)
    assert all((t == 7).all() for t in grads)


def test_non_finite_values_are_reported_and_stay_in_their_head():
    q, k, v, lam, do = inputs(131, 200, 4, 2, 128, "bf16")
    cfg = lh.make_diff_config(1, 200, 4, 128, "bf16", 2)
    ref = run(cfg, q, k, v, lam, do)
    v2 = v.clone()
    v2[77, 1, 5] = float("nan")
    ws, o = lh.DiffWorkspace(cfg, DEV), torch.empty_like(q)
    lh.diff_attn_fwd(cfg, q, k, v2, lam, o, ws)
    assert lh.get_device_error() == ((0, 0) if os.environ.get("LH_ATTN_SIMT", "").startswith("1") else (9, 102))
    assert torch.equal(o[:, :2], ref["o"][:, :2]) and o[77:, 2:].isnan().any(-1).all()
    assert torch.equal(run(cfg, q, k, v, lam, do)["dk"], ref["dk"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_short_sequences(dtype):
    """1,500 sequences of 0 to 3 tokens."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (1500,), generator=g)
    ends = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T = int(ends[-1])
    q, k, v, lam, do = inputs(141, T, 1, 1, 64, dtype)
    cfg = lh.make_diff_config(1500, 0, 1, 64, dtype, rows=T)
    got = run(cfg, q, k, v, lam, do, cu=ends.to(torch.int32).to(DEV))
    check(got, q, k, v, lam, do, list(zip(ends.tolist(), ends[1:].tolist())), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_offsets_past_32_bits(dtype):
    """Token rows 2^24 elements apart: the last ones start beyond element 2^31."""
    N, D, ld = 140, 64, 1 << 24
    q, k, v, lam, do = inputs(151, N, 1, 1, D, dtype)
    far = torch.empty((N - 1) * ld + D, dtype=DT[dtype], device=DEV).as_strided((N, D), (ld, 1))
    far.copy_(k[:, 0])
    want = run(lh.make_diff_config(1, N, 1, D, dtype), q, k, v, lam, do)["o"]
    cfg = lh.make_diff_config(1, N, 1, D, dtype, ldk=ld)
    o = torch.empty_like(q)
    lh.diff_attn_fwd(cfg, q, far, v, lam, o, lh.DiffWorkspace(cfg, DEV))
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_without_gradients_nothing_is_kept_for_them(dtype, monkeypatch):
    q, k, v, lam, do = inputs(161, 130, 2, 1, 64, dtype)
    q, k, v = (t[None] for t in (q, k, v))
    made, make = [], lh.make_diff_config
    monkeypatch.setattr(lh, "make_diff_config", lambda *a, **kw: made.append(make(*a, **kw)) or made[-1])
    a = lh.differential_attention(q, k, v, lam)
    with torch.no_grad():
        b = lh.differential_attention(q.clone().requires_grad_(), k, v, lam)
    c = lh.differential_attention(q, k, v, lam.clone().requires_grad_())
    c.backward(do[None])
    assert [m.train for m in made] == [0, 0, 1]
    assert torch.equal(a, b) and torch.equal(a, c.detach()) and lh.get_device_error() == (0, 0)


@pytest.mark.parametrize("dtype,G", [("fp32", 1), ("bf16", 1), ("bf16", 2)])
def test_heads_that_do_not_fit_l2_together(dtype, G):
    """400 sequences of 200 tokens: the tiles of three key/value heads are taken in more than one group. Each head by
    itself gives the same bits."""
    B, N, Hk, D = 400, 200, 3, 64
    q, k, v, lam, do = inputs(171, B * N, Hk * G, Hk, D, dtype)
    got = run(lh.make_diff_config(B, N, Hk * G, D, dtype, Hk), q, k, v, lam, do)
    one = lh.make_diff_config(B, N, G, D, dtype, 1)
    for h in range(Hk):
        heads, kv = slice(h * G, h * G + G), slice(h, h + 1)
        ref = run(one, q[:, heads].contiguous(), k[:, kv].contiguous(), v[:, kv].contiguous(), lam[heads].clone(),
                  do[:, heads].contiguous())
        for n, at in (("o", heads), ("dq", heads), ("dk", kv), ("dv", kv)):
            assert torch.equal(got[n][:, at], ref[n]), (n, h)
        assert torch.equal(got["dlam"][heads], ref["dlam"])
