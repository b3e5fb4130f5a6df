"""Layer norm, forward and backward, against its 64-bit form."""

import ctypes
import threading

import pytest
import torch

from layertest import DT, HALF, assert_within, norm_ref
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
EPS = 1e-5


def rand(seed, *shape, dtype="fp32", mean=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) + mean).to(DT[dtype]).to(DEV)


def run(x, w, b, dy, dtype, wdtype, eps=EPS, ldx=0, ldy=0, M=None, d=None):
    M, d = x.shape[0] if M is None else M, x.shape[1] if d is None else d
    cfg = lh.make_norm_config(M, d, dtype, wdtype, eps, ldx, ldy)
    y, dx = torch.full_like(dy, 7.0), torch.full_like(x, 7.0)
    mean, rstd = (torch.empty(M, device=DEV) for _ in range(2))
    dw, db = (None if t is None else torch.full((d,), 7.0, dtype=DT[wdtype], device=DEV) for t in (w, b))
    lh.norm_fwd(cfg, x, w, b, y, mean, rstd)
    lh.norm_bwd(cfg, dy, x, w, mean, rstd, dx, dw, db, lh.norm_workspace(cfg, DEV))
    torch.cuda.synchronize()
    return dict(y=y, dx=dx, dw=dw, db=db)


def check(got, x, w, b, dy, dtype, wdtype, eps=EPS):
    for n, (ref, err) in norm_ref(x, w, b, eps, dy).items():
        if got[n] is not None:
            u = HALF[wdtype if n in ("dw", "db") else dtype]
            # a result below the type's normal range keeps an absolute half step
            assert_within(got[n], ref, u * ref.abs() + (1 + u) * err + 2.0 ** -134, n)


@pytest.mark.parametrize("M,d", [(1, 1), (3, 1), (5, 2), (7, 3), (1, 8), (33, 31), (64, 32), (65, 33), (130, 64), (1000, 128),
                                 (9, 255), (17, 256), (17, 257), (300, 1024), (50, 1537), (11, 2048), (5, 8192), (3, 8193), (4, 8200),
                                 (3, 16383), (5, 16384)])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_against_64_bits(M, d, dtype, wdtype):
    x, dy = rand(1, M, d, dtype=dtype, mean=0.5), rand(2, M, d, dtype=dtype)
    w, b = rand(3, d, dtype=wdtype, mean=1.0), rand(4, d, dtype=wdtype)
    check(run(x, w, b, dy, dtype, wdtype), x, w, b, dy, dtype, wdtype)


@pytest.mark.parametrize("M,d", [(40000, 32), (20000, 40), (5000, 512), (3000, 36)])
def test_many_rows(M, d):
    """More rows than resident groups: several passes of every block."""
    x, dy = rand(1, M, d, dtype="bf16"), rand(2, M, d, dtype="bf16")
    w, b = rand(3, d, mean=1.0), rand(4, d)
    check(run(x, w, b, dy, "bf16", "fp32"), x, w, b, dy, "bf16", "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_weight_or_bias(dtype):
    x, dy = rand(1, 37, 100, dtype=dtype), rand(2, 37, 100, dtype=dtype)
    w, b = rand(3, 100, dtype=dtype), rand(4, 100, dtype=dtype)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check(run(x, ww, bb, dy, dtype, dtype), x, ww, bb, dy, dtype, dtype)


@pytest.mark.parametrize("ldx,ldy", [(72, 80), (67, 0), (0, 129), (64, 64)])
def test_row_strides_leave_the_gaps_alone(ldx, ldy):
    M, d = 21, 64
    xs, ys = rand(1, M, ldx or d, dtype="bf16"), rand(2, M, ldy or d, dtype="bf16")
    w, b = rand(3, d, dtype="bf16"), rand(4, d, dtype="bf16")
    got = run(xs, w, b, ys, "bf16", "bf16", ldx=ldx, ldy=ldy, M=M, d=d)
    assert (got["y"][:, d:] == 7).all() and (got["dx"][:, d:] == 7).all()
    got["y"], got["dx"] = got["y"][:, :d], got["dx"][:, :d]
    check(got, xs[:, :d], w, b, ys[:, :d], "bf16", "bf16")


def test_large_mean_and_constant_rows():
    """A mean 1000 times the deviation; rows of one value (variance 0); infinities and NaN stay in their row."""
    x, dy = rand(1, 12, 96, mean=0.0), rand(2, 12, 96)
    x[:4] += 1000.0
    x[4:6] = 3.25
    w, b = rand(3, 96), rand(4, 96)
    check(run(x, w, b, dy, "fp32", "fp32"), x, w, b, dy, "fp32", "fp32")
    bad = x.clone()
    bad[7, 5], bad[8, 6] = float("inf"), float("nan")
    got, ref = run(bad, w, b, dy, "fp32", "fp32"), run(x, w, b, dy, "fp32", "fp32")
    keep = [i for i in range(12) if i not in (7, 8)]
    assert torch.equal(got["y"][keep], ref["y"][keep]) and torch.equal(got["dx"][keep], ref["dx"][keep])
    assert got["y"][7:9].isnan().any(1).all()


def test_no_rows_give_zero_gradients():
    w = rand(3, 40, dtype="bf16")
    cfg = lh.make_norm_config(0, 40)
    e = torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    f = torch.empty(0, device=DEV)
    dw, db = torch.full_like(w, 7.0), torch.full_like(w, 7.0)
    lh.norm_fwd(cfg, e, w, w, e, f, f)
    lh.norm_bwd(cfg, e, e, w, f, f, e, dw, db, None)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_in_place():
    x, dy = rand(1, 300, 128, dtype="bf16"), rand(2, 300, 128, dtype="bf16")
    w, b = rand(3, 128, dtype="bf16"), rand(4, 128, dtype="bf16")
    ref = run(x, w, b, dy, "bf16", "bf16")
    cfg = lh.make_norm_config(300, 128)
    mean, rstd = (torch.empty(300, device=DEV) for _ in range(2))
    x2, dy2, dw, db = x.clone(), dy.clone(), torch.empty_like(w), torch.empty_like(b)
    lh.norm_fwd(cfg, x2, w, b, x2, mean, rstd)
    lh.norm_bwd(cfg, dy2, x, w, mean, rstd, dy2, dw, db, lh.norm_workspace(cfg, DEV))
    torch.cuda.synchronize()
    assert torch.equal(x2, ref["y"]) and torch.equal(dy2, ref["dx"]) and torch.equal(dw, ref["dw"]) and torch.equal(db, ref["db"])


def test_same_bits_every_run_and_in_a_graph():
    x, dy = rand(1, 5000, 384, dtype="bf16"), rand(2, 5000, 384, dtype="bf16")
    w, b = rand(3, 384), rand(4, 384)
    ref = run(x, w, b, dy, "bf16", "fp32")
    cfg = lh.make_norm_config(5000, 384, "bf16", "fp32", EPS)
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    mean, rstd, ws = torch.empty(5000, device=DEV), torch.empty(5000, device=DEV), lh.norm_workspace(cfg, DEV)

    def step():
        lh.norm_fwd(cfg, x, w, b, y, mean, rstd)
        lh.norm_bwd(cfg, dy, x, w, mean, rstd, dx, dw, db, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (y, dx, dw, db):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for n, t in dict(y=y, dx=dx, dw=dw, db=db).items():
            assert torch.equal(t, ref[n]), n


def test_autograd_and_differences():
    """The autograd function against the formula's gradients, and against central differences of the 64-bit form."""
    x, w, b = rand(1, 2, 3, 40), rand(3, 40, mean=1.0), rand(4, 40)
    dy = rand(2, 2, 3, 40)
    xg, wg, bg = (t.clone().requires_grad_() for t in (x, w, b))
    lh.layer_norm(xg, wg, bg, EPS).backward(dy)
    check(dict(y=None, dx=xg.grad.view(6, 40), dw=wg.grad, db=bg.grad), x.view(6, 40), w, b, dy.view(6, 40), "fp32", "fp32")
    f = lambda x, w, b: float((norm_ref(x.view(6, 40), w, b, EPS)["y"][0] * dy.view(6, 40).double().cpu()).sum())  # noqa: E731
    h = 2.0 ** -13
    for grad, at, args in ((xg.grad.view(6, 40), (1, 7), 0), (wg.grad, (5,), 1), (bg.grad, (9,), 2)):
        a = [t.double().cpu().clone() for t in (x.view(6, 40), w, b)]
        a[args][at] += h
        up = f(*a)
        a[args][at] -= 2 * h
        # the difference's own error: h^2 / 6 of a third derivative of order 10, 64-bit rounding / h
        assert abs((up - f(*a)) / (2 * h) - float(grad[at])) < 1e-5
    # a frozen weight, a strided input and an odd offset
    y = lh.layer_norm(x.transpose(0, 1), w, None)
    assert_within(y.reshape(6, 40), norm_ref(x.transpose(0, 1).reshape(6, 40), w, None, EPS)["y"][0],
                  torch.full((6, 40), 1e-5), "strided")
    flat = rand(5, 1 + 3 * 33)
    y = lh.layer_norm(flat[1:].view(3, 33))
    assert_within(y, norm_ref(flat[1:].view(3, 33), None, None, EPS)["y"][0], torch.full((3, 33), 1e-5), "odd offset")


def test_another_stream():
    x, dy = rand(1, 4000, 256, dtype="bf16"), rand(2, 4000, 256, dtype="bf16")
    w = rand(3, 256, dtype="bf16")
    ref = run(x, w, w, dy, "bf16", "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(x, w, w, dy, "bf16", "bf16")
    assert all(torch.equal(got[n], ref[n]) for n in ref)


def test_offsets_past_32_bits():
    """Rows 2^25 elements apart: the last ones start beyond element 2^31."""
    M, d, ld = 70, 320, 1 << 25
    x, w = rand(1, M, d, dtype="bf16"), rand(3, d, dtype="bf16")
    far = torch.empty((M - 1) * ld + d, dtype=torch.bfloat16, device=DEV).as_strided((M, d), (ld, 1))
    far.copy_(x)
    a, b = torch.empty_like(x), torch.empty_like(x)
    lh.norm_fwd(lh.make_norm_config(M, d), x, w, None, a)
    lh.norm_fwd(lh.make_norm_config(M, d, ldx=ld), far, w, None, b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_two_host_threads_with_rows_of_unlike_length():
    """Rows of more than 8,192 values keep their columns' sums in shared memory, as much as their length takes: calls of
    two lengths from two host threads at once do not get in each other's way. (The C function itself: the binding's own
    work between two calls would keep the threads apart.)"""
    f, keep = lh.lib().lh_norm_bwd, []

    def job(d):
        x, dy, w = rand(1, 2, d, dtype="bf16"), rand(2, 2, d, dtype="bf16"), rand(3, d, dtype="bf16")
        cfg, one = lh.make_norm_config(2, d), torch.ones(2, device=DEV)
        ts = (dy, x, w, one, one, torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), lh.norm_workspace(cfg, DEV))
        stream = torch.cuda.Stream()
        keep.append((cfg, ts, stream))
        return ctypes.byref(cfg), *(t.data_ptr() for t in ts), ts[-1].numel(), stream.cuda_stream

    jobs = [job(16384), job(8200)]
    states, go = [set(), set()], threading.Barrier(len(jobs))
    torch.cuda.synchronize()

    def loop(args, seen):
        go.wait()
        for _ in range(20000):
            seen.add(f(*args))

    threads = [threading.Thread(target=loop, args=a) for a in zip(jobs, states)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert states == [{0}, {0}]
