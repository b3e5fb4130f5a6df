"""Gradients of differential attention whose rows differ by many powers of two: every row, and every key, is held to
its own size. bf16 runs on fp16 copies, so this is where a power shared by rows that do not belong together would show.

Bounds. As in layertest.diff_ref, with the absolute part row by row. fp16 subnormals are off by 2^-25 in the units
that a kernel holds a value in:
- the copies: a row's (do) or a head's (v) largest value lies in [1/8, 256), so an element is off by 2^-25 of 8 times
  that largest value at most, 2^-22 of it, and so are the saved outputs A v;
- dq: dS is held at 2^sh = 2^14 / (2^x 2^y) with 2^x <= 2 |do row|_1 and 2^y <= 2 max |v|, so it is off by
  2^-25 2^-14 4 |do row|_1 max |v| = 2^-37 |do row|_1 max |v|;
- dk: the same with the largest do row that its key's 128-key tile sees, and with max(1, |lam|) (a power of two again);
- dv: the maps are held at 2^sp times the row's power over the walk's largest, 2^sp (1 + |lam|) >= 2^12; two
  roundings (A1, then the difference), each 2^-25 2^-12 (1 + |lam|) of the copy's 8 and of 8 times the walk's largest do.
"""

import math
import os

import pytest
import torch

from layertest import DT, HALF, U, assert_within
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
SIMT = os.environ.get("LH_ATTN_SIMT", "").startswith("1")      # bf16 in fp32 arithmetic, which reports nothing
OP = {"fp32": 0.0, "bf16": torch.finfo(torch.float16).eps / 2}


def rand(seed, *shape, dtype="fp32"):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).to(DEV)


def gradients(q, k, v, lam, do, dtype, cu=None):
    T, H, D = q.shape
    cfg = lh.make_diff_config(1 if cu is None else cu.numel() - 1, T, H, D, dtype, k.shape[1], rows=None if cu is None else T)
    ws = lh.DiffWorkspace(cfg, DEV)
    ws.saved.fill_(255)
    if ws.ws is not None:
        ws.ws.fill_(255)
    o, dq, dk, dv, dlam = (torch.full_like(t, 7.0) for t in (q, q, k, v, lam))
    lh.diff_attn_fwd(cfg, q, k, v, lam, o, ws, cu=cu)
    lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, dq, dk, dv, dlam, cu=cu)
    torch.cuda.synchronize()
    assert lh.get_device_error() == (0, 0)
    return dict(dq=dq, dk=dk, dv=dv, dlam=dlam)


def reference(q, k, v, lam, do, op):
    """One sequence: gradients in 64 bits, and the bounds of their errors without the last rounding."""
    q, k, v, lam, do = (t.double() for t in (q, k, v, lam, do))
    n, H, D = q.shape
    h, G, sc = D // 2, H // k.shape[1], 1 / math.sqrt(D // 2)
    keep = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
    live = keep & (torch.arange(n, device=DEV)[:, None] > 0)     # a query that sees one key: its dS is zero by rule
    val = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v), dlam=torch.zeros_like(lam))
    err = {x: torch.zeros_like(t) for x, t in val.items()}
    sums = (n / 8 + 96) * U
    first = torch.arange(n, device=DEV) // 128 * 128              # the first query of a key's walk
    for kv in range(k.shape[1]):
        heads = range(kv * G, kv * G + G)
        V, mv = v[:, kv], v[:, kv].abs().max()
        lm = float(lam[kv * G:kv * G + G].abs().max())
        # the largest row of do, by its 1-norm and by its largest value, that the walk of each key sees
        size = torch.stack([do[:, x].abs().sum(-1) for x in heads]).amax(0)
        top = torch.stack([do[:, x].abs().amax(-1) for x in heads]).amax(0)
        walk = lambda t: t.flip(0).cummax(0).values.flip(0)[first]  # noqa: E731
        wn, wt = walk(size), walk(top)
        for x in heads:
            g, la = do[:, x], lam[x]
            A, eA = [], []
            for m in (0, 1):
                a, b = q[:, x, m * h:m * h + h], k[:, kv, m * h:m * h + h]
                s = (a @ b.T * sc).masked_fill(~keep, -math.inf)
                mag = (a.abs() @ b.abs().T * sc).masked_fill(~keep, 0).amax(-1, keepdim=True)
                A.append(s.softmax(-1))
                eA.append(A[m] * (2 * (h + 4) * U * mag + 2.0 ** -21 + (n / 64 + 96) * U))
            both, absB = A[0] - la * A[1], A[0] + la.abs() * A[1]
            dP, mP = g @ V.T, g.abs() @ V.abs().T
            small = bool(op) * 2.0 ** -22
            eP = (D + 8) * U * mP + small * (g.abs().sum(-1, keepdim=True) * mv + g.abs().amax(-1, keepdim=True) * V.abs().sum(-1))
            val["dv"][:, kv] += both.T @ g
            eB = eA[0] + la.abs() * eA[1] + (2 * op + sums) * absB
            err["dv"][:, kv] += eB.T @ g.abs()
            err["dv"][:, kv] += bool(op) * n * 2 * 2.0 ** -37 * (1 + lm) * 64 * wt[:, None]
            err["dv"][:, kv] += small * (both.abs().T @ g.abs().amax(-1, keepdim=True))
            for m, f in ((0, 1.0), (1, -la)):
                delta = (A[m] * dP).sum(-1, keepdim=True)
                eD = (g.abs() * ((eA[m] + (op + sums) * A[m]) @ V.abs())).sum(-1, keepdim=True) \
                    + (g.abs() * (A[m] @ V).abs()).sum(-1, keepdim=True) * (op + (D + 8) * U) \
                    + 2 * small * g.abs().sum(-1, keepdim=True) * mv
                dS = (A[m] * (dP - delta) * f * sc).masked_fill(~live, 0)
                eS = (eA[m] * (dP - delta).abs() + A[m] * (eP + eD)) * abs(f) * sc + (op + 4 * U) * dS.abs()
                tiny = bool(op) * 2.0 ** -37 * mv * sc
                sl = slice(m * h, m * h + h)
                K, Q = k[:, kv, sl], q[:, x, sl]
                eq = (eS + tiny * abs(f) * g.abs().sum(-1, keepdim=True)).masked_fill(~live, 0)
                ek = (eS + tiny * max(1.0, 2 * lm) * wn).masked_fill(~live, 0)
                val["dq"][:, x, sl] = dS @ K
                err["dq"][:, x, sl] = (eq + sums * dS.abs()) @ K.abs()
                val["dk"][:, kv, sl] += dS.T @ Q
                err["dk"][:, kv, sl] += (ek + sums * dS.abs()).T @ Q.abs()
                if m == 1:
                    val["dlam"][x] -= delta.sum()
                    err["dlam"][x] += (eD + (A[m] * eP).sum(-1, keepdim=True)).sum() + sums * delta.abs().sum()
    return val, err


def check(got, q, k, v, lam, do, dtype):
    val, err = reference(q, k, v, lam, do, OP[dtype])
    u = HALF[dtype]
    for n in val:
        assert_within(got[n], val[n], u * val[n].abs() + (1 + u) * err[n], n)


def spread(kind, T, H):
    """Powers of two of do's rows."""
    i = torch.arange(T)
    e = {"mixed": -((i * 7) % 41), "late rows small": -40 * (i >= T // 2), "late rows large": -40 * (i < T // 2),
         "one large": -30 * (i != 5), "falling": -(i * 50 // T)}[kind]
    e = e[:, None].repeat(1, H)
    e[:, 1:] = e[:, 1:].flip(0)          # another head, the other way round
    return torch.exp2(e.float())[..., None].to(DEV)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["mixed", "late rows small", "late rows large", "one large", "falling"])
@pytest.mark.parametrize("T,H,Hk,D,outlier", [(700, 2, 1, 128, 100.0), (515, 2, 2, 64, 1.0)])
def test_every_row_to_its_own_size(kind, T, H, Hk, D, outlier, dtype):
    q, k, v = rand(1, T, H, D, dtype=dtype), rand(2, T, Hk, D, dtype=dtype), rand(3, T, Hk, D, dtype=dtype)
    v[T // 3, :, 9] = outlier
    lam = torch.tensor([0.4, -0.7], dtype=DT[dtype], device=DEV)
    do = (rand(4, T, H, D) * spread(kind, T, H)).to(DT[dtype])
    check(gradients(q, k, v, lam, do, dtype), q, k, v, lam, do, dtype)


def steps(seed, *shape):
    """Values that fp16 holds exactly whatever the power of two: +- (1 .. 7) / 4."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(1, 8, shape, generator=g) * (2 * torch.randint(0, 2, shape, generator=g) - 1) / 4).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("T,H,Hk,D", [(900, 2, 1, 128), (900, 4, 2, 64)])
def test_a_row_times_a_power_of_two(T, H, Hk, D):
    """do's rows times powers of two of their own: dq's rows come out times the same powers, bit for bit; and keys
    that only see rows of one common power take it too."""
    q, k, v, do = rand(1, T, H, D, dtype="bf16"), rand(2, T, Hk, D, dtype="bf16"), rand(3, T, Hk, D, dtype="bf16"), steps(4, T, H, D)
    lam = torch.linspace(0.2, 0.8, H).to(torch.bfloat16).to(DEV)
    ref = gradients(q, k, v, lam, do, "bf16")
    p = torch.exp2(torch.randint(-40, 41, (T, H, 1), generator=torch.Generator().manual_seed(9)).float()).to(DEV)
    got = gradients(q, k, v, lam, (do * p).to(torch.bfloat16), "bf16")
    assert torch.equal(got["dq"], (ref["dq"] * p).to(torch.bfloat16))
    p = torch.ones(T, 1, 1, device=DEV)
    p[384:] = 2.0 ** -40
    got = gradients(q, k, v, lam, (do * p).to(torch.bfloat16), "bf16")
    for n in ("dk", "dv"):
        assert torch.equal(got[n][384:], (ref[n][384:] * p[384:]).to(torch.bfloat16)), n


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_zeros_and_no_gradient_at_all(D):
    """Zero rows among tiny ones leave the tiny ones their bits; all zeros give zeros."""
    T, H, Hk = 600, 2, 1
    q, k, v = rand(1, T, H, D, dtype="bf16"), rand(2, T, Hk, D, dtype="bf16"), rand(3, T, Hk, D, dtype="bf16")
    lam = torch.full((H,), 0.5, dtype=torch.bfloat16, device=DEV)
    do = (rand(4, T, H, D) * 2.0 ** -45).to(torch.bfloat16)
    do[::3] = 0
    do[256:384] = 0
    got = gradients(q, k, v, lam, do, "bf16")
    check(got, q, k, v, lam, do, "bf16")
    assert not got["dq"][::3].any()
    got = gradients(q, k, v, lam, torch.zeros_like(do), "bf16")
    assert not any(t.any() for t in got.values())


def test_packed_sequences_of_unlike_size():
    """A sequence whose do is 2^40 times another's, tiles of one next to tiles of the other."""
    T, H, Hk, D = 1000, 4, 2, 64
    ends = [0, 130, 131, 400, 400, 717, 1000]
    q, k, v, do = rand(1, T, H, D, dtype="bf16"), rand(2, T, Hk, D, dtype="bf16"), rand(3, T, Hk, D, dtype="bf16"), rand(4, T, H, D)
    lam = torch.linspace(0.2, 0.8, H).to(torch.bfloat16).to(DEV)
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        do[lo:hi] *= 2.0 ** (-20 * (i % 3))
    do = do.to(torch.bfloat16)
    got = gradients(q, k, v, lam, do, "bf16", cu=torch.tensor(ends, dtype=torch.int32, device=DEV))
    for lo, hi in zip(ends, ends[1:]):
        if hi > lo:
            part = [t[lo:hi] for t in (q, k, v)]
            val, err = reference(*part, lam, do[lo:hi], OP["bf16"])
            for n in ("dq", "dk", "dv"):
                assert_within(got[n][lo:hi], val[n], HALF["bf16"] * val[n].abs() + 1.01 * err[n], (n, lo))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mul", [1.0, 2.0 ** 20, 2.0 ** -20])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_not_finite_stays_in_its_row(bad, mul, dtype):
    """Whatever size the other queries have: their outputs and gradients keep their bits."""
    T, H, Hk, D, row = 300, 4, 2, 64, 171
    q, k, v, do = (rand(i, T, n, D, dtype=dtype) for i, n in enumerate((H, Hk, Hk, H)))
    q, k, lam = q * mul, k / mul, torch.full((H,), 0.5, dtype=DT[dtype], device=DEV)
    cfg = lh.make_diff_config(1, T, H, D, dtype, Hk)

    def run(q, do):
        ws = lh.DiffWorkspace(cfg, DEV)
        o, dq, dk, dv, dlam = (torch.empty_like(t) for t in (q, q, k, v, lam))
        lh.diff_attn_fwd(cfg, q, k, v, lam, o, ws)
        lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, dq, dk, dv, dlam)
        torch.cuda.synchronize()
        return lh.get_device_error()[1], o, dq, dk, dv, dlam

    code, *ref = run(q, do)
    assert code == 0 and all(t.isfinite().all() for t in ref)
    q2, do2 = q.clone(), do.clone()
    q2[row, 1, 3] = do2[row, 1, 5] = bad
    same = torch.ones(T, H, dtype=torch.bool, device=DEV)
    same[row, 1] = False
    for args in ((q2, do), (q, do2)):
        code, o, dq, dk, dv, dlam = run(*args)
        assert code in ((0,) if dtype == "fp32" or SIMT else (101, 102))
        assert torch.equal(o[same], ref[0][same]) and torch.equal(dq[same], ref[1][same])
        assert not dq[~same].isfinite().all()
        assert torch.equal(dk[:, 1], ref[2][:, 1]) and torch.equal(dv[:, 1], ref[3][:, 1])
        keep = [0, 2, 3]
        assert torch.equal(dlam[keep], ref[4][keep])
