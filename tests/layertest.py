"""Plain 64-bit forms of the layer operators and bounds on their rounding errors.

U is the half step of fp32, HALF[t] of the output type: a result rounded once
is off by at most HALF[t] times itself. The bounds below count the roundings
of the fp32 arithmetic on the way, each as at most U times the magnitude it
acts on; an accumulation of n values in any order is off by at most n U times
the sum of their magnitudes.
"""

import math

import torch

U = torch.finfo(torch.float32).eps / 2
HALF = {"fp32": U, "bf16": torch.finfo(torch.bfloat16).eps / 2}
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def assert_within(got, ref, tol, what):
    got, ref, tol = got.detach().double().cpu(), ref.double().cpu(), tol.double().cpu()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(((got - ref).abs() / tol.clamp_min(1e-300)).flatten().nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst at {i}: got "
                             f"{got.flatten()[i].item()!r}, want {ref.flatten()[i].item()!r}, allowed {tol.flatten()[i].item():.3g}")


def norm_ref(x, w, b, eps, dy=None):
    """(y, dx, dw, db) in 64 bits and the bounds of their errors without the last rounding."""
    x = x.double().cpu()
    M, d = x.shape
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double().cpu()
    b = torch.zeros(d, dtype=torch.float64) if b is None else b.double().cpu()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    z = (x - mean) * rstd
    y = z * w + b
    # a row's sum: at most 32 values added by a thread, then 5 + 5 levels of a
    # tree, one product with 1/d (itself rounded): the mean is off by 44 U
    # mean|x|; the variance by 44 U of itself plus 2 roundings, rstd by half of
    # that plus its root and quotient: 26 U. z: the mean's error times rstd,
    # rstd's, and the rounding of x - mean and of the product.
    ez = 44 * U * rstd * x.abs().mean(-1, keepdim=True) + 30 * U * z.abs()
    # ... and the variance of a row whose mean is off by e is off by e^2
    ey = ez * w.abs() + 2 * U * ((z * w).abs() + b.abs())
    out = dict(y=(y, ey))
    if dy is not None:
        dy = dy.double().cpu()
        g = dy * w
        c1, c2 = g.mean(-1, keepdim=True), (g * z).mean(-1, keepdim=True)
        dx = rstd * (g - c1 - z * c2)
        a1, a2 = g.abs().mean(-1, keepdim=True), (g * z).abs().mean(-1, keepdim=True)
        e2 = (g.abs() * ez).mean(-1, keepdim=True) + 46 * U * a2
        edx = rstd * (46 * U * a1 + z.abs() * e2 + ez * c2.abs() + 4 * U * (g.abs() + c1.abs() + (z * c2).abs())) + 26 * U * dx.abs()
        # columns: a thread adds at most the rows that fall to it (148 blocks at
        # least when there are more rows than that), then the blocks' partial sums
        n = M / 148 + 64 + 32
        out.update(dx=(dx, edx),
                   dw=((dy * z).sum(0), (dy.abs() * ez).sum(0) + n * U * (dy * z).abs().sum(0)),
                   db=(dy.sum(0), n * U * dy.abs().sum(0)))
    return out


def rope_ref(x, pos, freq, axis, pairs, rot, inverse):
    """x [B, N, heads, D] rotated in 64 bits, and the bound of the error without the last rounding."""
    R = rot // 2
    x = x.double().cpu()
    ang = pos.double().cpu()[axis.long().cpu()].movedim(0, -1) * freq.double().cpu()      # [B, N, R]
    ang = ang[:, :, None]
    c, s = ang.cos(), ang.sin() * (-1 if inverse else 1)
    out, mag = x.clone(), x.abs().clone()
    a = x[..., :R] if pairs == "half" else x[..., 0:rot:2]
    b = x[..., R:rot] if pairs == "half" else x[..., 1:rot:2]
    lo, hi, m = a * c - b * s, b * c + a * s, a.abs() + b.abs()
    # cosine and sine: the reduced angle rounded to fp32 (at most U/2 of a
    # quarter turn), sincospif within 2 steps, so 4 U; the angle in turns within
    # 2^-51 of itself on both sides; two products and a sum: 2 U
    e = (6 * U + 2.0 ** -51 * ang.abs()) * m
    err = torch.zeros_like(x)
    if pairs == "half":
        out[..., :R], out[..., R:rot] = lo, hi
        err[..., :R], err[..., R:rot] = e, e
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = lo, hi
        err[..., 0:rot:2], err[..., 1:rot:2] = e, e
    return out, err


def diff_ref(q, k, v, lam, spans, do=None, op=0.0):
    """Differential attention over token rows: q [T, H, D], k, v [T, Hk, D], spans the (first row, end) of each
    sequence. 64-bit (o, dq, dk, dv, dlam) and the bounds of their errors without the last rounding.

    op: the half step of the rounding that the maps and their gradients get as operands of a matrix product
    (fp16: 2^-11; 0 for fp32 arithmetic). Bounds: a score is a sum of D/2 exact products, off by (D/2 + 4) U of the
    sum of its magnitudes (the scale and the exponent's argument among the 4); twice that, for its row's
    denominator too, plus the exponential (2^-22), is the relative error of a map's value; the sums over keys and
    the rescaling of a running sum add (n/64 + 96) U. Subnormal fp16 operands are off by 2^-25 2^-10 absolutely at
    the scale at which the kernels hold them (the maps times 2^10)."""
    q, k, v, lam = (t.double().cpu() for t in (q, k, v, lam))
    T, H, D = q.shape
    Hk, h = k.shape[1], D // 2
    G, sc = H // Hk, 1 / math.sqrt(h)
    z = lambda t: torch.zeros_like(t)  # noqa: E731
    val = dict(o=z(q), dq=z(q), dk=z(k), dv=z(v), dlam=torch.zeros(H, dtype=torch.float64))
    err = {n: z(t) for n, t in val.items()}
    do = None if do is None else do.double().cpu()
    tiny = 2.0 ** -35 if op else 0.0
    for lo, hi in spans:
        n = hi - lo
        if n == 0:
            continue
        keep = torch.ones(n, n, dtype=torch.bool).tril()
        for hd in range(H):
            Q, K, V = q[lo:hi, hd], k[lo:hi, hd // G], v[lo:hi, hd // G]
            A, R = [], []
            for m in (0, 1):
                a, b = Q[:, m * h:m * h + h], K[:, m * h:m * h + h]
                s = (a @ b.T * sc).masked_fill(~keep, -math.inf)
                mag = (a.abs() @ b.abs().T * sc).masked_fill(~keep, 0).amax(-1, keepdim=True)
                A.append(s.softmax(-1))
                R.append(2 * (h + 4) * U * mag + 2.0 ** -21 + (n / 64 + 96) * U)
            la = lam[hd]
            both = A[0] - la * A[1]
            # what the maps are off by: fp32 first, then as operands
            eA = [A[m] * R[m] for m in (0, 1)]
            eB = eA[0] + la.abs() * eA[1]
            absB = A[0] + la.abs() * A[1]
            eBo = eB + op * absB + tiny * keep
            sums = (n / 8 + 96) * U
            val["o"][lo:hi, hd] = both @ V
            err["o"][lo:hi, hd] = (eBo + sums * absB) @ V.abs()
            if do is None:
                continue
            g = do[lo:hi, hd]
            dP = g @ V.T
            mP = g.abs() @ V.abs().T
            eP = (D + 8) * U * mP
            val["dv"][lo:hi, hd // G] += both.T @ g
            err["dv"][lo:hi, hd // G] += (eBo + sums * absB).T @ g.abs()
            for m, f in ((0, torch.ones((), dtype=torch.float64)), (1, -la)):
                delta = (A[m] * dP).sum(-1, keepdim=True)
                # d = <do, A v>, with the saved A v off like o (and stored in 11 bits where op is set)
                eD = (g.abs() * ((eA[m] + (op + sums) * A[m] + tiny * keep) @ V.abs())).sum(-1, keepdim=True) \
                    + (g.abs() * (A[m] @ V).abs()).sum(-1, keepdim=True) * (op + (D + 8) * U)
                # a query that sees one key: its dS is zero by rule
                live = keep & (torch.arange(n)[:, None] > 0)
                dS = (A[m] * (dP - delta) * f * sc).masked_fill(~live, 0)
                eS = ((eA[m] * (dP - delta).abs() + A[m] * (eP + eD)) * f.abs() * sc + (op + 4 * U) * dS.abs()
                      + tiny * (1 + mP.amax())).masked_fill(~live, 0)
                sl = slice(m * h, m * h + h)
                val["dq"][lo:hi, hd, sl] = dS @ K[:, sl]
                err["dq"][lo:hi, hd, sl] = (eS + sums * dS.abs()) @ K[:, sl].abs()
                val["dk"][lo:hi, hd // G, sl] += dS.T @ Q[:, sl]
                err["dk"][lo:hi, hd // G, sl] += (eS + sums * dS.abs()).T @ Q[:, sl].abs()
                if m == 1:
                    val["dlam"][hd] -= delta.sum()
                    err["dlam"][hd] += eD.sum() + (n / 8 + 96) * U * delta.abs().sum()
    return val, err
