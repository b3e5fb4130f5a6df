"""dlam, the sum over all rows and keys of -A2 dP, where the sum nearly cancels: its terms have to be fp32."""

import pytest
import torch

from layertest import DT, HALF
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_dlam_is_as_exact_as_fp32_terms_make_it(dtype):
    """dout is turned so that each head's sum is about -0.2, of terms whose magnitudes add up to some 30,000.

    What fp32 leaves: a score of order 1 is a sum of 64 products added up in at most 64 steps (order sqrt(64) / 4 half
    steps of 2^-24 at random); its exponent's argument, of order -12, is rounded to 2^-21; the exponential is off by
    2^-22: 2^-21 of a term in all, in the root mean square, doubled here for what the row's denominator adds. These
    errors are independent from term to term, or common to a row (the denominator), so they add up to 2^-20 times the
    2-norms of the terms and of the rows' sums; four times that is allowed, and the rounding of the result. A sum over
    outputs A2 v that were saved in 16 bits is off by far more, and so is 0."""
    N, H, D = 3000, 8, 128
    g = torch.Generator().manual_seed(17)
    q, k, v = (torch.randn(N, H, D, generator=g).to(DT[dtype]).to(DEV) for _ in range(3))
    # 64 bits until it is turned: on the type's grid already, the small turns would round back
    wide = torch.randn(N, H, D, generator=g, dtype=torch.float64).to(DEV)
    do = torch.empty_like(q)
    lam = torch.full((H,), 0.5, dtype=DT[dtype], device=DEV)
    late = torch.ones(N, N, dtype=torch.bool, device=DEV).triu(1)
    want, tol, saved = [], [], {torch.float16: [], torch.bfloat16: []}
    for h in range(H):
        Q, K, V, G = (t[:, h].double() for t in (q, k, v, wide))
        a2 = (Q[:, 64:] @ K[:, 64:].T / 8).masked_fill(late, -torch.inf).softmax(-1)
        o2 = a2 @ V
        G = G - ((G * o2).sum() - 0.2) / (o2 * o2).sum() * o2
        do[:, h] = G.to(DT[dtype])
        G = do[:, h].double()
        want.append(-(G * o2).sum())
        tol.append(4 * 2.0 ** -20 * ((a2 * (G @ V.T)).norm() + (G * o2).sum(-1).norm()) + HALF[dtype] * want[-1].abs())
        for t, e in saved.items():
            e.append(-(G * o2.to(t).double()).sum())
    want, tol = torch.stack(want), torch.stack(tol)
    cfg = lh.make_diff_config(1, N, H, D, dtype)
    ws = lh.DiffWorkspace(cfg, DEV)
    o, dq, dk, dv, dlam = (torch.empty_like(t) for t in (q, q, k, v, lam))
    lh.diff_attn_fwd(cfg, q, k, v, lam, o, ws)
    lh.diff_attn_bwd(cfg, do, q, k, v, lam, ws, dq, dk, dv, dlam)
    torch.cuda.synchronize()
    # the bound tells the forms apart that are not good enough
    for t, e in saved.items():
        assert (torch.stack(e) - want).abs().gt(tol).any(), t
    assert (want.abs() > 10 * tol).all()
    assert ((dlam.double() - want).abs() <= tol).all(), ((dlam.double() - want) / tol).tolist()
