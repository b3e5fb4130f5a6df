"""The operators around the attention of a layer, as a training program runs them, with their plain forms.

Three operators, which one differential attention layer over long contexts runs in this order:

  norm    layer norm of the rows of a matrix, y = (x - mean) / sqrt(var + eps) * w + b, in front of the
          projections (one row per token) and on each head's attention output (one row per token and head),
          with its backward pass and the reduction of the weight's and the bias's gradient;
  rope    rotary positions of the queries and keys over one or several axes (a text position; or time, height
          and width of a video token), and the inverse rotation, which is its backward pass;
  diff    causal differential attention: each head's q and k rows hold two maps (first and second half of the
          row); o = softmax(q1 k1^T / sqrt(D/2)) v - lam[h] softmax(q2 k2^T / sqrt(D/2)) v, over a batch of
          equal sequences or over sequences packed one behind the other (cu: their offsets), query heads
          sharing key/value heads, with its backward pass (dq, dk, dv, dlam).

`listed()` names the cases that stand for the real ranges, `draw()` gives others. `own` False: the plain
forms, in elementary torch operations. `own` True: the calls of long_context_symmetric_b200.lh.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # 64 tokens of a short validation prompt at the width of the 98K-context layer (16 heads of 64): latency
        {"name": "norm_prompt", "op": "norm", "rows": 64, "d": 1024, "dtype": "bf16", "wdtype": "bf16", "train": False},
        # the norm in front of the projections of a 98K-context layer with 16 heads of 128, training, fp32 weights
        {"name": "norm_98k", "op": "norm", "rows": 98304, "d": 2048, "dtype": "bf16", "wdtype": "fp32", "train": True},
        # head-wise norm of the attention output: 131,072 tokens of 8 heads of 128, one row per token and head
        {"name": "norm_heads", "op": "norm", "rows": 1048576, "d": 128, "dtype": "bf16", "wdtype": "bf16", "train": True},
        # an odd width and an odd number of rows in fp32, as in a parity run against a small model
        {"name": "norm_odd", "op": "norm", "rows": 5003, "d": 1537, "dtype": "fp32", "wdtype": "fp32", "train": True},
        # one short prompt, text positions: latency
        {"name": "rope_prompt", "op": "rope", "B": 1, "N": 256, "H": 16, "Hk": 16, "D": 128, "rot": 128, "axes": 1,
         "pairs": "half", "dtype": "bf16", "inverse": False},
        # the 512K-context sequence of 16 heads of 128 with time, height and width of video tokens
        {"name": "rope_512k", "op": "rope", "B": 1, "N": 524288, "H": 16, "Hk": 16, "D": 128, "rot": 128, "axes": 3,
         "pairs": "half", "dtype": "bf16", "inverse": False},
        # the gradient's way back: shared key heads, partly rotated rows, neighbouring pairs, fp32, an odd length
        {"name": "rope_back", "op": "rope", "B": 2, "N": 8191, "H": 8, "Hk": 2, "D": 64, "rot": 48, "axes": 2,
         "pairs": "next", "dtype": "fp32", "inverse": True},
        # forward only over a short prompt of 8 heads of 128: latency
        {"name": "diff_prompt", "op": "diff", "B": 1, "N": 200, "seqs": 0, "H": 8, "Hk": 8, "D": 128, "dtype": "bf16", "train": False},
        # the 8K training step: 2 sequences of 8 heads of 128
        {"name": "diff_8k", "op": "diff", "B": 2, "N": 8192, "seqs": 0, "H": 8, "Hk": 8, "D": 128, "dtype": "bf16", "train": True},
        # one head of a long sequence, as a rank of a head-parallel job holds it
        {"name": "diff_32k", "op": "diff", "B": 1, "N": 32768, "seqs": 0, "H": 1, "Hk": 1, "D": 128, "dtype": "bf16", "train": True},
        # documents packed into one row of 7,001 tokens, 16 query heads of 64 on 4 key/value heads
        {"name": "diff_packed", "op": "diff", "B": 1, "N": 7001, "seqs": 9, "H": 16, "Hk": 4, "D": 64, "dtype": "bf16", "train": True},
        # the fp32 path at an odd length
        {"name": "diff_fp32", "op": "diff", "B": 1, "N": 1021, "seqs": 0, "H": 4, "Hk": 4, "D": 64, "dtype": "fp32", "train": True},
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("norm", "rope", "diff"))
    if op == "norm":
        d = _log(rng, 32, 16384)
        return {"op": op, "rows": _log(rng, 1, min(1048576, (1 << 27) // d)), "d": d, "dtype": rng.choice(("bf16", "bf16", "fp32")),
                "wdtype": rng.choice(("bf16", "fp32")), "train": rng.random() < 0.7}
    if op == "rope":
        H = rng.choice((1, 3, 4, 8, 16, 24))
        Hk = rng.choice([h for h in (1, 2, 3, 4, 8, 16, 24) if H % h == 0])
        D = rng.choice((32, 64, 72, 96, 128, 256))
        axes = rng.choice((1, 1, 2, 3))
        rot = 2 * rng.randint(axes, D // 2) if rng.random() < 0.3 else D
        B = rng.choice((1, 1, 2, 3))
        return {"op": op, "B": B, "N": _log(rng, 1, min(524288, (1 << 29) // (B * (H + Hk) * D))), "H": H, "Hk": Hk, "D": D, "rot": rot,
                "axes": axes, "pairs": rng.choice(("half", "next")), "dtype": rng.choice(("bf16", "bf16", "fp32")), "inverse": rng.random() < 0.5}
    D = rng.choice((64, 128))
    H = rng.choice((1, 2, 4, 6, 8, 16))
    Hk = rng.choice([h for h in (1, 2, 3, 4, 8, 16) if H % h == 0])
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    B = rng.choice((1, 1, 2, 3))
    most = (1 << 30) if dtype == "bf16" else (1 << 26)
    N = _log(rng, 1, int(math.sqrt(most / (B * H))))
    return {"op": op, "B": 1, "N": N * B, "seqs": rng.randint(2, 12), "H": H, "Hk": Hk, "D": D, "dtype": dtype, "train": rng.random() < 0.7} \
        if rng.random() < 0.4 and N * B <= 8192 else \
        {"op": op, "B": B, "N": N, "seqs": 0, "H": H, "Hk": Hk, "D": D, "dtype": dtype, "train": rng.random() < 0.7}


def _lengths(case):
    """Lengths of the packed sequences: they add up to N, some are short, one may be empty (fixed by the case)."""
    r = random.Random(case["N"] * 31 + case["seqs"])
    cuts = sorted(r.randint(0, case["N"]) for _ in range(case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["N"]])]


# --------------------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _inputs(case, seed):
    """The tensors that a program holds before the call."""
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 13)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = {}
    if case["op"] == "norm":
        M, d, wt = case["rows"], case["d"], TYPES[case["wdtype"]]
        # a residual stream: channels of unlike size with a mean of their own
        chan = torch.exp(0.5 * torch.randn(d, generator=g, device=dev))
        off = 0.3 * torch.randn(d, generator=g, device=dev)
        s["x"] = torch.randn(M, d, generator=g, device=dev).mul_(chan).add_(off).to(dt)
        s["w"] = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(wt)
        s["b"] = (0.1 * torch.randn(d, generator=g, device=dev)).to(wt)
        if case["train"]:
            s["dy"] = normal(M, d)
        return s
    if case["op"] == "rope":
        B, N, R, A = case["B"], case["N"], case["rot"] // 2, case["axes"]
        s["q"], s["k"] = normal(B, N, case["H"], case["D"]), normal(B, N, case["Hk"], case["D"])
        # tokens of a grid: time, height, width; one axis: a text's running position
        t = torch.arange(N, device=dev, dtype=torch.int32) + torch.randint(0, 4096, (B, 1), generator=g, device=dev, dtype=torch.int32)
        grid = (t,) if A == 1 else (t // 32, t % 32) if A == 2 else (t // 576, (t // 32) % 18, t % 32)
        s["pos"] = torch.stack(grid).contiguous()
        # one ladder of frequencies over the pairs, cut into one run of pairs per axis
        s["freq"] = torch.tensor([10000.0 ** (-2.0 * i / case["rot"]) for i in range(R)], dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor([i * A // R for i in range(R)], dtype=torch.int32, device=dev)
        return s
    B, N, H, Hk, D = case["B"], case["N"], case["H"], case["Hk"], case["D"]
    s["q"], s["k"], s["v"] = normal(B, N, H, D), normal(B, N, Hk, D), normal(B, N, Hk, D)
    s["lam"] = (0.2 + 0.6 * torch.rand(H, generator=g, device=dev)).to(dt)
    if case["train"]:
        s["do"] = normal(B, N, H, D)
    s["cu"] = None
    if case["seqs"]:
        ends = torch.tensor([0] + _lengths(case), dtype=torch.int64).cumsum(0)
        s["cu"] = ends.to(torch.int32).to(dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from long_context_symmetric_b200 import lh
        s["lh"] = lh
        dev = _device()
        if case["op"] == "norm":
            M = case["rows"]
            s["cfg"] = lh.make_norm_config(M, case["d"], case["dtype"], case["wdtype"], EPS)
            s["y"] = torch.empty_like(s["x"])
            if case["train"]:
                s["mean"], s["rstd"] = (torch.empty(M, dtype=torch.float32, device=dev) for _ in range(2))
                s["dx"], s["dw"], s["db"] = torch.empty_like(s["x"]), torch.empty_like(s["w"]), torch.empty_like(s["b"])
                s["ws"] = lh.norm_workspace(s["cfg"], dev)
        elif case["op"] == "rope":
            s["cfg"] = lh.make_rope_config(case["B"], case["N"], case["H"], case["Hk"], case["D"], case["rot"], case["axes"],
                                           case["dtype"], case["pairs"])
            s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        else:
            s["cfg"] = lh.make_diff_config(case["seqs"] or case["B"], case["N"], case["H"], case["D"], case["dtype"], case["Hk"],
                                           rows=case["N"] if case["seqs"] else None, train=case["train"])
            s["ws"] = lh.DiffWorkspace(s["cfg"], dev)
            s["o"] = torch.empty_like(s["q"])
            if case["train"]:
                s["dq"], s["dk"], s["dv"], s["dlam"] = (torch.empty_like(s[n]) for n in ("q", "k", "v", "lam"))
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return {"norm": _norm, "rope": _rope, "diff": _diff}[s["case"]["op"]](s)


def _norm(s):
    if own:
        lh, cfg = s["lh"], s["cfg"]
        if not s["case"]["train"]:
            lh.norm_fwd(cfg, s["x"], s["w"], s["b"], s["y"])
            return {"y": s["y"]}
        lh.norm_fwd(cfg, s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"])
        lh.norm_bwd(cfg, s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"], s["ws"])
        return {"y": s["y"], "dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    x, w = s["x"].float(), s["w"].float()
    xc = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    xhat = xc * rstd
    out = {"y": (xhat * w + s["b"].float()).to(s["x"].dtype)}
    if s["case"]["train"]:
        dy = s["dy"].float()
        g = dy * w
        dx = (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)) * rstd
        out.update(dx=dx.to(s["x"].dtype), dw=(dy * xhat).sum(0).to(s["w"].dtype), db=dy.sum(0).to(s["b"].dtype))
    return out


def _rope(s):
    c = s["case"]
    if own:
        s["lh"].rope(s["cfg"], s["q"], s["k"], s["pos"], s["freq"], s["axis"], s["qo"], s["ko"], inverse=c["inverse"])
        return {"q": s["qo"], "k": s["ko"]}
    # angles in 64 bits: at position 500,000 a rounding of 2^-24 would move the fastest pair by 0.03
    ang = s["pos"].double()[s["axis"].long()].movedim(0, -1) * s["freq"]
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    sin = -sin if c["inverse"] else sin
    R = c["rot"] // 2

    def turn(x):
        xf = x.float()
        out = xf.clone()
        a, b = (xf[..., :R], xf[..., R:2 * R]) if c["pairs"] == "half" else (xf[..., 0:2 * R:2], xf[..., 1:2 * R:2])
        lo, hi = a * cos - b * sin, b * cos + a * sin
        if c["pairs"] == "half":
            out[..., :R], out[..., R:2 * R] = lo, hi
        else:
            out[..., 0:2 * R:2], out[..., 1:2 * R:2] = lo, hi
        return out.to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _diff(s):
    c = s["case"]
    if own:
        lh, cfg = s["lh"], s["cfg"]
        lh.diff_attn_fwd(cfg, s["q"], s["k"], s["v"], s["lam"], s["o"], s["ws"], cu=s["cu"])
        if not c["train"]:
            return {"o": s["o"]}
        lh.diff_attn_bwd(cfg, s["do"], s["q"], s["k"], s["v"], s["lam"], s["ws"], s["dq"], s["dk"], s["dv"], s["dlam"], cu=s["cu"])
        return {"o": s["o"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dlam": s["dlam"]}
    B, N, H, Hk, D = c["B"], c["N"], c["H"], c["Hk"], c["D"]
    G, h = H // Hk, D // 2
    scale = 1 / math.sqrt(h)
    # [B, Hk, G, map, N, D/2], [B, Hk, 1, map, N, D/2], [B, Hk, 1, N, D]
    q = s["q"].float().view(B, N, Hk, G, 2, h).permute(0, 2, 3, 4, 1, 5)
    k = s["k"].float().view(B, N, Hk, 1, 2, h).permute(0, 2, 3, 4, 1, 5)
    v = s["v"].float().view(B, N, Hk, 1, D).permute(0, 2, 3, 1, 4)
    i = torch.arange(N, device=q.device)
    keep = i[:, None] >= i[None, :]
    if s["cu"] is not None:
        doc = torch.searchsorted(s["cu"][1:].long(), i, right=True)
        keep = keep & (doc[:, None] == doc[None, :])
    lam = s["lam"].float().view(1, Hk, G, 1, 1)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~keep, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p[:, :, :, 0] - lam * p[:, :, :, 1], v)

    def rows(x, width):
        return x.movedim(-2, 1).reshape(B, N, -1, width)

    out = {"o": rows(o, D).to(s["q"].dtype)}
    if c["train"]:
        do = s["do"].float().view(B, N, Hk, G, D).permute(0, 2, 3, 1, 4)
        dv = torch.matmul((p[:, :, :, 0] - lam * p[:, :, :, 1]).transpose(-1, -2), do).sum(2)
        dp = torch.matmul(do, v.transpose(-1, -2)).unsqueeze(3)
        delta = (p * dp).sum(-1, keepdim=True)
        sign = torch.stack([torch.ones_like(lam), -lam], 3)
        ds = p.mul_(dp - delta).mul_(sign).mul_(scale)
        del dp
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
        out.update(dq=rows(dq.movedim(3, -2).flatten(-2), D).to(s["q"].dtype), dk=rows(dk.movedim(2, -2).flatten(-2), D).to(s["q"].dtype),
                   dv=rows(dv, D).to(s["q"].dtype), dlam=-delta[:, :, :, 1].double().sum((0, 3, 4)).view(H).to(s["lam"].dtype))
    return out


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "norm":
        M, d, we = case["rows"], case["d"], BYTES[case["wdtype"]]
        # x and w, b in, y out; training: dy (and x again, behind the forward pass) in, dx and dw, db out
        b = 2 * M * d * e + 2 * d * we
        f = 8 * M * d
        if case["train"]:
            b += 3 * M * d * e + 3 * d * we + 16 * M
            f += 14 * M * d
        return {"bytes": b, "flops": f}
    if case["op"] == "rope":
        n = case["B"] * case["N"]
        rows = n * (case["H"] + case["Hk"])
        return {"bytes": 2 * rows * case["D"] * e + 4 * n * case["axes"] + 12 * (case["rot"] // 2), "flops": 3 * rows * case["rot"]}
    H, Hk, D, T = case["H"], case["Hk"], case["D"], case["B"] * case["N"]
    pairs = sum(n * (n + 1) // 2 for n in (_lengths(case) if case["seqs"] else [case["N"]] * case["B"]))
    # per (query, key) pair and head: two products over D/2 for the scores, two over D for the outputs
    f = pairs * H * (2 * D + 4 * D)
    b = T * D * e * (2 * H + 2 * Hk)
    if case["train"]:
        # scores again, dO V^T, P^T dO, dS K and dS^T Q (D in all for each of the two)
        f += pairs * H * 10 * D
        b += T * D * e * (4 * H + 4 * Hk)
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if not torch.cuda.is_available() and work(case)["flops"] > 2e10:
        return None
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "diff": _exact_diff}[case["op"]](case, s)


def _exact_norm(case, s):
    M, d = case["rows"], case["d"]
    w, b = s["w"].double(), s["b"].double()
    y = torch.empty(M, d, dtype=torch.float64, device=w.device)
    dx, dw, db = torch.empty_like(y), torch.zeros_like(w), torch.zeros_like(b)
    step = max(1, (1 << 25) // d)
    for r in range(0, M, step):
        x = s["x"][r:r + step].double()
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        z = (x - mean) / (var + EPS).sqrt()
        y[r:r + step] = z * w + b
        if case["train"]:
            dy = s["dy"][r:r + step].double()
            dw += torch.einsum("md,md->d", dy, z)
            db += dy.sum(0)
            # the Jacobian's product: what is left of w dy across the mean and across z, over the deviation
            u = dy * w
            u = u - z * (u * z).sum(-1, keepdim=True) / d
            dx[r:r + step] = (u - u.sum(-1, keepdim=True) / d) / (var + EPS).sqrt()
    return {"y": y, "dx": dx, "dw": dw, "db": db} if case["train"] else {"y": y}


def _exact_rope(case, s):
    R = case["rot"] // 2
    at = s["pos"].double().permute(1, 2, 0).index_select(2, s["axis"].long()) * s["freq"]
    z = torch.polar(torch.ones_like(at), -at if case["inverse"] else at)[:, :, None]

    def turn(x):
        y = x.double()
        part = y[..., :2 * R].unflatten(-1, (2, R)).transpose(-1, -2) if case["pairs"] == "half" else y[..., :2 * R].unflatten(-1, (R, 2))
        w = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z)
        w = w.transpose(-1, -2).flatten(-2) if case["pairs"] == "half" else w.flatten(-2)
        return torch.cat([w, y[..., 2 * R:]], -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _exact_diff(case, s):
    B, N, H, Hk, D = case["B"], case["N"], case["H"], case["Hk"], case["D"]
    h, G = D // 2, H // Hk
    names = ("o", "dq", "dk", "dv")
    out = {n: torch.zeros(B, N, Hk if n in ("dk", "dv") else H, D, dtype=torch.float64, device=s["q"].device) for n in names}
    dlam = torch.zeros(H, dtype=torch.float64, device=s["q"].device)
    spans = [(b, 0, N) for b in range(B)]
    if case["seqs"]:
        ends = s["cu"].tolist()
        spans = [(0, lo, hi) for lo, hi in zip(ends, ends[1:]) if hi > lo]
    for b, lo, hi in spans:
        for head in range(H):
            q, k, v = s["q"][b, lo:hi, head].double(), s["k"][b, lo:hi, head // G].double(), s["v"][b, lo:hi, head // G].double()
            lam = float(s["lam"][head].double())
            for r in range(0, hi - lo, 4096):  # query rows r .. e see the keys before e
                e = min(r + 4096, hi - lo)
                late = torch.ones(e - r, e, dtype=torch.bool, device=q.device).triu(r + 1)
                a = [((q[r:e, m * h:m * h + h] @ k[:e, m * h:m * h + h].T) / math.sqrt(h)).masked_fill(late, -math.inf).softmax(-1) for m in (0, 1)]
                both = a[0] - lam * a[1]
                out["o"][b, lo + r:lo + e, head] = both @ v[:e]
                if case["train"]:
                    do = s["do"][b, lo + r:lo + e, head].double()
                    out["dv"][b, lo:lo + e, head // G] += both.T @ do
                    dboth = do @ v[:e].T
                    dlam[head] -= (a[1] * dboth).sum()
                    for m, c in ((0, 1.0), (1, -lam)):
                        ds = a[m] * (c * dboth)
                        ds = (ds - a[m] * ds.sum(-1, keepdim=True)) / math.sqrt(h)
                        out["dq"][b, lo + r:lo + e, head, m * h:m * h + h] = ds @ k[:e, m * h:m * h + h]
                        out["dk"][b, lo:lo + e, head // G, m * h:m * h + h] += ds.T @ q[r:e, m * h:m * h + h]
    if not case["train"]:
        return {"o": out["o"]}
    return dict(out, dlam=dlam)
