"""Thin ctypes binding over liblh (include/lh.h).

Argument marshalling only: every step of the hot path runs in liblh's CUDA
kernels. Tensors are torch tensors on a CUDA device (PyTorch supplies device
memory and streams); each wrapper passes their data pointers and the current
stream to the C entry point of the same name and raises LHError on a non-zero
status. The library is loaded on first use; if it is missing the call raises
(there is no fallback implementation).
"""

from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblh.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "lh.h")

LH_BF16, LH_FP32 = 0, 1
LH_ACC_FP32, LH_ACC_FIXED64 = 0, 1
LH_ERR_NULL = 1
MAX_LEVELS = 8
MAX_K = 4096

c_int, c_void_p, c_size_t = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t


class LHError(RuntimeError):
    def __init__(self, status: int, name: str):
        super().__init__(f"{name}: {status_string(status)} (status {status})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("B", c_int), ("H", c_int), ("N", c_int), ("D", c_int), ("p", c_int),
                ("L", c_int), ("K", c_int), ("dtype", c_int), ("accum", c_int),
                ("score", c_int), ("ties", c_int), ("order", c_int), ("weight", c_int),
                ("inclusion", c_int)]


SCORES = {"max": 0, "k": 1, "sum": 2, "prod": 3, "maxpool": 4}
TIES = {"low": 0, "high": 1}
ORDERS = {"post": 0, "pre": 1}
WEIGHTS = {"one": 0, "mean": 1}
INCLUSIONS = {"nested": 0, "partition": 1}


class Plan(ctypes.Structure):
    _fields_ = [("S", c_int), ("E", c_int), ("n", c_int * MAX_LEVELS), ("k", c_int * MAX_LEVELS),
                ("c", c_int * MAX_LEVELS), ("lvl_off", c_int * MAX_LEVELS), ("ws_bytes", c_size_t)]


class CPPlan(ctypes.Structure):
    _fields_ = [("world", c_int), ("rank", c_int), ("n_loc", c_int), ("E_loc", c_int),
                ("lvl_off_loc", c_int * MAX_LEVELS), ("glob", Plan)]


class Buffers(ctypes.Structure):
    _fields_ = [("pyr_q", c_void_p), ("pyr_k", c_void_p), ("pyr_v", c_void_p), ("sq", c_void_p),
                ("sel", c_void_p), ("map", c_void_p), ("slot", c_void_p), ("qs", c_void_p),
                ("ks", c_void_p), ("vs", c_void_p), ("os", c_void_p), ("lse", c_void_p),
                ("ws", c_void_p), ("ws_bytes", c_size_t), ("dos", c_void_p), ("delta", c_void_p),
                ("dqs", c_void_p), ("dks", c_void_p), ("dvs", c_void_p), ("scale", c_void_p)]


class NormConfig(ctypes.Structure):
    _fields_ = [("M", ctypes.c_longlong), ("d", c_int), ("dtype", c_int), ("wdtype", c_int),
                ("ldx", ctypes.c_longlong), ("ldy", ctypes.c_longlong), ("eps", ctypes.c_float)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("B", c_int), ("N", c_int), ("H", c_int), ("Hk", c_int), ("D", c_int), ("rot", c_int), ("axes", c_int),
                ("dtype", c_int), ("pairs", c_int), ("pos64", c_int)] + [
                    (n, ctypes.c_longlong) for n in ("q_ld", "q_bs", "k_ld", "k_bs", "qo_ld", "qo_bs", "ko_ld", "ko_bs",
                                                     "pos_as", "pos_bs")]


class DiffConfig(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("H", c_int), ("Hk", c_int), ("D", c_int), ("dtype", c_int),
                ("packed", c_int), ("train", c_int)] + [(n, ctypes.c_longlong) for n in ("ldq", "ldk", "ldv", "ldo")]


class DiffPlan(ctypes.Structure):
    _fields_ = [("saved_bytes", c_size_t), ("ws_bytes", c_size_t)]


_lib = None

_SIGS = {
    "lh_version": ([], c_int),
    "lh_status_string": ([c_int], ctypes.c_char_p),
    "lh_plan": ([ctypes.POINTER(Config), ctypes.POINTER(Plan)], c_int),
    "lh_pool": ([ctypes.POINTER(Config)] + [c_void_p] * 9, c_int),
    "lh_score_topk": ([ctypes.POINTER(Config), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                       c_size_t, c_void_p], c_int),
    "lh_gather": ([ctypes.POINTER(Config)] + [c_void_p] * 12, c_int),
    "lh_attn_fwd": ([ctypes.POINTER(Config)] + [c_void_p] * 7, c_int),
    "lh_scatter": ([ctypes.POINTER(Config)] + [c_void_p] * 4, c_int),
    "lh_scatter_bwd": ([ctypes.POINTER(Config)] + [c_void_p] * 7, c_int),
    "lh_attn_bwd": ([ctypes.POINTER(Config)] + [c_void_p] * 11, c_int),
    "lh_spread": ([ctypes.POINTER(Config)] + [c_void_p] * 8, c_int),
    "lh_forward": ([ctypes.POINTER(Config)] + [c_void_p] * 4 + [ctypes.POINTER(Buffers), c_void_p], c_int),
    "lh_backward": ([ctypes.POINTER(Config)] + [c_void_p] * 4 + [ctypes.POINTER(Buffers), c_void_p], c_int),
    "lh_get_device_error": ([c_void_p, ctypes.POINTER(c_int)], c_int),
    "lh_launch_count": ([], ctypes.c_ulonglong),
    "lh_selftest_timeout": ([ctypes.c_longlong, c_void_p, c_void_p], c_int),
    "lh_score_topk_noalloc": ([ctypes.POINTER(Config)] + [c_void_p] * 5, c_int),
    "lh_selftest_exp2": ([c_void_p, c_void_p, c_void_p, c_int, c_void_p], c_int),
    "lh_pool_range": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 9, c_int),
    "lh_scatter_range": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 4, c_int),
    "lh_cp_plan": ([ctypes.POINTER(Config), c_int, c_int, ctypes.POINTER(CPPlan)], c_int),
    "lh_cp_pool": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 9, c_int),
    "lh_cp_assemble_sq": ([ctypes.POINTER(Config), c_int] + [c_void_p] * 3, c_int),
    "lh_cp_segment": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 5, c_int),
    "lh_cp_gather": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 13, c_int),
    "lh_cp_attn_fwd": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 8, c_int),
    "lh_cp_scatter": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 4, c_int),
    "lh_cp_scatter_bwd": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 8, c_int),
    "lh_cp_attn_bwd": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 12, c_int),
    "lh_norm_plan": ([ctypes.POINTER(NormConfig), ctypes.POINTER(c_size_t)], c_int),
    "lh_norm_fwd": ([ctypes.POINTER(NormConfig)] + [c_void_p] * 7, c_int),
    "lh_norm_bwd": ([ctypes.POINTER(NormConfig)] + [c_void_p] * 9 + [c_size_t, c_void_p], c_int),
    "lh_rope": ([ctypes.POINTER(RopeConfig)] + [c_void_p] * 5 + [c_int] + [c_void_p] * 3, c_int),
    "lh_diff_plan": ([ctypes.POINTER(DiffConfig), ctypes.POINTER(DiffPlan)], c_int),
    "lh_diff_attn_fwd": ([ctypes.POINTER(DiffConfig)] + [c_void_p] * 7 + [c_size_t, c_void_p], c_int),
    "lh_diff_attn_bwd": ([ctypes.POINTER(DiffConfig)] + [c_void_p] * 7 + [c_size_t, c_void_p, c_size_t] +
                         [c_void_p] * 5, c_int),
    "lh_cp_spread": ([ctypes.POINTER(Config), c_int, c_int] + [c_void_p] * 8, c_int),
}


def lib():
    """Load liblh.so (once) and declare the entry points' signatures."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"liblh.so not found at {LIB_PATH}; build it with "
                               "`python -m long_context_symmetric_b200.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _lib = l
    return _lib


def header_functions() -> list[str]:
    """Names of the entry points declared in include/lh.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\w[\w\s\*]*?\b(lh_\w+)\s*\(", text, flags=re.M)))


def status_string(s: int) -> str:
    return lib().lh_status_string(s).decode()


def _check(status: int, name: str):
    if status != 0:
        raise LHError(status, name)


def _ptr(t):
    """Data pointer of a tensor (or None / int passthrough)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _p(t):
    """The same of a tensor on a CUDA device: host memory never reaches a kernel."""
    if isinstance(t, torch.Tensor) and not t.is_cuda:
        raise ValueError(f"a tensor is on {t.device}, a CUDA device is wanted")
    return _ptr(t)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_config(B, H, N, D, p, L, K, dtype="bf16", accum="fp", score="max", ties="low", order="post",
                weight="one", inclusion="nested") -> Config:
    """Problem sizes, element type, accumulation mode and the readings of the
    open points (defaults: the library's reading)."""
    return Config(B, H, N, D, p, L, K, {"bf16": LH_BF16, "fp32": LH_FP32}[dtype],
                  {"fp": LH_ACC_FP32, "fixed": LH_ACC_FIXED64}[accum], SCORES[score], TIES[ties],
                  ORDERS[order], WEIGHTS[weight], INCLUSIONS[inclusion])


def plan(cfg: Config) -> Plan:
    out = Plan()
    _check(lib().lh_plan(ctypes.byref(cfg), ctypes.byref(out)), "lh_plan")
    return out


def pool(cfg, q, k, v, pyr_q, pyr_k, pyr_v, sq, scale, stream=None):
    _check(lib().lh_pool(ctypes.byref(cfg), _p(q), _p(k), _p(v), _p(pyr_q), _p(pyr_k), _p(pyr_v),
                         _p(sq), _p(scale), _stream(stream)), "lh_pool")


def score_topk(cfg, sq, sel, map_, slot, ws, ws_bytes=None, stream=None):
    nbytes = ws_bytes if ws_bytes is not None else (ws.numel() * ws.element_size() if ws is not None else 0)
    _check(lib().lh_score_topk(ctypes.byref(cfg), _p(sq), _p(sel), _p(map_), _p(slot), _p(ws),
                               nbytes, _stream(stream)), "lh_score_topk")


def score_topk_noalloc(cfg, sq, sel, map_, slot, stream=None):
    """lh_score_topk with the descent's scratch in liblh's fixed device array (no workspace)."""
    _check(lib().lh_score_topk_noalloc(ctypes.byref(cfg), _p(sq), _p(sel), _p(map_), _p(slot),
                                       _stream(stream)), "lh_score_topk_noalloc")


def gather(cfg, q, k, v, pyr_q, pyr_k, pyr_v, map_, scale, qs, ks, vs, stream=None):
    _check(lib().lh_gather(ctypes.byref(cfg), _p(q), _p(k), _p(v), _p(pyr_q), _p(pyr_k), _p(pyr_v),
                           _p(map_), _p(scale), _p(qs), _p(ks), _p(vs), _stream(stream)), "lh_gather")


def attn_fwd(cfg, qs, ks, vs, scale, os_, lse, stream=None):
    _check(lib().lh_attn_fwd(ctypes.byref(cfg), _p(qs), _p(ks), _p(vs), _p(scale), _p(os_), _p(lse),
                             _stream(stream)), "lh_attn_fwd")


def scatter(cfg, os_, slot, o, stream=None):
    _check(lib().lh_scatter(ctypes.byref(cfg), _p(os_), _p(slot), _p(o), _stream(stream)), "lh_scatter")


def scatter_bwd(cfg, dout, os_, slot, dos, delta, scale, stream=None):
    _check(lib().lh_scatter_bwd(ctypes.byref(cfg), _p(dout), _p(os_), _p(slot), _p(dos), _p(delta), _p(scale),
                                _stream(stream)), "lh_scatter_bwd")


def attn_bwd(cfg, qs, ks, vs, dos, lse, delta, scale, dqs, dks, dvs, stream=None):
    _check(lib().lh_attn_bwd(ctypes.byref(cfg), _p(qs), _p(ks), _p(vs), _p(dos), _p(lse), _p(delta),
                             _p(scale), _p(dqs), _p(dks), _p(dvs), _stream(stream)), "lh_attn_bwd")


def spread(cfg, dqs, dks, dvs, slot, dq, dk, dv, stream=None):
    _check(lib().lh_spread(ctypes.byref(cfg), _p(dqs), _p(dks), _p(dvs), _p(slot), _p(dq), _p(dk),
                           _p(dv), _stream(stream)), "lh_spread")


def get_device_error(stream=None):
    detail = c_int(0)
    st = lib().lh_get_device_error(_stream(stream), ctypes.byref(detail))
    return st, detail.value


def launch_count() -> int:
    return int(lib().lh_launch_count())


def selftest_timeout(limit_cycles: int, gave_up: torch.Tensor, stream=None):
    """One warp waits, with the kernels' bounded wait, on an mbarrier nothing
    arrives on; after `limit_cycles` SM cycles it gives up and records
    LH_ERR_TIMEOUT (detail 900). `gave_up`: a device int32 tensor, set to 1."""
    _check(lib().lh_selftest_timeout(int(limit_cycles), _p(gave_up), _stream(stream)), "lh_selftest_timeout")


def selftest_exp2(x: torch.Tensor, y_fma: torch.Tensor, y_sfu: torch.Tensor, stream=None):
    """2^x of a device float32 tensor by the attention kernels' FMA-pipe
    polynomial (y_fma) and by the special-function unit's ex2.approx (y_sfu)."""
    _check(lib().lh_selftest_exp2(_p(x), _p(y_fma), _p(y_sfu), x.numel(), _stream(stream)), "lh_selftest_exp2")


def pool_range(cfg, t0, nt, q, k, v, pyr_q, pyr_k, pyr_v, sq, scale, stream=None):
    _check(lib().lh_pool_range(ctypes.byref(cfg), t0, nt, _p(q), _p(k), _p(v), _p(pyr_q), _p(pyr_k), _p(pyr_v),
                               _p(sq), _p(scale), _stream(stream)), "lh_pool_range")


def scatter_range(cfg, t0, nt, os_, slot, o, stream=None):
    _check(lib().lh_scatter_range(ctypes.byref(cfg), t0, nt, _p(os_), _p(slot), _p(o), _stream(stream)),
           "lh_scatter_range")


# ---------------------------------------------------------------------------
# sequence-sharded (context-parallel) path: the per-rank calls
# ---------------------------------------------------------------------------

def cp_plan(cfg, world: int, rank: int) -> CPPlan:
    out = CPPlan()
    _check(lib().lh_cp_plan(ctypes.byref(cfg), world, rank, ctypes.byref(out)), "lh_cp_plan")
    return out


def cp_pool(cfg, world, rank, q, k, v, pyr_q, pyr_k, pyr_v, sq_loc, scale, stream=None):
    _check(lib().lh_cp_pool(ctypes.byref(cfg), world, rank, _p(q), _p(k), _p(v), _p(pyr_q), _p(pyr_k),
                            _p(pyr_v), _p(sq_loc), _p(scale), _stream(stream)), "lh_cp_pool")


def cp_assemble_sq(cfg, world, sq_gathered, sq, stream=None):
    _check(lib().lh_cp_assemble_sq(ctypes.byref(cfg), world, _p(sq_gathered), _p(sq), _stream(stream)),
           "lh_cp_assemble_sq")


def cp_segment(cfg, world, rank, map_, slot, slot_loc, seg, stream=None):
    _check(lib().lh_cp_segment(ctypes.byref(cfg), world, rank, _p(map_), _p(slot), _p(slot_loc), _p(seg),
                               _stream(stream)), "lh_cp_segment")


def cp_gather(cfg, world, rank, q, k, v, pyr_q, pyr_k, pyr_v, map_, seg, scale, qs, ks, vs, stream=None):
    _check(lib().lh_cp_gather(ctypes.byref(cfg), world, rank, _p(q), _p(k), _p(v), _p(pyr_q), _p(pyr_k),
                              _p(pyr_v), _p(map_), _p(seg), _p(scale), _p(qs), _p(ks), _p(vs), _stream(stream)),
           "lh_cp_gather")


def cp_attn_fwd(cfg, world, rank, seg, qs, ks, vs, scale, os_, lse, stream=None):
    _check(lib().lh_cp_attn_fwd(ctypes.byref(cfg), world, rank, _p(seg), _p(qs), _p(ks), _p(vs), _p(scale),
                                _p(os_), _p(lse), _stream(stream)), "lh_cp_attn_fwd")


def cp_scatter(cfg, world, rank, os_, slot_loc, o, stream=None):
    _check(lib().lh_cp_scatter(ctypes.byref(cfg), world, rank, _p(os_), _p(slot_loc), _p(o), _stream(stream)),
           "lh_cp_scatter")


def cp_scatter_bwd(cfg, world, rank, dout, os_, slot_loc, seg, dos, delta, scale, stream=None):
    _check(lib().lh_cp_scatter_bwd(ctypes.byref(cfg), world, rank, _p(dout), _p(os_), _p(slot_loc), _p(seg),
                                   _p(dos), _p(delta), _p(scale), _stream(stream)), "lh_cp_scatter_bwd")


def cp_attn_bwd(cfg, world, rank, seg, qs, ks, vs, dos, lse, delta, scale, dqs, dks, dvs, stream=None):
    _check(lib().lh_cp_attn_bwd(ctypes.byref(cfg), world, rank, _p(seg), _p(qs), _p(ks), _p(vs), _p(dos),
                                _p(lse), _p(delta), _p(scale), _p(dqs), _p(dks), _p(dvs), _stream(stream)),
           "lh_cp_attn_bwd")


def cp_spread(cfg, world, rank, dqs, dks, dvs, slot_loc, dq, dk, dv, stream=None):
    _check(lib().lh_cp_spread(ctypes.byref(cfg), world, rank, _p(dqs), _p(dks), _p(dvs), _p(slot_loc), _p(dq),
                              _p(dk), _p(dv), _stream(stream)), "lh_cp_spread")


# ---------------------------------------------------------------------------
# buffers of one forward + backward (PyTorch allocates; liblh never does)
# ---------------------------------------------------------------------------

class Workspace:
    """Every intermediate buffer of one forward+backward, sized by lh_plan."""

    def __init__(self, cfg: Config, device, backward: bool = True):
        self.cfg = cfg
        self.plan = pl = plan(cfg)
        B, H, D = cfg.B, cfg.H, cfg.D
        S, E = pl.S, pl.E
        dt = torch.bfloat16 if cfg.dtype == LH_BF16 else torch.float32
        L, K = cfg.L, cfg.K
        f32, i32 = torch.float32, torch.int32
        z = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=device)
        e1 = max(E, 1)
        self.pyr_q, self.pyr_k, self.pyr_v = (z(B, H, e1, D) for _ in range(3))
        self.sq = z(2, B, H, e1, dtype=torch.float64)
        self.sel = z(B, H, max(L - 1, 1), K, dtype=i32)
        self.map = z(B, H, S, dtype=i32)
        self.slot = z(B, H, e1, dtype=i32)
        # attention operand type of the sub-sequence: fp16 for bf16 I/O
        bop = torch.float16 if cfg.dtype == LH_BF16 else dt
        self.qs, self.ks, self.vs = (z(B, H, S, D, dtype=bop) for _ in range(3))
        self.os = z(B, H, S, D, dtype=f32)
        self.lse = z(B, H, S, dtype=f32)
        self.ws = z(max(pl.ws_bytes, 16), dtype=torch.uint8)
        # per-head operand magnitudes [4][B][H] (uint32 bit patterns, held as int32)
        self.scale = torch.zeros(4, B, H, dtype=torch.int32, device=device)
        if backward:
            self.dos = z(B, H, S, D, dtype=bop)
            self.delta = z(B, H, S, dtype=f32)
            self.dqs, self.dks, self.dvs = (z(B, H, S, D, dtype=f32) for _ in range(3))
        else:
            self.dos = self.delta = self.dqs = self.dks = self.dvs = None
        self.c = Buffers(
            _p(self.pyr_q), _p(self.pyr_k), _p(self.pyr_v), _p(self.sq), _p(self.sel), _p(self.map),
            _p(self.slot), _p(self.qs), _p(self.ks), _p(self.vs), _p(self.os), _p(self.lse),
            _p(self.ws), self.ws.numel(), _p(self.dos), _p(self.delta), _p(self.dqs), _p(self.dks),
            _p(self.dvs), _p(self.scale))


def forward(cfg, q, k, v, o, ws: Workspace, stream=None):
    _check(lib().lh_forward(ctypes.byref(cfg), _p(q), _p(k), _p(v), _p(o), ctypes.byref(ws.c),
                            _stream(stream)), "lh_forward")


def backward(cfg, dout, dq, dk, dv, ws: Workspace, stream=None):
    _check(lib().lh_backward(ctypes.byref(cfg), _p(dout), _p(dq), _p(dk), _p(dv), ctypes.byref(ws.c),
                             _stream(stream)), "lh_backward")


class LighthouseAttention(torch.autograd.Function):
    """Autograd wrapper: o = lighthouse(q, k, v) with q, k, v [B, N, H, D] on a CUDA device.

    The selection is frozen in the forward pass and takes no gradient.
    """

    @staticmethod
    def forward(ctx, q, k, v, p: int, L: int, K: int, accum: str = "fp"):
        B, N, H, D = q.shape
        dtype = {torch.bfloat16: "bf16", torch.float32: "fp32"}[q.dtype]
        cfg = make_config(B, H, N, D, p, L, K, dtype, accum)
        ws = Workspace(cfg, q.device, backward=True)
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o = torch.empty_like(q)
        forward(cfg, q, k, v, o, ws)
        ctx.cfg, ctx.ws = cfg, ws
        return o

    @staticmethod
    def backward(ctx, do):
        do = do.contiguous()
        dq, dk, dv = (torch.empty_like(do) for _ in range(3))
        backward(ctx.cfg, do, dq, dk, dv, ctx.ws)
        return dq, dk, dv, None, None, None, None


def lighthouse_attention(q, k, v, p: int, L: int, K: int, accum: str = "fp"):
    return LighthouseAttention.apply(q, k, v, p, L, K, accum)


# ---------------------------------------------------------------------------
# operators of the layer around the attention: layer norm, rotary positions,
# differential attention
#
# The functions can be captured into CUDA graphs, backward pass included, behind
# one call outside of the capture. As with any torch operation no eager autograd
# graph of the same leaves may live then (its gradient nodes belong to the stream
# that it was made on, and torch would wait for that stream inside the capture).
# ---------------------------------------------------------------------------

_DTYPES = {"bf16": LH_BF16, "fp32": LH_FP32}
_TORCH = {LH_BF16: torch.bfloat16, LH_FP32: torch.float32}
_NAMES = {torch.bfloat16: "bf16", torch.float32: "fp32"}


# The current stream's handle and the current device without the objects that
# torch.cuda.current_stream() builds around them (4 of the 12 us that a small
# call took on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name, dev, stream, *args):
    """One entry point, on the device that the tensors live on."""
    f = getattr(_lib or lib(), name)
    if dev.type != "cuda":
        # host memory never reaches a kernel: asked without pointers, the library
        # names what is wrong with the configuration and launches nothing
        st = f(*(None if t is c_void_p else a for a, t in zip((*args, None), f.argtypes)))
        if st in (0, LH_ERR_NULL):
            raise ValueError(f"{name}: the tensors are on {dev}, a CUDA device is wanted")
    elif dev.index == _raw_device():
        st = f(*args, _raw_stream(dev.index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _stream(stream))
    if st != 0:
        raise LHError(st, name)


def _need(name, dev, label, t, dt, n):
    """t is None, or contiguous, of type dt, on dev and at least n elements long."""
    if t is None or (t.dtype is dt and t.device == dev and t.numel() >= n and t.is_contiguous()):
        return
    _refuse(name, dev, label, t, dt)
    raise ValueError(f"{name}: {label} of shape {tuple(t.shape)}: {n} contiguous elements are wanted")


def _walks_as(t, width, rows, ld, per, bs):
    """A tensor that is not contiguous steps as the call will: dense rows of `width` elements, ld apart, each `per`
    of them bs apart. (A dense stretch longer than a row is taken as a buffer that the call's strides cut up.)"""
    want, nxt, seen = 1, None, 1
    steps = ([ld] if per > 1 else []) + ([bs] if rows > per else [])
    for size, stride in zip(reversed(t.shape), reversed(t.stride())):
        if size == 1:
            continue
        if want < width:
            if stride != want:
                return False
            want *= size
        elif want > width or seen >= rows:
            return True
        else:
            # the next level, or this one's continuation in a tensor of more axes
            if steps and stride == steps[0]:
                steps.pop(0)
            elif stride != nxt:
                return False
            nxt = stride * size
            seen *= size
    return True


def _rows_fit(name, dev, label, t, dt, rows, ld, width, per=0, bs=0):
    """rows x width elements, ld apart (each `per` of them bs apart), lie in the tensor's storage, and its strides are
    the call's."""
    if not per:
        n = (rows - 1) * ld + width if rows else 0
    else:
        n = (rows // per - 1) * bs + (per - 1) * ld + width
    if t.dtype is dt and t.device == dev:
        # a contiguous tensor of that size, or room enough behind a view's first element
        if t.is_contiguous():
            if t.numel() >= n:
                return
        elif not _walks_as(t, width, rows, ld, per or rows, bs):
            raise ValueError(f"{name}: {label} has strides {tuple(t.stride())}, the call's rows of {width} are {ld} apart")
        if n <= t.untyped_storage().nbytes() // t.element_size() - t.storage_offset():
            return
    _refuse(name, dev, label, t, dt)
    raise ValueError(f"{name}: {label} ends before row {rows - 1} of {width} elements, {ld} apart")


def _refuse(name, dev, label, t, dt):
    if t.dtype != dt:
        raise ValueError(f"{name}: {label} has type {t.dtype}, {dt} is wanted")
    if t.device != dev:
        raise ValueError(f"{name}: {label} is on {t.device}, the call is on {dev}")


def make_norm_config(M, d, dtype="bf16", wdtype=None, eps=1e-5, ldx=0, ldy=0) -> NormConfig:
    """M rows of d values; ldx (ldy): elements between rows of x and dx (y and dy), 0: d."""
    return NormConfig(M, d, _DTYPES[dtype], _DTYPES[wdtype or dtype], ldx, ldy, eps)


def norm_ws_bytes(cfg: NormConfig) -> int:
    n = c_size_t(0)
    _check(lib().lh_norm_plan(ctypes.byref(cfg), ctypes.byref(n)), "lh_norm_plan")
    return n.value


def norm_workspace(cfg: NormConfig, device):
    """Scratch of norm_bwd (any buffer of norm_ws_bytes(cfg) bytes serves)."""
    return torch.empty(max(norm_ws_bytes(cfg), 16), dtype=torch.uint8, device=device)


def norm_fwd(cfg, x, w, b, y, mean=None, rstd=None, stream=None):
    dev, dt, wt, M, d, f = x.device, _TORCH[cfg.dtype], _TORCH[cfg.wdtype], cfg.M, cfg.d, "lh_norm_fwd"
    _rows_fit(f, dev, "x", x, dt, M, cfg.ldx or d, d)
    _rows_fit(f, dev, "y", y, dt, M, cfg.ldy or d, d)
    _need(f, dev, "w", w, wt, d)
    _need(f, dev, "b", b, wt, d)
    _need(f, dev, "mean", mean, torch.float32, M)
    _need(f, dev, "rstd", rstd, torch.float32, M)
    _call(f, dev, stream, ctypes.byref(cfg), _ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd))


def norm_bwd(cfg, dy, x, w, mean, rstd, dx, dw, db, ws, stream=None):
    dev, dt, wt, M, d, f = x.device, _TORCH[cfg.dtype], _TORCH[cfg.wdtype], cfg.M, cfg.d, "lh_norm_bwd"
    _rows_fit(f, dev, "x", x, dt, M, cfg.ldx or d, d)
    _rows_fit(f, dev, "dx", dx, dt, M, cfg.ldx or d, d)
    _rows_fit(f, dev, "dy", dy, dt, M, cfg.ldy or d, d)
    _need(f, dev, "w", w, wt, d)
    _need(f, dev, "mean", mean, torch.float32, M)
    _need(f, dev, "rstd", rstd, torch.float32, M)
    _need(f, dev, "dw", dw, wt, d)
    _need(f, dev, "db", db, wt, d)
    _need(f, dev, "ws", ws, torch.uint8, 0)
    _call(f, dev, stream, ctypes.byref(cfg), _ptr(dy), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws),
          ws.numel() if ws is not None else 0)


ROPE_PAIRS = {"half": 0, "next": 1}


def make_rope_config(B, N, H, Hk, D, rot=None, axes=1, dtype="bf16", pairs="half", pos64=False, shared_pos=False,
                     q_ld=0, q_bs=0, k_ld=0, k_bs=0, qo_ld=0, qo_bs=0, ko_ld=0, ko_bs=0, pos_as=None,
                     pos_bs=None) -> RopeConfig:
    """q [B][N][H][D] and k [B][N][Hk][D], the first `rot` elements of a row rotated; positions [axes][B][N]
    ([axes][N] if the sequences share them). *_ld, *_bs: elements between tokens and sequences, 0: contiguous."""
    return RopeConfig(B, N, H, Hk, D, D if rot is None else rot, axes, _DTYPES[dtype], ROPE_PAIRS[pairs], int(pos64),
                      q_ld, q_bs, k_ld, k_bs, qo_ld, qo_bs, ko_ld, ko_bs,
                      (N if shared_pos else B * N) if pos_as is None else pos_as,
                      (0 if shared_pos else N) if pos_bs is None else pos_bs)


def rope(cfg, q, k, pos, freq, axis, qo, ko, inverse=False, stream=None):
    """qo, ko: q and k rotated (q and k themselves: in place). inverse: the backward pass, dq and dk for q and k."""
    dev, dt, B, N, D, R, f = q.device, _TORCH[cfg.dtype], cfg.B, cfg.N, cfg.D, cfg.rot // 2, "lh_rope"
    if B and N:
        for label, t, heads, ld, bs in (("q", q, cfg.H, cfg.q_ld, cfg.q_bs), ("qo", qo, cfg.H, cfg.qo_ld, cfg.qo_bs),
                                        ("k", k, cfg.Hk, cfg.k_ld, cfg.k_bs), ("ko", ko, cfg.Hk, cfg.ko_ld, cfg.ko_bs)):
            if heads:
                ld = ld or heads * D
                _rows_fit(f, dev, label, t, dt, B * N, ld, heads * D, N, bs or N * ld)
        # rows of N positions, pos_bs apart, in axes * B (shared: axes) of them
        if cfg.pos_bs:
            _rows_fit(f, dev, "pos", pos, torch.int64 if cfg.pos64 else torch.int32, cfg.axes * B, cfg.pos_bs, N, B, cfg.pos_as)
        else:
            _rows_fit(f, dev, "pos", pos, torch.int64 if cfg.pos64 else torch.int32, cfg.axes, cfg.pos_as, N)
    _need(f, dev, "freq", freq, torch.float64, R)
    _need(f, dev, "axis", axis, torch.int32, R)
    _call(f, dev, stream, ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(pos), _ptr(freq), _ptr(axis), int(inverse), _ptr(qo), _ptr(ko))


def make_diff_config(B, N, H, D, dtype="bf16", Hk=None, rows=None, train=True, ldq=0, ldk=0, ldv=0, ldo=0) -> DiffConfig:
    """B sequences of N tokens, H query heads of D elements (two maps of D/2) on Hk key/value heads. rows: B
    sequences packed in that many token rows, their offsets given to each call as cu (N is then not used)."""
    return DiffConfig(B, B * N if rows is None else rows, H, H if Hk is None else Hk, D, _DTYPES[dtype],
                      int(rows is not None), int(train), ldq, ldk, ldv, ldo)


def diff_plan(cfg: DiffConfig) -> DiffPlan:
    out = DiffPlan()
    _check(lib().lh_diff_plan(ctypes.byref(cfg), ctypes.byref(out)), "lh_diff_plan")
    return out


class DiffWorkspace:
    """Buffers of one differential attention: what the forward pass leaves for the backward (saved: a forward pass's
    buffer, otherwise a new one), and the backward's scratch (False: none). One forward + backward at a time: calls that
    overlap each need their own."""

    def __init__(self, cfg: DiffConfig, device, saved=None, scratch: bool = True):
        self.plan = pl = diff_plan(cfg)
        new = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=device)  # noqa: E731
        self.saved = new(pl.saved_bytes) if saved is None else saved
        self.ws = new(pl.ws_bytes) if cfg.train and scratch else None


def _diff_check(f, dev, cfg, cu, lam, ws, rows):
    dt, T, D = _TORCH[cfg.dtype], cfg.T, cfg.D
    for label, t, ld, heads in rows:
        _rows_fit(f, dev, label, t, dt, T, ld or heads * D, heads * D)
    _need(f, dev, "lam", lam, dt, cfg.H)
    _need(f, dev, "saved", ws.saved, torch.uint8, 0)
    if cfg.packed:
        if cu is None:
            raise ValueError(f"{f}: packed sequences need cu")
        _need(f, dev, "cu", cu, torch.int32, cfg.B + 1)


def diff_attn_fwd(cfg, q, k, v, lam, o, ws: DiffWorkspace, cu=None, stream=None):
    f, dev = "lh_diff_attn_fwd", q.device
    _diff_check(f, dev, cfg, cu, lam, ws, (("q", q, cfg.ldq, cfg.H), ("k", k, cfg.ldk, cfg.Hk),
                                           ("v", v, cfg.ldv, cfg.Hk), ("o", o, cfg.ldo, cfg.H)))
    _call(f, dev, stream, ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(cu), _ptr(o), _ptr(ws.saved), ws.saved.numel())


def diff_attn_bwd(cfg, dout, q, k, v, lam, ws: DiffWorkspace, dq, dk, dv, dlam, cu=None, stream=None):
    f, dev = "lh_diff_attn_bwd", q.device
    _diff_check(f, dev, cfg, cu, lam, ws,
                (("dout", dout, cfg.ldo, cfg.H), ("q", q, cfg.ldq, cfg.H), ("dq", dq, cfg.ldq, cfg.H),
                 ("k", k, cfg.ldk, cfg.Hk), ("dk", dk, cfg.ldk, cfg.Hk), ("v", v, cfg.ldv, cfg.Hk), ("dv", dv, cfg.ldv, cfg.Hk)))
    _need(f, dev, "dlam", dlam, _TORCH[cfg.dtype], cfg.H)
    _need(f, dev, "ws", ws.ws, torch.uint8, 0)
    _call(f, dev, stream, ctypes.byref(cfg), _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(cu), _ptr(ws.saved),
          ws.saved.numel(), _ptr(ws.ws), ws.ws.numel() if ws.ws is not None else 0, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam))


def type_name(t, what):
    """The library's name of a tensor's type."""
    if t.dtype not in _NAMES:
        raise ValueError(f"{what}: {t.dtype} is not supported (bfloat16, float32)")
    return _NAMES[t.dtype]


def _whole(t):
    """Contiguous and 16-byte aligned."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class LayerNorm(torch.autograd.Function):
    """y = layer norm of the last axis of x, weight w and bias b (either None)."""

    @staticmethod
    def forward(ctx, x, w, b, eps: float):
        d = x.shape[-1]
        for label, t in (("w", w), ("b", b)):
            if t is not None and tuple(t.shape) != (d,):
                raise ValueError(f"layer_norm: {label} has shape {tuple(t.shape)}, ({d},) is wanted")
        if w is not None and b is not None and w.dtype != b.dtype:
            raise ValueError("layer_norm: w and b have unlike types")
        x = _whole(x)
        w, b = (None if t is None else _whole(t) for t in (w, b))
        p = w if w is not None else b
        M = x.numel() // d if d else 0
        cfg = make_norm_config(M, d, type_name(x, "layer_norm"), type_name(x if p is None else p, "layer_norm"), eps)
        y = torch.empty_like(x)
        mean, rstd = (torch.empty(M, dtype=torch.float32, device=x.device) for _ in range(2))
        norm_fwd(cfg, x, w, b, y, mean, rstd)
        ctx.save_for_backward(x, w, b, mean, rstd)
        ctx.cfg = cfg
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, b, mean, rstd = ctx.saved_tensors
        dy, dx = _whole(dy), torch.empty_like(x)
        dw = torch.empty_like(w) if w is not None and ctx.needs_input_grad[1] else None
        db = torch.empty_like(b) if b is not None and ctx.needs_input_grad[2] else None
        norm_bwd(ctx.cfg, dy, x, w, mean, rstd, dx, dw, db, norm_workspace(ctx.cfg, x.device))
        return dx, dw, db, None


def layer_norm(x, w=None, b=None, eps: float = 1e-5):
    return LayerNorm.apply(x, w, b, eps)


class RopePlan:
    """The device tables of a rotary embedding: a frequency (radians per position) and an axis for each pair.

    sections: pairs per axis (their sum is rot/2; one axis: None). order: "runs" (the first sections[0] pairs turn
    with axis 0, and so on) or "cycle" (pairs dealt to the axes in turn, an axis dropping out once it has its
    share). ladder: "shared" (pair i has base^(-2i/rot), whatever its axis) or "own" (each axis has its own ladder
    from 1 down, over its own pairs). freq: the frequencies themselves instead, for a scaled ladder."""

    def __init__(self, rot, sections=None, base=10000.0, device="cuda", order="runs", ladder="shared", freq=None):
        R = rot // 2
        sections = [R] if sections is None else list(sections)
        if rot < 2 or rot % 2 or sum(sections) != R or min(sections) < 0:
            raise ValueError(f"RopePlan: sections {sections} do not add up to {rot}/2 pairs")
        if order not in ("runs", "cycle") or ladder not in ("shared", "own"):
            raise ValueError(f"RopePlan: unknown order {order!r} or ladder {ladder!r}")
        axis, left = [], list(sections)
        if order == "runs":
            axis = [a for a, n in enumerate(sections) for _ in range(n)]
        else:
            while len(axis) < R:
                for a, n in enumerate(left):
                    if n:
                        axis.append(a)
                        left[a] -= 1
        seen = [0] * len(sections)
        own_place = []
        for a in axis:
            own_place.append(seen[a])
            seen[a] += 1
        if freq is None:
            freq = [base ** (-2.0 * i / rot) if ladder == "shared" else base ** (-float(own_place[i]) / sections[axis[i]])
                    for i in range(R)]
        self.rot, self.axes = rot, len(sections)
        self.freq = torch.as_tensor(freq, dtype=torch.float64).to(device)
        self.axis = torch.tensor(axis, dtype=torch.int32, device=device)
        if self.freq.shape != (R,):
            raise ValueError(f"RopePlan: {tuple(self.freq.shape)} frequencies, ({R},) are wanted")

    def positions(self, pos, B, N):
        """pos as [axes][B][N] or [axes][N] (shared by the sequences; [B][N], [N] with one axis), int32 or int64."""
        if pos.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"rotary: positions have type {pos.dtype}, int32 or int64 are wanted")
        if self.axes == 1 and (pos.ndim == 1 or (pos.ndim == 2 and tuple(pos.shape) == (B, N) != (1, N))):
            pos = pos[None]
        if tuple(pos.shape) not in ((self.axes, B, N), (self.axes, N)):
            raise ValueError(f"rotary: positions of shape {tuple(pos.shape)} for {self.axes} axes, {B} x {N} tokens")
        return _whole(pos)


class Rotary(torch.autograd.Function):
    """(q, k) rotated by their tokens' positions; the gradient turns back."""

    @staticmethod
    def forward(ctx, q, k, pos, plan: RopePlan, pairs: str):
        B, N, H, D = q.shape
        if k.shape[:2] != (B, N) or k.shape[3] != D or k.dtype != q.dtype:
            raise ValueError(f"rotary: q {tuple(q.shape)} {q.dtype} and k {tuple(k.shape)} {k.dtype} do not belong together")
        q, k, pos = _whole(q), _whole(k), plan.positions(pos, B, N)
        cfg = make_rope_config(B, N, H, k.shape[2], D, plan.rot, plan.axes, type_name(q, "rotary"), pairs,
                               pos64=pos.dtype == torch.int64, shared_pos=pos.ndim == 2)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        rope(cfg, q, k, pos, plan.freq, plan.axis, qo, ko)
        ctx.cfg, ctx.plan = cfg, plan
        ctx.save_for_backward(pos)
        return qo, ko

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        (pos,) = ctx.saved_tensors
        dq, dk = _whole(dq), _whole(dk)
        gq, gk = torch.empty_like(dq), torch.empty_like(dk)
        rope(ctx.cfg, dq, dk, pos, ctx.plan.freq, ctx.plan.axis, gq, gk, inverse=True)
        return gq, gk, None, None, None


def rotary(q, k, pos, plan: RopePlan, pairs: str = "half", maps: int = 1):
    """q [B, N, H, D], k [B, N, Hk, D] rotated by positions pos (see RopePlan.positions).

    maps: a row holds that many maps of D/maps elements, each rotated by itself (plan.rot <= D/maps). In front of
    differential_attention: 2. Rotated as a whole, a "half" pair would join an element of the first map with one of the
    second, and a map's scores would depend on where its tokens stand, not on their distance alone."""
    if maps == 1:
        return Rotary.apply(q, k, pos, plan, pairs)
    if maps < 1 or q.shape[-1] % maps or k.shape[-1] != q.shape[-1]:
        raise ValueError(f"rotary: {maps} maps in rows of {q.shape[-1]} (q) and {k.shape[-1]} (k) elements")
    cut = lambda t: t.reshape(*t.shape[:-2], t.shape[-2] * maps, t.shape[-1] // maps)  # noqa: E731
    qo, ko = Rotary.apply(cut(q), cut(k), pos, plan, pairs)
    return qo.view(q.shape), ko.view(k.shape)


class DifferentialAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lam, cu, train=True):
        packed = cu is not None
        if q.ndim != (3 if packed else 4) or k.shape != v.shape or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
            raise ValueError(f"differential_attention: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} do not "
                             f"belong together ([B, N, heads, D], or [T, heads, D] with cu)")
        H, D = q.shape[-2:]
        Hk = k.shape[-2]
        if any(t.dtype != q.dtype for t in (k, v, lam)) or tuple(lam.shape) != (H,):
            raise ValueError("differential_attention: k, v and lam [H] have q's type")
        q, k, v, lam = (_whole(t) for t in (q, k, v, lam))
        name = type_name(q, "differential_attention")
        cfg = (make_diff_config(cu.numel() - 1, 0, H, D, name, Hk, rows=q.shape[0], train=train) if packed
               else make_diff_config(q.shape[0], q.shape[1], H, D, name, Hk, train=train))
        ws = DiffWorkspace(cfg, q.device, scratch=False)
        # packed: rows outside the sequences are not written by the kernels
        o = torch.zeros_like(q) if packed else torch.empty_like(q)
        diff_attn_fwd(cfg, q, k, v, lam, o, ws, cu=cu)
        if train:
            ctx.cfg = cfg
            ctx.save_for_backward(q, k, v, lam, cu, ws.saved)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, lam, cu, saved = ctx.saved_tensors
        new = torch.zeros_like if ctx.cfg.packed else torch.empty_like
        dq, dk, dv, dlam = new(q), new(k), new(v), torch.empty_like(lam)
        diff_attn_bwd(ctx.cfg, _whole(do), q, k, v, lam, DiffWorkspace(ctx.cfg, q.device, saved), dq, dk, dv, dlam, cu=cu)
        return dq, dk, dv, dlam, None, None


def differential_attention(q, k, v, lam, cu=None):
    """o = (softmax map 1 - lam * softmax map 2) v, causal; q [B, N, H, D], k, v [B, N, Hk, D], lam [H]. A head's q and k
    rows hold map 1 in their first half and map 2 in the second (positions: rotary with maps=2). With cu (int32
    [sequences + 1], device): q [T, H, D] and so on, the sequences packed one behind the other."""
    # without a backward pass to come nothing is kept for one
    train = torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v, lam))
    return DifferentialAttention.apply(q, k, v, lam, cu, train)
