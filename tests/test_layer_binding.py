"""The binding against a stand-in for the library: what it passes on, and what it never does."""

import pytest
import torch

from long_context_symmetric_b200 import lh

BF = torch.bfloat16


class Recorder:
    """Entry points that note their arguments and launch nothing. A call with any pointer besides the configuration
    counts as a launch; without pointers the answer is the library's own (status 1: a null pointer)."""

    def __init__(self, library):
        self.library, self.launched = library, []

    def __getattr__(self, name):
        real = getattr(self.library, name)
        if name.endswith("_plan") or name == "lh_status_string":
            return real

        def call(*args):
            if any(a for a, t in zip(args[1:], real.argtypes[1:]) if t is lh.c_void_p):
                self.launched.append(name)
                return 0
            return real(*args)

        call.argtypes = real.argtypes
        return call


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder(lh.lib())
    monkeypatch.setattr(lh, "_lib", r)
    monkeypatch.setattr(lh, "lib", lambda: r)
    monkeypatch.setattr(lh, "_stream", lambda s: 0)
    return r


def calls(dev):
    """Every operator's calls on tensors of a device."""
    x, f32 = torch.zeros(4, 64, dtype=BF, device=dev), torch.zeros(4, device=dev)
    w, ncfg = torch.zeros(64, dtype=BF, device=dev), lh.make_norm_config(4, 64)
    ws = torch.zeros(lh.norm_ws_bytes(ncfg), dtype=torch.uint8, device=dev)
    yield "norm_fwd", lambda: lh.norm_fwd(ncfg, x, w, w, x, f32, f32)
    yield "norm_bwd", lambda: lh.norm_bwd(ncfg, x, x, w, f32, f32, x, w, w, ws)
    yield "layer_norm", lambda: lh.layer_norm(x, w, w)
    q, pos = torch.zeros(1, 4, 2, 64, dtype=BF, device=dev), torch.zeros(1, 1, 4, dtype=torch.int32, device=dev)
    plan, rcfg = lh.RopePlan(64, device=dev), lh.make_rope_config(1, 4, 2, 2, 64)
    yield "rope", lambda: lh.rope(rcfg, q, q, pos, plan.freq, plan.axis, q, q)
    yield "rotary", lambda: lh.rotary(q, q, pos, plan)
    lam, dcfg = torch.zeros(2, dtype=BF, device=dev), lh.make_diff_config(1, 4, 2, 64)
    dws = lh.DiffWorkspace(dcfg, dev)
    yield "diff_attn_fwd", lambda: lh.diff_attn_fwd(dcfg, q, q, q, lam, q, dws)
    yield "diff_attn_bwd", lambda: lh.diff_attn_bwd(dcfg, q, q, q, q, lam, dws, q, q, q, lam)
    yield "differential_attention", lambda: lh.differential_attention(q, q, q, lam)


@pytest.mark.parametrize("name", [n for n, _ in calls("cpu")])
def test_host_memory_never_reaches_a_kernel(recorder, name):
    with pytest.raises(ValueError, match="on cpu"):
        dict(calls("cpu"))[name]()
    assert recorder.launched == []


def test_no_rows_on_the_host_are_refused_too(recorder):
    e = torch.zeros(0, 64, dtype=BF)
    with pytest.raises(ValueError, match="on cpu"):
        lh.norm_fwd(lh.make_norm_config(0, 64), e, None, None, e)
    assert recorder.launched == []


def test_a_bad_configuration_is_named_first(recorder):
    x = torch.zeros(4, 64, dtype=BF)
    with pytest.raises(lh.LHError, match="status 2"):
        lh.norm_fwd(lh.make_norm_config(4, 64, eps=-1.0), x, None, None, x)
    assert recorder.launched == []


def test_maps_have_to_fit_the_rows(recorder):
    q, pos, plan = torch.zeros(1, 4, 2, 64, dtype=BF), torch.arange(4, dtype=torch.int32), lh.RopePlan(32, device="cpu")
    for maps in (0, -1, 3):
        with pytest.raises(ValueError, match="maps"):
            lh.rotary(q, q, pos, plan, maps=maps)
    with pytest.raises(lh.LHError, match="status 2"):       # tables of a whole row on half of one
        lh.rotary(q, q, pos, lh.RopePlan(64, device="cpu"), maps=2)
    assert recorder.launched == []


def test_the_path_refuses_host_memory_too(recorder):
    t, f = torch.zeros(1, 256, 2, 64, dtype=BF), torch.zeros(1024)
    cfg = lh.make_config(1, 2, 256, 64, 4, 2, 16)
    for call in (lambda: lh.lighthouse_attention(t, t, t, 4, 2, 16), lambda: lh.Workspace(cfg, "cpu"),
                 lambda: lh.pool(cfg, t, t, t, t, t, t, f.double(), f.int()), lambda: lh.gather(cfg, t, t, t, t, t, t, f.int(), f, t, t, t),
                 lambda: lh.attn_fwd(cfg, t, t, t, f, f, f), lambda: lh.scatter_range(cfg, 0, 16, f, f.int(), t),
                 lambda: lh.cp_pool(cfg, 2, 0, t, t, t, t, t, t, f.double(), f.int()),
                 lambda: lh.selftest_exp2(f, f, f), lambda: lh.selftest_timeout(1000, f.int())):
        with pytest.raises(ValueError, match="on cpu"):
            call()
    assert recorder.launched == []
