"""What lh.differential_attention holds on the device between its passes, and for how long."""

import pytest
import torch

from layertest import DT
from long_context_symmetric_b200 import lh

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
B, N, H, Hk, D = 2, 2048, 4, 2, 128


def leaves(dtype):
    g = torch.Generator().manual_seed(3)
    r = lambda n: torch.randn(B, N, n, D, generator=g).to(DT[dtype]).to(DEV)  # noqa: E731
    return [r(H).requires_grad_(), r(Hk).requires_grad_(), r(Hk).requires_grad_(),
            torch.full((H,), 0.5, dtype=DT[dtype], device=DEV, requires_grad=True)], r(H)


def size(t):
    return t.numel() * t.element_size()


def held():
    """Bytes asked for and not let go (memory_allocated counts what the allocator's blocks are too large by)."""
    return torch.cuda.memory_stats()["requested_bytes.all.current"]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_scratch_is_not_held_and_what_is_saved_goes_with_the_pass(dtype):
    args, do = leaves(dtype)
    lh.differential_attention(*args).backward(do)
    plan = lh.diff_plan(lh.make_diff_config(B, N, H, D, dtype, Hk))
    grads = sum(size(t.grad) for t in args)
    for t in args:
        t.grad = None
    torch.cuda.synchronize()
    start = held()
    o = lh.differential_attention(*args)
    assert held() - start <= size(o) + plan.saved_bytes + 1024
    o.backward(do)
    # o and its graph still live: the node has run, and holds nothing any more
    assert held() - start <= size(o) + grads + 1024
    assert lh.get_device_error() == (0, 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_saved_tensor_hooks_see_all_of_it(dtype):
    """Kept on the host between the passes (as offloading does): the same gradients."""
    args, do = leaves(dtype)
    lh.differential_attention(*args).backward(do)
    want = [t.grad.clone() for t in args]
    for t in args:
        t.grad = None
    seen = []

    def pack(t):
        seen.append(t.numel() * t.element_size())
        return t.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.to(DEV)):
        o = lh.differential_attention(*args)
    torch.empty(1 << 28, dtype=torch.uint8, device=DEV).fill_(255)      # whatever was let go is overwritten
    o.backward(do)
    assert lh.diff_plan(lh.make_diff_config(B, N, H, D, dtype, Hk)).saved_bytes in seen
    assert all(torch.equal(t.grad, w) for t, w in zip(args, want)) and lh.get_device_error() == (0, 0)


def test_a_graph_that_is_kept_can_run_again():
    args, do = leaves("bf16")
    o = lh.differential_attention(*args)
    a = torch.autograd.grad(o, args, do, retain_graph=True)
    b = torch.autograd.grad(o, args, do)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
