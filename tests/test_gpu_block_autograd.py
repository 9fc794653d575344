"""The example block (examples/mamba2_block.py) as a part of a training program:
when its checkpoints are freed, what it refuses, what it skips."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mamba2_block.py")


@pytest.fixture(scope="module")
def setup():
    spec = importlib.util.spec_from_file_location("mamba2_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    torch.manual_seed(5)
    block = m.Mamba2Block(256, 4, dstate=64)
    x = torch.randn(2, 512, 256, device="cuda").bfloat16().requires_grad_(True)
    residual = torch.randn(2, 512, 256, device="cuda").requires_grad_(True)
    return m, block, x, residual


def step(block, x, residual):
    out, res = block(x, residual)
    torch.autograd.backward([out, res], [torch.ones_like(out), torch.ones_like(res)])
    return out, res


def test_checkpoints_are_freed_by_the_backward_pass(setup):
    """With the step's outputs still held, nothing but they stays allocated."""
    _, block, x, residual = setup
    step(block, x, residual)  # gradients and libraries' buffers exist from here on
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    held = step(block, x, residual)
    torch.cuda.synchronize()
    kept = torch.cuda.memory_allocated() - before
    assert kept == sum(t.numel() * t.element_size() for t in held)  # whole multiples of the allocator's 512 bytes


def test_second_derivatives_are_refused(setup):
    _, block, x, residual = setup
    out, _ = block(x, residual)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out.float().sum(), x, create_graph=True)


def test_without_gradients_nothing_is_packed(setup, monkeypatch):
    m, block, x, residual = setup
    out, res = block(x, residual)

    def refuse(*_):
        raise AssertionError("a checkpoint was made")

    monkeypatch.setattr(m.mss.norms, "_empty_packed", refuse)
    with torch.no_grad():
        got = block(x, residual)
    assert torch.equal(got[0], out) and torch.equal(got[1], res)
    with pytest.raises(AssertionError):
        block(x, residual)
