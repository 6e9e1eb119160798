"""The feed-forward example runs the operators together: training with kept activations lowers the loss,
and the 4-bit block answers single tokens close to the trained one."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_feed_forward_block_example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import feed_forward_block as e
    print("[example] M=512 K=256 F=704", flush=True)
    losses, error = e.main(M=512, K=256, F=704, steps=20)
    assert all(b < a for a, b in zip(losses, losses[1:])) and losses[-1] < 0.9 * losses[0]
    # INT4 steps are a seventh of a group's largest weight: some 10% of a Gaussian weight's spread, and three layers
    assert error < 0.3


def test_example_gradients_with_kept_activations():
    """The block's gradients against autograd of the same formula in 64 bits on the CPU: off by the 8-bit
    steps of the kept activations and bf16 roundings, a few percent of each gradient's norm."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import feed_forward_block as e
    print("[example gradients] M=200 K=128 F=320", flush=True)
    b = e.Block(200, 128, 320, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((200, 128), generator=g, device="cuda").bfloat16()
    dy = (torch.randn((200, 128), generator=g, device="cuda") * 0.01).bfloat16()
    b.forward(x)
    dx = b.backward(x, dy)
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in b.w.items()}
    x6 = x.double().cpu().requires_grad_()
    n = torch.nn.functional.layer_norm(x6, (128,), p["gamma"], p["beta"], e.EPS)
    y = x6 + (torch.nn.functional.silu(n @ p["wg"].T) * (n @ p["wu"].T)) @ p["wd"].T
    y.backward(dy.double().cpu())
    got = dict(b.grad, x=dx)
    for k, want in dict({k: v.grad for k, v in p.items()}, x=x6.grad).items():
        err = (got[k].double().cpu() - want).norm() / want.norm()
        assert err < 0.03, (k, float(err))
