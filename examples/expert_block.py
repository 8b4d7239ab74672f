"""Train a pre-norm expert block on a synthetic target and print the loss: layer norm, the sort of
the tokens by expert, dispatch, the experts' FP8 linears, combine, and all their gradients.

    python examples/expert_block.py --tokens 4096 --cols 1024 --hidden 2048 --experts 8 --topk 2
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scaled_fp8_linear_amd as m  # noqa: E402


def train(tokens=4096, cols=1024, hidden=2048, experts=8, topk=2, steps=10, lr=1e-3, fp8=True,
          seed=0, log=print):
    """The losses of ``steps`` steps of Adam on a fixed random target."""
    torch.manual_seed(seed)
    m.fp8_state().reset()
    block = m.ExpertBlock(cols, hidden, experts, topk, device="cuda")
    x = torch.randn(tokens, cols, device="cuda", dtype=torch.bfloat16)
    target = x + 0.5 * torch.tanh(x.roll(1, 1).float()).bfloat16()
    opt = torch.optim.Adam(block.parameters(), lr=lr)
    losses = []
    for step in range(steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        with m.fp8_autocast(enabled=fp8):
            y = block(x)
        loss = (y.float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        log(f"step {step:3d}  loss {losses[-1]:.5f}  {1e3 * (time.perf_counter() - t0):.2f} ms")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("cols", 1024), ("hidden", 2048), ("experts", 8),
                        ("topk", 2), ("steps", 10)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--bf16", action="store_true", help="experts in bf16 instead of FP8")
    a = ap.parse_args()
    train(a.tokens, a.cols, a.hidden, a.experts, a.topk, a.steps, fp8=not a.bf16)
