"""The example runs the operators together: training brings the loss down, and
generation token by token agrees with the scan over the same tokens."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_recurrent_layer_example():
    import torch

    from triangular_solve_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import recurrent_layer as ex
    finally:
        sys.path.pop(0)
    model, losses = ex.train(steps=80, width=64, rows=16, length=64, log=None)
    # the task's own uncertainty (where a marker comes: 0.2 of the tokens) is
    # 0.45 nats a token; untrained it is log 16 = 2.8
    assert losses[0] > 2.0 and sum(losses[-5:]) / 5 < 1.2
    prompts = ex.batch(5, 33, torch.Generator().manual_seed(9)).cuda()
    tokens = ex.generate(model, prompts, 20)
    with torch.no_grad():
        logits = model(torch.cat([prompts, tokens[:, :-1]], 1))[0][:, 32:]
    best = logits.max(-1).values
    chosen = logits.gather(-1, tokens.unsqueeze(-1)).squeeze(-1)
    # the same arithmetic in another order: the choice may differ where two
    # logits are within rounding of each other
    assert (best - chosen).max().item() <= 1e-3
