"""The operators together, as the example's language model uses them: training
steps whose loss falls, and generation by single tokens that follows the pass
over the whole sequence."""
import importlib.util
import os

import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    spec = importlib.util.spec_from_file_location("example_lm", os.path.join(ROOT, "examples", "lm.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss(lm):
    """From about ln(vocabulary) to well below it within 80 steps: the task's
    targets follow from the two tokens before them."""
    torch.manual_seed(0)
    model = lm.Model(vocab=64, dim=64, inner=128).cuda()
    losses = lm.train(model, 80)
    assert abs(losses[0] - 4.16) < 1.0                 # ln 64
    assert sum(losses[-5:]) / 5 < 0.5 * losses[0]
    for name, p in model.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all(), name


def test_single_tokens_follow_the_prompt(lm):
    """Logits token by token equal the whole prompt's within bf16 rounding of the
    activations (the projections round at different sizes)."""
    torch.manual_seed(1)
    model = lm.Model(vocab=300, dim=64, inner=128).cuda()
    tokens = torch.randint(0, 300, (3, 20), device="cuda")
    whole, _ = model.prompt(tokens)
    logits, states = model.prompt(tokens[:, :7])
    assert torch.allclose(logits, whole[:, :7], atol=0.05, rtol=0.05)
    for i in range(7, 20):
        logits = model.step(tokens[:, i], states)
        assert torch.allclose(logits, whole[:, i], atol=0.05, rtol=0.05), i
    S.check_device_errors()
