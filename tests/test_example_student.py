"""The student of the example: gated recurrences between an embedding and a
distillation, running, with gradients for every parameter, and generating by single
tokens that follow the pass over the whole sequence."""
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


def test_the_student_learns_from_the_teacher(lm):
    torch.manual_seed(0)
    teacher = lm.Model(vocab=64, dim=64, inner=128).cuda()
    student = lm.Model(vocab=64, dim=32, inner=64, gated=True).cuda()
    before = {k: v.detach().clone() for k, v in student.named_parameters()}
    losses = lm.teach(teacher, student, 5)
    assert all(v == v and abs(v) != float("inf") for v in losses)
    for name, p in student.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and (p.grad != 0).any(), name
        assert not torch.equal(p, before[name]), name
    assert all(p.grad is None for p in teacher.parameters())


def test_single_tokens_follow_the_prompt(lm):
    """Logits token by token equal the whole prompt's within bf16 rounding of the
    activations (the projections round at different sizes)."""
    torch.manual_seed(1)
    model = lm.Model(vocab=300, dim=64, inner=128, gated=True).cuda()
    tokens = torch.randint(0, 300, (3, 20), device="cuda")
    whole, _ = model.prompt(tokens)
    logits, states = model.prompt(tokens[:, :7])
    assert torch.allclose(logits, whole[:, :7], atol=0.05, rtol=0.05)
    for i in range(7, 20):
        logits = model.step(tokens[:, i], states)
        assert torch.allclose(logits, whole[:, i], atol=0.05, rtol=0.05), i
    assert model.generate(tokens, 4).shape == (3, 4)
    S.check_device_errors()
