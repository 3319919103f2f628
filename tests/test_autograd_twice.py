"""The differentiable functions differentiated twice: the first gradients are the
usual ones, and a second derivative is refused, whether it would come through the
incoming gradient or through what the forward saved."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def leaf(*shape, dtype=torch.float32, seed=0, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(*shape, generator=g) * scale + shift).to(dtype).cuda()).requires_grad_(True)


def conv():
    x, w, b = leaf(2, 20, 16, seed=1), leaf(16, 4, seed=2), leaf(16, seed=3)
    return (x, w, b), lambda: S.causal_conv(x, w, b)


def norm():
    x, w, r = leaf(6, 32, seed=1), leaf(32, seed=2), leaf(6, 32, seed=3)
    return (x, w, r), lambda: S.layer_norm(x, w, residual=r)[0]


def stream():  # only the residual stream's output is used
    x, w, r = leaf(6, 32, seed=1), leaf(32, seed=2), leaf(6, 32, seed=3)
    return (x, r), lambda: S.layer_norm(x, w, residual=r)[1] ** 2


def loss():
    h, w = leaf(5, 64, dtype=torch.bfloat16, seed=1), leaf(50, 64, dtype=torch.bfloat16, seed=2, scale=0.2)
    targets = torch.tensor([3, 4, -100, 0, 49], device="cuda")
    return (h, w), lambda: S.linear_cross_entropy(h, w, targets, reduction="none")


def scan():
    x, dt = leaf(1, 64, 32, seed=1), leaf(1, 64, 32, seed=2, scale=0.1, shift=0.5)
    a, b, c = leaf(32, 16, seed=3, scale=0.1, shift=-1.0), leaf(1, 64, 16, seed=4), leaf(1, 64, 16, seed=5)
    return (x, dt, a, b, c), lambda: S.selective_scan(x, dt, a, b, c, chunk_len=16)


@pytest.mark.parametrize("linear", [True, False], ids=["saved", "incoming"])
@pytest.mark.parametrize("make", [conv, norm, stream, loss, scan])
def test_second_derivatives_are_refused(make, linear):
    leaves, f = make()

    def total():
        y = f().float()
        return y.sum() if linear else (y * y).sum()

    want = torch.autograd.grad(total(), leaves)
    got = torch.autograd.grad(total(), leaves, create_graph=True)
    for a, b in zip(want, got):
        # the scan's dB and dC are summed by atomics, in any order
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-5) if make is scan else torch.equal(a, b)
    # beside a path that is differentiable, as in a penalty on the gradient
    penalty = sum((g.float() ** 2).sum() for g in got) + sum((v.float() ** 2).sum() for v in leaves)
    with pytest.raises(RuntimeError, match="differentiated again"):
        penalty.backward()


def test_gradients_accumulate_as_before():
    """create_graph=True with gradients added up over two calls, in .grad."""
    leaves, f = conv()
    f().sum().backward()
    once = [v.grad.clone() for v in leaves]
    for v in leaves:
        v.grad = None
    for _ in range(2):
        f().sum().backward(create_graph=True)
    for v, g in zip(leaves, once):
        assert torch.equal(v.grad, g + g)
