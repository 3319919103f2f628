"""The digits of the gated linear recurrence's decays, against 64 bits.

Bounds, with u = 2^-24.  e^g is off, relatively, by at most 7 u (the exponential 2^-22 =
4 u, its argument's remainder and its product with it 3 u), whatever g;
sigmoid(-g) = 1 / (1 + e^g) by 7 + 1 + 2 = 10 u; b = (1 - floor) sigmoid(-g) by 12 u."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_recur import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


@pytest.mark.parametrize("D", [1024, 1023])
def test_sigmoids_keep_their_digits_far_out(D):
    """b and a's derivative relative to themselves, for gates up to +-80."""
    gate = torch.linspace(-80, 80, 16 * D, device="cuda").view(16, 1, D)
    g = gate[:, 0].double()
    zero, ones = torch.zeros(16, D, device="cuda"), torch.ones(16, D, device="cuda")
    y, _, states = S.recur_fwd(gate, torch.ones_like(gate), state0=zero, want_states=True)
    b, a = torch.sigmoid(-g), torch.sigmoid(g)
    assert ((y[:, 0].double() / b - 1).abs() <= 14 * U).all()
    r = S.recur_bwd(gate, torch.full_like(gate, -1.0), states=states, dy=torch.zeros_like(gate), dfinal=ones)
    assert ((r["dgate"][:, 0].double() / (a * b) - 1).abs() <= 36 * U).all()
    out = S.recur_step(gate[:, 0], torch.ones_like(gate[:, 0]), state=zero)
    assert ((out.double() / b - 1).abs() <= 14 * U).all()
