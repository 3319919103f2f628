"""The gated linear recurrence where a state is kept for long or thrown away at once,
against its definition h <- a h + b v in 64 bits.

Bounds, with u = 2^-24.  e^g is off, relatively, by at most 7 u (the exponential 2^-22 =
4 u, its argument's remainder and its product with it 3 u), whatever g;
sigmoid(-g) = 1 / (1 + e^g) by 7 + 1 + 2 = 10 u; b = (1 - floor) sigmoid(-g) by 12 u; a by 13 u where it is 1 - b >= b, and by 20 u where it
is floor + (1 - floor) e^g sigmoid(-g).  Below 2^-126 all are 0, an error of TINY.
A step then rounds its two terms and their sum, a stretch's maps round as often as its
steps and three times more where they are composed: an error E of the state obeys
E = a E' + 28 u (a M' + b |v|), M = a M' + b |v| bounding |h|.  What is thrown away with
a = 0 leaves no error.  The backward runs the same recurrence over dy."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_recur import DTYPES, TINY, U, _walk, assert_close, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def reference(t):
    """Values, gradients and their bounds (before the outputs' own rounding), in 64 bits."""
    g, v = t["gate"].double(), t["value"].double()
    B, L, D = g.shape
    floor = 0.0 if t["floor"] is None else t["floor"].double()
    open_, hold = torch.sigmoid(-g), torch.sigmoid(g)
    a, b = floor + (1 - floor) * hold, (1 - floor) * open_
    start = t["state0"].double()
    h = _walk(a, b * v, start)
    M = _walk(a, b * v.abs(), start.abs())
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    Mb = torch.cat([start.abs()[:, None], M[:, :-1]], 1)
    E = _walk(a, 28 * U * M + TINY * (Mb + v.abs() + 1), torch.zeros_like(start))
    Eb = torch.cat([torch.zeros_like(start)[:, None], E[:, :-1]], 1)
    r = {"y": h, "y_bound": E, "final": h[:, -1], "final_bound": E[:, -1],
         "states": before[:, ::64], "states_bound": Eb[:, ::64]}
    dy, size = t["dy"].double(), t["dy"].double().abs()
    dy[:, -1] += t["dfinal"].double()
    size[:, -1] += t["dfinal"].double().abs()
    up = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    none = torch.zeros_like(start)
    lam, Ml = _walk(up, dy.flip(1), none).flip(1), _walk(up, size.flip(1), none)
    El = _walk(up, 28 * U * Ml + TINY * (Ml + 1), none).flip(1)
    Ml = Ml.flip(1)
    apart, Ea = before - v, Eb + 2 * U * (Mb + v.abs())
    slope = b * hold
    r["dvalue"], r["dvalue_bound"] = lam * b, El * b + Ml * (14 * U * b + TINY)
    r["dgate"] = lam * apart * slope
    r["dgate_bound"] = slope * (El * (apart.abs() + Ea) + Ml * Ea + 34 * U * Ml * apart.abs()) + TINY * Ml * (apart.abs() + 1)
    r["dstate0"], r["dstate0_bound"] = a[:, 0] * lam[:, 0], a[:, 0] * (El + 22 * U * Ml)[:, 0] + TINY * (Ml[:, 0] + 1)
    return r


SHAPES = [
    (1, 1, 32), (2, 5, 33), (3, 16, 64), (2, 50, 64), (2, 150, 40), (2, 150, 33),
    (1, 3000, 32), (1, 3000, 33),      # a cluster along time
    (24, 300, 1000), (24, 300, 1001),  # more CTAs than the GPU holds
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", SHAPES)
@pytest.mark.parametrize("floor", [False, True])
def test_resets_from_large_states(dtype, B, L, D, floor):
    """Gates that throw most or all of the state away, among values of 10^-4 to 10^8."""
    t = make(dtype, B, L, D, floor=floor, carry=True, seed=B + L + D)
    g = torch.Generator(device="cuda").manual_seed(7)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    resets = torch.tensor([-float("inf"), -80.0, -30.0, -18.0, -12.0, -5.0], device="cuda")
    which = (uniform(B, L, D) * len(resets)).long()
    t["gate"] = torch.where(uniform(B, L, D) < 0.25, resets[which].to(t["gate"].dtype), t["gate"])
    t["value"] = (t["value"].float() * 10 ** (uniform(B, L, D) * 12 - 4)).to(t["value"].dtype)
    t["state0"] = t["state0"] * 1e8
    t["dy"] = (t["dy"].float() * 10 ** (uniform(B, L, D) * 8 - 4)).to(t["dy"].dtype)
    if floor:  # some channels without
        t["floor"] = torch.where(torch.arange(D, device="cuda") % 2 == 0, t["floor"], 0.0)
    ref, got = reference(t), run(t)
    for name in ("y", "final", "states", "dvalue", "dgate", "dstate0"):
        assert_close(got[name], ref, name)
    state = t["state0"].clone()
    y = S.recur_step(t["gate"][:, 0], t["value"][:, 0], t["floor"], state=state)
    one = {k: v[:, 0] for k, v in ref.items() if k in ("y", "y_bound")}
    assert_close(y, one, "y")
    assert_close(state, one, "y")


@pytest.mark.parametrize("L,D", [(1, 64), (20, 64), (20, 33), (3000, 64), (3000, 33)])
@pytest.mark.parametrize("big,v", [(1e8, 1.0), (3e4, 1e-3), (-1e3, 1e-3), (3e38, -3e38)])
def test_an_open_gate_forgets(L, D, big, v):
    """With gates of -infinity every state is its step's value, in every bit."""
    gate = torch.full((2, L, D), -float("inf"), device="cuda")
    value = torch.full((2, L, D), v, device="cuda")
    state = torch.full((2, D), big, device="cuda")
    y, final, states = S.recur_fwd(gate, value, state0=state, want_final=True, want_states=True)
    assert (y == value).all() and (final == value[:, 0]).all()
    if abs(big) < 1e38:  # else the distance of state and value, which dgate takes, is infinite
        dy = torch.ones_like(y)
        g = S.recur_bwd(gate, value, states=states, dy=dy, want_dstate0=True)
        assert torch.equal(g["dvalue"], dy) and (g["dgate"] == 0).all() and (g["dstate0"] == 0).all()
    out = S.recur_step(gate[:, 0], value[:, 0], state=state)
    assert (out == value[:, 0]).all() and (state == value[:, 0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,D", [(1, 64), (20, 33), (3000, 64)])
def test_a_closed_gate_takes_nothing(dtype, L, D):
    """With gates of infinity, or far out, every state is the first, whatever the values."""
    dt = DTYPES[dtype]
    top = torch.finfo(dt).max
    gate = torch.tensor([float("inf"), top, 1e4, 100.0], device="cuda").to(dt).repeat(D)[:D].expand(2, L, D).contiguous()
    value = torch.full((2, L, D), -top, device="cuda", dtype=dt)
    state = torch.linspace(-1, 1, D, device="cuda").to(dt).float().expand(2, D).contiguous()
    y, final, states = S.recur_fwd(gate, value, state0=state, want_final=True, want_states=True)
    assert (y.float() == state[:, None]).all() and torch.equal(final, state)
    g = S.recur_bwd(gate, value.sign(), states=states, dy=torch.ones_like(y), want_dstate0=True)
    assert (g["dvalue"] == 0).all() and (g["dgate"] == 0).all() and (g["dstate0"] == L).all()
    S.recur_step(gate[:, 0], value[:, 0], state=state)
    assert torch.equal(state, final)


STEADY = [(11.0, 0.0), (18.0, 0.0), (6.0, 0.99), (6.0, 0.999), (9.0, 0.5), (4.0, 0.0), (0.5, 0.0), (14.0, 0.9)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [
    (1, 65536, 64), (1, 65536, 33),      # clusters
    (8, 16384, 1024), (5, 16384, 1025),  # more CTAs than the GPU holds, or half of them
])
def test_steady_gates_hold_a_steady_state(dtype, B, L, D):
    """A state equal to a steady value stays there, over all of a long sequence.

    A stretch's e and Q = 1 - P are formed alike; e is off from Q v by 33 u (16 steps of two
    roundings, the product b v), by 24 u more where 8 stretches are composed, P by 40 u:
    a state that enters is moved towards a value within 97 u of v, never past it but for
    its own rounding.  Within a stretch a step rounds twice: 26 u.  128 u in all.
    Backward the same holds for l = dy / b, whose b is off by 12 u, and the share of l that
    goes to the value is dy: 256 u with the products."""
    dt = DTYPES[dtype]
    pick = torch.arange(D, device="cuda") % len(STEADY)
    steady = torch.tensor(STEADY, device="cuda")
    gate = steady[pick, 0].to(dt).expand(B, L, D).contiguous()
    floor = steady[pick, 1].contiguous()
    v = torch.linspace(-2, 2, D, device="cuda").to(dt)
    value = v.expand(B, L, D).contiguous()
    state0 = v.float().expand(B, D).contiguous()
    y, final, states = S.recur_fwd(gate, value, floor, state0=state0, want_final=True, want_states=True)
    bound = 128 * U * state0.abs()
    assert ((final - state0).abs() <= bound).all()
    assert ((states - state0[:, None]).abs() <= bound[:, None]).all()
    if dtype == "f32":
        assert ((y - value).abs() <= 128 * U * value.abs()).all()
    else:  # the value itself is the nearest
        assert torch.equal(y, value)
    b = (1 - floor.double()) * torch.sigmoid(-gate[:, 0].double())
    dfinal = ((1 - b) / b).float()  # what goes back to a step when dy is 1 for ever
    dy = torch.ones_like(gate)
    g = S.recur_bwd(gate, value, floor, states=states, dy=dy, dfinal=dfinal, want_dstate0=True)
    assert ((g["dstate0"].double() * b / (1 - b) - 1).abs() <= 256 * U).all()
    assert ((g["dvalue"].double() - 1).abs() <= 256 * U).all()


@pytest.mark.parametrize("D", [1024, 1023])
def test_sigmoids_keep_their_digits_far_out(D):
    """b, a and a's derivative relative to themselves, for gates up to +-80."""
    gate = torch.linspace(-80, 80, 16 * D, device="cuda").view(16, 1, D)
    g = gate[:, 0].double()
    zero, ones = torch.zeros(16, D, device="cuda"), torch.ones(16, D, device="cuda")
    y, _, states = S.recur_fwd(gate, torch.ones_like(gate), state0=zero, want_states=True)
    b, a = torch.sigmoid(-g), torch.sigmoid(g)
    assert ((y[:, 0].double() / b - 1).abs() <= 14 * U).all()
    r = S.recur_bwd(gate, torch.full_like(gate, -1.0), states=states, dy=torch.zeros_like(gate), dfinal=ones, want_dstate0=True)
    assert ((r["dstate0"].double() / a - 1).abs() <= 24 * U).all()
    assert ((r["dgate"][:, 0].double() / (a * b) - 1).abs() <= 36 * U).all()
    out = S.recur_step(gate[:, 0], torch.ones_like(gate[:, 0]), state=zero)
    assert ((out.double() / b - 1).abs() <= 14 * U).all()
    S.recur_step(gate[:, 0], torch.zeros_like(gate[:, 0]), state=ones)
    assert ((ones.double() / a - 1).abs() <= 24 * U).all()
