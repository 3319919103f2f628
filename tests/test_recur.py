"""The gated linear recurrence (forward, gradients, single steps) against its
definition in 64 bits.

Bounds, with u = 2^-24.  1 - a = (1 - floor) sigmoid(-g) is off, relatively, by at
most d = (|g| + 8) 2^-22: the exponential's argument by 2 |g| u, the exponential
by 2^-22, its sum with 1, the reciprocal and the two products by 8 u together;
below 2^-126 it is 0, which adds an error of TINY.
The state obeys h = a h' + b v, so an error E of it obeys
E = a E' + d b (|v| + M) + rounding, M = a M' + b |v| bounding |h|.  A step
rounds at most twice; the maps of a tile of 64 steps compose in at most 8 + 16
places with two roundings of at most M each, less than one per step; the last
places, which later steps do not inherit, are 16 u M.  The backward runs the same
recurrence over dy."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

U, TINY = 2.0 ** -24, 2.0 ** -126
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def make(dtype, B, L, D, floor=False, valid=None, carry=False, packed=False, seed=0, spread=3.0, shift=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    both = torch.cat([randn(B, L, D) * spread + shift, randn(B, L, D)], -1).to(dt)
    t = {"gate": both[..., :D], "value": both[..., D:]}
    if not packed:
        t = {k: v.contiguous() for k, v in t.items()}
    t["floor"] = torch.rand(D, generator=g, device="cuda") * 0.95 if floor else None
    t["valid"] = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    t["state0"] = randn(B, D) if carry else None
    t["dy"] = randn(B, L, D).to(dt)
    t["dfinal"] = randn(B, D) if carry else None
    return t


def _walk(a, add, start):
    """x_t = a_t x_{t-1} + add_t along axis 1, x_{-1} = start."""
    out = torch.empty_like(add)
    x = start
    for i in range(add.shape[1]):
        x = a[:, i] * x + add[:, i]
        out[:, i] = x
    return out


def reference(t):
    """Values, gradients and their bounds (before the outputs' own rounding), in 64 bits."""
    g, v = t["gate"].double(), t["value"].double()
    B, L, D = g.shape
    keep = 1.0 if t["floor"] is None else 1.0 - t["floor"].double()
    live = torch.ones(B, L, 1, dtype=torch.bool, device="cuda")
    if t["valid"] is not None:
        live = (torch.arange(L, device="cuda") < t["valid"][:, None])[..., None]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    g, v = torch.where(live, g, zero), torch.where(live, v, zero)
    side = torch.sigmoid(-g)
    b = torch.where(live, keep * side, zero)
    a = 1 - b
    d = (g.abs() + 8) * 2.0 ** -22
    start = torch.zeros(B, D, dtype=torch.float64, device="cuda") if t["state0"] is None else t["state0"].double()
    h = _walk(a, b * v, start)
    M = _walk(a, b * v.abs(), start.abs())
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    Mb = torch.cat([start.abs()[:, None], M[:, :-1]], 1)
    E = _walk(a, (d * b + TINY) * (v.abs() + Mb) + 3 * U * (M + Mb), torch.zeros_like(start))
    Eb = torch.cat([torch.zeros_like(start)[:, None], E[:, :-1]], 1) + 16 * U * Mb
    E = E + 16 * U * M
    r = {"y": torch.where(live, h, zero), "y_bound": torch.where(live, E, zero), "final": h[:, -1], "final_bound": E[:, -1],
         "before": before}
    # backward: l_t = dy_t + a_{t+1} l_{t+1}
    dy = torch.where(live, t["dy"].double(), zero)
    if t["dfinal"] is not None:
        dy[:, -1] += t["dfinal"].double()
    size = torch.where(live, t["dy"].double().abs(), zero)
    if t["dfinal"] is not None:
        size[:, -1] += t["dfinal"].double().abs()
    up = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    none = torch.zeros_like(start)
    lam = _walk(up, dy.flip(1), none).flip(1)
    Ml = _walk(up, size.flip(1), none)
    # E_t = a_{t+1} E_{t+1} + (d b)_{t+1} |l_{t+1}| + rounding: the error of a step's decay
    # meets what comes back from that step
    later = ((d * b + TINY).flip(1) * Ml + 3 * U * Ml)[:, :-1]
    El = _walk(up, torch.cat([none[:, None], later], 1) + 3 * U * Ml, none).flip(1) + 16 * U * Ml.flip(1)
    Ml = Ml.flip(1)
    apart, Ea = before - v, Eb + 2 * U * (Mb + v.abs())
    slope = b * (1 - side)
    few = 2 * d + 8 * U
    r["dvalue"], r["dvalue_bound"] = lam * b, El * b + Ml * (b * few + TINY)
    r["dgate"] = lam * apart * slope
    r["dgate_bound"] = slope * (El * (apart.abs() + Ea) + Ml * Ea + Ml * apart.abs() * few) + TINY * Ml * apart.abs()
    part = torch.where(live, side, zero)
    r["dfloor"] = (lam * apart * part).sum((0, 1))
    # the sum: 8 steps, then a thread's tiles, 8 warps and the CTAs' sums, one after the other
    n = 8 + L // 64 + 1 + 8 + 16 * B
    r["dfloor_bound"] = (part * (El * (apart.abs() + Ea) + Ml * Ea + Ml * apart.abs() * (few + n * U))).sum((0, 1))
    r["dstate0"], r["dstate0_bound"] = a[:, 0] * lam[:, 0], a[:, 0] * El[:, 0] + Ml[:, 0] * (d * b)[:, 0] + 16 * U * Ml[:, 0]
    return r


def assert_close(got, ref, name):
    want, bound = ref[name], ref[name + "_bound"]
    if got.dtype is torch.bfloat16:
        bound = bound + torch.finfo(got.dtype).eps / 2 * (want.abs() + bound) + 2.0 ** -134  # half the least number
    else:
        bound = bound + U * (want.abs() + bound) + 2.0 ** -126  # results below are flushed to 0
    assert torch.isfinite(got).all(), name
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), f"{name}: {off.max().item():.3e} over its bound at {int(off.argmax())}"


def run(t, **kw):
    y, final, states = S.recur_fwd(t["gate"], t["value"], t["floor"], t["valid"], state0=t["state0"], want_final=True,
                                   want_states=True)
    g = S.recur_bwd(t["gate"], t["value"], t["floor"], t["valid"], states=states, dy=t["dy"], dfinal=t["dfinal"],
                    want_dstate0=True, **kw)
    return {"y": y, "final": final, "states": states, **g}


NAMES = ("y", "final", "dvalue", "dgate", "dstate0")
CASES = [
    # B, L, D, valid lengths
    (1, 1, 1, None),
    (2, 1, 7, [0, 1]),
    (3, 2, 64, [0, 1, 2]),
    (2, 8, 33, None),
    (3, 9, 130, [9, 8, 1]),
    (2, 63, 64, None),
    (2, 64, 65, [64, 63]),
    (2, 65, 96, None),
    (5, 129, 200, [129, 128, 65, 64, 0]),
    (1, 700, 64, None),
    (4, 300, 513, [300, 1, 0, 257]),
    (1, 3000, 32, None),             # a cluster of 16 CTAs along time
    (2, 2049, 100, [2049, 1025]),
    (1, 1100, 256, [77]),
    (24, 70, 1000, None),            # more CTAs than the GPU holds
    (40, 130, 512, [3 * i for i in range(40)]),
    (300, 16, 72, None),             # short sequences: one warp per CTA
    (70, 17, 72, [i % 18 for i in range(70)]),
    (30, 61, 40, None),
    (1, 3000, 32, [0]),              # a cluster with nothing, or one step, to do
    (1, 3000, 32, [1]),
    (33, 40, 64, [i for i in range(33)]),  # more rows than are sorted by their lengths
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,valid", CASES)
@pytest.mark.parametrize("form", ["plain", "all"])
def test_values_and_gradients(dtype, B, L, D, valid, form):
    every = form == "all"
    t = make(dtype, B, L, D, floor=every, valid=valid, carry=every, packed=every, seed=B + L + D)
    ref, got = reference(t), run(t)
    for name in NAMES + (("dfloor",) if every else ()):
        assert_close(got[name], ref, name)
    assert every or got["dfloor"] is None
    kept = ref["before"][:, ::64]
    assert got["states"].shape == kept.shape
    assert torch.allclose(got["states"].double(), kept, rtol=1e-3, atol=1e-3)
    if valid is not None:
        gone = torch.arange(L, device="cuda") >= t["valid"][:, None]
        for name in ("y", "dvalue", "dgate"):
            assert (got[name][gone] == 0).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_memories(dtype):
    """Decays within 10^-4 of 1 over thousands of steps keep their digits."""
    t = make(dtype, 1, 6000, 40, carry=True, spread=0.5, shift=9.0, seed=5)
    ref, got = reference(t), run(t)
    for name in NAMES:
        assert_close(got[name], ref, name)
    # far inside what a rounded decay would lose: a constant gate, against the closed form
    gate = torch.full((1, 6000, 40), 11.0, device="cuda")
    value = torch.ones_like(gate)
    y, _, _ = S.recur_fwd(gate, value)
    b = torch.sigmoid(torch.tensor(-11.0, dtype=torch.float64))
    steps = torch.arange(1, 6001, dtype=torch.float64)
    want = -torch.expm1(steps * torch.log1p(-b)).cuda()[None, :, None]
    # b is off by at most 19 2^-22; a step and its share of the compositions round
    # within 3 u of the state, which forgets 1.7e-5 a step
    bound = want * (19 * 2.0 ** -22 + steps.cuda()[None, :, None] * 1.5 * U + 16 * U)
    assert ((y.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_saturated_gates(dtype):
    """Gates at +-infinity, at the type's limits and far out: closed, open, and no NaN."""
    inf, top = float("inf"), torch.finfo(DTYPES[dtype]).max
    row = torch.tensor([inf, -inf, top, -top, 100.0, -100.0, 88.9, -88.9, 0.0], device="cuda")
    t = make(dtype, 2, 9 * 20, 64, carry=True, floor=True, seed=3)
    t["gate"] = row.repeat(20)[None, :, None].expand(2, 180, 64).to(DTYPES[dtype]).contiguous()
    got = run(t)
    sane = dict(t, gate=t["gate"].clamp(-200, 200))
    ref = reference(sane)
    for name in NAMES + ("dfloor",):
        assert_close(got[name], ref, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(3, 200, 64), (3, 200, 33), (2, 1100, 64)])
def test_masked_steps_take_no_part(dtype, B, L, D):
    valid = [L // 2 + 1, 0, L][:B]
    t = make(dtype, B, L, D, valid=valid, carry=True, floor=True, packed=True, seed=1)
    clean = run(t)
    gone = torch.arange(L, device="cuda") >= t["valid"][:, None]
    for name, bad in (("gate", float("nan")), ("value", float("inf")), ("dy", float("nan"))):
        t[name] = t[name].clone()
        t[name][gone] = bad
    dirty = run(t)
    for name in clean:
        assert torch.equal(clean[name], dirty[name]), name
    # a row's valid steps alone give the same
    n = valid[0]
    y, final, _ = S.recur_fwd(t["gate"][:1, :n], t["value"][:1, :n], t["floor"], state0=t["state0"][:1], want_final=True)
    assert torch.equal(y, clean["y"][:1, :n])
    empty = [i for i in range(B) if valid[i] == 0]
    assert torch.equal(clean["final"][empty], t["state0"][empty])
    assert torch.equal(clean["dstate0"][empty], t["dfinal"][empty])


@pytest.mark.parametrize("D", [32, 33])
def test_many_short_rows(D):
    """More batch rows than a grid's second axis could hold."""
    t = make("f32", 70000, 3, D, seed=14)
    ref, got = reference(t), run(t)
    for name in NAMES:
        assert_close(got[name], ref, name)


def test_two_streams_at_once():
    """Calls on two streams, each with clusters and workspaces of its own, interleaved."""
    ts = [make("bf16", 1, 4000, 64, carry=True, floor=True, seed=s) for s in (1, 2)]
    want = [run(t) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (t, s) in enumerate(zip(ts, streams)):
            with torch.cuda.stream(s):
                got[i].append(run(t))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for k in g:
                assert torch.equal(g[k], want[i][k]), k


def test_lengths_outside_the_sequence_are_clamped():
    t = make("f32", 3, 100, 64, valid=[-5, 1000, 2 ** 31 - 1])
    u = dict(t, valid=torch.tensor([0, 100, 100], dtype=torch.int32, device="cuda"))
    a, b = run(t), run(u)
    for name in a:
        if a[name] is not None:
            assert torch.equal(a[name], b[name]), name


def strided(B, L, D, batch, step, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = (B - 1) * batch + (L - 1) * step + D
    return torch.randn(n, generator=g).to(dtype).cuda().as_strided((B, L, D), (batch, step, 1))


LAYOUTS = [
    ("time-major", 3, 70, 64, 64, 3 * 64),
    ("wider rows, odd", 3, 70, 64, 71 * 67, 67),
    ("batch rows off a boundary", 3, 70, 64, 70 * 64 + 1, 64),
    ("one step for all of time", 3, 70, 64, 64, 0),
    ("one row for the batch", 3, 70, 64, 0, 64),
    ("overlapping steps", 1, 70, 64, 64, 2),
    ("one step, odd rows", 5, 1, 64, 67, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name,B,L,D,batch,step", LAYOUTS, ids=[v[0] for v in LAYOUTS])
@pytest.mark.parametrize("which", ["gate", "value"])
def test_layouts(name, B, L, D, batch, step, which, dtype):
    t = make(dtype, B, L, D, carry=True, seed=2)
    t[which] = strided(B, L, D, batch, step, DTYPES[dtype], seed=4)
    u = dict(t, **{which: t[which].contiguous()})
    a, b = run(t), run(u)
    ref = reference(u)
    for k in NAMES:
        assert_close(a[k], ref, k)
        assert_close(b[k], ref, k)
    if L == 1:
        state = t["state0"].clone()
        y = S.recur_step(t["gate"][:, 0], t["value"][:, 0], state=state)
        assert_close(y, {"y": ref["y"][:, 0], "y_bound": ref["y_bound"][:, 0]}, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tensors_off_a_boundary(dtype):
    """Tensors that start one element into a buffer: another kernel takes them, which
    splits time otherwise, so that its results are the definition's within the same
    bounds, not the same bits."""
    B, L, D = 2, 90, 64
    t = make(dtype, B, L, D, carry=True, seed=6)
    want = reference(t)

    def shifted(v):
        buf = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
        return buf[1:].view(v.shape).copy_(v)

    out = shifted(torch.zeros_like(t["gate"]))
    y, _, states = S.recur_fwd(shifted(t["gate"]), shifted(t["value"]), state0=shifted(t["state0"]), out=out, want_states=True)
    assert y is out
    assert_close(y, want, "y")
    g = S.recur_bwd(t["gate"], t["value"], states=shifted(states), dy=shifted(t["dy"]), dfinal=t["dfinal"], want_dstate0=True)
    for k in ("dgate", "dvalue", "dstate0"):
        assert_close(g[k], want, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 2048), (3, 33), (130, 64), (1024, 2048), (77, 1000), (5, 513)])
def test_steps(dtype, B, D):
    """A step against the definition, and steps after a prompt against the whole."""
    t = make(dtype, B, 1, D, carry=True, floor=D % 2 == 0, packed=True, seed=D)
    ref = reference(t)
    guard = torch.full((2, D), 7.0, device="cuda")
    held = torch.cat([t["state0"], guard])
    y = S.recur_step(t["gate"][:, 0], t["value"][:, 0], t["floor"], state=held[:B])
    assert_close(y, {"y": ref["y"][:, 0], "y_bound": ref["y_bound"][:, 0]}, "y")
    assert_close(held[:B], {"s": ref["final"], "s_bound": ref["final_bound"]}, "s")
    assert (held[B:] == 7).all()  # nothing is written past the last row


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_steps(dtype):
    B, L, D = 3, 150, 96
    t = make(dtype, B, L, D, carry=True, floor=True, seed=8)
    ref = reference(t)
    n = 131
    y, state, _ = S.recur_fwd(t["gate"][:, :n], t["value"][:, :n], t["floor"], state0=t["state0"], want_final=True)
    rows = [y]
    for i in range(n, L):
        rows.append(S.recur_step(t["gate"][:, i], t["value"][:, i], t["floor"], state=state)[:, None])
    assert_close(torch.cat(rows, 1), ref, "y")
    assert_close(state, ref, "final")
    # the sequence in two calls
    _, state, _ = S.recur_fwd(t["gate"][:, :77], t["value"][:, :77], t["floor"], state0=t["state0"], want_final=True)
    y, final, _ = S.recur_fwd(t["gate"][:, 77:], t["value"][:, 77:], t["floor"], state0=state, want_final=True)
    assert_close(y, {k: v[:, 77:] for k, v in ref.items() if k in ("y", "y_bound")}, "y")
    assert_close(final, ref, "final")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B, L, D, valid", [
    (2, 1, 64, None), (3, 40, 96, [40, 0, 1]), (1, 5000, 64, None), (2, 3000, 33, [2999, 0]), (40, 300, 256, None),
])
def test_a_state_is_carried_in_place(dtype, B, L, D, valid):
    """state0 and out_final in the same memory: the bits of two tensors."""
    t = make(dtype, B, L, D, floor=True, valid=valid, carry=True, seed=11)
    a = (t["gate"], t["value"], t["floor"], t["valid"])
    y, final, states = S.recur_fwd(*a, state0=t["state0"], want_final=True, want_states=True)
    for _ in range(3):
        carried = t["state0"].clone()
        y1, same, states1 = S.recur_fwd(*a, state0=carried, out_final=carried, want_states=True)
        assert same.data_ptr() == carried.data_ptr()
        assert torch.equal(y1, y) and torch.equal(carried, final) and torch.equal(states1, states)


def test_gradients_match_central_differences():
    """Against differences of the 64-bit definition (step 2^-10: truncation of order
    2^-20 of the third derivatives, each at most the sums of the absolute values
    below)."""
    B, L, D = 2, 5, 3
    t = make("f32", B, L, D, carry=True, floor=True, valid=[5, 3], seed=9, spread=1.0, shift=0.0)
    got = run(t)
    live = (torch.arange(L, device="cuda") < t["valid"][:, None])[..., None]

    def total(gate, value, floor, state0):
        b = torch.where(live, (1 - floor) * torch.sigmoid(-gate), 0.0)
        h, s = state0, 0.0
        for i in range(L):
            h = h + b[:, i] * (value[:, i] - h)
            s = s + torch.where(live[:, i], h * t["dy"][:, i].double(), 0.0).sum()
        return s + (h * t["dfinal"].double()).sum()

    base = {k: t[k].double() for k in ("gate", "value", "floor", "state0")}
    step = 2.0 ** -10
    bound = 2.0 ** -18 * (t["dy"].double().abs().sum() + t["dfinal"].double().abs().sum()) * (
        1 + t["value"].abs().max() + t["state0"].abs().max())
    for name in base:
        diff = torch.empty_like(base[name])
        for i in range(diff.numel()):
            side = []
            for sign in (1, -1):
                moved = base[name].clone()
                moved.view(-1)[i] += sign * step
                side.append(total(**dict(base, **{name: moved})))
            diff.view(-1)[i] = (side[0] - side[1]) / (2 * step)
        assert ((got["d" + name].double() - diff).abs() <= bound).all(), name


def test_a_floor_of_one_holds_the_state():
    t = make("f32", 2, 100, 64, carry=True, seed=4)
    t["floor"] = torch.ones(64, device="cuda")
    got, ref = run(t), reference(t)
    assert (got["y"] == t["state0"][:, None]).all() and (got["dgate"] == 0).all() and (got["dvalue"] == 0).all()
    assert_close(got["dfloor"], ref, "dfloor")


def test_the_same_every_time_and_with_dirty_workspaces():
    t = make("bf16", 3, 1500, 128, carry=True, floor=True, valid=[1500, 3, 700], seed=11)
    a = run(t)
    for fill in (0, 255):  # 255: NaN in every type
        ws = torch.full((1 << 20,), fill, dtype=torch.uint8, device="cuda")
        b = run(t, workspace=ws)
        for k in a:
            assert torch.equal(a[k], b[k]), k


def test_another_stream_and_a_graph():
    t = make("f32", 2, 1500, 64, carry=True, floor=True, seed=12)
    want = run(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, final, states = S.recur_fwd(t["gate"], t["value"], t["floor"], state0=t["state0"], want_final=True, want_states=True,
                                   stream=side)
    g = S.recur_bwd(t["gate"], t["value"], t["floor"], states=states, dy=t["dy"], dfinal=t["dfinal"], stream=side)
    side.synchronize()
    assert torch.equal(y, want["y"]) and torch.equal(final, want["final"]) and torch.equal(g["dfloor"], want["dfloor"])
    graph = torch.cuda.CUDAGraph()
    state = t["state0"].clone()
    with torch.cuda.graph(graph):
        got = run(t)
        step = S.recur_step(t["gate"][:, 0], t["value"][:, 0], t["floor"], state=state)
    t["gate"].copy_(t["gate"].flip(1))
    fresh = run(t)
    state.copy_(t["state0"])
    graph.replay()
    torch.cuda.synchronize()
    for k in fresh:
        assert torch.equal(got[k], fresh[k]), k
    again = t["state0"].clone()
    assert torch.equal(S.recur_step(t["gate"][:, 0], t["value"][:, 0], t["floor"], state=again), step)
    assert torch.equal(again, state)


@pytest.mark.parametrize("use", ["y", "final", "both"])
def test_autograd(use):
    t = make("f32", 2, 150, 64, carry=True, floor=True, valid=[150, 70], packed=True, seed=13)
    leaves = {k: t[k].clone().requires_grad_(True) for k in ("floor", "state0")}
    both = torch.cat([t["gate"], t["value"]], -1).requires_grad_(True)
    gate, value = both.split(64, dim=-1)
    y, final = S.gated_recurrence(gate, value, leaves["floor"], t["valid"], state0=leaves["state0"], want_final=True)
    total = 0.0
    if use != "final":
        total = total + (y * t["dy"]).sum()
    else:
        t["dy"] = torch.zeros_like(t["dy"])
    if use != "y":
        total = total + (final * t["dfinal"]).sum()
    else:
        t["dfinal"] = None
    total.backward()
    want = run(t)
    assert torch.equal(both.grad, torch.cat([want["dgate"], want["dvalue"]], -1))
    assert torch.equal(leaves["floor"].grad, want["dfloor"]) and torch.equal(leaves["state0"].grad, want["dstate0"])
    assert torch.equal(S.gated_recurrence(gate, value, leaves["floor"], t["valid"], state0=leaves["state0"]), y)


def test_second_derivatives_are_refused():
    t = make("f32", 1, 20, 32)
    gate = t["gate"].requires_grad_(True)
    y = S.gated_recurrence(gate, t["value"])
    (g,) = torch.autograd.grad((y * y).sum(), gate, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (g * g).sum().backward()


def test_elements_past_32_bits():
    """More than 2^31 elements of y, and of the gradients: one step's gate and value
    for all of time (stride 0), so that every state is known: v (1 - a^t)."""
    D, L = 64, 2 ** 31 // 64 + 100
    gate = torch.linspace(-1, 3, D, device="cuda").to(torch.bfloat16)
    value = torch.linspace(-2, 2, D, device="cuda").to(torch.bfloat16)
    g, v = (x.as_strided((1, L, D), (0, 0, 1)) for x in (gate, value))
    y, final, states = S.recur_fwd(g, v, want_final=True, want_states=True)
    b = torch.sigmoid(-gate.double())
    # the state settles at the value: 3000 steps forget e^-140
    settled = value.double()
    bound = 2.0 ** -8 * settled.abs() + 2.0 ** -18
    for at in (slice(3000, 3100), slice(L // 2, L // 2 + 100), slice(L - 100, L)):
        assert ((y[0, at].double() - settled).abs() <= bound).all()
    first = settled * (1 - (1 - b) ** torch.arange(1, 101, device="cuda")[:, None])
    assert ((y[0, :100].double() - first).abs() <= 2.0 ** -8 * first.abs() + 2.0 ** -18).all()
    assert ((final[0].double() - settled).abs() <= 2.0 ** -18).all()
    y.fill_(1.0)  # dy
    r = S.recur_bwd(g, v, states=states, dy=y, want_dstate0=True)
    # l = sum of a^k = (1 - a^n) / b, n steps from the end; dv = l b
    n = torch.arange(100, 0, -1, device="cuda")[:, None]
    want = 1 - (1 - b) ** n
    assert ((r["dvalue"][0, -100:].double() - want).abs() <= 2.0 ** -8 * want + 2.0 ** -18).all()
    assert ((r["dvalue"][0, :3100].double() - 1).abs() <= 2.0 ** -8 + 2.0 ** -18).all()
    assert ((r["dstate0"][0].double() - (1 - b) / b).abs() <= 2.0 ** -18 * (1 - b) / b).all()


def test_refusals():
    t = make("f32", 2, 30, 64, carry=True, floor=True)
    g, v, f = t["gate"], t["value"], t["floor"]
    _, _, states = S.recur_fwd(g, v, f, want_states=True)
    for call, error in [
        (lambda: S.recur_fwd(g.cpu(), v, f), ValueError),
        (lambda: S.recur_fwd(g, v.cpu(), f), ValueError),
        (lambda: S.recur_fwd(g.half(), v.half(), f), TypeError),
        (lambda: S.recur_fwd(g, v.bfloat16(), f), TypeError),
        (lambda: S.recur_fwd(g, v[:, :5], f), ValueError),
        (lambda: S.recur_fwd(g[0], v[0], f), ValueError),
        (lambda: S.recur_fwd(g.transpose(1, 2), v.transpose(1, 2)), ValueError),
        (lambda: S.recur_fwd(g, v, f[:5]), ValueError),
        (lambda: S.recur_fwd(g, v, f.double()), TypeError),
        (lambda: S.recur_fwd(g, v, f, torch.tensor([1, 2], device="cuda")), TypeError),
        (lambda: S.recur_fwd(g, v, f, state0=t["state0"].bfloat16()), TypeError),
        (lambda: S.recur_fwd(g, v, f, out=torch.empty_like(g)[:, :3]), ValueError),
        (lambda: S.recur_bwd(g, v, f, states=states[:1], dy=t["dy"]), ValueError),
        (lambda: S.recur_bwd(g, v, f, states=states, dy=t["dy"].transpose(0, 1)), ValueError),
        (lambda: S.recur_step(g, v, f, state=t["state0"]), ValueError),
        (lambda: S.recur_step(g[:, 0], v[:, 0], f, state=t["state0"][:1]), ValueError),
        (lambda: S.recur_step(g[:, 0], v[:, 0], f, state=t["state0"].bfloat16()), TypeError),
    ]:
        with pytest.raises(error):
            call()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for call, status in [
        (lambda: S.recur_fwd(g[:, :0], v[:, :0], f), S.Status.ERR_SHAPE),
        (lambda: S.recur_fwd(g[:0], v[:0], f), S.Status.ERR_SHAPE),
        (lambda: S.recur_bwd(g, v, f, states=states, dy=t["dy"], workspace=small), S.Status.ERR_SHAPE),
    ]:
        with pytest.raises(S.SsmError) as e:
            call()
        assert e.value.status == status
