"""Softmax cross entropy where parts of the vocabulary are masked, tokens are
certain, or logits are far from 0.

A mask over unused entries of the vocabulary is a constant feature: h[:, 0] = 1,
and weight[v, 0] is the masking value for masked entries and 0 for others.  The
masked entries' probabilities are exactly 0 (the masks are 10^10 and more below
the other logits), so everything else is that of the remaining vocabulary, to the
bounds of test_xent.py."""
import math

import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_xent import IGNORE, assert_close, make, reference, run

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.bfloat16).min


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield
    S.check_device_errors()


@pytest.mark.parametrize("T", [1, 12, 70, 300])
@pytest.mark.parametrize("value", [-math.inf, LOWEST])
def test_an_infinite_weight_leaves_the_gradient_finite(T, value):
    """One masked entry: its probability is 0, and so is its row of dweight; the other
    rows are those of the vocabulary without it.  (dh of the feature that holds an
    infinite weight is 0 * inf, by the formula.)"""
    V, D = 300, 64
    t = make(T, V, D, seed=T)
    t["h"][:, 0] = 1.0
    t["w"][:, 0] = 0.0
    t["w"][7, 0] = value
    left = torch.tensor([v for v in range(V) if v != 7], device="cuda")
    t["targets"] = left[t["targets"] % left.numel()]
    small = dict(t, w=t["w"][left].contiguous(), targets=t["targets"] - (t["targets"] > 7).long())
    for dloss in (t["dloss"], torch.full_like(t["dloss"], 0.25)):  # each token's own, and a shared one
        t["dloss"] = small["dloss"] = dloss
        ref, got = reference(small), run(t)
        for name in ("loss", "lse"):
            assert_close(got[name], ref, name)
        first = 1 if math.isinf(value) else 0
        ref["dh"], ref["dh_bound"] = ref["dh"][:, first:], ref["dh_bound"][:, first:]
        assert_close(got["dh"][:, first:], ref, "dh")
        assert_close(got["dweight"][left], ref, "dweight")
        assert (got["dweight"][7] == 0).all()


def spans(V):
    """Masked stretches: the first columns of the vocabulary, a whole tile of 256, a
    stretch that starts or ends inside a tile, the vocabulary's end, all but one."""
    return {"first 32": [(0, 32)], "first tile": [(0, 256)], "first 40": [(0, 40)],
            "middle": [(256, 300), (512, 800)], "end": [(V - 70, V)],
            "all but one": [(0, 600), (601, V)], "every second": [(i, i + 1) for i in range(0, V, 2)]}


def masked(T, V, D, stretches, value, seed):
    t = make(T, V, D, seed=seed)
    t["h"][:, 0] = 1.0
    t["w"][:, 0] = 0.0
    out = torch.zeros(V, dtype=torch.bool, device="cuda")
    for a, b in stretches:
        out[a:b] = True
    t["w"][out, 0] = value
    left = torch.nonzero(~out)[:, 0]
    t["targets"] = left[t["targets"] % left.numel()]
    place = torch.cumsum((~out).long(), 0) - 1
    small = dict(t, w=t["w"][left].contiguous(), targets=place[t["targets"]])
    return t, out, left, small


@pytest.mark.parametrize("value", [-math.inf, LOWEST, -1e30, -1e10, -9e9])
@pytest.mark.parametrize("where", list(spans(1000)))
@pytest.mark.parametrize("T", [12, 40, 300])
def test_masked_vocabulary(T, where, value):
    V, D = 1000, 64
    t, out, left, small = masked(T, V, D, spans(V)[where], value, seed=T)
    ref = reference(small)
    got = run(t)
    for name in ("loss", "lse"):
        assert_close(got[name], ref, name)
    # an infinite weight makes dh of its own feature 0 * inf; the others stand
    first = 1 if math.isinf(value) else 0
    ref["dh"], ref["dh_bound"] = ref["dh"][:, first:], ref["dh_bound"][:, first:]
    assert_close(got["dh"][:, first:], ref, "dh")
    assert_close(got["dweight"][left], ref, "dweight")
    assert (got["dweight"][out] == 0).all()


def exact_logits(T, V, top, seed, D=64):
    """Logits that are exact in fp32 whatever the order of the sums: one feature is 1
    and all others 0, so that S[t, v] = weight[v, 0].  The targets' entry is at `top`,
    the others 16 to 40 below."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = 1.0
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = top - 16 - torch.randint(0, 4, (V,), generator=g, device="cuda") * 8
    target = int(torch.randint(0, V, (1,), generator=g, device="cuda"))
    w[target, 0] = top
    assert (w[:, 0] % 8 == 0).all()  # no entry was rounded: bf16 steps by 8 up to 2048
    return {"h": h, "w": w, "targets": torch.full((T,), target, device="cuda"),
            "dloss": torch.randn(T, generator=g, device="cuda")}


@pytest.mark.parametrize("top", [0.0, 40.0, -1024.0, 1024.0])
@pytest.mark.parametrize("T,V", [(3, 1000), (40, 1000), (300, 700), (20, 1), (50, 1)])
def test_a_certain_tokens_loss_keeps_its_digits(T, V, top):
    """Losses of 1e-5 under an lse of up to 1024: never negative, and within the
    rounding of the sum of exponentials, not of lse.  The sum is 1 and less than
    2^-9; each of its additions is off by at most 2^-24 and at most 64 follow one
    another (1000 columns in steps of 32 and the joins), each exponential by 2^-20
    of itself."""
    t = exact_logits(T, V, top, seed=V + T)
    loss, lse = S.xent_fwd(t["h"], t["w"], t["targets"])
    s = t["w"][:, 0].double()
    # log sum exp(s - top) without the top entry's 1, which log1p takes apart
    rest = torch.exp(s - top).sum() - 1.0
    want = torch.log1p(rest)
    assert (loss >= 0).all()
    assert ((loss.double() - want).abs() <= 64 * 2.0 ** -24 + 2.0 ** -20 * want).all()
    assert ((lse.double() - (top + want)).abs() <= 64 * 2.0 ** -24 + 2.0 ** -22 * abs(top)).all()


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("level", [LOWEST, -1e30, -1e10, 1e10, 1e30])
def test_a_vocabulary_that_is_masked_as_a_whole(T, level):
    """All logits equal, at the mask's value: the loss is the vocabulary's logarithm,
    not the difference of two numbers of the mask's size."""
    V = 1000
    t = make(T, V, 64, seed=T)
    t["h"][:, 1:] = 0
    t["h"][:, 0] = 1.0
    t["w"][:, 0] = level
    loss, lse = S.xent_fwd(t["h"], t["w"], t["targets"])
    assert ((loss.double() - math.log(V)).abs() <= 2.0 ** -18).all()
    assert (lse == t["w"][0, 0].float()).all()


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("level", [-1e30, -1e10, -3.3e9, 3.3e9, 1e10, 1e30])
def test_gradients_of_logits_far_from_0(T, level):
    """G is dloss (exp(S - lse) - onehot) of the lse that the forward returned: with
    one entry at `level` and the others, at twice the distance from 0 below it, of
    probability 0, dweight is -dloss h at the targets and dloss h at that entry."""
    V, D = 600, 64
    t = make(T, V, D, seed=T)
    t["h"][:, 1:] = 0
    t["h"][:, 0] = 1.0
    t["w"][:, 1:] = 0
    t["w"][:, 0] = 2 * level if level < 0 else -level
    t["w"][77, 0] = level
    t["targets"][t["targets"] == 77] = 78
    for dloss in (t["dloss"], torch.full_like(t["dloss"], 0.25)):
        got = run(dict(t, dloss=dloss))
        assert (got["lse"] == t["w"][77, 0].float()).all()
        at = torch.zeros(V, dtype=torch.double, device="cuda")
        at.index_add_(0, t["targets"], -dloss.double())
        at[77] = dloss.double().sum()
        size = torch.zeros_like(at).index_add_(0, t["targets"], dloss.double().abs())
        size[77] = dloss.double().abs().sum()
        # bf16 G, at most 2^-8 of each term, and the result's own rounding
        assert ((got["dweight"][:, 0].double() - at).abs() <= 2 * 2.0 ** -8 * size).all()
        assert (got["dweight"][:, 1:] == 0).all()
        # dh of feature 0: dloss (w[77] - w[target]), each term rounded in G
        want = dloss.double() * (t["w"][77, 0].double() - t["w"][t["targets"], 0].double())
        size = dloss.double().abs() * (abs(t["w"][77, 0].double()) + t["w"][t["targets"], 0].double().abs())
        assert ((got["dh"][:, 0].double() - want).abs() <= 2 * 2.0 ** -8 * size).all()


def test_targets_in_another_order_of_axes_are_refused():
    """Targets [length, batch] for h [batch, length, dim] have the right number of
    elements in the wrong places."""
    t = make(60, 200, 64)
    h, targets = t["h"].view(3, 20, 64), t["targets"].view(3, 20)
    want = S.linear_cross_entropy(h, t["w"], targets)
    assert torch.equal(S.linear_cross_entropy(h, t["w"], t["targets"]), want)  # flat, in order
    for wrong in (targets.T, targets.reshape(20, 3), targets[:, :10], targets[None]):
        with pytest.raises(ValueError):
            S.linear_cross_entropy(h, t["w"], wrong)
    with pytest.raises(ValueError):
        S.linear_cross_entropy(h, t["w"], t["targets"][:59])


@pytest.mark.parametrize("shared", [False, True])
def test_seams_of_the_vocabulary(shared):
    """Several pieces of the vocabulary, with nearly all of each token's probability on
    one column beside a seam: the first and last columns of pieces, tiles and the
    vocabulary.  A column lost or doubled there is an error of the size of dh
    itself."""
    T, V, D = 8000, 70001, 64
    rows = (T + 255) // 256 * 256
    most = (512 << 20) // (2 * rows) // 256                   # tiles of 256 columns in a piece of 512 MiB
    tiles = (V + 255) // 256
    pieces = -(-tiles // most)
    step = -(-tiles // pieces) * 256
    assert pieces > 2
    at = [0, 255, 256, V - 1, V // 64 * 64 - 1] + [c + d for c in range(step, V, step) for d in (-1, 0)]
    at = torch.tensor(sorted(set(at)), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)
    w = (torch.randint(0, 2, (V, D), generator=g, device="cuda") * 2 - 1).to(torch.bfloat16)
    column = at[torch.arange(T, device="cuda") % len(at)]
    t = {"h": w[column] * 0.5, "w": w, "targets": torch.randint(0, V, (T,), generator=g, device="cuda"),
         "dloss": torch.full((T,), 1.0 / T, device="cuda") if shared else
                  torch.randn(T, generator=g, device="cuda")}
    t["targets"] = torch.where(t["targets"] == column, (column + 1000) % V, t["targets"])
    t["targets"][5::50] = IGNORE
    ref, got = reference(t), run(t)
    for name in ("loss", "lse", "dh", "dweight"):
        assert_close(got[name], ref, name)
    if shared:
        for name in ("dh", "dweight"):
            off = (got[name].double() - ref[name]).norm()
            # outputs round by at most 2^-8, 2^-9 on average over a tensor
            assert off <= 2.0 ** -9 * 1.25 * ref[name].norm(), name
