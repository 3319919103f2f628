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
from test_xent import assert_close, make, reference, run

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
