"""The distillation's logits are the products h W^T themselves.

Rows of h with one nonzero value make every logit one exact product, so that only the softmax's own
arithmetic is left.  Bounds, with u = 2^-24 and x a logit's distance to the largest one,
over the temperature: an exponential is off by 10 u |x| + 4 u of itself (its argument
twice, in a tile and where tiles are joined; 2^-22), the sum of the positive terms by 40 u
(8 in a group of 32 columns, 8 groups, the tiles), its logarithm by 2 u of itself; the
maximum over the temperature and the sum with it round 3 times."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_distill import assert_close, make, reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


@pytest.mark.parametrize("tokens", [1, 100, 700])
@pytest.mark.parametrize("vocab,dim", [(1000, 2048), (513, 64)])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 4.0])
def test_exact_products(tokens, vocab, dim, temperature):
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    at = torch.randint(0, dim, (tokens,), generator=g, device="cuda")
    h = torch.zeros(tokens, dim, device="cuda", dtype=torch.bfloat16)
    h[torch.arange(tokens, device="cuda"), at] = 4.0
    w = ((torch.rand(vocab, dim, generator=g, device="cuda") * 2 - 1) * 15).bfloat16()
    ids = torch.randint(0, vocab, (tokens, 5), generator=g, device="cuda")
    logits = torch.randn(tokens, 5, generator=g, device="cuda")
    loss, lse = S.distill_fwd(h, w, ids, logits, temperature=temperature)
    s = 4 * w.double().T[at] / temperature
    want = torch.logsumexp(s, 1)
    p, x = torch.softmax(s, 1), s.amax(1, keepdim=True) - s
    bound = U * ((10 * x * p).sum(1) + 44 + 4 * (want - s.amax(1)) + 2 * s.amax(1).abs() + want.abs())
    assert ((lse.double() - want).abs() <= bound).all()
    q = torch.softmax(logits.double() / temperature, 1)
    terms = q * (torch.log(q) - (s.gather(1, ids) - want[:, None]))
    # q is off by 10 u |x'| + 12 u, its logarithm by as much, a difference of logits by 3 u
    far = (logits.amax(1, keepdim=True) - logits).double() / temperature
    rel = U * (10 * far + 12)
    each = q * (rel * (1 + (torch.log(q) - (s.gather(1, ids) - want[:, None])).abs())
                + U * (4 * torch.log(q).abs() + 6 * (s.amax(1, keepdim=True) - s.gather(1, ids))) + bound[:, None]) + 8 * U * terms.abs()
    assert ((loss.double() - terms.sum(1)).abs() <= each.sum(1)).all()
    if temperature == 1.0:  # the cross entropy's denominator is the same
        _, other = S.xent_fwd(h, w, ids[:, 0].contiguous())
        assert ((other.double() - lse.double()).abs() <= 2 * bound).all()


@pytest.mark.parametrize("tokens", [40, 700])
def test_long_products_are_summed_in_ranges(tokens):
    """The tensor cores cut off a share of an accumulator at every 16 products, so that a logit is
    off by that share of half its size for each of 128 steps; in three ranges of 44 steps, a
    third of the logit each, by 45 / 129 of that.  0.6 leaves room for the rest."""
    V, D = 4000, 2048
    g = torch.Generator(device="cuda").manual_seed(tokens)
    h = torch.randn(tokens, D, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") * 4 / D ** 0.5).bfloat16()
    ids = torch.randint(0, V, (tokens, 3), generator=g, device="cuda")
    want = torch.logsumexp(h.double() @ w.double().T, 1)
    _, whole = S.xent_fwd(h, w, ids[:, 0].contiguous())
    _, lse = S.distill_fwd(h, w, ids, torch.zeros(tokens, 3, device="cuda"))
    assert (lse.double() - want).abs().mean() <= 0.6 * (whole.double() - want).abs().mean()


SEAMS = [
    # tokens, vocab, dim, top, and what differs: around 768 dimensions, half tiles and tiles of the vocabulary
    (1, 1, 776, 1, {}),
    (3, 127, 776, 127, {}),
    (129, 128, 784, 100, dict(ragged=True)),
    (128, 129, 768, 129, {}),
    (257, 257, 1000, 16, dict(ignored=0.4)),
    (40, 385, 832, 300, dict(temp=0.5)),
    (300, 600, 2056, 64, dict(teacher=torch.bfloat16)),
    (100, 700, 4104, 5, dict(temp=3.0)),
    (600, 5000, 1536, 120, dict(low=True)),                  # all entries in the first tile
    (2500, 9001, 776, 9, dict(ragged=True, ignored=0.2)),    # many tiles per cluster
]


@pytest.mark.parametrize("T,V,D,K,more", SEAMS)
def test_values_around_the_seams(T, V, D, K, more):
    t = make(T, V, D, K, seed=T + V, **more)
    ref = reference(t)
    a = (t["h"], t["w"], t["ids"], t["logits"])
    loss, lse = S.distill_fwd(*a, temperature=t["temp"])
    assert_close(loss, ref, "loss")
    assert_close(lse, ref, "lse")
    for fill in (0, 255):  # whatever a workspace holds
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        again = S.distill_fwd(*a, temperature=t["temp"], workspace=ws)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    S.check_device_errors()
