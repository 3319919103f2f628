"""Distillation from a teacher's top logits (values and gradients) against its
definition in 64 bits.

Bounds, with u = 2^-24 and T the temperature.  A student's logit is off by at most
e = dim 2^-23 max_v sum_d |h w|, over T by that and 2 u of itself; lse and log p
follow within twice that, plus 2^-20 of the values for exponentials, logarithm and
differences.  A probability q of the teacher is off, relatively, by the
exponential (2^-22 and 2 u of its argument) and the sum of `top` terms:
dq = (|z - max| / T + top + 8) 2^-23.  The loss adds q |log q - log p| dq and its
factors' errors.  An entry of G = (p - q) dloss / T is off by p (2 e / T + 2^-20) +
q dq and rounded to bf16, at most 2^-8 of it; dh and dweight add those errors
times |weight| or |h|, the accumulation of vocab (or tokens) terms, 2^-23 each, and
their own rounding to bf16."""
import math

import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

IGNORE = -100
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield
    S.check_device_errors()


def make(T, V, D, K, ignored=0.0, ragged=False, scale=2.0, temp=1.0, teacher=torch.float32, near=0.5, low=False, seed=0):
    """low: all entries among the first ids, so that one tile of columns holds them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    t = {"h": torch.randn(T, D, **kw).to(torch.bfloat16),
         "w": (torch.randn(V, D, **kw) * scale / D ** 0.5).to(torch.bfloat16), "dloss": torch.randn(T, **kw), "temp": temp}
    z = (t["h"].float() + near * torch.randn(T, D, **kw)).to(torch.bfloat16).float() @ t["w"].float().T
    if low:
        z[:, 2 * K:] = -INF
    z, ids = z.topk(K, dim=1)
    order = torch.rand(T, K, **kw).argsort(1)  # in any order
    t["logits"], t["ids"] = z.gather(1, order).to(teacher), ids.gather(1, order)
    if ragged:
        t["ids"][torch.rand(T, K, **kw) < 0.4] = IGNORE
    if ignored:
        t["ids"][torch.rand(T, **kw) < ignored] = IGNORE
    return t


def reference(t, ignore=IGNORE):
    h, w = t["h"].double(), t["w"].double()
    T, D = h.shape
    V, temp = w.shape[0], t["temp"]
    z = t["logits"].double()
    entry = (t["ids"] != ignore) & (z != -INF)
    K = z.shape[1]
    keep = entry.any(1)
    h = torch.where(keep[:, None], h, 0.0)
    at = torch.where(entry, t["ids"], 0)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    z = torch.where(entry, z, -INF)
    z = torch.where(keep[:, None], z, zero)
    far = torch.where(entry, (z.amax(1, keepdim=True) - z) / temp, zero)
    logq = torch.log_softmax(z / temp, 1)
    q = torch.where(entry, logq.exp(), zero)
    dq = (far + K + 8) * 2.0 ** -23
    S64 = h @ w.T / temp
    size = h.abs() @ w.abs().T
    e = D * 2.0 ** -23 * size.amax(1) / temp + 2.0 ** -23 * S64.abs().amax(1)
    lse = torch.logsumexp(S64, 1)
    logit = S64.gather(1, at)
    small = 2.0 ** -20 * (1 + lse.abs())
    none = torch.zeros_like(lse)
    apart = torch.where(entry & (q > 0), logq - (logit - lse[:, None]), zero)
    loss = (q * apart).sum(1)
    part = (2 * e + small)[:, None] + 2.0 ** -20 * logit.abs() + dq + 2.0 ** -22 * logq.abs()
    eloss = (q * (apart.abs() * (dq + (K + 4) * 2.0 ** -24) + torch.where(q > 0, part, zero))).sum(1)
    g = torch.where(keep, t["dloss"].double(), zero) / temp
    p = torch.exp(S64 - lse[:, None])
    G = p
    eG = p * (2 * e + small)[:, None]
    G = G.scatter_add(1, at, -q)
    eG = eG.scatter_add(1, at, q * dq)
    G, eG = G * g[:, None], eG * g.abs()[:, None]
    eG = eG + 2.0 ** -8 * (G.abs() + eG)
    dh, dw = G @ w, G.T @ h
    edh = eG @ w.abs() + V * 2.0 ** -23 * (G.abs() @ w.abs())
    edw = eG.T @ h.abs() + T * 2.0 ** -23 * (G.abs().T @ h.abs())
    return {"loss": loss, "loss_bound": torch.where(keep, eloss, none), "lse": torch.where(keep, lse, none),
            "lse_bound": torch.where(keep, e + small, none),
            "dh": dh, "dh_bound": edh + 2.0 ** -8 * (dh.abs() + edh),
            "dweight": dw, "dweight_bound": edw + 2.0 ** -8 * (dw.abs() + edw)}


def assert_close(got, ref, name):
    assert torch.isfinite(got).all(), name
    off = (got.double() - ref[name]).abs() - ref[name + "_bound"]
    assert (off <= 0).all(), f"{name}: {off.max().item():.3e} over its bound at {int(off.argmax())}"


def run(t, **kw):
    a = (t["h"], t["w"], t["ids"], t["logits"])
    loss, lse = S.distill_fwd(*a, temperature=t["temp"], **kw)
    return {"loss": loss, "lse": lse, **S.distill_bwd(*a, lse=lse, dloss=t["dloss"], temperature=t["temp"], **kw)}


NAMES = ("loss", "lse", "dh", "dweight")
CASES = [
    # tokens, vocab, dim, top, and what differs
    (1, 1, 8, 1, {}),
    (1, 5, 8, 5, {}),
    (3, 257, 64, 2, {}),
    (2, 40, 72, 40, dict(temp=0.7)),
    (130, 1000, 72, 33, dict(ignored=0.3)),
    (256, 256, 64, 256, dict(ragged=True)),           # every column an entry
    (257, 513, 200, 64, dict(temp=2.0)),              # one row and one column past a tile
    (511, 255, 520, 7, dict(ignored=0.9)),
    (300, 20000, 64, 16, dict(ragged=True, temp=4.0)),
    (1000, 3001, 768, 100, dict(ignored=0.5, teacher=torch.bfloat16)),
    (700, 5000, 1000, 8, dict(scale=30.0)),           # peaked: most probabilities underflow
    (33, 2000, 136, 1000, dict(ragged=True)),
    (40, 3000, 64, 1024, {}),
    (64, 33000, 2048, 32, dict(teacher=torch.bfloat16, temp=0.5)),
    (600, 5000, 64, 120, dict(low=True)),             # all entries in the first tile
    (400, 5000, 64, 1, {}),                           # the cross entropy of the likeliest
    (8000, 70001, 64, 16, dict(ragged=True, ignored=0.1)),  # several pieces of the vocabulary
]


@pytest.mark.parametrize("T,V,D,K,more", CASES)
def test_values_and_gradients(T, V, D, K, more):
    t = make(T, V, D, K, seed=T + K, **more)
    ref, got = reference(t), run(t)
    S.check_device_errors()
    for name in NAMES:
        assert_close(got[name], ref, name)
    gone = (t["ids"] == IGNORE).all(1)
    assert (got["loss"][gone] == 0).all() and (got["lse"][gone] == 0).all() and (got["dh"][gone] == 0).all()


def test_one_entry_is_the_cross_entropy():
    t = make(300, 4000, 128, 1, ignored=0.2)
    loss, lse = S.xent_fwd(t["h"], t["w"], t["ids"][:, 0])
    got = run(t)
    # two results within the bounds of the same definition
    ref = reference(t)
    assert ((got["lse"] - lse).double().abs() <= 2 * ref["lse_bound"]).all()
    assert ((got["loss"] - loss).double().abs() <= 2 * ref["loss_bound"]).all()
    g = S.xent_bwd(t["h"], t["w"], t["ids"][:, 0], lse=lse, dloss=t["dloss"])
    for k in ("dh", "dweight"):
        assert ((g[k].double() - got[k].double()).abs() <= 2 * ref[k + "_bound"]).all(), k


def test_a_student_that_agrees():
    """All of the vocabulary as entries with the student's own logits: a loss and
    gradients of 0, up to the bounds."""
    t = make(40, 300, 64, 300, near=0.0)
    logits = t["h"].float() @ t["w"].float().T
    t["ids"] = torch.arange(300, device="cuda").expand(40, 300).contiguous()
    t["logits"] = logits
    ref, got = reference(t), run(t)
    for name in NAMES:
        assert_close(got[name], ref, name)
    assert got["loss"].abs().max() < 1e-5


def test_the_order_of_entries_does_not_matter_beyond_rounding():
    t = make(200, 1000, 64, 20, ragged=True, seed=4)
    a = run(t)
    perm = torch.randperm(20, device="cuda")
    b = run(dict(t, ids=t["ids"][:, perm].contiguous(), logits=t["logits"][:, perm].contiguous()))
    ref = reference(t)
    for name in NAMES:
        assert_close(b[name], ref, name)
    assert torch.equal(a["lse"], b["lse"])


def test_ids_that_come_twice_count_twice():
    t = make(60, 400, 64, 12, seed=5)
    t["ids"][:, 3] = t["ids"][:, 4]
    t["ids"][::2, 5] = t["ids"][::2, 4]
    t["ids"][:, 6:] = t["ids"][:, 6:7]
    ref, got = reference(t), run(t)
    for name in NAMES:
        assert_close(got[name], ref, name)


@pytest.mark.parametrize("T", [12, 300])
def test_entries_without_weight(T):
    """Logits of -infinity take no part, as ids that are ignored; logits at the type's
    lowest beside others underflow; a token with all of them lowest is uniform."""
    t = make(T, 600, 64, 10, seed=6)
    low = torch.finfo(torch.float32).min
    t["logits"][:, 4] = -INF
    t["logits"][::3] = -INF
    t["logits"][1::3, 5] = low
    t["logits"][2::3] = low
    ref, got = reference(t), run(t)
    for name in NAMES:
        assert_close(got[name], ref, name)
    assert (got["loss"][::3] == 0).all() and (got["dh"][::3] == 0).all()
    u = dict(t, ids=t["ids"].clone(), logits=t["logits"].clone())
    u["ids"][t["logits"] == -INF] = IGNORE
    u["logits"][t["logits"] == -INF] = float("nan")  # of an ignored entry: without effect
    again = run(u)
    for name in NAMES:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("T", [100, 700])
def test_tokens_without_entries_take_no_part(T):
    t = make(T, 1000, 128, 16, ignored=0.4)
    a = run(t)
    gone = (t["ids"] == IGNORE).all(1)
    dirty = dict(t, h=t["h"].clone(), dloss=t["dloss"].clone(), logits=t["logits"].clone())
    dirty["h"][gone] = float("nan")
    dirty["dloss"][gone] = INF
    dirty["logits"][gone] = float("nan")
    b = run(dirty)
    for k in a:
        if T <= 256 and k in ("loss", "lse"):
            assert torch.equal(a[k][~gone], b[k][~gone]) and (b[k][gone] == 0).all()
        else:
            assert torch.equal(a[k], b[k]), k
    few = {k: (v if k in ("w", "temp") else v[~gone]) for k, v in t.items()}
    c = run(few)
    assert torch.equal(c["dh"], a["dh"][~gone]) and torch.equal(c["dweight"], a["dweight"])
    none = dict(t, ids=torch.full_like(t["ids"], IGNORE), h=torch.full_like(t["h"], float("nan")))
    for k, v in run(none).items():
        assert (v == 0).all(), k


@pytest.mark.parametrize("T", [100, 300])
def test_ids_outside_the_vocabulary_give_nan(T):
    t = make(T, 300, 64, 9)
    want = run(t)
    keep = torch.arange(T, device="cuda") != 5
    for bad in (300, 511, -1, 2 ** 31, 2 ** 40, -2 ** 40):
        u = dict(t, ids=t["ids"].clone())
        u["ids"][5, 3] = bad
        got = run(u)
        assert got["loss"][5].isnan() and got["dh"][5].isnan().all() and got["dweight"].isnan().all()
        assert torch.equal(got["loss"][keep], want["loss"][keep]) and torch.equal(got["dh"][keep], want["dh"][keep])
    # a NaN of the teacher stays with its token
    u = dict(t, logits=t["logits"].clone())
    u["logits"][5, 3] = float("nan")
    got = run(u)
    assert got["loss"][5].isnan() and got["dh"][5].isnan().all()
    assert torch.equal(got["loss"][keep], want["loss"][keep]) and torch.equal(got["dh"][keep], want["dh"][keep])
    # and one of the student
    u = dict(t, h=t["h"].clone())
    u["h"][5, 3] = float("nan")
    got = run(u)
    assert got["loss"][5].isnan() and torch.equal(got["loss"][keep], want["loss"][keep])
    assert torch.equal(got["dh"][keep], want["dh"][keep])
    S.check_device_errors()


def test_another_ignore_index():
    t = make(100, 300, 64, 12)
    t["ids"][::3, 2:7] = 7
    a = run(t, ignore_index=7)
    ref = reference(t, ignore=7)
    for name in NAMES:
        assert_close(a[name], ref, name)


@pytest.mark.parametrize("value", [-INF, torch.finfo(torch.bfloat16).min, -1e10])
@pytest.mark.parametrize("T", [40, 300])
def test_masked_vocabulary(T, value):
    """Part of the vocabulary masked by a constant feature: the rest is as without it."""
    V, D = 1000, 64
    t = make(T, V, D, 12, seed=T)
    t["h"][:, 0] = 1.0
    t["w"][:, 0] = 0.0
    out = torch.zeros(V, dtype=torch.bool, device="cuda")
    out[:300] = True
    out[512:700] = True
    t["w"][out, 0] = value
    left = torch.nonzero(~out)[:, 0]
    place = torch.cumsum((~out).long(), 0) - 1
    t["ids"] = left[t["ids"] % left.numel()]
    small = dict(t, w=t["w"][left].contiguous(), ids=place[t["ids"]])
    ref, got = reference(small), run(t)
    for name in ("loss", "lse"):
        assert_close(got[name], ref, name)
    first = 1 if math.isinf(value) else 0
    ref["dh"], ref["dh_bound"] = ref["dh"][:, first:], ref["dh_bound"][:, first:]
    assert_close(got["dh"][:, first:], ref, "dh")
    assert_close(got["dweight"][left], ref, "dweight")
    assert (got["dweight"][out] == 0).all()


def test_gradients_match_central_differences():
    """Against differences of the 64-bit loss (step 2^-12, truncation of order
    2^-24); what is left is the rounding of G and of the results to bf16, at most
    2^-8 each of terms that the scales below bound."""
    t = make(3, 7, 8, 4, scale=4.0, temp=1.5, seed=2)
    got = run(t)
    h, w = t["h"].double(), t["w"].double()
    logq = torch.log_softmax(t["logits"].double() / 1.5, 1)

    def total(h, w):
        logp = torch.log_softmax(h @ w.T / 1.5, 1)
        return ((logq.exp() * (logq - logp.gather(1, t["ids"]))).sum(1) * t["dloss"].double()).sum()

    step = 2.0 ** -12
    bounds = {"dh": t["dloss"].abs().max() * 2 * w.abs().sum(0).max(),
              "dweight": t["dloss"].abs().max() * h.abs().sum(0).max()}
    for name, base in (("dh", h), ("dweight", w)):
        diff = torch.empty_like(base)
        for i in range(base.numel()):
            moved = [base.clone(), base.clone()]
            moved[0].view(-1)[i] += step
            moved[1].view(-1)[i] -= step
            side = [total(m, w) if name == "dh" else total(h, m) for m in moved]
            diff.view(-1)[i] = (side[0] - side[1]) / (2 * step)
        assert (got[name].double() - diff).abs().max() <= 2 * 2.0 ** -8 * bounds[name], name


def test_a_shared_loss_weight_is_not_rounded():
    t = make(40, 3001, 256, 8, temp=3.0, seed=7)
    t["dloss"] = torch.full((40,), 1 / 40, device="cuda")
    ref, got = reference(t), run(t)
    for name in ("dh", "dweight"):
        assert_close(got[name], ref, name)


def test_the_same_every_time_and_with_dirty_workspaces():
    t = make(700, 9000, 256, 24, ignored=0.2, ragged=True)
    a = run(t)
    for fill in (0, 255):  # 255: NaN in every type
        big = torch.full((1 << 28,), fill, dtype=torch.uint8, device="cuda")
        loss, lse = S.distill_fwd(t["h"], t["w"], t["ids"], t["logits"], workspace=big)
        g = S.distill_bwd(t["h"], t["w"], t["ids"], t["logits"], lse=lse, dloss=t["dloss"], workspace=big.fill_(fill))
        assert torch.equal(loss, a["loss"]) and torch.equal(lse, a["lse"])
        assert torch.equal(g["dh"], a["dh"]) and torch.equal(g["dweight"], a["dweight"])


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd(reduction):
    t = make(60, 500, 96, 6, ignored=0.3, temp=2.0)
    h = t["h"].view(3, 20, 96).clone().requires_grad_(True)
    w = t["w"].clone().requires_grad_(True)
    ids, logits = t["ids"].view(3, 20, 6), t["logits"].view(3, 20, 6)
    loss = S.linear_distillation(h, w, ids, logits, temperature=2.0, reduction=reduction)
    kept = (t["ids"] != IGNORE).any(1)
    value, lse = S.distill_fwd(t["h"], t["w"], t["ids"], t["logits"], temperature=2.0)
    if reduction == "none":
        assert torch.equal(loss.view(-1), value)
        (loss * t["dloss"].view(3, 20)).sum().backward()
        dloss = t["dloss"]
    else:
        scale = 1.0 if reduction == "sum" else 1.0 / float(kept.sum())
        assert torch.allclose(loss, value.sum() * scale, rtol=1e-6)
        loss.backward()
        dloss = torch.full_like(t["dloss"], scale)
    g = S.distill_bwd(t["h"], t["w"], t["ids"], t["logits"], lse=lse, dloss=dloss, temperature=2.0)
    assert torch.allclose(h.grad.view(60, 96).float(), g["dh"].float(), rtol=2 ** -6, atol=1e-6)
    assert torch.allclose(w.grad.float(), g["dweight"].float(), rtol=2 ** -6, atol=1e-6)
    assert S.linear_distillation(h, w, torch.full_like(ids, IGNORE), logits).item() == 0.0
    (once,) = torch.autograd.grad(S.linear_distillation(h, w, ids, logits) ** 2, h, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        once.float().sum().backward()


def test_another_stream_and_a_graph():
    t = make(300, 4000, 128, 10, ignored=0.2)
    want = run(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = (t["h"], t["w"], t["ids"], t["logits"])
    loss, lse = S.distill_fwd(*a, stream=side)
    g = S.distill_bwd(*a, lse=lse, dloss=t["dloss"], stream=side)
    side.synchronize()
    assert torch.equal(loss, want["loss"]) and torch.equal(g["dweight"], want["dweight"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(t)
    t["ids"].copy_(t["ids"].roll(1, 0))
    t["logits"].copy_(t["logits"].roll(1, 0))
    fresh = run(t)
    graph.replay()
    torch.cuda.synchronize()
    for k in fresh:
        assert torch.equal(got[k], fresh[k]), k


def test_a_vocabulary_past_32_bits():
    """More than 2^31 elements in the weight and its gradient.  All rows but the last
    300 are zero: the exact values need those alone and the number of the others."""
    D, n, T, K = 2048, 300, 40, 8
    V = 2 ** 31 // D + n
    t = make(T, n, D, K, seed=5)
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[-n:] = t["w"]
    got = run(dict(t, w=w, ids=t["ids"] + (V - n)))
    S.check_device_errors()
    h, wt = t["h"].double(), t["w"].double()
    s = h @ wt.T
    lse = torch.log(torch.exp(s).sum(1) + (V - n))
    e = D * 2.0 ** -23 * (h.abs() @ wt.abs().T).amax(1)
    # the sum of as many equal exponentials: at most 512 additions after one another
    small = 2.0 ** -20 * (1 + lse.abs()) + 512 * 2.0 ** -24
    assert ((got["lse"].double() - lse).abs() <= e + small).all()
    logq = torch.log_softmax(t["logits"].double(), 1)
    loss = (logq.exp() * (logq - s.gather(1, t["ids"]) + lse[:, None])).sum(1)
    assert ((got["loss"].double() - loss).abs() <= 2 * e + 4 * small).all()
    # a zero row's G is dloss p, rounded to bf16: 2^-8 of each term, and as much again
    # for p's own error (which is far below that)
    G = (torch.exp(-lse) * t["dloss"].double())[:, None]
    ref = (G * h).sum(0)
    assert ((got["dweight"][0].double() - ref).abs() <= 2.0 ** -7 * (G.abs() * h.abs()).sum(0) + 2.0 ** -8 * ref.abs()).all()
    G = torch.exp(s - lse[:, None]).scatter_add(1, t["ids"], -logq.exp()) * t["dloss"].double()[:, None]
    ref = G.T @ h
    bound = 2.0 ** -7 * (G.abs().T @ h.abs()) + 2.0 ** -8 * ref.abs()
    assert ((got["dweight"][-n:].double() - ref).abs() <= bound).all()


def test_refusals():
    t = make(10, 50, 64, 4)
    h, w, ids, z = t["h"], t["w"], t["ids"], t["logits"]
    _, lse = S.distill_fwd(h, w, ids, z)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for call, error in [
        (lambda: S.distill_fwd(h.cpu(), w, ids, z), ValueError),
        (lambda: S.distill_fwd(h.half(), w, ids, z), TypeError),
        (lambda: S.distill_fwd(h, w.float(), ids, z), TypeError),
        (lambda: S.distill_fwd(h, w[:, :32], ids, z), ValueError),
        (lambda: S.distill_fwd(h, w, ids.int(), z), TypeError),
        (lambda: S.distill_fwd(h, w, ids[:5], z), ValueError),
        (lambda: S.distill_fwd(h, w, ids[:, 0], z), ValueError),
        (lambda: S.distill_fwd(h, w, ids, z[:, :3]), ValueError),
        (lambda: S.distill_fwd(h, w, ids, z.half()), TypeError),
        (lambda: S.distill_fwd(h, w, ids.T.contiguous().T, z), ValueError),
        (lambda: S.distill_bwd(h, w, ids, z, lse=lse[:3], dloss=t["dloss"]), ValueError),
        (lambda: S.distill_bwd(h, w, ids, z, lse=lse, dloss=t["dloss"].double()), TypeError),
        (lambda: S.linear_distillation(h, w, ids, z, reduction="max"), ValueError),
        (lambda: S.linear_distillation(h, w, ids, z.clone().requires_grad_(True)), ValueError),
        (lambda: S.linear_distillation(h.view(2, 5, 64), w, ids, z), ValueError),
    ]:
        with pytest.raises(error):
            call()
    many = torch.zeros(10, 1025, dtype=torch.int64, device="cuda")
    for call, status in [
        (lambda: S.distill_fwd(h.float(), w.float(), ids, z), S.Status.ERR_UNSUPPORTED),
        (lambda: S.distill_fwd(h[:, :60].contiguous(), w[:, :60].contiguous(), ids, z), S.Status.ERR_UNSUPPORTED),
        (lambda: S.distill_fwd(h, w, many, many.float()), S.Status.ERR_UNSUPPORTED),
        (lambda: S.distill_fwd(h[:0], w, ids[:0], z[:0]), S.Status.ERR_SHAPE),
        (lambda: S.distill_fwd(h, w, ids[:, :0], z[:, :0]), S.Status.ERR_SHAPE),
        (lambda: S.distill_fwd(h, w, ids, z, temperature=0.0), S.Status.ERR_SHAPE),
        (lambda: S.distill_fwd(h, w, ids, z, workspace=small), S.Status.ERR_SHAPE),
        (lambda: S.distill_bwd(h, w, ids, z, lse=lse, dloss=t["dloss"], workspace=small), S.Status.ERR_SHAPE),
    ]:
        with pytest.raises(S.SsmError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("T,K", [(1, 1), (1, 3), (24, 2), (128, 4), (100, 64)])
@pytest.mark.parametrize("shared", [True, False])
def test_gradients_of_few_tokens_keep_their_digits(T, K, shared):
    """Up to 128 tokens G is kept in two halves of 8 bits each, off by 2^-16: dh and
    dweight are off by their own rounding (at most 2^-8, 2^-9 on average over a
    tensor) and a little."""
    t = make(T, 3001, 256, K, seed=T + K, ragged=K > 2)
    if shared:
        t["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
    ref, got = reference(t), run(t)
    for name in ("dh", "dweight"):
        assert_close(got[name], ref, name)
        off = (got[name].double() - ref[name]).norm()
        assert off <= 2.0 ** -9 * 1.25 * ref[name].norm(), (name, float(off / ref[name].norm()))


@pytest.mark.parametrize("T,ignored", [(127, 0.0), (128, 0.0), (129, 0.0), (300, 0.6)])
def test_around_half_a_tile_of_tokens(T, ignored):
    """The count of tokens with entries decides, also where others are left out."""
    t = make(T, 700, 136, 12, ignored=ignored, seed=T)
    ref, got = reference(t), run(t)
    for name in NAMES:
        assert_close(got[name], ref, name)
