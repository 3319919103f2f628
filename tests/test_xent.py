"""Softmax cross entropy over the vocabulary (forward and gradients) against its
definition in 64 bits.

Bounds.  The logits are sums of `dim` exact bf16 products accumulated in fp32,
each addition off by at most 2^-23 of the running magnitude: a logit is within
e = dim 2^-23 max_v sum_d |h w| of the exact one.  lse and loss follow within e
and 2 e, plus 2^-20 of the values themselves for the exponentials, logarithm
and differences.  An entry of G = dloss (p - onehot) is off by dloss p (2 e +
2^-20) and rounded to bf16, at most 2^-8 of it; dh and dweight add those errors
times |weight| or |h|, the accumulation of vocab (or tokens) terms, 2^-23 each,
and their own rounding to bf16."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield
    S.check_device_errors()


def make(T, V, D, ignored=0.0, scale=2.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    t = {"h": torch.randn(T, D, **kw).to(torch.bfloat16),
         "w": (torch.randn(V, D, **kw) * scale / D ** 0.5).to(torch.bfloat16),
         "targets": torch.randint(0, V, (T,), **kw), "dloss": torch.randn(T, **kw)}
    if ignored:
        t["targets"][torch.rand(T, **kw) < ignored] = IGNORE
    return t


def reference(t):
    """The values, the gradients and their bounds, in 64 bits."""
    h, w = t["h"].double(), t["w"].double()
    keep = t["targets"] != IGNORE
    h = torch.where(keep[:, None], h, 0.0)
    T, D = h.shape
    V = w.shape[0]
    S64 = h @ w.T
    size = (h.abs() @ w.abs().T)
    e = D * 2.0 ** -23 * size.amax(1)
    lse = torch.logsumexp(S64, 1)
    at = torch.where(keep, t["targets"], 0)[:, None]
    logit = S64.gather(1, at)[:, 0]
    zero = torch.zeros_like(lse)
    small = 2.0 ** -20 * (1 + lse.abs() + logit.abs())
    g = torch.where(keep, t["dloss"].double(), 0.0)
    p = torch.exp(S64 - lse[:, None])
    del S64, size
    G = p * g[:, None]
    eG = G.abs() * (2 * e + 2.0 ** -20)[:, None]
    G.scatter_add_(1, at, -g[:, None])
    eG += 2.0 ** -8 * (G.abs() + eG)
    dh, dw = G @ w, G.T @ h
    edh = eG @ w.abs() + V * 2.0 ** -23 * (G.abs() @ w.abs())
    edw = eG.T @ h.abs() + T * 2.0 ** -23 * (G.abs().T @ h.abs())
    return {"loss": torch.where(keep, lse - logit, zero), "loss_bound": torch.where(keep, 2 * e + small, zero),
            "lse": torch.where(keep, lse, zero), "lse_bound": torch.where(keep, e + small, zero),
            "dh": dh, "dh_bound": edh + 2.0 ** -8 * (dh.abs() + edh),
            "dweight": dw, "dweight_bound": edw + 2.0 ** -8 * (dw.abs() + edw)}


def assert_close(got, ref, name):
    assert torch.isfinite(got).all(), name
    off = (got.double() - ref[name]).abs() - ref[name + "_bound"]
    assert (off <= 0).all(), f"{name}: {off.max().item():.3e} over its bound at {int(off.argmax())}"


def run(t, **kw):
    loss, lse = S.xent_fwd(t["h"], t["w"], t["targets"], **kw)
    g = S.xent_bwd(t["h"], t["w"], t["targets"], lse=lse, dloss=t["dloss"], **kw)
    return {"loss": loss, "lse": lse, **g}


CASES = [
    # tokens, vocab, dim, ignored, scale
    (1, 1, 8, 0.0, 2.0),
    (1, 5, 8, 0.0, 2.0),
    (3, 257, 64, 0.0, 2.0),
    (2, 40, 72, 0.5, 2.0),
    (130, 1000, 72, 0.3, 2.0),
    (256, 256, 64, 0.0, 2.0),
    (257, 513, 200, 0.0, 2.0),       # one row and one column past a tile
    (511, 255, 520, 0.9, 2.0),
    (300, 20000, 64, 0.1, 2.0),      # dh split along the vocabulary
    (1000, 3001, 768, 0.5, 2.0),
    (700, 5000, 1000, 0.2, 30.0),    # peaked: most probabilities underflow
    (16, 129, 136, 0.2, 2.0),        # up to 32 tokens the forward streams the vocabulary
    (17, 30001, 72, 0.0, 2.0),
    (32, 700, 136, 0.0, 30.0),
    (33, 20000, 64, 0.3, 2.0),
    (64, 33000, 2048, 0.0, 2.0),
    (65, 700, 64, 0.0, 2.0),
    (8000, 70001, 64, 0.1, 2.0),     # several pieces of the vocabulary
]


@pytest.mark.parametrize("T,V,D,ignored,scale", CASES)
def test_values_and_gradients(T, V, D, ignored, scale):
    t = make(T, V, D, ignored, scale)
    ref = reference(t)
    got = run(t)
    S.check_device_errors()
    for name in ("loss", "lse", "dh", "dweight"):
        assert_close(got[name], ref, name)
    gone = t["targets"] == IGNORE
    assert (got["loss"][gone] == 0).all() and (got["dh"][gone] == 0).all()


def test_gradients_match_central_differences():
    """Against differences of the 64-bit loss (step 2^-12, truncation of order
    2^-24); what is left is the rounding of G and of the results to bf16, at
    most 2^-8 each of terms that the scales below bound."""
    t = make(3, 7, 8, scale=4.0, seed=2)
    got = run(t)
    h, w = t["h"].double(), t["w"].double()

    def total(h, w):
        s = h @ w.T
        loss = torch.logsumexp(s, 1) - s.gather(1, t["targets"][:, None])[:, 0]
        return (loss * t["dloss"].double()).sum()

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
        off = (got[name].double() - diff).abs().max()
        assert off <= 2 * 2.0 ** -8 * bounds[name], (name, float(off))


def test_ignored_tokens_take_no_part():
    """What the ignored tokens' rows hold changes nothing; all of them ignored is
    a loss of 0 with zero gradients."""
    t = make(300, 1000, 128, 0.4)
    a = run(t)
    gone = t["targets"] == IGNORE
    dirty = dict(t, h=t["h"].clone(), dloss=t["dloss"].clone())
    dirty["h"][gone] = float("nan")
    dirty["dloss"][gone] = float("inf")
    b = run(dirty)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    # the kept tokens alone give the same
    few = {k: (v if k == "w" else v[~gone]) for k, v in t.items()}
    c = run(few)
    assert torch.equal(c["loss"], a["loss"][~gone]) and torch.equal(c["dh"], a["dh"][~gone])
    assert torch.equal(c["dweight"], a["dweight"])
    none = dict(t, targets=torch.full_like(t["targets"], IGNORE))
    none["h"] = torch.full_like(t["h"], float("nan"))
    d = run(none)
    for k in d:
        assert (d[k] == 0).all(), k


def test_another_ignore_index():
    t = make(200, 300, 64)
    t["targets"][::3] = 7
    kept = t["targets"] != 7
    a = run(t, ignore_index=7)
    assert (a["loss"][~kept] == 0).all()
    few = {k: (v if k == "w" else v[kept]) for k, v in t.items()}
    b = run(few)
    assert torch.equal(a["loss"][kept], b["loss"]) and torch.equal(a["dweight"], b["dweight"])


@pytest.mark.parametrize("T", [100, 12, 40])
def test_targets_outside_the_vocabulary_give_nan(T):
    t = make(T, 300, 64)
    want = run(t)
    for bad in (300, -1, 2 ** 40, -2 ** 40):
        u = dict(t, targets=t["targets"].clone())
        u["targets"][5] = bad
        got = run(u)
        assert got["loss"][5].isnan() and got["dh"][5].isnan().all()
        keep = torch.arange(T, device="cuda") != 5
        assert torch.equal(got["loss"][keep], want["loss"][keep])
        assert torch.equal(got["dh"][keep], want["dh"][keep])
        assert got["dweight"].isnan().all()
    S.check_device_errors()


@pytest.mark.parametrize("T", [100, 12, 40])
def test_nan_rows_stay_apart(T):
    """A token whose hidden state is NaN has a NaN loss; the others' values and dh
    do not change."""
    t = make(T, 300, 64)
    want = run(t)
    u = dict(t, h=t["h"].clone())
    u["h"][9, 3] = float("nan")
    got = run(u)
    keep = torch.arange(T, device="cuda") != 9
    assert got["loss"][9].isnan()
    assert torch.equal(got["loss"][keep], want["loss"][keep])
    assert torch.equal(got["dh"][keep], want["dh"][keep])


def test_the_same_every_time_and_with_dirty_workspaces():
    t = make(700, 9000, 256, 0.2)
    a = run(t)
    lib, dev = S.load(), t["h"].device
    for fill in (0, 255):  # 255: NaN in every type
        big = torch.full((1 << 28,), fill, dtype=torch.uint8, device=dev)
        loss, lse = S.xent_fwd(t["h"], t["w"], t["targets"], workspace=big)
        g = S.xent_bwd(t["h"], t["w"], t["targets"], lse=lse, dloss=t["dloss"], workspace=big.fill_(fill))
        assert torch.equal(loss, a["loss"]) and torch.equal(lse, a["lse"])
        assert torch.equal(g["dh"], a["dh"]) and torch.equal(g["dweight"], a["dweight"])


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd(reduction):
    t = make(60, 500, 96, 0.3)
    h = t["h"].view(3, 20, 96).clone().requires_grad_(True)
    w = t["w"].clone().requires_grad_(True)
    targets = t["targets"].view(3, 20)
    loss = S.linear_cross_entropy(h, w, targets, reduction=reduction)
    kept = t["targets"] != IGNORE
    value, lse = S.xent_fwd(t["h"], t["w"], t["targets"])
    if reduction == "none":
        assert torch.equal(loss.view(-1), value)
        (loss * t["dloss"].view(3, 20)).sum().backward()
        dloss = t["dloss"]
    else:
        scale = 1.0 if reduction == "sum" else 1.0 / float(kept.sum())
        assert torch.allclose(loss, value.sum() * scale, rtol=1e-6)
        loss.backward()
        dloss = torch.full_like(t["dloss"], scale)
    g = S.xent_bwd(t["h"], t["w"], t["targets"], lse=lse, dloss=dloss)
    assert torch.allclose(h.grad.view(60, 96).float(), g["dh"].float(), rtol=2 ** -6, atol=1e-6)
    assert torch.allclose(w.grad.float(), g["dweight"].float(), rtol=2 ** -6, atol=1e-6)
    gone = S.linear_cross_entropy(h, w, torch.full_like(targets, IGNORE))
    assert gone.item() == 0.0


def test_another_stream_and_a_graph():
    t = make(300, 4000, 128, 0.2)
    want = run(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = S.xent_fwd(t["h"], t["w"], t["targets"], stream=side)
    g = S.xent_bwd(t["h"], t["w"], t["targets"], lse=lse, dloss=t["dloss"], stream=side)
    side.synchronize()
    assert torch.equal(loss, want["loss"]) and torch.equal(g["dweight"], want["dweight"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(t)
    t["targets"].copy_(t["targets"].roll(1))
    fresh = run(t)
    graph.replay()
    torch.cuda.synchronize()
    for k in fresh:
        assert torch.equal(got[k], fresh[k]), k


def test_refusals():
    t = make(10, 50, 64)
    h, w, c = t["h"], t["w"], t["targets"]
    _, lse = S.xent_fwd(h, w, c)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for call, error in [
        (lambda: S.xent_fwd(h.cpu(), w, c), ValueError),
        (lambda: S.xent_fwd(h.half(), w, c), TypeError),
        (lambda: S.xent_fwd(h, w.float(), c), TypeError),
        (lambda: S.xent_fwd(h, w[:, :32], c), ValueError),
        (lambda: S.xent_fwd(h, w, c.int()), TypeError),
        (lambda: S.xent_fwd(h, w, c[:5]), ValueError),
        (lambda: S.xent_fwd(h.T, w, c), ValueError),
        (lambda: S.xent_bwd(h, w, c, lse=lse[:3], dloss=t["dloss"]), ValueError),
        (lambda: S.xent_bwd(h, w, c, lse=lse, dloss=t["dloss"].double()), TypeError),
        (lambda: S.linear_cross_entropy(h, w, c, reduction="max"), ValueError),
    ]:
        with pytest.raises(error):
            call()
    for call, status in [
        (lambda: S.xent_fwd(h.float(), w.float(), c), S.Status.ERR_UNSUPPORTED),
        (lambda: S.xent_fwd(h[:, :60].contiguous(), w[:, :60].contiguous(), c), S.Status.ERR_UNSUPPORTED),
        (lambda: S.xent_fwd(h[:0], w, c[:0]), S.Status.ERR_SHAPE),
        (lambda: S.xent_fwd(h, w[:0], c), S.Status.ERR_SHAPE),
        (lambda: S.xent_fwd(h, w, c, workspace=small), S.Status.ERR_SHAPE),
        (lambda: S.xent_bwd(h, w, c, lse=lse, dloss=t["dloss"], workspace=small), S.Status.ERR_SHAPE),
        (lambda: S.xent_fwd(h.view(-1)[4:4 + 8 * 64].view(8, 64), w, c[:8]), S.Status.ERR_ALIGN),
    ]:
        with pytest.raises(S.SsmError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("T,scale", [(1, 1.0), (24, 1 / 24), (40, 3.7e-3), (300, 1 / 300), (24, 0.0)])
def test_a_shared_loss_weight_is_not_rounded(T, scale):
    """With one dloss for all tokens (a mean) the gradients are within their own
    rounding and that of the probabilities: no common factor is lost.  The bound
    is that of `reference` without the rounding of G at the target, p - 1, but for
    the 2^-9 that it loses when p is not small."""
    t = make(T, 3001, 256, 0.2 if T > 1 else 0.0, seed=T)
    t["dloss"] = torch.full((T,), scale, device="cuda")
    ref = reference(t)
    got = run(t)
    for name in ("dh", "dweight"):
        assert_close(got[name], ref, name)
        norm = ref[name].norm()
        off = (got[name].double() - ref[name]).norm()
        # outputs round by at most 2^-8, 2^-9 on average over a tensor
        assert off <= 2.0 ** -9 * 1.25 * norm, (name, float(off / norm))


@pytest.mark.parametrize("T", [8, 40])
def test_a_vocabulary_past_32_bits(T):
    """More than 2^31 elements in the weight and its gradient.  All of its rows
    but the last 300 are zero, so the exact values need those alone.  To the
    bounds at the top comes the sum of as many equal exponentials: at most 512
    additions one after the other (256 columns, then the tiles' sums), 2^-24
    of the sum each."""
    D, n = 2048, 300
    V = 2 ** 31 // D + n
    t = make(T, n, D, seed=5)
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[-n:] = t["w"]
    t["targets"] += V - n
    t["targets"][0] = 0
    got = run(dict(t, w=w))
    S.check_device_errors()
    h, wt, g = t["h"].double(), t["w"].double(), t["dloss"].double()
    s = h @ wt.T
    e = D * 2.0 ** -23 * (h.abs() @ wt.abs().T).amax(1)
    long = 512 * 2.0 ** -24
    lse = torch.log(torch.exp(s).sum(1) + (V - n))
    at = (t["targets"] - (V - n)).clamp_min(0)[:, None]
    logit = torch.where(t["targets"] == 0, 0.0, s.gather(1, at)[:, 0])
    small = 2.0 ** -20 * (1 + lse.abs() + logit.abs()) + long
    for name, ref, bound in (("lse", lse, e + small), ("loss", lse - logit, 2 * e + small)):
        assert ((got[name].double() - ref).abs() <= bound).all(), name
    off_p = (2 * e + long + 2.0 ** -20)[:, None]

    def grads(p, hit):
        G = p * g[:, None]
        eG = G.abs() * off_p
        G = G - hit * g[:, None]
        return G, eG + 2.0 ** -8 * (G.abs() + eG)

    zero = torch.zeros(T, 2, dtype=torch.double, device="cuda")  # the vocabulary's first row, another zero one
    zero[0, 0] = 1.0
    tail = torch.zeros_like(s).scatter_(1, at, (t["targets"] > 0).double()[:, None])
    Gz, eGz = grads(torch.exp(-lse)[:, None].expand(T, 2), zero)
    Gt, eGt = grads(torch.exp(s - lse[:, None]), tail)

    def check(got, G, eG, a, terms, name):
        ref = G @ a
        bound = eG @ a.abs() + terms * 2.0 ** -23 * (G.abs() @ a.abs())
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        off = (got.double() - ref).abs() - bound
        assert (off <= 0).all(), f"{name}: {off.max().item():.3e} over its bound"

    check(got["dh"], Gt, eGt, wt, V, "dh")
    check(got["dweight"][-n:], Gt.T, eGt.T, h, T, "dweight")
    check(got["dweight"][:1], Gz[:, :1].T, eGz[:, :1].T, h, T, "dweight, first row")
    same = got["dweight"][1:2]
    check(same, Gz[:, 1:].T, eGz[:, 1:].T, h, T, "dweight, a zero row")
    assert (got["dweight"][1:-n] == same).all()


@pytest.mark.parametrize("ignored", [False, True])
def test_tokens_past_32_bits(ignored):
    """More than 2^31 elements in h and its gradient; all rows of h but the last
    ones are zero, and where `ignored` out of the loss."""
    D, V, n = 2048, 512, 70
    T = 2 ** 31 // D + n
    small = make(n + 30, V, D, seed=6)
    small["h"][:30] = 0
    small["dloss"][:] = 2.0 ** -10
    if ignored:
        small["targets"][:30] = IGNORE
    g = torch.Generator(device="cuda").manual_seed(7)
    t = {"h": torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"), "w": small["w"],
         "targets": torch.full((T,), IGNORE, device="cuda") if ignored else
                    torch.randint(0, V, (T,), generator=g, device="cuda"),
         "dloss": torch.full((T,), 2.0 ** -10, device="cuda")}
    t["h"][-n:] = small["h"][-n:]
    sample = torch.cat([torch.arange(30, device="cuda"), torch.arange(T - n, T, device="cuda")])
    t["targets"][sample] = small["targets"]
    ref = reference(small)
    got = run(t)
    S.check_device_errors()
    for name in ("loss", "lse", "dh"):
        assert_close(got[name][sample], ref, name)
    assert_close(got["dweight"], ref, "dweight")
    if ignored:
        assert (got["dh"][:-n] == 0).all() and (got["loss"][:-n] == 0).all()
