"""The embedding, the gated recurrence and the distillation in one graph, as a
student model runs them: every stage's values and gradients against its definition
in 64 bits, given what the stage before it handed on (the bounds are those of the
stages' own tests)."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
import test_distill
import test_recur
from test_embed import check_gradient, check_lookup

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield
    S.check_device_errors()


def make(B, L, D, V, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    valid = torch.randint(1, L + 1, (B,), **kw, dtype=torch.int32)
    tokens = torch.randint(0, V, (B, L), **kw)
    past = torch.arange(L, device="cuda") >= valid[:, None]
    tokens[past] = IGNORE
    ids = torch.randint(0, V, (B, L, K), **kw)
    ids[past] = IGNORE
    return {"tokens": tokens, "valid": valid, "past": past, "ids": ids, "logits": torch.randn(B, L, K, **kw) * 2,
            "embed": torch.randn(V, D, **kw) * 0.5, "a": torch.randn(D, 2 * D, **kw) / D ** 0.5,
            "floor": torch.rand(D, **kw) * 0.9, "out": (torch.randn(V, D, **kw) * 2 / D ** 0.5).to(torch.bfloat16)}


def forward(t, p):
    x = S.embedding(t["tokens"], p["embed"], scale=2.0)
    gate, value = (x @ p["a"]).chunk(2, dim=-1)                  # read in place, strided
    y = S.gated_recurrence(gate, value, p["floor"], t["valid"])
    h = y.to(torch.bfloat16)
    loss = S.linear_distillation(h, p["out"], t["ids"], t["logits"], temperature=1.5, reduction="none")
    return {"x": x, "gate": gate, "value": value, "y": y, "h": h, "loss": loss}


def check(t, p, f, dloss):
    D, V, K = t["embed"].shape[1], t["embed"].shape[0], t["ids"].shape[2]
    check_lookup({"ids": t["tokens"], "w": t["embed"]}, f["x"].detach(), 2.0)
    r = {"gate": f["gate"].detach(), "value": f["value"].detach(), "floor": t["floor"], "valid": t["valid"],
         "state0": None, "dy": f["y"].grad, "dfinal": None}
    ref = test_recur.reference(r)
    got = {"y": f["y"].detach(), "dgate": f["gate"].grad, "dvalue": f["value"].grad, "dfloor": p["floor"].grad}
    for name in got:
        test_recur.assert_close(got[name], ref, name)
    d = {"h": f["h"].detach().view(-1, D), "w": t["out"], "ids": t["ids"].view(-1, K), "logits": t["logits"].view(-1, K),
         "dloss": dloss.view(-1), "temp": 1.5}
    ref = test_distill.reference(d)
    got = {"loss": f["loss"].detach().view(-1), "dh": f["h"].grad.view(-1, D), "dweight": p["out"].grad}
    for name in got:
        test_distill.assert_close(got[name], ref, name)
    check_gradient({"ids": t["tokens"].view(-1), "w": t["embed"], "dy": f["x"].grad.view(-1, D)}, p["embed"].grad, 2.0)
    assert (f["h"].grad[t["past"]] == 0).all() and (f["gate"].grad[t["past"]] == 0).all()


@pytest.mark.parametrize("B,L,D,V,K", [(3, 150, 64, 300, 8), (2, 1100, 32, 1000, 20), (1, 1, 8, 5, 3), (5, 40, 136, 77, 1)])
def test_training_step(B, L, D, V, K):
    t = make(B, L, D, V, K, seed=B + L)
    p = {k: t[k].clone().requires_grad_(True) for k in ("embed", "a", "floor", "out")}
    f = forward(t, p)
    for k in ("x", "gate", "value", "y", "h"):
        f[k].retain_grad()
    dloss = torch.full((B, L), 1.0 / (B * L), device="cuda")
    f["loss"].backward(dloss)
    check(t, p, f, dloss)


def test_a_captured_training_step():
    """Forward and backward in one graph, replayed on other inputs, give an eager run's
    bits."""
    t, u = make(3, 200, 64, 300, 8, seed=1), make(3, 200, 64, 300, 8, seed=2)
    names = ("embed", "a", "floor", "out")

    def step(v, p):
        f = forward(v, p)
        return f["loss"], torch.autograd.grad(f["loss"].sum(), [p[k] for k in names])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held = {k: v.clone() for k, v in t.items()}
        p = {k: held[k].clone().requires_grad_(True) for k in names}
        step(held, p)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loss, grads = step(held, p)
    torch.cuda.current_stream().wait_stream(side)
    for v in (u, t):
        for k in held:
            held[k].copy_(v[k])
        with torch.no_grad():
            for k in names:
                p[k].copy_(v[k])
        graph.replay()
        torch.cuda.synchronize()
        want, wgrads = step(v, {k: v[k].clone().requires_grad_(True) for k in names})
        assert torch.equal(loss, want)
        for k, a, b in zip(names, grads, wgrads):
            assert torch.equal(a, b), k


def test_a_tied_embedding_gets_both_gradients():
    """The weight at both ends: distill's dweight, and the embedding's added onto it."""
    B, L, D, V, K = 2, 64, 64, 200, 5
    t = make(B, L, D, V, K, seed=4)
    w, tokens = t["out"], t["tokens"].view(-1)
    x = S.embed_fwd(tokens, w)
    loss, lse = S.distill_fwd(x, w, t["ids"].view(-1, K), t["logits"].view(-1, K))
    g = S.distill_bwd(x, w, t["ids"].view(-1, K), t["logits"].view(-1, K), lse=lse, dloss=torch.ones_like(loss))
    first = g["dweight"].clone()
    both = S.embed_bwd(tokens, g["dh"], add_to=g["dweight"])
    check_gradient({"ids": tokens, "w": w, "dy": g["dh"]}, both, 1.0, add=first)
    assert both is g["dweight"]
