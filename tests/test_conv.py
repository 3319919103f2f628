"""The short causal convolution (forward, backward, single steps) against its
formulas in 64 bits.

Bounds.  With u = 2^-24, pre is a sum of at most five products, each rounded
once, so it is within 8 u S of the exact one, S = |bias| + sum |w x|.  silu has
slope at most 1.1 and is evaluated with a 2-ulp exponential and quotient, so y
is within 2^-20 S; bf16 outputs add half an ulp, at most 2^-8 |y|.  In the backward
silu'' <= 0.5 carries the error of pre: dpre is within 2^-20 |dy| (1 + S), dx
within the same times sum |w|.  The weight sums add n terms, at most `n` of
them one after the other: n u on top of each term's own error."""
import numpy as np
import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def make(dtype, B, L, D, K, *, bias=True, valid=None, carry=False, pad=0, seed=0):
    """Inputs on the GPU; `pad` > 0 gives x as columns [pad, pad + D) of wider rows."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    wide = torch.randn(B, L, D + 2 * pad, generator=g).to(dt).cuda()
    t = {"x": wide[:, :, pad:pad + D] if pad else wide,
         "w": (torch.rand(D, K, generator=g) * 2 - 1).cuda(),
         "b": torch.randn(D, generator=g).cuda() if bias else None,
         "valid": torch.tensor(valid, dtype=torch.int32).cuda() if valid is not None else None,
         "state0": torch.randn(B, K - 1, D, generator=g).to(dt).cuda() if carry else None,
         "dy": torch.randn(B, L, D, generator=g).to(dt).cuda()}
    return t


def f64(t):
    return t.detach().double().cpu().numpy()


def reference(t, silu, dy=None):
    """Outputs, error scales and gradients by the formulas, step by step."""
    x, w = f64(t["x"]), f64(t["w"])
    B, L, D = x.shape
    K = w.shape[1]
    b = f64(t["b"]) if t["b"] is not None else np.zeros(D)
    head = f64(t["state0"]) if t["state0"] is not None else np.zeros((B, K - 1, D))
    vl = [L] * B if t["valid"] is None else [min(max(int(v), 0), L) for v in t["valid"].cpu()]
    y, scale = np.zeros((B, L, D)), np.zeros((B, L, D))
    final = np.zeros((B, K - 1, D))
    dxp = np.zeros((B, L + K - 1, D))
    dxs = np.zeros((B, L + K - 1, D))
    dw, dws, db, dbs = np.zeros((D, K)), np.zeros((D, K)), np.zeros(D), np.zeros(D)
    for i in range(B):
        n = vl[i]
        xp = np.concatenate([head[i], x[i, :n]])
        final[i] = xp[n:n + K - 1]
        if n == 0:
            continue
        win = np.stack([xp[k:k + n] for k in range(K)], -1)            # [n, D, K]
        pre = b + (win * w).sum(-1)
        scale[i, :n] = np.abs(b) + (np.abs(win) * np.abs(w)).sum(-1)
        s = 1 / (1 + np.exp(-pre))
        y[i, :n] = pre * s if silu else pre
        if dy is None:
            continue
        g = dy[i, :n] * (s * (1 + pre * (1 - s)) if silu else 1)
        e = np.abs(dy[i, :n]) * (1 + scale[i, :n])
        for k in range(K):
            dxp[i, k:k + n] += g * w[:, k]
            dxs[i, k:k + n] += e * np.abs(w[:, k])
        dw += (g[:, :, None] * win).sum(0)
        dws += (e[:, :, None] * np.abs(win)).sum(0)
        db += g.sum(0)
        dbs += e.sum(0)
    return {"y": y, "scale": scale, "final": final, "dx": dxp[:, K - 1:], "dx_scale": dxs[:, K - 1:],
            "dstate0": dxp[:, :K - 1], "dstate0_scale": dxs[:, :K - 1], "dw": dw, "dw_scale": dws,
            "db": db, "db_scale": dbs}


def assert_close(got, want, bound, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), f"{what}: {off.max():.3e} over its bound at {np.unravel_index(off.argmax(), off.shape)}"


def half_ulp(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0


CASES = [
    # dtype, B, L, D, K, silu, bias, valid, carry, pad
    ("f32", 1, 1, 1, 4, True, True, None, False, 0),
    ("f32", 2, 2, 8, 4, True, True, None, True, 0),       # shorter than the taps
    ("bf16", 3, 130, 64, 4, True, True, [130, 0, 2], True, 0),
    ("bf16", 2, 257, 200, 3, False, False, [257, 256], False, 200),  # x inside wider rows
    ("f32", 2, 100, 33, 2, True, True, [1, 99], True, 0),  # an odd width: single elements
    ("bf16", 2, 77, 264, 4, True, False, None, True, 4),   # rows that start off a 16-byte boundary
    ("bf16", 1, 700, 513, 4, True, True, None, False, 513),
    ("f32", 4, 64, 1024, 4, False, True, [64, 5, 63, 8], False, 0),
    ("f32", 1, 4000, 260, 3, True, True, None, True, 0),
    ("bf16", 40, 9, 48, 2, True, True, [9] * 20 + [-3, 12] * 10, False, 0),  # lengths outside [0, L]
]


@pytest.mark.parametrize("dtype,B,L,D,K,silu,bias,valid,carry,pad", CASES)
def test_forward_and_backward_match_the_formulas(dtype, B, L, D, K, silu, bias, valid, carry, pad):
    t = make(dtype, B, L, D, K, bias=bias, valid=valid, carry=carry, pad=pad)
    ref = reference(t, silu, f64(t["dy"]))
    y, final = S.conv_fwd(t["x"], t["w"], t["b"], t["valid"], state0=t["state0"], silu=silu,
                          want_final=True)
    g = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=t["dy"], state0=t["state0"], silu=silu,
                   want_dstate0=carry)
    assert_close(y, ref["y"], half_ulp(dtype, ref["y"]) + 2.0 ** -20 * ref["scale"], "y")
    assert (f64(final) == ref["final"]).all()
    if valid is not None:
        n = t["valid"].clamp(0, L)
        past = torch.arange(L, device="cuda") >= n[:, None]
        assert (y[past] == 0).all() and (g["dx"][past] == 0).all()
    assert_close(g["dx"], ref["dx"], half_ulp(dtype, ref["dx"]) + 2.0 ** -20 * ref["dx_scale"], "dx")
    if carry:
        assert_close(g["dstate0"], ref["dstate0"],
                     half_ulp(dtype, ref["dstate0"]) + 2.0 ** -20 * ref["dstate0_scale"], "dstate0")
    n = min(B * L, 1024)
    assert_close(g["dweight"], ref["dw"], (2.0 ** -20 + n * U) * ref["dw_scale"], "dweight")
    if bias:
        assert_close(g["dbias"], ref["db"], (2.0 ** -20 + n * U) * ref["db_scale"], "dbias")
    else:
        assert g["dbias"] is None


@pytest.mark.parametrize("silu", [True, False])
def test_gradients_match_central_differences(silu):
    """The kernel's gradients against differences of the 64-bit forward: a step
    of 2^-12 leaves a truncation error of order 2^-24 and, in 64 bits, no
    rounding to speak of; the kernel's own error is of order 2^-20 per term."""
    t = make("f32", 2, 11, 6, 4, valid=[11, 7], carry=True, seed=5)
    g = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=t["dy"], state0=t["state0"], silu=silu,
                   want_dstate0=True)
    dy, h = f64(t["dy"]), 2.0 ** -12
    for name, grad in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("state0", "dstate0")):
        base = t[name].double().cpu()
        got, diff = f64(g[grad]), np.empty(base.shape)
        for at in np.ndindex(*base.shape):
            side = []
            for sign in (1, -1):
                moved = base.clone()
                moved[at] += sign * h
                side.append((reference({**t, name: moved}, silu)["y"] * dy).sum())
            diff[at] = (side[0] - side[1]) / (2 * h)
        assert np.abs(got - diff).max() <= 1e-5 * max(1.0, np.abs(diff).max()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_steps_are_not_read(dtype):
    """NaN and infinities past valid_len change nothing, in x or in dy."""
    t = make(dtype, 3, 150, 72, 4, valid=[150, 70, 0], carry=True)
    clean = S.conv_fwd(t["x"], t["w"], t["b"], t["valid"], state0=t["state0"], want_final=True)
    kw = dict(state0=t["state0"], want_dstate0=True)
    g = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=t["dy"], **kw)
    x, dy = t["x"].clone(), t["dy"].clone()
    for i, n in enumerate([150, 70, 0]):
        x[i, n:] = float("nan")
        dy[i, n:] = float("inf")
        dy[i, n + 1:] = torch.finfo(dy.dtype).min
    dirty = S.conv_fwd(x, t["w"], t["b"], t["valid"], state0=t["state0"], want_final=True)
    gd = S.conv_bwd(x, t["w"], t["b"], t["valid"], dy=dy, **kw)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    for k in g:
        assert torch.equal(g[k], gd[k]), k


@pytest.mark.parametrize("dtype,D,K", [("f32", 40, 4), ("bf16", 2048, 4), ("bf16", 37, 3),
                                       ("f32", 5, 2)])
def test_steps_and_pieces_follow_the_whole(dtype, D, K):
    """Single steps on the carried state, and a call over the rest from the
    first call's final state, give the bits of one call."""
    B, L, cut = 3, 23, 9
    t = make(dtype, B, L, D, K, seed=3)
    whole, final = S.conv_fwd(t["x"], t["w"], t["b"], want_final=True)
    first, state = S.conv_fwd(t["x"][:, :cut], t["w"], t["b"], want_final=True)
    assert torch.equal(first, whole[:, :cut])
    rest, end = S.conv_fwd(t["x"][:, cut:], t["w"], t["b"], state0=state, want_final=True)
    assert torch.equal(rest, whole[:, cut:]) and torch.equal(end, final)
    state = torch.zeros(B, K - 1, D, dtype=t["x"].dtype, device="cuda")
    for i in range(L):
        y = S.conv_step(t["x"][:, i], t["w"], t["b"], state=state)
        assert torch.equal(y, whole[:, i]), i
    assert torch.equal(state, final)


def test_backward_is_the_same_every_time():
    t = make("bf16", 5, 900, 320, 4, valid=[900, 1, 333, 0, 899])
    a = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=t["dy"])
    for _ in range(3):
        b = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=t["dy"])
        assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


def test_broadcast_rows():
    """x may be one row seen by every batch row (stride 0): its gradient is
    still one per batch row."""
    t = make("f32", 1, 50, 24, 4)
    x = t["x"].expand(4, 50, 24)
    y = S.conv_fwd(x, t["w"], t["b"])
    one = S.conv_fwd(t["x"], t["w"], t["b"])
    assert torch.equal(y, one.expand(4, 50, 24))


def test_autograd():
    """causal_conv under autograd returns the library's backward, for a strided x
    and a broadcast incoming gradient."""
    t = make("bf16", 2, 60, 32, 4, carry=True, valid=[60, 31], pad=32)
    leaves = {k: t[k].detach().clone().requires_grad_(True) for k in ("x", "w", "b", "state0")}
    y = S.causal_conv(leaves["x"], leaves["w"], leaves["b"], t["valid"], state0=leaves["state0"])
    y.sum().backward()
    g = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=torch.ones_like(y), state0=t["state0"],
                   want_dstate0=True)
    for k, grad in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("state0", "dstate0")):
        assert torch.equal(leaves[k].grad, g[grad]), k


def test_another_stream_and_a_graph():
    t = make("bf16", 2, 300, 128, 4)
    want = S.conv_fwd(t["x"], t["w"], t["b"])
    gwant = S.conv_bwd(t["x"], t["w"], t["b"], dy=t["dy"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        got = S.conv_fwd(t["x"], t["w"], t["b"], stream=handle)
        ggot = S.conv_bwd(t["x"], t["w"], t["b"], dy=t["dy"], stream=handle)
        side.synchronize()
        assert torch.equal(got, want)
        assert all(torch.equal(gwant[k], ggot[k]) for k in ("dx", "dweight", "dbias"))
    state = torch.zeros(2, 3, 128, dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty(2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, o in enumerate(outs):
            S.conv_step(t["x"][:, i], t["w"], t["b"], state=state, out=o)
    state.zero_()
    g.replay()
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[:, i])


def test_offsets_past_32_bits():
    """More than 2^31 elements in x and y: the last steps are where they belong."""
    B, D = 2, 2048
    L = (2 ** 31 // D) // B + 40  # the second row ends past 2^31 elements
    x = torch.zeros(B, L, D, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(D, 4, device="cuda")
    tail = torch.randn(20, D, device="cuda").to(torch.bfloat16)
    x[1, -20:] = tail
    y, final = S.conv_fwd(x, w, None, want_final=True)
    short = torch.cat([torch.zeros(1, 3, D, dtype=torch.bfloat16, device="cuda"), tail[None]], 1)
    want = S.conv_fwd(short, w, None)
    assert torch.equal(y[1, -20:], want[0, 3:]) and torch.equal(final[1], tail[-3:])
    assert (y[0, -20:] == 0).all() and (y[1, :100] == 0).all()
    del y
    g = S.conv_bwd(x, w, None, dy=x)
    gs = S.conv_bwd(short, w, None, dy=short)
    assert torch.equal(g["dx"][1, -20:], gs["dx"][0, 3:])
    assert torch.allclose(g["dweight"], gs["dweight"], rtol=1e-5, atol=1e-5)


def test_refusals():
    t = make("f32", 2, 10, 16, 4)
    x, w, b = t["x"], t["w"], t["b"]
    for call, error in [
        (lambda: S.conv_fwd(x.half(), w, b), TypeError),
        (lambda: S.conv_fwd(x.cpu(), w, b), ValueError),
        (lambda: S.conv_fwd(x[0], w, b), ValueError),
        (lambda: S.conv_fwd(x, w.double(), b), TypeError),
        (lambda: S.conv_fwd(x, w[:8], b), ValueError),
        (lambda: S.conv_fwd(x, w, b[:8]), ValueError),
        (lambda: S.conv_fwd(x.transpose(1, 2), w, b), ValueError),
        (lambda: S.conv_fwd(x, w, b, torch.tensor([1, 2], device="cuda")), TypeError),
        (lambda: S.conv_fwd(x, w, b, state0=x[:, :2]), ValueError),
        (lambda: S.conv_fwd(x, w, b, out=x.transpose(0, 1)), ValueError),
        (lambda: S.conv_bwd(x, w, b, dy=x[:, :5]), ValueError),
        (lambda: S.conv_bwd(x, w, b, dy=x, workspace=torch.empty(4, device="cuda")), ValueError),
        (lambda: S.conv_step(x, w, b, state=x[:, :3].contiguous()), ValueError),
        (lambda: S.conv_step(x[:, 0], w, b, state=x[:, :2].contiguous()), ValueError),
    ]:
        with pytest.raises(error):
            call()
    for call, status in [
        (lambda: S.conv_fwd(x, torch.zeros(16, 5, device="cuda"), b), S.Status.ERR_UNSUPPORTED),
        (lambda: S.conv_fwd(x[:, :0], w, b), S.Status.ERR_SHAPE),
        (lambda: S.conv_bwd(x, w, b, dy=x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
         S.Status.ERR_SHAPE),
    ]:
        with pytest.raises(S.SsmError) as e:
            call()
        assert e.value.status == status
