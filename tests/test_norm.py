"""The norm of the residual stream (forward and backward) against its formulas
in 64 bits.

Bounds.  With u = 2^-24 and m the largest |r| of a row: the mean of the row is
within d u m of the exact one for at most d additions one after another (16 per
thread, then a tree: d = 32 covers both and the roundings of the division), and
the centred values, squares and their sum follow, so xhat is within 2^-18 (m
rstd + |xhat|) of the exact one.  y scales that by |w| and adds the bias; bf16
outputs add half an ulp.  The backward's two row means are sums of |g| and
|g xhat| with the same relative error.  The weight sums add one term per row."""
import numpy as np
import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

E = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(dtype, rows, dim, residual, bias=True, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    t = {"x": (torch.randn(rows, dim, generator=g) + offset).to(DT[dtype]).cuda(),
         "w": (torch.randn(dim, generator=g) * 0.2 + 1).cuda(),
         "b": torch.randn(dim, generator=g).cuda() if bias else None,
         "dy": torch.randn(rows, dim, generator=g).to(DT[dtype]).cuda(), "res": None, "dr": None}
    if residual:
        t["res"] = (torch.randn(rows, dim, generator=g) * 2).to(DT[residual]).cuda()
        t["dr"] = torch.randn(rows, dim, generator=g).to(DT[residual]).cuda()
    return t


def f64(t):
    return t.detach().double().cpu().numpy()


def forward(r, w, b, rms, eps):
    mean = 0.0 if rms else r.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((r - mean) ** 2).mean(-1, keepdims=True) + eps)
    xhat = (r - mean) * rstd
    return xhat * w + b, xhat, rstd


def half_ulp(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 2.0 ** -23 * np.abs(ref)


def assert_close(got, want, bound, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), f"{what}: {off.max():.3e} over its bound at {np.unravel_index(off.argmax(), off.shape)}"


CASES = [
    # dtype, rows, dim, residual, rms, bias
    ("f32", 1, 1, None, True, False),
    ("f32", 3, 7, None, False, True),
    ("bf16", 5, 64, "bf16", False, True),
    ("bf16", 1, 2048, "f32", True, False),
    ("bf16", 1000, 1024, "bf16", False, True),
    ("f32", 700, 1537, None, False, False),
    ("bf16", 650, 1000, "f32", True, True),
    ("f32", 2000, 132, "f32", False, True),
    ("bf16", 900, 2047, None, False, True),
    ("f32", 9, 8192, "f32", False, True),
    ("bf16", 1300, 8191, "bf16", True, False),
    ("bf16", 1300, 8192, "f32", False, True),
    ("bf16", 40000, 33, "bf16", False, True),
    # rows that start off a 16-byte boundary
    ("bf16", 650, 1001, "f32", False, True),
    ("bf16", 7, 3, "bf16", False, True),
    ("bf16", 9, 1, "f32", True, False),
    ("f32", 21, 2, "f32", False, True),
    ("f32", 611, 8189, None, False, True),
    ("bf16", 2000, 1030, None, True, False),
    ("bf16", 333, 4500, "bf16", False, True),
]


@pytest.mark.parametrize("dtype,rows,dim,residual,rms,bias", CASES)
def test_forward_and_backward_match_the_formulas(dtype, rows, dim, residual, rms, bias):
    t = make(dtype, rows, dim, residual, bias)
    eps = 1e-5
    y, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], rms=rms, eps=eps,
                             want_stats=True)
    if residual:
        total = f64(t["x"]) + f64(t["res"])
        assert_close(r, total, half_ulp(residual, total), "r")
        assert r.dtype == t["res"].dtype
    else:
        assert r is None
        r = t["x"]
    r64, w, b = f64(r), f64(t["w"]), f64(t["b"]) if bias else 0.0
    want, xhat, rstd = forward(r64, w, b, rms, eps)
    top = np.abs(r64).max(-1, keepdims=True) * rstd
    ex = E * (top + np.abs(xhat))                          # error of xhat
    assert_close(y, want, half_ulp(dtype, want) + ex * np.abs(w) + E * np.abs(b), "y")
    assert_close(stats[1], rstd[:, 0], E * rstd[:, 0], "rstd")
    if rms:
        assert (stats[0] == 0).all()
    again = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], rms=rms, eps=eps)
    assert torch.equal(again[0], y) and again[2] is None

    g = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"], rms=rms, want_dbias=bias)
    dy, dr = f64(t["dy"]), f64(t["dr"]) if residual else 0.0
    gw = dy * w
    mg = 0.0 if rms else gw.mean(-1, keepdims=True)
    mx = (gw * xhat).mean(-1, keepdims=True)
    dx = rstd * (gw - mg - xhat * mx) + dr
    size = rstd * (np.abs(gw) + np.abs(gw).mean(-1, keepdims=True)
                   + (np.abs(xhat) + top) * (np.abs(gw) * (np.abs(xhat) + top)).mean(-1, keepdims=True))
    bound = 4 * E * (size + np.abs(dr))
    assert_close(g["dx"], dx, half_ulp(dtype, dx) + bound, "dx")
    if residual:
        assert_close(g["dresidual"], dx, half_ulp(residual, dx) + bound, "dresidual")
        assert g["dresidual"].dtype == t["res"].dtype
    n = min(rows, 1024) * 2.0 ** -24
    assert_close(g["dweight"], (dy * xhat).sum(0),
                 (np.abs(dy) * (ex + n * np.abs(xhat))).sum(0), "dweight")
    if bias:
        assert_close(g["dbias"], dy.sum(0), n * np.abs(dy).sum(0), "dbias")
    else:
        assert g["dbias"] is None


@pytest.mark.parametrize("dim", [96, 97])
def test_tensors_off_a_boundary(dim):
    """Contiguous tensors that start off a 16-byte boundary give what aligned
    copies of them give, up to the order of the sums."""
    t = make("bf16", 40, dim, "bf16")

    def moved(v):
        buf = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
        buf[1:] = v.reshape(-1)
        return buf[1:].view(v.shape)

    y, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True)
    y2, r2, stats2 = S.norm_fwd(moved(t["x"]), moved(t["w"]), moved(t["b"]),
                                residual=moved(t["res"]), want_stats=True)
    assert torch.equal(r, r2)
    assert torch.allclose(y.float(), y2.float(), rtol=2 ** -7, atol=2 ** -14)
    g = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"], want_dbias=True)
    g2 = S.norm_bwd(moved(r), moved(t["w"]), stats=stats, dy=moved(t["dy"]), dr=moved(t["dr"]),
                    want_dbias=True)
    assert torch.allclose(g["dx"].float(), g2["dx"].float(), rtol=2 ** -7, atol=2 ** -12)
    for k in ("dweight", "dbias"):
        assert torch.allclose(g[k], g2[k], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_match_central_differences(rms):
    """The kernel's gradients against differences of the 64-bit forward (step
    2^-12: truncation of order 2^-24 times the third derivative)."""
    t = make("f32", 3, 10, "f32", True, seed=4)
    eps = 1e-5
    _, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], rms=rms, eps=eps,
                             want_stats=True)
    g = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"], rms=rms, want_dbias=True)
    dy, dr, h = f64(t["dy"]), f64(t["dr"]), 2.0 ** -12
    base = {"r": f64(r), "w": f64(t["w"]), "b": f64(t["b"])}

    def objective(v):
        return (forward(v["r"], v["w"], v["b"], rms, eps)[0] * dy).sum() + (v["r"] * dr).sum()

    for name, grad in (("r", "dx"), ("w", "dweight"), ("b", "dbias")):
        diff = np.empty(base[name].shape)
        for at in np.ndindex(*diff.shape):
            side = []
            for sign in (1, -1):
                moved = base[name].copy()
                moved[at] += sign * h
                side.append(objective({**base, name: moved}))
            diff[at] = (side[0] - side[1]) / (2 * h)
        assert np.abs(f64(g[grad]) - diff).max() <= 2e-5 * max(1.0, np.abs(diff).max()), name


def test_constant_rows_and_large_means():
    """A constant row has no variance: xhat is 0 and the result the bias.  A mean
    a thousand times the spread is subtracted before anything is squared."""
    dim = 512
    x = torch.full((2, dim), 3.25, device="cuda")
    w, b = torch.ones(dim, device="cuda"), torch.linspace(-1, 1, dim, device="cuda")
    y, _, stats = S.norm_fwd(x, w, b, want_stats=True)
    assert torch.equal(y, b.expand(2, dim)) and (stats[0] == 3.25).all()
    t = make("f32", 64, dim, None, offset=1000.0)
    y, _, _ = S.norm_fwd(t["x"], t["w"], t["b"])
    want, xhat, rstd = forward(f64(t["x"]), f64(t["w"]), f64(t["b"]), False, 1e-5)
    bound = E * (np.abs(f64(t["x"])).max(-1, keepdims=True) * rstd + np.abs(xhat)) * np.abs(f64(t["w"]))
    assert_close(y, want, bound + 2.0 ** -22 * (1 + np.abs(want)), "y")


def test_rows_do_not_touch_each_other():
    """NaN and infinities in one row stay in it; row groups at the end of the
    grid that hold no row change nothing."""
    for rows, dim in ((5, 96), (700, 1024), (3, 8192)):
        t = make("bf16", rows, dim, "bf16")
        y, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True)
        g = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"])
        x = t["x"].clone()
        x[1, 3], x[2, 5] = float("nan"), float("inf")
        y2, r2, s2 = S.norm_fwd(x, t["w"], t["b"], residual=t["res"], want_stats=True)
        g2 = S.norm_bwd(r2, t["w"], stats=s2, dy=t["dy"], dr=t["dr"])
        keep = torch.ones(rows, dtype=torch.bool)
        keep[1] = keep[2] = False
        assert torch.equal(y[keep], y2[keep]) and torch.equal(g["dx"][keep], g2["dx"][keep])
        assert y2[1].isnan().all() and y2[2].isnan().any()


def test_in_place_stream_and_determinism():
    t = make("bf16", 333, 768, "f32")
    y, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True)
    res = t["res"].clone()
    y2, r2, _ = S.norm_fwd(t["x"], t["w"], t["b"], residual=res, out_r=res)
    assert r2.data_ptr() == res.data_ptr() and torch.equal(r2, r) and torch.equal(y2, y)
    a = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"], want_dbias=True)
    for _ in range(3):
        b = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"], want_dbias=True)
        assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype,residual", [("bf16", "f32"), ("bf16", "bf16"), ("f32", None)])
def test_autograd(dtype, residual):
    """layer_norm under autograd returns the library's backward, with and
    without a gradient along the stream; leading dimensions are kept."""
    t = make(dtype, 12, 40, residual)
    shape = (3, 4, 40)
    leaf = {k: t[k].reshape(shape if t[k].dim() == 2 else -1).clone().requires_grad_(True)
            for k in ("x", "w", "b", "res") if t[k] is not None}
    for along in ((False, True) if residual else (False,)):
        for v in leaf.values():
            v.grad = None
        out = S.layer_norm(leaf["x"], leaf["w"], leaf["b"], residual=leaf.get("res"))
        y, r = out if residual else (out, None)
        assert y.shape == shape
        total = (y * t["dy"].view(shape)).sum()
        if along:
            total = total + (r * t["dr"].view(shape)).sum()
        total.backward()
        _, r1, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True)
        g = S.norm_bwd(t["x"] if r1 is None else r1, t["w"], stats=stats, dy=t["dy"],
                       dr=t["dr"] if along else None, want_dbias=True)
        assert torch.equal(leaf["x"].grad.view(12, 40), g["dx"])
        assert torch.equal(leaf["w"].grad, g["dweight"]) and torch.equal(leaf["b"].grad, g["dbias"])
        if residual:
            assert torch.equal(leaf["res"].grad.view(12, 40), g["dresidual"])
    if residual:  # only the stream is used: no gradient arrives at y
        for v in leaf.values():
            v.grad = None
        S.layer_norm(leaf["x"], leaf["w"], leaf["b"], residual=leaf["res"])[1].float().sum().backward()
        assert (leaf["res"].grad == 1).all() and (leaf["x"].grad == 1).all()
        assert (leaf["w"].grad == 0).all()


def test_another_stream_and_a_graph():
    t = make("bf16", 64, 512, "bf16")
    y, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True)
    g = S.norm_bwd(r, t["w"], stats=stats, dy=t["dy"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, r2, s2 = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True, stream=side)
    g2 = S.norm_bwd(r2, t["w"], stats=s2, dy=t["dy"], stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(g["dx"], g2["dx"])
    assert torch.equal(g["dweight"], g2["dweight"])
    out, out_r = torch.empty_like(y), torch.empty_like(r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], out=out, out_r=out_r)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y) and torch.equal(out_r, r)


def test_offsets_past_32_bits():
    dim = 2048
    rows = 2 ** 31 // dim + 5
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(7, dim, device="cuda").to(torch.bfloat16)
    x[-7:] = tail
    w = torch.rand(dim, device="cuda")
    y, _, stats = S.norm_fwd(x, w, want_stats=True)
    y7, _, s7 = S.norm_fwd(tail, w, want_stats=True)
    # the short call holds a row in twice the threads: equal up to the sums' order
    assert (y[:-7] == 0).all()
    assert torch.allclose(y[-7:].float(), y7.float(), rtol=2 ** -7, atol=1e-6)
    del y
    g = S.norm_bwd(x, w, stats=stats, dy=x)
    g7 = S.norm_bwd(tail, w, stats=s7, dy=tail)
    assert torch.allclose(g["dx"][-7:].float(), g7["dx"].float(), rtol=2 ** -7, atol=1e-2)
    assert torch.allclose(g["dweight"], g7["dweight"], rtol=1e-5, atol=1e-4)


def test_refusals():
    t = make("bf16", 4, 32, "bf16")
    x, w, b, res = t["x"], t["w"], t["b"], t["res"]
    _, r, stats = S.norm_fwd(x, w, b, residual=res, want_stats=True)
    for call, error in [
        (lambda: S.norm_fwd(x.half(), w, b), TypeError),
        (lambda: S.norm_fwd(x.cpu(), w, b), ValueError),
        (lambda: S.norm_fwd(x.T, w, b), ValueError),
        (lambda: S.norm_fwd(x, w.to(torch.bfloat16), b), TypeError),
        (lambda: S.norm_fwd(x, w[:16], b), ValueError),
        (lambda: S.norm_fwd(x, w, b, residual=res[:2]), ValueError),
        (lambda: S.norm_fwd(x, w, b, residual=res.half()), TypeError),
        (lambda: S.norm_fwd(x, w, b, out_r=res), ValueError),
        (lambda: S.norm_bwd(r, w, stats=stats[0], dy=t["dy"]), ValueError),
        (lambda: S.norm_bwd(r, w, stats=stats, dy=t["dy"][:2]), ValueError),
        (lambda: S.norm_bwd(r, w, stats=stats, dy=t["dy"], dr=t["dr"].float()), TypeError),
    ]:
        with pytest.raises(error):
            call()
    big = torch.zeros(2, 8200, device="cuda")
    for call, status in [
        (lambda: S.norm_fwd(big, torch.ones(8200, device="cuda")), S.Status.ERR_UNSUPPORTED),
        (lambda: S.norm_fwd(x[:0], w, b), S.Status.ERR_SHAPE),
        (lambda: S.norm_fwd(x, w, b, eps=-1.0), S.Status.ERR_SHAPE),
        (lambda: S.norm_fwd(x, w, b, eps=float("nan")), S.Status.ERR_SHAPE),
        (lambda: S.norm_fwd(x.float(), w, b, residual=res), S.Status.ERR_UNSUPPORTED),
        (lambda: S.norm_bwd(r, w, stats=stats, dy=t["dy"],
                            workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
         S.Status.ERR_SHAPE),
    ]:
        with pytest.raises(S.SsmError) as e:
            call()
        assert e.value.status == status
