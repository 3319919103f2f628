"""The embedding lookup and the gradient of its weight against their definitions in
64 bits.

Bounds.  The lookup multiplies once and rounds once: u = 2^-24 of the value, and
half a step of the output's type.  The gradient adds n rows in fp32: each of
n - 1 additions is off by at most u times the sum of the absolute values, the
product with the scale (and the sum with what is there) by u each, and the result
is rounded to its type."""
import math

import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def make(T, V, D, dtype=BF16, io=None, ids="zipf", ignored=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    if ids == "zipf":
        i = (torch.exp(torch.rand(T, **kw) * math.log(V + 1)).long() - 1).clamp(0, V - 1)
    elif ids == "one":
        i = torch.full((T,), V // 2, device="cuda")
    elif ids == "last":
        i = torch.where(torch.rand(T, **kw) < 0.5, V - 1, 0)
    else:
        i = torch.randint(0, V, (T,), **kw)
    if ignored:
        i[torch.rand(T, **kw) < ignored] = IGNORE
    return {"ids": i, "w": torch.randn(V, D, **kw).to(dtype), "dy": torch.randn(T, D, **kw).to(io or dtype),
            "dw": torch.randn(V, D, **kw).to(dtype)}


def half(t):
    return torch.finfo(t.dtype).eps / 2


def check_lookup(t, y, scale, ignore=IGNORE):
    kept = (t["ids"] != ignore) & (t["ids"] >= 0) & (t["ids"] < t["w"].shape[0])
    want = t["w"].double()[t["ids"][kept]] * scale
    bound = U * want.abs() + half(y) * want.abs() * (1 + U)
    assert ((y[kept].double() - want).abs() <= bound).all()
    assert (y[t["ids"] == ignore] == 0).all()


def check_gradient(t, dw, scale, add=None, ignore=IGNORE):
    V = t["w"].shape[0]
    kept = (t["ids"] != ignore) & (t["ids"] >= 0) & (t["ids"] < V)
    ids, dy = t["ids"][kept], t["dy"][kept].double()
    zero = torch.zeros(V, dy.shape[1], dtype=torch.float64, device="cuda")
    want = zero.index_add(0, ids, dy) * scale
    size = zero.index_add(0, ids, dy.abs()) * abs(scale)
    count = torch.bincount(ids, minlength=V)[:, None]
    if add is not None:
        want, size = want + add.double(), size + add.double().abs()
    bound = (count + 1) * U * size
    bound = bound + half(dw) * (want.abs() + bound)
    off = (dw.double() - want).abs() - bound
    assert (off <= 0).all(), f"{off.max().item():.3e} over the bound at {int(off.argmax())}"
    gone = count[:, 0] == 0
    assert torch.equal(dw[gone], torch.zeros_like(dw[gone]) if add is None else add[gone])


TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
CASES = [
    # tokens, vocab, dim, ids, ignored
    (1, 1, 1, "zipf", 0.0),
    (1, 70000, 64, "any", 0.0),
    (2, 3, 7, "one", 0.0),
    (5, 600, 8, "zipf", 0.5),
    (33, 511, 130, "zipf", 0.2),     # one digit
    (64, 512, 64, "any", 0.0),       # two
    (257, 1000, 513, "zipf", 0.3),
    (1000, 50257, 768, "zipf", 0.1),
    (1023, 65536, 200, "last", 0.0),
    (1025, 300, 1537, "one", 0.0),   # one run over all windows
    (8193, 5000, 96, "zipf", 0.0),
    (5000, 300000, 64, "any", 0.1),  # three digits
    (70001, 2000, 64, "zipf", 0.1),  # more keys per CTA than a tile of the sort holds
    (40000, 3000, 2048, "zipf", 0.0),
    (66000, 700, 72, "one", 0.0),
    (300, 50, 6000, "zipf", 0.0),
    (8191, 300, 64, "zipf", 0.1),    # up to 8192 tokens are placed by counting
    (8192, 300, 72, "one", 0.0),
    (8193, 511, 64, "any", 0.1),     # sorted by one digit, two, three
    (9000, 512, 40, "zipf", 0.1),
    (9000, 300000, 24, "any", 0.1),
    (16385, 262144, 8, "any", 0.0),
    (131073, 3, 8, "zipf", 0.5),
]


@pytest.mark.parametrize("dtype,io", TYPES, ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("T,V,D,ids,ignored", CASES)
def test_values_and_gradients(T, V, D, ids, ignored, dtype, io):
    t = make(T, V, D, dtype, io, ids, ignored, seed=T + D)
    for scale in (1.0, D ** 0.5):
        check_lookup(t, S.embed_fwd(t["ids"], t["w"], scale=scale, dtype=io), scale)
    dw = S.embed_bwd(t["ids"], t["dy"], vocab=V, scale=scale, dtype=dtype)
    assert dw.dtype is dtype
    check_gradient(t, dw, scale)
    there = t["dw"].clone()
    assert S.embed_bwd(t["ids"], t["dy"], scale=scale, add_to=there) is there
    check_gradient(t, there, scale, add=t["dw"])


@pytest.mark.parametrize("T", [1, 100, 9000])
def test_nothing_kept(T):
    """All tokens ignored: rows of zeros, a gradient of zeros, and nothing added."""
    t = make(T, 50, 64)
    t["ids"][:] = IGNORE
    t["dy"][:] = float("nan")
    assert (S.embed_fwd(t["ids"], t["w"]) == 0).all()
    assert (S.embed_bwd(t["ids"], t["dy"], vocab=50) == 0).all()
    there = t["dw"].clone()
    S.embed_bwd(t["ids"], t["dy"], add_to=there)
    assert torch.equal(there, t["dw"])


@pytest.mark.parametrize("D", [64, 33])
def test_ids_outside_the_vocabulary(D):
    """NaN rows that are noticed; no part in the gradient; neighbours as without them."""
    t = make(200, 300, D, seed=3)
    bad = torch.tensor([300, -1, 2 ** 31, 2 ** 32 + 5, -2 ** 40, 2 ** 62], device="cuda")
    u = dict(t, ids=t["ids"].clone(), dy=t["dy"].clone())
    at = torch.arange(7, 7 + 6 * 9, 9, device="cuda")
    u["ids"][at] = bad
    u["dy"][at] = float("nan")
    y = S.embed_fwd(u["ids"], u["w"])
    rest = torch.ones(200, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert y[at].isnan().all() and torch.equal(y[rest], S.embed_fwd(t["ids"], t["w"])[rest])
    check_gradient(u, S.embed_bwd(u["ids"], u["dy"], vocab=300), 1.0)


def test_another_ignore_index():
    t = make(500, 40, 64, ids="any")
    y = S.embed_fwd(t["ids"], t["w"], ignore_index=7)
    check_lookup(t, y, 1.0, ignore=7)
    dw = S.embed_bwd(t["ids"], t["dy"], vocab=40, ignore_index=7)
    check_gradient(t, dw, 1.0, ignore=7)
    assert (dw[7] == 0).all()


@pytest.mark.parametrize("dtype,io", TYPES, ids=["f32", "bf16", "mixed"])
def test_tensors_off_a_boundary(dtype, io):
    """Tensors that start one element into a buffer, whose neighbours stay."""
    t = make(300, 90, 64, dtype, io, seed=6)

    def shifted(v, fill=7.0):
        buf = torch.full((v.numel() + 40,), fill, dtype=v.dtype, device="cuda")
        return buf, buf[1:1 + v.numel()].view(v.shape).copy_(v)

    _, w = shifted(t["w"])
    _, dy = shifted(t["dy"])
    buf, out = shifted(t["dy"])
    y = S.embed_fwd(t["ids"], w, dtype=io, out=out)
    assert y is out and torch.equal(y, S.embed_fwd(t["ids"], t["w"], dtype=io))
    assert buf[0] == 7 and (buf[1 + y.numel():] == 7).all()
    want = S.embed_bwd(t["ids"], t["dy"], add_to=t["dw"].clone())
    buf, there = shifted(t["dw"])
    assert torch.equal(S.embed_bwd(t["ids"], dy, add_to=there), want)
    assert buf[0] == 7 and (buf[1 + there.numel():] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,D", [(1, 1), (3, 5), (9, 17), (1000, 33)])
def test_gradients_of_odd_sizes_are_written_as_a_whole(dtype, V, D):
    """Every byte of a gradient at any offset, and no byte around it."""
    lib = S.load()
    import ctypes
    from selective_state_space_fwd_gb300._binding import EmbedShapes
    t = make(40, V, D, dtype, seed=D)
    code = 1 if dtype is BF16 else 0
    s = EmbedShapes(40, V, D, IGNORE, 1.0, code, code)
    ws = torch.empty(lib.ssm_embed_bwd_workspace_bytes(ctypes.byref(s)), dtype=torch.uint8, device="cuda")
    want = S.embed_bwd(t["ids"], t["dy"], vocab=V)
    for shift in range(9):
        buf = torch.full((V * D + 40,), 7.0, dtype=dtype, device="cuda")
        out = buf[shift:shift + V * D]
        st = lib.ssm_embed_bwd(t["ids"].data_ptr(), t["dy"].data_ptr(), out.data_ptr(), 0, ws.data_ptr(), ws.numel(),
                               ctypes.byref(s), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(out.view(V, D), want)
        assert (buf[:shift] == 7).all() and (buf[shift + V * D:] == 7).all()


def test_the_same_every_time_and_with_dirty_workspaces():
    t = make(20000, 900, 256, ignored=0.2, seed=8)
    a = S.embed_bwd(t["ids"], t["dy"], vocab=900)
    for fill in (0, 255):  # 255: NaN in every type
        ws = torch.full((1 << 27,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(S.embed_bwd(t["ids"], t["dy"], vocab=900, workspace=ws), a)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, interleaved."""
    ts = [make(20000, 3000, 256, seed=s) for s in (1, 2)]
    want = [S.embed_bwd(t["ids"], t["dy"], vocab=3000) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (t, s) in enumerate(zip(ts, streams)):
            with torch.cuda.stream(s):
                got[i].append(S.embed_bwd(t["ids"], t["dy"], vocab=3000))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])


def test_shapes_of_ids():
    t = make(60, 90, 64)
    ids = t["ids"].view(3, 20)
    y = S.embed_fwd(ids, t["w"])
    assert y.shape == (3, 20, 64) and torch.equal(y.view(60, 64), S.embed_fwd(t["ids"], t["w"]))
    assert torch.equal(S.embed_bwd(ids, t["dy"].view(3, 20, 64), vocab=90), S.embed_bwd(t["ids"], t["dy"], vocab=90))
    one = S.embed_fwd(t["ids"][0], t["w"])
    assert one.shape == (64,) and torch.equal(one, y[0, 0])
    assert S.embed_bwd(t["ids"][0], t["dy"][0], vocab=90).shape == (90, 64)


def test_another_stream_and_a_graph():
    t = make(700, 4000, 128, ignored=0.2)
    want = S.embed_bwd(t["ids"], t["dy"], vocab=4000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = S.embed_fwd(t["ids"], t["w"], stream=side)
    dw = S.embed_bwd(t["ids"], t["dy"], vocab=4000, stream=side)
    side.synchronize()
    assert torch.equal(dw, want) and torch.equal(y, S.embed_fwd(t["ids"], t["w"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = S.embed_fwd(t["ids"], t["w"])
        dw = S.embed_bwd(t["ids"], t["dy"], vocab=4000)
    t["ids"].copy_(t["ids"].roll(1))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, S.embed_fwd(t["ids"], t["w"])) and torch.equal(dw, S.embed_bwd(t["ids"], t["dy"], vocab=4000))


@pytest.mark.parametrize("dtype,io", TYPES, ids=["f32", "bf16", "mixed"])
def test_autograd(dtype, io):
    t = make(60, 90, 64, dtype, io, ignored=0.2)
    w = t["w"].clone().requires_grad_(True)
    y = S.embedding(t["ids"].view(3, 20), w, scale=8.0, dtype=io)
    assert torch.equal(y.view(60, 64), S.embed_fwd(t["ids"], t["w"], scale=8.0, dtype=io))
    (y * t["dy"].view(3, 20, 64)).sum().backward()
    assert w.grad.dtype is dtype
    wide = torch.stack([t["ids"], t["ids"]], 1)[:, 0]  # strided
    assert torch.equal(S.embedding(wide, w), S.embed_fwd(t["ids"], t["w"]))
    assert torch.equal(w.grad, S.embed_bwd(t["ids"], t["dy"], vocab=90, scale=8.0, dtype=dtype))
    (g,) = torch.autograd.grad((S.embedding(t["ids"], w) ** 2).sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        g.sum().backward()


def test_gradients_match_differences():
    """The lookup is linear in the weight: the difference of two calls along a
    direction is the gradient's product with it, up to the rounding of both."""
    t = make(50, 20, 16, F32, seed=5)
    move = torch.randn_like(t["w"])
    dw = S.embed_bwd(t["ids"], t["dy"], vocab=20, scale=3.0)
    moved = S.embed_fwd(t["ids"], t["w"] + move, scale=3.0).double() - S.embed_fwd(t["ids"], t["w"], scale=3.0).double()
    left, right = (moved * t["dy"].double()).sum(), (dw.double() * move.double()).sum()
    size = 3 * (t["dy"].double().abs() * (t["w"].abs() + move.abs()).double()[t["ids"]]).sum()
    assert (left - right).abs() <= 60 * U * size


def test_elements_past_32_bits():
    """More than 2^31 elements in the weight and its gradient, and in the rows."""
    D = 2048
    V = 2 ** 31 // D + 300
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.zeros(V, D, dtype=BF16, device="cuda")
    w[-300:] = torch.randn(300, D, generator=g, device="cuda").to(BF16)
    ids = torch.randint(V - 300, V, (1000,), generator=g, device="cuda")
    assert torch.equal(S.embed_fwd(ids, w), w[ids])
    dy = torch.randn(1000, D, generator=g, device="cuda").to(BF16)
    dw = S.embed_bwd(ids, dy, vocab=V)
    small = S.embed_bwd(ids - (V - 300), dy, vocab=300)
    assert torch.equal(dw[-300:], small) and (dw[:-300] == 0).all()
    T = V
    ids = torch.randint(0, 300, (T,), generator=g, device="cuda")
    y = S.embed_fwd(ids, w[-300:].contiguous())
    assert torch.equal(y[-1000:], w[-300:][ids[-1000:]])
    dy = torch.zeros(T, D, dtype=BF16, device="cuda")
    dy[-1000:] = y[-1000:]
    dw = S.embed_bwd(ids, dy, vocab=300)
    # the sums' partial results are zeros but for the last rows'
    check_gradient({"ids": ids[-1000:], "w": w[-300:], "dy": y[-1000:]}, dw, 1.0)


def test_refusals():
    t = make(10, 50, 64)
    ids, w, dy = t["ids"], t["w"], t["dy"]
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for call, error in [
        (lambda: S.embed_fwd(ids.cpu(), w), ValueError),
        (lambda: S.embed_fwd(ids, w.cpu()), ValueError),
        (lambda: S.embed_fwd(ids.int(), w), TypeError),
        (lambda: S.embed_fwd(ids, w.half()), TypeError),
        (lambda: S.embed_fwd(ids, w, dtype=torch.float16), TypeError),
        (lambda: S.embed_fwd(ids, w[:, ::2]), ValueError),
        (lambda: S.embed_fwd(ids[::2], w), ValueError),
        (lambda: S.embed_fwd(ids, w[0]), ValueError),
        (lambda: S.embed_fwd(ids, w, out=torch.empty_like(dy)[:5]), ValueError),
        (lambda: S.embed_bwd(ids, dy), ValueError),
        (lambda: S.embed_bwd(ids, dy[:5], vocab=50), ValueError),
        (lambda: S.embed_bwd(ids, dy.half(), vocab=50), TypeError),
        (lambda: S.embed_bwd(ids, dy, vocab=49, add_to=t["dw"]), ValueError),
        (lambda: S.embed_bwd(ids, dy, dtype=F32, add_to=t["dw"]), TypeError),
        (lambda: S.embed_bwd(ids, dy, add_to=t["dw"][:, :32]), ValueError),
    ]:
        with pytest.raises(error):
            call()
    for call, status in [
        (lambda: S.embed_fwd(ids[:0], w), S.Status.ERR_SHAPE),
        (lambda: S.embed_fwd(ids, w[:0]), S.Status.ERR_SHAPE),
        (lambda: S.embed_fwd(ids, w, scale=float("inf")), S.Status.ERR_SHAPE),
        (lambda: S.embed_fwd(ids, w.float(), dtype=BF16), S.Status.ERR_UNSUPPORTED),
        (lambda: S.embed_bwd(ids, dy, vocab=50, dtype=F32), S.Status.ERR_UNSUPPORTED),
        (lambda: S.embed_bwd(ids, dy, vocab=0), S.Status.ERR_SHAPE),
        (lambda: S.embed_bwd(ids, dy, vocab=50, workspace=small), S.Status.ERR_SHAPE),
    ]:
        with pytest.raises(S.SsmError) as e:
            call()
        assert e.value.status == status
