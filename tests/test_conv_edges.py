"""The short causal convolution on x as it may lie in memory: time-major, inside
wider rows, with padding that fits no multiple, overlapping, and of single steps or
rows.  The layout must not change a value."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_conv import U, assert_close, f64, half_ulp, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield
    S.check_device_errors()


def strided(B, L, D, batch, step, dtype, seed):
    """[B, L, D] with those strides in elements, over a buffer of random values."""
    g = torch.Generator().manual_seed(seed)
    n = (B - 1) * batch + (L - 1) * step + D
    return torch.randn(n, generator=g).to(dtype).cuda().as_strided((B, L, D), (batch, step, 1))


LAYOUTS = [
    # name, B, L, D, batch stride, step stride
    ("time-major", 3, 70, 64, 64, 3 * 64),
    ("time-major, wider rows", 3, 70, 64, 96, 4 * 96),
    ("time-major, no multiple", 3, 70, 64, 96, 3 * 96 + 8),
    ("batch rows with padding of no multiple", 3, 70, 64, 70 * 64 + 8, 64),
    ("batch rows with padding of whole steps", 3, 70, 64, 75 * 96, 96),
    ("one batch row in wider rows", 1, 90, 64, 64, 104),
    ("one batch row, stride 0", 1, 90, 64, 0, 64),
    ("one step, batch rows of no multiple", 5, 1, 64, 104, 64),
    ("one step, one row", 1, 1, 64, 64, 64),
    ("overlapping windows of time", 4, 40, 64, 8 * 64, 64),
    ("overlapping windows of channels", 1, 40, 64, 64, 8),
    ("steps and rows alike", 3, 40, 64, 64, 64),
    ("one row for the batch", 3, 40, 64, 0, 64),
    ("one step for all of time", 3, 40, 64, 64, 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("name,B,L,D,batch,step", LAYOUTS, ids=[v[0] for v in LAYOUTS])
def test_layouts_of_x(name, B, L, D, batch, step, masked, dtype):
    t = make(dtype, B, L, D, 4, valid=[L - 7 * i if L > 7 * i else 1 for i in range(B)] if masked else None,
             carry=True, seed=B + L)
    t["x"] = strided(B, L, D, batch, step, t["dy"].dtype, seed=3)
    ref = reference(t, True, f64(t["dy"]))
    kw = dict(state0=t["state0"])
    y, final = S.conv_fwd(t["x"], t["w"], t["b"], t["valid"], want_final=True, **kw)
    y1, final1 = S.conv_fwd(t["x"].contiguous(), t["w"], t["b"], t["valid"], want_final=True, **kw)
    assert torch.equal(y, y1) and torch.equal(final, final1)
    assert_close(y, ref["y"], half_ulp(dtype, ref["y"]) + 2.0 ** -20 * ref["scale"], "y")
    g = S.conv_bwd(t["x"], t["w"], t["b"], t["valid"], dy=t["dy"], want_dstate0=True, **kw)
    n = min(B * L, 1024)
    for k, r in (("dx", "dx"), ("dstate0", "dstate0")):
        assert_close(g[k], ref[r], half_ulp(dtype, ref[r]) + 2.0 ** -20 * ref[r + "_scale"], k)
    for k, r in (("dweight", "dw"), ("dbias", "db")):
        assert_close(g[k], ref[r], (2.0 ** -20 + n * U) * ref[r + "_scale"], k)
    if L == 1:
        state = t["state0"].clone()
        step_y = S.conv_step(t["x"][:, 0], t["w"], t["b"], state=state)
        if not masked:
            assert torch.equal(step_y, y[:, 0]) and torch.equal(state, final)


@pytest.mark.parametrize("dtype,B,D", [("bf16", 1021, 2048), ("bf16", 1022, 2048), ("bf16", 1023, 2048),
                                       ("bf16", 1024, 2048), ("f32", 1023, 1024), ("f32", 1024, 1024),
                                       ("bf16", 700, 2048), ("f32", 513, 1000)])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_steps_of_large_batches(dtype, B, D, K):
    """Single steps whose threads hold one batch row or four, with remainders of one
    to three rows: the bits of conv_fwd from the same state."""
    t = make(dtype, B, 1, D, K, bias=K != 3, carry=True, seed=K)
    for silu in (True, False):
        want, final = S.conv_fwd(t["x"], t["w"], t["b"], state0=t["state0"], silu=silu, want_final=True)
        guard = torch.full((3, K - 1, D), 7.0, dtype=t["state0"].dtype, device="cuda")
        held = torch.cat([t["state0"], guard])
        y = S.conv_step(t["x"][:, 0], t["w"], t["b"], state=held[:B], silu=silu)
        assert torch.equal(y, want[:, 0]) and torch.equal(held[:B], final)
        assert (held[B:] == 7).all()  # nothing is written past the last row
