"""The gated linear recurrence where clusters of CTAs share the time: strided inputs, and numbers
of channel groups around what the GPU holds.  Bounds: those of test_recur.py."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_recur import DTYPES, NAMES, assert_close, make, reference, run, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


LAYOUTS = [
    # name, B, L, D, stride of the batch rows, of the steps
    ("time-major", 2, 1100, 64, 64, 2 * 64),
    ("wider rows", 2, 1100, 64, 1100 * 96, 96),
    ("wider rows, odd", 2, 1100, 64, 1100 * 67, 67),
    ("one row for the batch", 3, 1100, 64, 0, 64),
    ("one step for all of time", 1, 3000, 32, 32, 0),
    ("overlapping steps", 1, 3000, 32, 32, 2),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name,B,L,D,batch,step", LAYOUTS, ids=[v[0] for v in LAYOUTS])
@pytest.mark.parametrize("which", ["gate", "value"])
def test_layouts(name, B, L, D, batch, step, which, dtype):
    t = make(dtype, B, L, D, carry=True, floor=True, valid=[L, L - 77, 1][:B], seed=2)
    t[which] = strided(B, L, D, batch, step, DTYPES[dtype], seed=4)
    got, ref = run(t), reference(dict(t, **{which: t[which].contiguous()}))
    for k in NAMES + ("dfloor",):
        assert_close(got[k], ref, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 225), (1, 257), (1, 513), (1, 601), (3, 515), (1, 1025), (2, 2001), (1, 448), (1, 480), (1, 1216)])
def test_channel_groups_around_what_the_gpu_holds(dtype, B, D):
    t = make(dtype, B, 1300, D, carry=True, floor=True, seed=D)
    got, ref = run(t), reference(t)
    for k in NAMES + ("dfloor",):
        assert_close(got[k], ref, k)
