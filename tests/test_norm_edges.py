"""The norm of the residual stream where rows meet: what one row holds must not
reach its neighbours, whatever the groups of columns in which rows are read."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_norm import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


# Row lengths off a 16-byte boundary: groups of 4 (fp32) or 8 (bf16) columns then
# reach over the ends of rows.  8189 and 8191 are the widest; with 1, 2 and 3
# columns one group holds several rows.
DIMS = [("bf16", 97), ("bf16", 1001), ("bf16", 3), ("bf16", 1), ("bf16", 8189), ("bf16", 1030),
        ("f32", 97), ("f32", 1537), ("f32", 3), ("f32", 2), ("f32", 1), ("f32", 8191)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("stream", ["none", "same", "f32"])
@pytest.mark.parametrize("dtype,dim", DIMS)
def test_a_row_of_nan_or_infinities_stays_apart(dtype, dim, stream, rms):
    """NaN, infinities and the type's lowest value in the first and last columns of
    a row change no bit of any other row: not of y, r, the statistics or dx."""
    if stream == "f32" and dtype == "f32":
        pytest.skip("the same as a stream of x's type")
    residual = {"none": None, "same": dtype, "f32": "f32"}[stream]
    vec = 16 // (2 if dtype == "bf16" else 4)
    ends = sorted({c for c in [*range(vec), *range(dim - vec, dim)] if 0 <= c < dim})
    for rows in (41, 700):  # few rows, and more than four per SM
        t = make(dtype, rows, dim, residual)
        kw = dict(residual=t["res"], rms=rms, want_stats=True)

        def run(x):
            y, r, stats = S.norm_fwd(x, t["w"], t["b"], **kw)
            g = S.norm_bwd(x if r is None else r, t["w"], stats=stats, dy=t["dy"], dr=t["dr"], rms=rms)
            return {"y": y, "r": r, "stats": stats.T, "dx": g["dx"], "dresidual": g["dresidual"]}

        want = run(t["x"])
        low = torch.finfo(t["x"].dtype).min
        for n, bad in enumerate((float("nan"), float("inf"), -float("inf"), low)):
            x = t["x"].clone()
            hit = torch.tensor([0, 11 + n, 12 + 9 * n, rows - 1], device="cuda")
            for c in ends:
                x[hit, c] = bad
            got = run(x)
            keep = torch.ones(rows, dtype=torch.bool, device="cuda")
            keep[hit] = False
            for k, v in want.items():
                if v is not None:
                    assert torch.equal(got[k][keep], v[keep]), (k, rows, bad)
