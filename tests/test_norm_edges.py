"""The norm of the residual stream where rows meet: what one row holds must not
reach its neighbours, whatever the groups of columns in which rows are read."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S
from test_norm import make
from test_norm import test_forward_and_backward_match_the_formulas as formulas

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


@pytest.mark.parametrize("rows", [5, 900])
@pytest.mark.parametrize("dim", [1300, 1700, 2561, 3000, 4089, 4096])
@pytest.mark.parametrize("dtype,residual", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_wide_rows_match_the_formulas(dtype, residual, dim, rows):
    """Row lengths that take the backward's CTAs of 161 to 512 threads with 8 columns
    each."""
    formulas(dtype, rows, dim, residual, rms=dim % 2 == 1, bias=True)


@pytest.mark.parametrize("dtype,residual", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("dim", [1, 3, 97, 1001, 1537, 4089, 8189])
def test_in_place_stream_off_a_boundary(dtype, residual, dim):
    """The stream updated in place where groups of columns reach into the rows before
    and after, which other threads are writing."""
    rows = 3001 if dim < 2000 else 1200
    t = make(dtype, rows, dim, residual)
    y, r, stats = S.norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], want_stats=True)
    for _ in range(5):
        res = t["res"].clone()
        y2, r2, stats2 = S.norm_fwd(t["x"], t["w"], t["b"], residual=res, out_r=res, want_stats=True)
        assert r2.data_ptr() == res.data_ptr()
        assert torch.equal(r2, r) and torch.equal(y2, y) and torch.equal(stats2, stats)


@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("dtype,dim", [("bf16", 1000), ("bf16", 1001), ("bf16", 96), ("f32", 1500), ("f32", 1537)])
@pytest.mark.parametrize("column", [0, 50, -1])
def test_an_infinity_in_a_root_mean_square_row(dtype, dim, column, rows):
    """The mean square is infinite and its reciprocal root 0: the row's finite columns
    are 0 wherever the infinity stands, also in the last group of columns, which
    threads past the row's end hold too."""
    t = make(dtype, rows, dim, None, bias=False)
    t["x"][1, column] = float("inf")
    y, _, stats = S.norm_fwd(t["x"], t["w"], rms=True, want_stats=True)
    assert stats[1, 1] == 0
    rest = torch.ones(dim, dtype=torch.bool, device="cuda")
    rest[column] = False
    assert (y[1, rest] == 0).all() and y[1, column].isnan()
