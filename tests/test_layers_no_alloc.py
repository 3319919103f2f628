"""The operators around the scan allocate nothing: with outputs and workspaces of the
caller's, calls through the C ABI leave the device's free memory as it was."""
import ctypes

import pytest
import torch

import selective_state_space_fwd_gb300 as S
from selective_state_space_fwd_gb300._binding import ConvShapes, NormShapes, XentShapes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def new(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype)


def conv_calls(lib, dim, code, dtype):
    B, L, K = 4, 300, 4
    x, y, dy, dx = (new(B, L, dim, dtype=dtype) for _ in range(4))
    w, b, dw, db = new(dim, K), new(dim), new(dim, K), new(dim)
    state, final = new(B, K - 1, dim, dtype=dtype), new(B, K - 1, dim, dtype=dtype)
    s = ConvShapes(B, L, dim, K, L * dim, dim, 1)
    one = ConvShapes(B, 1, dim, K, L * dim, dim, 1)
    ws = torch.empty(lib.ssm_conv_bwd_workspace_bytes(ctypes.byref(s)), dtype=torch.uint8, device="cuda")
    p = [v.data_ptr() for v in (x, w, b, state, y, final, dy, dx, dw, db, ws)]
    x_, w_, b_, st_, y_, f_, dy_, dx_, dw_, db_, ws_ = p

    def run(stream):
        return [lib.ssm_conv_fwd(x_, w_, b_, None, st_, y_, f_, ctypes.byref(s), code, stream),
                lib.ssm_conv_bwd(x_, w_, b_, None, st_, dy_, dx_, dw_, db_, f_, ws_, ws.numel(),
                                 ctypes.byref(s), code, stream),
                lib.ssm_conv_step(x_, w_, b_, st_, y_, ctypes.byref(one), code, stream)]
    return run, (x, y, dy, dx, w, b, dw, db, state, final, ws)


def norm_calls(lib, dim, code, dtype):
    rows = 2000
    x, y, res, r, dx = (new(rows, dim, dtype=dtype) for _ in range(5))
    w, b, dw, db, stats = new(dim), new(dim), new(dim), new(dim), new(2, rows)
    s = NormShapes(rows, dim, 0, 1e-5, code, code)
    ws = torch.empty(lib.ssm_norm_bwd_workspace_bytes(ctypes.byref(s)), dtype=torch.uint8, device="cuda")
    x_, y_, res_, r_, dx_, w_, b_, dw_, db_, st_, ws_ = (
        v.data_ptr() for v in (x, y, res, r, dx, w, b, dw, db, stats, ws))

    def run(stream):
        return [lib.ssm_norm_fwd(x_, res_, w_, b_, y_, r_, st_, ctypes.byref(s), stream),
                lib.ssm_norm_bwd(r_, w_, st_, y_, res_, dx_, None, dw_, db_, ws_, ws.numel(),
                                 ctypes.byref(s), stream)]
    return run, (x, y, res, r, dx, w, b, dw, db, stats, ws)


def xent_calls(lib, tokens):
    V, D = 5000, 128
    h, w, dh, dw = (new(n, D, dtype=torch.bfloat16) for n in (tokens, V, tokens, V))
    targets = torch.randint(0, V, (tokens,), device="cuda")
    loss, lse, dloss = new(tokens), new(tokens), new(tokens)
    s = XentShapes(tokens, V, D, -100)
    size = [lib.ssm_xent_workspace_bytes(ctypes.byref(s), k) for k in (0, 1)]
    ws = torch.empty(max(size), dtype=torch.uint8, device="cuda")
    h_, w_, dh_, dw_, t_, loss_, lse_, dl_, ws_ = (
        v.data_ptr() for v in (h, w, dh, dw, targets, loss, lse, dloss, ws))

    def run(stream):
        return [lib.ssm_xent_fwd(h_, w_, t_, loss_, lse_, ws_, size[0], ctypes.byref(s), 1, stream),
                lib.ssm_xent_bwd(h_, w_, t_, lse_, dl_, dh_, dw_, ws_, size[1], ctypes.byref(s), 1, stream)]
    return run, (h, w, dh, dw, targets, loss, lse, dloss, ws)


def test_calls_allocate_nothing():
    lib = S.load()
    bf16 = torch.bfloat16
    made = [conv_calls(lib, 64, 0, torch.float32), conv_calls(lib, 129, 1, bf16),
            norm_calls(lib, 512, 1, bf16), norm_calls(lib, 513, 0, torch.float32),
            xent_calls(lib, 10), xent_calls(lib, 700)]
    stream = torch.cuda.current_stream().cuda_stream
    for run, _ in made:  # the first call of a kernel loads it
        assert all(status == 0 for status in run(stream))
    torch.cuda.synchronize()
    before, _ = torch.cuda.mem_get_info()
    for _ in range(20):
        for run, _ in made:
            assert all(status == 0 for status in run(stream))
    torch.cuda.synchronize()
    after, _ = torch.cuda.mem_get_info()
    assert after == before, "a call allocated device memory"
    S.check_device_errors()
