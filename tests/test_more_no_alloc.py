"""The gated recurrence, the embedding lookup and the distillation allocate nothing:
with outputs and workspaces of the caller's, calls through the C ABI leave the
device's free memory as it was."""
import ctypes

import pytest
import torch

import selective_state_space_fwd_gb300 as S
from selective_state_space_fwd_gb300._binding import DistillShapes, EmbedShapes, RecurShapes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


def new(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype)


def space(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def recur_calls(lib, L, dim, code, dtype):
    B = 2
    t = [new(B, L, dim, dtype=dtype) for _ in range(6)]
    floor, state, final, df = torch.rand(dim, device="cuda"), new(B, dim), new(B, dim), new(dim)
    s = RecurShapes(B, L, dim, L * dim, dim, L * dim, dim)
    one = RecurShapes(B, 1, dim, L * dim, dim, L * dim, dim)
    states = new(B, lib.ssm_recur_chunks(ctypes.byref(s)), dim)
    ws = space(lib.ssm_recur_bwd_workspace_bytes(ctypes.byref(s)))
    g, v, y, dy, dg, dv = (x.data_ptr() for x in t)
    f_, s_, e_, df_, st_, w_ = (x.data_ptr() for x in (floor, state, final, df, states, ws))

    def run(stream):
        return [lib.ssm_recur_fwd(g, v, f_, None, s_, y, e_, st_, ctypes.byref(s), code, stream),
                lib.ssm_recur_bwd(g, v, f_, None, st_, dy, e_, dg, dv, df_, s_, w_, ws.numel(), ctypes.byref(s), code, stream),
                lib.ssm_recur_step(g, v, f_, s_, y, ctypes.byref(one), code, stream)]
    return run, (t, floor, state, final, df, states, ws)


def embed_calls(lib, tokens, vocab, dim, code, dtype):
    ids = torch.randint(0, vocab, (tokens,), device="cuda")
    w, y, dy, dw = new(vocab, dim, dtype=dtype), new(tokens, dim, dtype=dtype), new(tokens, dim, dtype=dtype), new(vocab, dim, dtype=dtype)
    s = EmbedShapes(tokens, vocab, dim, -100, 1.0, code, code)
    ws = space(lib.ssm_embed_bwd_workspace_bytes(ctypes.byref(s)))
    i_, w_, y_, dy_, dw_, ws_ = (x.data_ptr() for x in (ids, w, y, dy, dw, ws))

    def run(stream):
        return [lib.ssm_embed_fwd(i_, w_, y_, ctypes.byref(s), stream),
                lib.ssm_embed_bwd(i_, dy_, dw_, 0, ws_, ws.numel(), ctypes.byref(s), stream),
                lib.ssm_embed_bwd(i_, dy_, dw_, 1, ws_, ws.numel(), ctypes.byref(s), stream)]
    return run, (ids, w, y, dy, dw, ws)


def distill_calls(lib, tokens, top):
    V, D = 5000, 128
    h, w, dh, dw = (new(n, D, dtype=torch.bfloat16) for n in (tokens, V, tokens, V))
    ids, z = torch.randint(0, V, (tokens, top), device="cuda"), new(tokens, top)
    loss, lse, dloss = new(tokens), new(tokens), new(tokens)
    s = DistillShapes(tokens, V, D, top, -100, 2.0, 0)
    size = [lib.ssm_distill_workspace_bytes(ctypes.byref(s), k) for k in (0, 1)]
    ws = space(max(size))
    h_, w_, i_, z_, lo_, ls_, dl_, dh_, dw_, ws_ = (x.data_ptr() for x in (h, w, ids, z, loss, lse, dloss, dh, dw, ws))

    def run(stream):
        return [lib.ssm_distill_fwd(h_, w_, i_, z_, lo_, ls_, ws_, size[0], ctypes.byref(s), 1, stream),
                lib.ssm_distill_bwd(h_, w_, i_, z_, ls_, dl_, dh_, dw_, ws_, size[1], ctypes.byref(s), 1, stream)]
    return run, (h, w, dh, dw, ids, z, loss, lse, dloss, ws)


def test_calls_allocate_nothing():
    lib = S.load()
    bf16 = torch.bfloat16
    made = [recur_calls(lib, 300, 64, 0, torch.float32), recur_calls(lib, 3000, 128, 1, bf16),
            recur_calls(lib, 70, 33, 1, bf16), embed_calls(lib, 100, 500, 64, 1, bf16),
            embed_calls(lib, 20000, 500, 65, 0, torch.float32), distill_calls(lib, 20, 7), distill_calls(lib, 700, 40)]
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


def test_the_first_calls_may_be_captured():
    """Nothing a first call does (loading, asking what the GPU holds) breaks a capture:
    sizes that no call before had."""
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, value = (torch.randn(1, 5000, 72, generator=g, device="cuda") for _ in range(2))
    ids = torch.randint(0, 700, (9000,), generator=g, device="cuda")
    dy = torch.randn(9000, 40, generator=g, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, states = S.recur_fwd(gate, value, want_states=True)
        r = S.recur_bwd(gate, value, states=states, dy=gate)
        dw = S.embed_bwd(ids, dy, vocab=700)
    graph.replay()
    torch.cuda.synchronize()
    y2, _, states = S.recur_fwd(gate, value, want_states=True)
    assert torch.equal(y, y2) and torch.equal(r["dgate"], S.recur_bwd(gate, value, states=states, dy=gate)["dgate"])
    assert torch.equal(dw, S.embed_bwd(ids, dy, vocab=700))
