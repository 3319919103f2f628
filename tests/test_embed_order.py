"""The embedding's gradient adds the rows of a token in an order that the ids fix: the
same bits wherever the tensors start."""
import pytest
import torch

import selective_state_space_fwd_gb300 as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(ssmlib):
    assert torch.cuda.is_available(), "these tests need a CUDA GPU"
    yield


@pytest.mark.parametrize("T,V,D,dtype,io", [
    (20000, 300, 256, torch.bfloat16, torch.bfloat16),
    (20000, 300, 256, torch.bfloat16, torch.float32),
    (5001, 40, 1536, torch.float32, torch.float32),
    (9000, 3, 1024, torch.float32, torch.float32),
    (20000, 300, 255, torch.bfloat16, torch.bfloat16),
])
@pytest.mark.parametrize("add", [False, True])
def test_the_same_bits_off_a_boundary(T, V, D, dtype, io, add):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    dy = torch.randn(T, D, generator=g, device="cuda").to(io)
    dw = torch.randn(V, D, generator=g, device="cuda").to(dtype)

    def shifted(v):
        buf = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
        return buf[1:].view(v.shape).copy_(v)

    def go(dy, dw):
        return S.embed_bwd(ids, dy, add_to=dw) if add else S.embed_bwd(ids, dy, vocab=V, dtype=dtype)

    want = go(dy, dw.clone())
    assert torch.equal(go(shifted(dy), dw.clone()), want)
    assert torch.equal(go(dy, shifted(dw)), want)
    assert torch.equal(go(shifted(dy), shifted(dw)), want)
