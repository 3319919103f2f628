"""C ABI checks of the embedding lookup that need no GPU: the symbols are exported,
and bad arguments are answered with a status before anything is launched (the
pointers here are never dereferenced)."""
import ctypes

import pytest

from selective_state_space_fwd_gb300 import _binding as Bd

FAKE = 0x10000
EXPECTED = {"ssm_embed_fwd", "ssm_embed_bwd", "ssm_embed_bwd_workspace_bytes"}
E = Bd.Status


def test_declared_and_exported(ssmlib):
    assert EXPECTED <= set(Bd.declared_functions())
    lib = ctypes.CDLL(Bd.LIB_PATH)
    for name in EXPECTED:
        assert hasattr(lib, name), name


def _embed(fn="fwd", ids=FAKE, x=FAKE, y=FAKE, add=0, ws=FAKE, nbytes=1 << 50, shapes=(4, 100, 64, -100, 1.0, 0, 0),
           no_shapes=False):
    lib, s = Bd.load(), Bd.EmbedShapes(*shapes)
    ref = None if no_shapes else ctypes.byref(s)
    if fn == "fwd":
        return lib.ssm_embed_fwd(ids, x, y, ref, None)
    return lib.ssm_embed_bwd(ids, x, y, add, ws, nbytes, ref, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(no_shapes=True), E.ERR_NULL),
    (dict(ids=None), E.ERR_NULL),
    (dict(x=None), E.ERR_NULL),
    (dict(y=None), E.ERR_NULL),
    (dict(shapes=(0, 100, 64, -100, 1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 0, 64, -100, 1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, -1, -100, 1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=((1 << 30) + 1, 100, 64, -100, 1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 1 << 31, 64, -100, 1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 1 << 30, 1 << 40, -100, 1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(1 << 30, 100, 1 << 20, -100, 1.0, 0, 0)), E.ERR_SHAPE),  # past the grid
    (dict(shapes=(4, 100, 64, -100, float("inf"), 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, -100, float("nan"), 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, -100, 1.0, 2, 0)), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 100, 64, -100, 1.0, 0, 1)), E.ERR_UNSUPPORTED),  # bf16 rows of an fp32 weight
    (dict(ids=FAKE + 4), E.ERR_ALIGN),
    (dict(x=FAKE + 2), E.ERR_ALIGN),
    (dict(y=FAKE + 2), E.ERR_ALIGN),
    (dict(y=FAKE + 1, shapes=(4, 100, 64, -100, 1.0, 1, 1)), E.ERR_ALIGN),
])
def test_embed_argument_errors(ssmlib, fn, kw, status):
    assert _embed(fn, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ws=None), E.ERR_NULL),
    (dict(ws=FAKE + 128), E.ERR_ALIGN),
    (dict(nbytes=100), E.ERR_SHAPE),
    (dict(add=2), E.ERR_UNSUPPORTED),
])
def test_embed_gradient_argument_errors(ssmlib, kw, status):
    assert _embed("bwd", **kw) == status


def test_workspace_sizes(ssmlib):
    """The sorted tokens twice, and at most two rows of fp32 per 8 tokens."""
    lib = Bd.load()
    for tokens in (1, 7, 8, 1000, 65536, 1 << 22):
        for dim in (1, 64, 1537, 4096):
            s = Bd.EmbedShapes(tokens, 50257, dim, -100, 1.0, 1, 1)
            n = lib.ssm_embed_bwd_workspace_bytes(ctypes.byref(s))
            assert 16 * tokens + 8 * dim <= n <= 16 * tokens + 8 * dim * (tokens // 8 + 1) + 3 * 256
    assert lib.ssm_embed_bwd_workspace_bytes(None) == 0
