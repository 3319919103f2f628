"""C ABI checks of the distillation that need no GPU: the symbols are exported, and
bad arguments are answered with a status before anything is launched (the pointers
here are never dereferenced)."""
import ctypes

import pytest

from selective_state_space_fwd_gb300 import _binding as Bd

FAKE = 0x10000
EXPECTED = {"ssm_distill_fwd", "ssm_distill_bwd", "ssm_distill_workspace_bytes"}
E = Bd.Status


def test_declared_and_exported(ssmlib):
    assert EXPECTED <= set(Bd.declared_functions())
    lib = ctypes.CDLL(Bd.LIB_PATH)
    for name in EXPECTED:
        assert hasattr(lib, name), name


def _distill(fn="fwd", h=FAKE, w=FAKE, ids=FAKE, logits=FAKE, loss=FAKE, lse=FAKE, dloss=FAKE, dw=FAKE, ws=FAKE,
             nbytes=1 << 60, shapes=(4, 100, 64, 8, -100, 1.0, 0), dtype=1, no_shapes=False):
    lib, s = Bd.load(), Bd.DistillShapes(*shapes)
    ref = None if no_shapes else ctypes.byref(s)
    if fn == "fwd":
        return lib.ssm_distill_fwd(h, w, ids, logits, loss, lse, ws, nbytes, ref, dtype, None)
    return lib.ssm_distill_bwd(h, w, ids, logits, lse, dloss, loss, dw, ws, nbytes, ref, dtype, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(no_shapes=True), E.ERR_NULL),
    (dict(h=None), E.ERR_NULL),
    (dict(w=None), E.ERR_NULL),
    (dict(ids=None), E.ERR_NULL),
    (dict(logits=None), E.ERR_NULL),
    (dict(loss=None), E.ERR_NULL),
    (dict(lse=None), E.ERR_NULL),
    (dict(ws=None), E.ERR_NULL),
    (dict(shapes=(0, 100, 64, 8, -100, 1.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 0, 64, 8, -100, 1.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, -8, 8, -100, 1.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 0, -100, 1.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(1 << 31, 100, 64, 8, -100, 1.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 8, -100, 0.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 8, -100, -1.0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 8, -100, float("nan"), 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 8, -100, float("inf"), 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 8, -100, 1e-40, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 64, 8, -100, 3e-39, 0)), E.ERR_SHAPE),  # 1/T is finite, log2(e)/T is not
    (dict(shapes=(4, 100, 60, 8, -100, 1.0, 0)), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 100, 64, 1025, -100, 1.0, 0)), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 100, 64, 8, -100, 1.0, 2)), E.ERR_UNSUPPORTED),
    (dict(dtype=0), E.ERR_UNSUPPORTED),
    (dict(h=FAKE + 8), E.ERR_ALIGN),
    (dict(w=FAKE + 2), E.ERR_ALIGN),
    (dict(ids=FAKE + 4), E.ERR_ALIGN),
    (dict(logits=FAKE + 2), E.ERR_ALIGN),
    (dict(lse=FAKE + 2), E.ERR_ALIGN),
    (dict(ws=FAKE + 128), E.ERR_ALIGN),
    (dict(nbytes=1000), E.ERR_SHAPE),
])
def test_distill_argument_errors(ssmlib, fn, kw, status):
    assert _distill(fn, **kw) == status


def test_distill_gradient_argument_errors(ssmlib):
    assert _distill("bwd", dloss=None) == E.ERR_NULL and _distill("bwd", dw=None) == E.ERR_NULL
    assert _distill("bwd", dw=FAKE + 8) == E.ERR_ALIGN and _distill("bwd", dloss=FAKE + 2) == E.ERR_ALIGN


def test_workspace_sizes(ssmlib):
    """The cross entropy's, the entries and, forward, their logits; never the vocabulary's."""
    lib = Bd.load()
    for tokens, vocab, top in ((1, 1, 1), (8192, 65536, 32), (4096, 50257, 1024)):
        s = Bd.DistillShapes(tokens, vocab, 64, top, -100, 1.0, 1)
        x = Bd.XentShapes(tokens, vocab, 64, -100)
        for backward in (0, 1):
            n = lib.ssm_distill_workspace_bytes(ctypes.byref(s), backward)
            more = n - lib.ssm_xent_workspace_bytes(ctypes.byref(x), backward)
            least = tokens * (8 * (top + 2) + 8 + (0 if backward else 4 * top))
            assert least <= more <= least + 3 * 256
    assert lib.ssm_distill_workspace_bytes(None, 0) == 0
