"""C ABI checks of the gated linear recurrence that need no GPU: the symbols are
exported, and bad arguments are answered with a status before anything is
launched (the pointers here are never dereferenced)."""
import ctypes

import pytest

from selective_state_space_fwd_gb300 import _binding as Bd

FAKE = 0x10000
EXPECTED = {"ssm_recur_fwd", "ssm_recur_bwd", "ssm_recur_step", "ssm_recur_bwd_workspace_bytes", "ssm_recur_chunks"}
E = Bd.Status


def test_declared_and_exported(ssmlib):
    assert EXPECTED <= set(Bd.declared_functions())
    lib = ctypes.CDLL(Bd.LIB_PATH)
    for name in EXPECTED:
        assert hasattr(lib, name), name


SHAPES = (2, 8, 16, 128, 16, 256, 32)


def _recur(fn="fwd", g=FAKE, v=FAKE, floor=None, valid=None, state=FAKE, y=FAKE, final=None, states=FAKE, dy=FAKE,
           dg=FAKE, dfloor=None, ws=None, nbytes=1 << 40, shapes=SHAPES, dtype=0, no_shapes=False):
    lib, s = Bd.load(), Bd.RecurShapes(*shapes)
    ref = None if no_shapes else ctypes.byref(s)
    if fn == "fwd":
        return lib.ssm_recur_fwd(g, v, floor, valid, state, y, final, states, ref, dtype, None)
    if fn == "step":
        return lib.ssm_recur_step(g, v, floor, state, y, ref, dtype, None)
    return lib.ssm_recur_bwd(g, v, floor, valid, states, dy, final, dg, y, dfloor, state, ws, nbytes, ref, dtype, None)


ONE = (2, 1, 16, 16, 16, 16, 16)


@pytest.mark.parametrize("kw,status", [
    (dict(no_shapes=True), E.ERR_NULL),
    (dict(g=None), E.ERR_NULL),
    (dict(v=None), E.ERR_NULL),
    (dict(y=None), E.ERR_NULL),
    (dict(fn="bwd", states=None), E.ERR_NULL),
    (dict(fn="bwd", dy=None), E.ERR_NULL),
    (dict(fn="bwd", dg=None), E.ERR_NULL),
    (dict(fn="bwd", y=None), E.ERR_NULL),
    (dict(fn="bwd", dfloor=FAKE), E.ERR_NULL),                   # a sum without a workspace
    (dict(fn="bwd", dfloor=FAKE, ws=FAKE, nbytes=64), E.ERR_SHAPE),
    (dict(fn="bwd", dfloor=FAKE, ws=FAKE + 4), E.ERR_ALIGN),
    (dict(fn="step", shapes=ONE, state=None), E.ERR_NULL),
    (dict(fn="step", shapes=ONE, y=None), E.ERR_NULL),
    (dict(fn="step"), E.ERR_SHAPE),                              # more than one step
    (dict(shapes=(0, 8, 16, 128, 16, 128, 16)), E.ERR_SHAPE),
    (dict(shapes=(2, 0, 16, 128, 16, 128, 16)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, -1, 128, 16, 128, 16)), E.ERR_SHAPE),
    (dict(shapes=(1 << 31, 1 << 31, 1 << 31, 128, 16, 128, 16)), E.ERR_SHAPE),
    (dict(shapes=(1 << 31, 1, 1, 1, 1, 1, 1)), E.ERR_SHAPE),     # past the grid
    (dict(shapes=(2, 8, 16, -128, 16, 128, 16)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, 16, 128, 16, 128, -16)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, 16, 128, 16, 1 << 62, 16)), E.ERR_SHAPE),
    (dict(dtype=2), E.ERR_UNSUPPORTED),
    (dict(g=FAKE + 2), E.ERR_ALIGN),
    (dict(v=FAKE + 1, dtype=1), E.ERR_ALIGN),
    (dict(floor=FAKE + 2, dtype=1), E.ERR_ALIGN),
    (dict(valid=FAKE + 2), E.ERR_ALIGN),
    (dict(state=FAKE + 2, dtype=1), E.ERR_ALIGN),
    (dict(states=FAKE + 2, dtype=1), E.ERR_ALIGN),
    (dict(fn="step", shapes=ONE, state=FAKE + 2), E.ERR_ALIGN),
])
def test_recur_argument_errors(ssmlib, kw, status):
    assert _recur(**kw) == status


def test_sizes(ssmlib):
    lib = Bd.load()
    for seqlen, chunks in ((1, 1), (64, 1), (65, 2), (65536, 1024)):
        s = Bd.RecurShapes(3, seqlen, 70, 0, 0, 0, 0)
        assert lib.ssm_recur_chunks(ctypes.byref(s)) == chunks
        n = lib.ssm_recur_bwd_workspace_bytes(ctypes.byref(s))
        assert n >= 3 * 70 * 4 and n % (70 * 4) == 0
    assert lib.ssm_recur_chunks(None) == 0 and lib.ssm_recur_bwd_workspace_bytes(None) == 0
