"""C ABI checks of the operators around the scan that need no GPU: the symbols
are exported, and bad arguments are answered with a status before anything is
launched (the pointers here are never dereferenced)."""
import ctypes

import pytest

from selective_state_space_fwd_gb300 import _binding as Bd

FAKE = 0x10000
EXPECTED = {"ssm_conv_fwd", "ssm_conv_bwd", "ssm_conv_step", "ssm_conv_bwd_workspace_bytes",
            "ssm_norm_fwd", "ssm_norm_bwd", "ssm_norm_bwd_workspace_bytes",
            "ssm_xent_fwd", "ssm_xent_bwd", "ssm_xent_workspace_bytes"}


def test_every_operator_is_declared_and_exported(ssmlib):
    assert EXPECTED <= set(Bd.declared_functions())
    lib = ctypes.CDLL(Bd.LIB_PATH)
    for name in EXPECTED:
        assert hasattr(lib, name), name


def _conv(fn="fwd", x=FAKE, w=FAKE, b=None, valid=None, state0=None, y=FAKE, final=None, dy=FAKE,
          ws=FAKE, nbytes=1 << 40, shapes=(2, 8, 16, 4, 128, 16, 1), dtype=0, no_shapes=False):
    lib, s = Bd.load(), Bd.ConvShapes(*shapes)
    ref = None if no_shapes else ctypes.byref(s)
    if fn == "fwd":
        return lib.ssm_conv_fwd(x, w, b, valid, state0, y, final, ref, dtype, None)
    if fn == "step":
        return lib.ssm_conv_step(x, w, b, state0, y, ref, dtype, None)
    return lib.ssm_conv_bwd(x, w, b, valid, state0, dy, y, FAKE, None, final, ws, nbytes, ref, dtype,
                            None)


E = Bd.Status


@pytest.mark.parametrize("kw,status", [
    (dict(no_shapes=True), E.ERR_NULL),
    (dict(x=None), E.ERR_NULL),
    (dict(w=None), E.ERR_NULL),
    (dict(y=None), E.ERR_NULL),
    (dict(fn="bwd", dy=None), E.ERR_NULL),
    (dict(fn="bwd", ws=None), E.ERR_NULL),
    (dict(fn="step", shapes=(2, 1, 16, 4, 16, 16, 1)), E.ERR_NULL),  # no state
    (dict(fn="step", state0=FAKE), E.ERR_SHAPE),                      # more than one step
    (dict(shapes=(0, 8, 16, 4, 128, 16, 1)), E.ERR_SHAPE),
    (dict(shapes=(2, 0, 16, 4, 128, 16, 1)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, -1, 4, 128, 16, 1)), E.ERR_SHAPE),
    (dict(shapes=(1 << 31, 1 << 31, 1 << 31, 4, 128, 16, 1)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, 16, 4, -128, 16, 1)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, 16, 4, 1 << 62, 16, 1)), E.ERR_SHAPE),
    (dict(shapes=(2, 8, 16, 1, 128, 16, 1)), E.ERR_UNSUPPORTED),
    (dict(shapes=(2, 8, 16, 5, 128, 16, 1)), E.ERR_UNSUPPORTED),
    (dict(shapes=(2, 8, 16, 4, 128, 16, 2)), E.ERR_UNSUPPORTED),
    (dict(dtype=3), E.ERR_UNSUPPORTED),
    (dict(x=FAKE + 2), E.ERR_ALIGN),
    (dict(x=FAKE + 1, dtype=1), E.ERR_ALIGN),
    (dict(w=FAKE + 2, dtype=1), E.ERR_ALIGN),
    (dict(valid=FAKE + 1), E.ERR_ALIGN),
    (dict(final=FAKE + 2), E.ERR_ALIGN),
    (dict(fn="bwd", ws=FAKE + 4), E.ERR_ALIGN),
    (dict(fn="bwd", nbytes=8), E.ERR_SHAPE),
])
def test_conv_argument_errors(ssmlib, kw, status):
    assert _conv(**kw) == status


def _norm(fn="fwd", x=FAKE, res=None, w=FAKE, b=None, y=FAKE, r=None, stats=FAKE, ws=FAKE,
          nbytes=1 << 40, shapes=(4, 64, 0, 1e-5, 0, 0), no_shapes=False):
    lib, s = Bd.load(), Bd.NormShapes(*shapes)
    ref = None if no_shapes else ctypes.byref(s)
    if fn == "fwd":
        return lib.ssm_norm_fwd(x, res, w, b, y, r, stats, ref, None)
    return lib.ssm_norm_bwd(x, w, stats, FAKE, res, y, r, FAKE, b, ws, nbytes, ref, None)


@pytest.mark.parametrize("kw,status", [
    (dict(no_shapes=True), E.ERR_NULL),
    (dict(x=None), E.ERR_NULL),
    (dict(w=None), E.ERR_NULL),
    (dict(y=None), E.ERR_NULL),
    (dict(res=FAKE), E.ERR_NULL),                              # a residual, nowhere to store the sum
    (dict(r=FAKE), E.ERR_NULL),                                # a sum without a residual
    (dict(fn="bwd", stats=None), E.ERR_NULL),
    (dict(fn="bwd", ws=None), E.ERR_NULL),
    (dict(shapes=(0, 64, 0, 1e-5, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 0, 0, 1e-5, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(1 << 60, 64, 0, 1e-5, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 64, 0, -1.0, 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 64, 0, float("inf"), 0, 0)), E.ERR_SHAPE),
    (dict(shapes=(4, 8193, 0, 1e-5, 0, 0)), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 64, 2, 1e-5, 0, 0)), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 64, 0, 1e-5, 2, 0)), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 64, 0, 1e-5, 0, 1), res=FAKE, r=FAKE), E.ERR_UNSUPPORTED),
    (dict(shapes=(4, 64, 0, 1e-5, 1, 0)), E.ERR_UNSUPPORTED),  # fp32 stream, but no stream
    (dict(x=FAKE + 2), E.ERR_ALIGN),
    (dict(w=FAKE + 1), E.ERR_ALIGN),
    (dict(stats=FAKE + 2), E.ERR_ALIGN),
    (dict(fn="bwd", nbytes=16), E.ERR_SHAPE),
])
def test_norm_argument_errors(ssmlib, kw, status):
    assert _norm(**kw) == status


def _xent(fn="fwd", h=FAKE, w=FAKE, t=FAKE, loss=FAKE, lse=FAKE, dloss=FAKE, dw=FAKE, ws=FAKE,
          nbytes=1 << 60, shapes=(4, 100, 64, -100), dtype=1, no_shapes=False):
    lib, s = Bd.load(), Bd.XentShapes(*shapes)
    ref = None if no_shapes else ctypes.byref(s)
    if fn == "fwd":
        return lib.ssm_xent_fwd(h, w, t, loss, lse, ws, nbytes, ref, dtype, None)
    return lib.ssm_xent_bwd(h, w, t, lse, dloss, loss, dw, ws, nbytes, ref, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(no_shapes=True), E.ERR_NULL),
    (dict(h=None), E.ERR_NULL),
    (dict(w=None), E.ERR_NULL),
    (dict(t=None), E.ERR_NULL),
    (dict(lse=None), E.ERR_NULL),
    (dict(ws=None), E.ERR_NULL),
    (dict(fn="bwd", dloss=None), E.ERR_NULL),
    (dict(fn="bwd", dw=None), E.ERR_NULL),
    (dict(shapes=(0, 100, 64, -100)), E.ERR_SHAPE),
    (dict(shapes=(4, 0, 64, -100)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, -8, -100)), E.ERR_SHAPE),
    (dict(shapes=(1 << 31, 100, 64, -100)), E.ERR_SHAPE),
    (dict(shapes=(4, 1 << 31, 64, -100)), E.ERR_SHAPE),
    (dict(shapes=(1 << 30, 1 << 30, 64, -100)), E.ERR_SHAPE),
    (dict(shapes=(4, 100, 60, -100)), E.ERR_UNSUPPORTED),
    (dict(dtype=0), E.ERR_UNSUPPORTED),
    (dict(dtype=9), E.ERR_UNSUPPORTED),
    (dict(h=FAKE + 8), E.ERR_ALIGN),
    (dict(w=FAKE + 2), E.ERR_ALIGN),
    (dict(t=FAKE + 4), E.ERR_ALIGN),
    (dict(lse=FAKE + 2), E.ERR_ALIGN),
    (dict(ws=FAKE + 128), E.ERR_ALIGN),
    (dict(fn="bwd", dw=FAKE + 8), E.ERR_ALIGN),
    (dict(nbytes=1000), E.ERR_SHAPE),
    (dict(fn="bwd", nbytes=1000), E.ERR_SHAPE),
])
def test_xent_argument_errors(ssmlib, kw, status):
    assert _xent(**kw) == status


def test_workspace_sizes(ssmlib):
    lib = Bd.load()
    conv = Bd.ConvShapes(8, 4096, 1024, 4, 0, 1024, 1)
    n = lib.ssm_conv_bwd_workspace_bytes(ctypes.byref(conv))
    assert n > 0 and n % (5 * 1024 * 4) == 0
    assert lib.ssm_conv_bwd_workspace_bytes(None) == 0
    assert lib.ssm_norm_bwd_workspace_bytes(ctypes.byref(Bd.NormShapes(1, 64, 0, 0.0, 0, 0))) == 512
    assert lib.ssm_norm_bwd_workspace_bytes(ctypes.byref(Bd.NormShapes(0, 64, 0, 0.0, 0, 0))) == 0
    for tokens, vocab in ((1, 1), (8192, 65536), (100000, 300000)):
        s = Bd.XentShapes(tokens, vocab, 64, -100)
        fwd = lib.ssm_xent_workspace_bytes(ctypes.byref(s), 0)
        bwd = lib.ssm_xent_workspace_bytes(ctypes.byref(s), 1)
        assert 0 < fwd < 2 ** 31 and 0 < bwd < 2 ** 31  # never the logits' size
    assert lib.ssm_xent_workspace_bytes(None, 0) == 0


def test_workspaces_cover_every_row_count(ssmlib):
    """The norm's workspace grows with its rows and never shrinks below what two
    rows per column take; the convolution's holds at least one partial sum."""
    lib = Bd.load()
    for dim in (1, 7, 64, 513, 1536, 8191, 8192):
        last = 0
        for rows in (1, 4, 5, 100, 5000, 1 << 20):
            n = lib.ssm_norm_bwd_workspace_bytes(ctypes.byref(Bd.NormShapes(rows, dim, 0, 0.0, 1, 1)))
            assert n % (8 * dim) == 0 and n >= last > -1
            last = n
    for batch, L, dim, width in ((1, 1, 1, 2), (3, 7, 33, 3), (32, 2048, 1536, 4)):
        s = Bd.ConvShapes(batch, L, dim, width, L * dim, dim, 1)
        n = lib.ssm_conv_bwd_workspace_bytes(ctypes.byref(s))
        assert n >= 4 * (width + 1) * dim and n % (4 * (width + 1) * dim) == 0
