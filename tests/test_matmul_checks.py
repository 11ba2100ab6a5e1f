"""Refusals of the NVFP4 matrix products on the host: the C entry points return
the documented status before any device work (pointers passed here are never
dereferenced), and the binding refuses operands that do not fit together (CPU
tensors stand in for device ones)."""
import ctypes

import pytest

import sink_window_video_b200 as swv

FAKE = 0x7F0000000000      # 256-byte aligned, never dereferenced
MAT, GRP = 0, 1


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(swv.LIB_PATH):
        from sink_window_video_b200 import build
        build.build()
    return swv.load()


def _call(L, which, M=64, N=96, K=128, E=4, X=None, W=None, ep=None, Y=FAKE, ldy=None, dt=swv.BF16,
          ws=FAKE, off=FAKE):
    X = swv.MatrixView(FAKE, FAKE, FAKE, swv.BLOCKS_1D) if X is None else X
    W = swv.MatrixView(FAKE, FAKE, FAKE, swv.TILES_2D) if W is None else W
    ldy = N if ldy is None else ldy
    if which == GRP:
        return L.nvfp4kv_grouped_matmul(X or None, W or None, E, M, N, K, off, ep, Y, ldy, dt, ws, None)
    return L.nvfp4kv_matmul(X or None, W or None, M, N, K, ep, Y, ldy, dt, ws, None)


def _ep(bias=None, act=0, gate=None, rpg=0, residual=None, ldr=0):
    return swv.Epilogue(bias, act, gate, rpg, residual, ldr)


@pytest.mark.parametrize("which", [MAT, GRP], ids=["dense", "grouped"])
def test_c_refusals(L, which):
    def call(**kw):
        return _call(L, which, **kw)
    view = swv.MatrixView
    inv, uns, ali = swv.ERR_INVALID_ARG, swv.ERR_UNSUPPORTED, swv.ERR_ALIGNMENT
    for kw in (dict(M=0), dict(M=-1), dict(N=0), dict(K=0), dict(M=1 << 25), dict(K=1 << 25),
               dict(N=1 << 25), dict(M=1 << 24, N=1 << 12, K=32), dict(M=1 << 20, K=1 << 16),
               dict(N=1 << 20, K=1 << 16), dict(Y=None), dict(ws=None), dict(ldy=95), dict(dt=2),
               dict(ldy=(1 << 40) + 1),
               dict(X=False), dict(W=False), dict(X=view(None, FAKE, FAKE, 1)),
               dict(X=view(FAKE, None, FAKE, 1)), dict(W=view(FAKE, FAKE, None, 2)),
               dict(W=view(FAKE, FAKE, FAKE, 0)), dict(X=view(FAKE, FAKE, FAKE, 3)),
               dict(ep=_ep(act=3)), dict(ep=_ep(act=-1)),
               dict(ep=_ep(residual=FAKE + (1 << 30), ldr=95)),
               # the residual on Y's elements, but not Y itself
               dict(ep=_ep(residual=FAKE + 2, ldr=96)), dict(ep=_ep(residual=FAKE, ldr=97)),
               dict(ep=_ep(residual=FAKE + 2 * 95, ldr=200), ldy=200)):
        assert call(**kw) == inv, kw
    for kw in (dict(K=48), dict(K=16), dict(N=90), dict(M=65, X=view(FAKE, FAKE, FAKE, 2))):
        assert call(**kw) == uns, kw
    for kw in (dict(X=view(FAKE + 8, FAKE, FAKE, 1)), dict(W=view(FAKE, FAKE + 8, FAKE, 2)),
               dict(X=view(FAKE, FAKE, FAKE + 2, 1)), dict(Y=FAKE + 1), dict(Y=FAKE + 2, dt=swv.F32),
               dict(ws=FAKE + 16), dict(ep=_ep(bias=FAKE + 2)),
               dict(ep=_ep(gate=FAKE + 1, rpg=1)),
               dict(ep=_ep(residual=FAKE + (1 << 30) + 1, ldr=96))):
        assert call(**kw) == ali, kw


def test_c_refusals_of_one_kind(L):
    assert _call(L, MAT, ep=_ep(gate=FAKE, rpg=0)) == swv.ERR_INVALID_ARG
    assert _call(L, MAT, ep=_ep(gate=FAKE, rpg=-3)) == swv.ERR_INVALID_ARG
    assert _call(L, GRP, off=None) == swv.ERR_INVALID_ARG
    assert _call(L, GRP, E=0) == swv.ERR_INVALID_ARG
    assert _call(L, GRP, E=1025) == swv.ERR_CAPACITY


def test_residual_beside_y_under_one_stride_is_no_overlap(L):
    """Columns [0, N) and [N, 2N) of one buffer share an address range but no
    element: the call passes the overlap check (and ends at the device check on
    a machine without the GPU; K = 48 stands for it where there is one)."""
    ep = _ep(residual=FAKE + 2 * 96, ldr=192)
    assert _call(L, MAT, ldy=192, ep=ep, K=48) == swv.ERR_UNSUPPORTED
    ep = _ep(residual=FAKE, ldr=96)           # Y itself
    assert _call(L, MAT, ep=ep, K=48) == swv.ERR_UNSUPPORTED


def _buf(M, K, mode=swv.BLOCKS_1D):
    return swv.MatrixBuffer(M, K, mode, device="cpu")


def test_binding_refusals():
    import torch
    X, W = _buf(5, 64), _buf(48, 64, swv.TILES_2D)
    ws = torch.zeros(256, dtype=torch.uint8)
    Y = torch.zeros(5, 48)

    def refused(exc, X=X, W=W, Y=Y, **kw):
        with pytest.raises(exc):
            swv.matmul(X, W, Y, ws, **kw)
    refused(ValueError, W=_buf(48, 96))                               # K differs
    refused(ValueError, Y=torch.zeros(5, 47))
    refused(ValueError, Y=torch.zeros(48, 5).t())                     # rows not contiguous
    refused(ValueError, Y=torch.zeros(1, 48).expand(5, 48))           # rows on one another
    refused(TypeError, Y=torch.zeros(5, 48, dtype=torch.float16))
    refused(ValueError, bias=torch.zeros(47))
    refused(ValueError, bias=torch.zeros(48, dtype=torch.bfloat16))
    refused(ValueError, gate=torch.zeros(2, 48))                      # no rows_per_gate
    refused(ValueError, gate=torch.zeros(2, 48), rows_per_gate=2)     # 3 rows needed
    refused(TypeError, residual=torch.zeros(5, 48, dtype=torch.bfloat16))
    refused(ValueError, residual=torch.zeros(4, 48))
    refused(ValueError)                                               # nothing on a GPU
    G = swv.GroupedMatrixBuffer(3, 48, 64, swv.TILES_2D, device="cpu")
    refused(TypeError, W=G)
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        swv.grouped_matmul(X, G, off[:3], Y, ws)
    with pytest.raises(ValueError):
        swv.grouped_matmul(X, G, off.long(), Y, ws)
    with pytest.raises(ValueError):
        swv.grouped_matmul(X, G, off, Y, ws, bias=torch.zeros(48))
    with pytest.raises(TypeError):
        swv.grouped_matmul(X, W, off, Y, ws)


def test_matrix_buffers_keep_their_view_in_step():
    import torch
    m = _buf(32, 64, swv.TILES_2D)
    assert (m.view.codes, m.view.scales, m.view.tensor_scale, m.view.mode) == \
        (m.codes.data_ptr(), m.scales.data_ptr(), m.tensor_scale.data_ptr(), swv.TILES_2D)
    m.codes = torch.zeros(32, 32, dtype=torch.uint8)
    assert m.view.codes == m.codes.data_ptr()
    g = swv.GroupedMatrixBuffer(2, 16, 32, swv.BLOCKS_1D, device="cpu")
    e = g.expert(1)
    assert e.codes.data_ptr() == g.codes.data_ptr() + 16 * 16
    assert e.scales.data_ptr() == g.scales.data_ptr() + 16 * 2
    assert e.tensor_scale.data_ptr() == g.tensor_scale.data_ptr() + 4
    with pytest.raises(ValueError):
        swv.MatrixBuffer(16, 32, 1, parts=(g.codes, g.scales[0], g.tensor_scale[:1]))


def test_struct_layouts_match_the_header(L):
    """The binding's structs have the header's fields at the offsets that a C
    compiler gives them."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "nvfp4kv.h"\nint main(void) {\n'
    for cname, cls in (("nvfp4kv_matrix_view", swv.MatrixView), ("nvfp4kv_epilogue", swv.Epilogue)):
        for f, _ in cls._fields_:
            src += f'printf("%zu ", offsetof({cname}, {f}));\n'
        src += f'printf("%zu\\n", sizeof({cname}));\n'
    src += "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        open(d + "/a.c", "w").write(src)
        subprocess.run(["gcc", "-I" + root + "/include", d + "/a.c", "-o", d + "/a"], check=True)
        lines = subprocess.run([d + "/a"], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, cls in zip(lines, (swv.MatrixView, swv.Epilogue)):
        want = [getattr(cls, f).offset for f, _ in cls._fields_] + [ctypes.sizeof(cls)]
        assert [int(x) for x in line.split()] == want
