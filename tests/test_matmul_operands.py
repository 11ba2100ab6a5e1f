"""Operands of the NVFP4 matrix products that the binding refuses before it calls
the library (CPU tensors stand in for device ones)."""
import pytest

import sink_window_video_b200 as swv


@pytest.fixture
def operands(monkeypatch):
    """Operands that fit together; a call that gets as far as the library fails."""
    import torch
    monkeypatch.setattr(swv, "load", lambda: pytest.fail("a call went on to the library"))
    X = swv.MatrixBuffer(5, 64, swv.BLOCKS_1D, device="cpu")
    W = swv.MatrixBuffer(48, 64, swv.TILES_2D, device="cpu")
    G = swv.GroupedMatrixBuffer(3, 48, 64, swv.TILES_2D, device="cpu")
    return X, W, G, torch.zeros(5, 48), torch.zeros(256, dtype=torch.uint8), \
        torch.zeros(4, dtype=torch.int32)


def test_activations_are_one_matrix(operands):
    """A set of matrices has the attributes of one; as X it is no activation."""
    import torch
    X, W, G, Y, ws, off = operands
    several = swv.GroupedMatrixBuffer(2, 5, 64, swv.BLOCKS_1D, device="cpu")
    for bad in (several, X.codes, None):
        with pytest.raises(TypeError):
            swv.matmul(bad, W, Y, ws)
        with pytest.raises(TypeError):
            swv.matmul(bad, W, Y, ws, gate=torch.zeros(1, 48), rows_per_gate=5)
        with pytest.raises(TypeError):
            swv.grouped_matmul(bad, G, off, Y, ws)


class _Library:
    """Stands in for the library and keeps what the products were called with."""

    def _call(self, *args):
        self.args = args
        return swv.OK

    nvfp4kv_matmul = nvfp4kv_grouped_matmul = _call


@pytest.fixture
def library(monkeypatch):
    L = _Library()
    monkeypatch.setattr(swv, "load", lambda: L)
    monkeypatch.setattr(swv, "_stream_on", lambda device, stream: 0)
    monkeypatch.setattr(swv, "_call_on", lambda device, where, fn, *args: fn(*args))
    return L


@pytest.mark.parametrize("rows", [5, 6, (1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 1, 1 << 70])
def test_one_gate_row_for_any_number_of_rows(operands, library, rows):
    """rows_per_gate beyond 32 bits: ctypes passes its low 32 bits on, which
    would send rows to gates that do not exist."""
    import torch
    X, W, _, Y, ws, _ = operands
    swv.matmul(X, W, Y, ws, gate=torch.zeros(1, 48), rows_per_gate=rows)
    ep = [a for a in library.args if isinstance(a, swv.Epilogue)][0]
    assert (X.M - 1) // ep.rows_per_gate == 0


@pytest.mark.parametrize("act", [-1, 3, 1 << 32, (1 << 32) + 1])
def test_activations_beyond_the_known_ones_are_refused(operands, act):
    X, W, G, Y, ws, off = operands
    with pytest.raises(swv.NvFp4KvError):
        swv.matmul(X, W, Y, ws, activation=act)
    with pytest.raises(swv.NvFp4KvError):
        swv.grouped_matmul(X, G, off, Y, ws, activation=act)


@pytest.mark.parametrize("mode", [0, 3, (1 << 32) + 1, (1 << 32) + 2])
def test_block_shapes_beyond_the_known_ones_are_refused(operands, mode):
    _, W, _, Y, ws, _ = operands
    X = swv.MatrixBuffer(5, 64, mode, device="cpu")
    with pytest.raises(swv.NvFp4KvError):
        swv.matmul(X, W, Y, ws)


def test_sizes_beyond_32_bits_are_refused(operands):
    """2^32 + 5 rows would be 5 to the library."""
    import torch

    class Parts(swv.MatrixBuffer):
        def _check_part(self, i, t):     # no memory of that size here
            pass
    _, W, _, Y, ws, _ = operands
    zero = torch.zeros(1, dtype=torch.uint8)
    X = Parts((1 << 32) + 5, 64, swv.BLOCKS_1D, parts=(zero, zero, zero))
    with pytest.raises(swv.NvFp4KvError):
        swv.matmul(X, W, Y, ws)
