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
