"""Buffers of quantized matrices on the host: what a call reads is what the
buffer's tensors are at that call, however they came to be so, and what does not
fit is refused (CPU tensors stand in for device ones)."""
import copy
import pickle

import pytest

import sink_window_video_b200 as swv


def _matrix(M=32, K=64, mode=swv.TILES_2D):
    return swv.MatrixBuffer(M, K, mode, device="cpu")


def _grouped(E=3, M=32, K=64, mode=swv.TILES_2D):
    return swv.GroupedMatrixBuffer(E, M, K, mode, device="cpu")


def _addresses(m):
    return m.codes.data_ptr(), m.scales.data_ptr(), m.tensor_scale.data_ptr()


def _view(m):
    v = m.view
    return v.codes, v.scales, v.tensor_scale


BOTH = pytest.mark.parametrize("make", [_matrix, _grouped], ids=["matrix", "grouped"])


@BOTH
def test_a_copy_has_a_view_of_its_own(make):
    a = make()
    first = _view(a)
    b = copy.copy(a)
    assert _view(b) == first                       # a copy shares the tensors
    b.codes = a.codes.clone()
    assert _view(b) == _addresses(b) != first
    assert _view(a) == _addresses(a) == first


@BOTH
@pytest.mark.parametrize("part", ["codes", "scales", "tensor_scale"])
def test_storage_replaced_in_place_is_seen(make, part):
    a = make()
    a.view
    t = getattr(a, part)
    old = t.data_ptr()
    other = t.clone()
    t.set_(other)
    assert getattr(a, part).data_ptr() == other.data_ptr() != old
    assert _view(a) == _addresses(a)
    third = t.clone()
    t.data = third
    assert t.data_ptr() == third.data_ptr()
    assert _view(a) == _addresses(a)


@BOTH
@pytest.mark.parametrize("part", ["codes", "scales", "tensor_scale"])
def test_parts_that_shrank_in_place_are_refused(make, part):
    """A smaller tensor, also one that starts at the same address, one of the full
    shape with other strides, and one of another type."""
    import torch
    for change in (lambda t: t[..., :t.shape[-1] // 2].contiguous(),
                   lambda t: t.view(-1)[:t.numel() // 2],
                   lambda t: t.as_strided(t.shape, (0,) * (t.dim() - 1) + (2,)),
                   lambda t: torch.zeros(t.shape, dtype=torch.float16)):
        a = make()
        a.view
        t = getattr(a, part)
        if part == "tensor_scale":
            t.set_(torch.zeros(2 * t.numel()).data[:t.numel()])
        else:
            t.set_(torch.zeros((2,) + t.shape, dtype=t.dtype)[0])
        a.view
        new = change(t.data)
        if new.shape == t.shape and new.is_contiguous() and new.dtype == t.dtype:
            continue                               # one element: no other strides
        t.data = new
        with pytest.raises(ValueError):
            a.view


@BOTH
def test_mode_and_sizes_are_those_at_the_call(make):
    import torch
    a = make()
    a.view
    a.mode = swv.BLOCKS_1D
    with pytest.raises(ValueError):                # the scales of tiles
        a.view
    a.scales = torch.zeros(a._shapes()[1], dtype=torch.uint8)
    assert a.view.mode == swv.BLOCKS_1D and _view(a) == _addresses(a)
    a.M = 48
    with pytest.raises(ValueError):
        a.view


@BOTH
def test_assigned_parts_are_checked_as_given_ones(make):
    import torch
    for part, bad in (("scales", torch.zeros(3)), ("scales", torch.zeros(3, dtype=torch.uint8)),
                      ("codes", torch.zeros(32, 64, dtype=torch.uint8)),
                      ("codes", torch.zeros(32, 32, dtype=torch.int8)),
                      ("tensor_scale", torch.zeros(4)),
                      ("tensor_scale", torch.zeros(1, dtype=torch.float64))):
        a = make()
        before = _addresses(a)
        with pytest.raises(ValueError):
            setattr(a, part, bad)
        assert _view(a) == _addresses(a) == before


def test_a_product_of_parts_that_do_not_fit_is_refused(monkeypatch):
    import torch
    monkeypatch.setattr(swv, "load", lambda: pytest.fail("a call went on to the library"))
    X, W = _matrix(5, 64, swv.BLOCKS_1D), _matrix(48, 64)
    ws, Y = torch.zeros(256, dtype=torch.uint8), torch.zeros(5, 48)
    for m in (X, W):
        keep = m.codes.data
        m.codes.data = torch.zeros(4, dtype=torch.uint8)
        with pytest.raises(ValueError, match="codes"):
            swv.matmul(X, W, Y, ws)
        m.codes.data = keep
    W.mode = swv.BLOCKS_1D
    with pytest.raises(ValueError, match="scales"):
        swv.matmul(X, W, Y, ws)
    with pytest.raises(ValueError, match="scales"):
        swv.quantize_matrix(torch.zeros(48, 64, dtype=torch.bfloat16), W, ws, stream=0)


@BOTH
@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
def test_copies_and_pickles_hold_the_values(make, how):
    import torch
    a = make()
    a.codes.random_(0, 256)
    a.scales.random_(0, 256)
    a.tensor_scale.fill_(0.5)
    a.view
    b = copy.deepcopy(a) if how == "deepcopy" else pickle.loads(pickle.dumps(a))
    assert type(b) is type(a) and (b.E, b.M, b.N, b.mode) == (a.E, a.M, a.N, a.mode)
    for part in ("codes", "scales", "tensor_scale"):
        x, y = getattr(a, part), getattr(b, part)
        assert torch.equal(x, y) and x.data_ptr() != y.data_ptr()
    assert _view(b) == _addresses(b) and _view(a) == _addresses(a)


def test_a_view_that_was_handed_out_does_not_change():
    a = _matrix()
    v, at = a.view, _addresses(a)
    a.codes = a.codes.clone()
    assert a.view.codes == a.codes.data_ptr()
    assert (v.codes, v.scales, v.tensor_scale) == at


def test_experts_by_any_index():
    g = _grouped()
    for e in (0, 2, -1, -3):
        m = g.expert(e)
        assert _addresses(m) == tuple(t[e].data_ptr() for t in (g.codes, g.scales, g.tensor_scale))
    for e in (3, -4):
        with pytest.raises(IndexError):
            g.expert(e)
