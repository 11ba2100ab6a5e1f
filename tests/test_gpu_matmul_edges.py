"""GPU NVFP4 matrix products at the edges of their kernel's tiles, roles and
groups, against float64 on the same codes and scales."""
import pytest

from test_gpu_matmul import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [1, 2, 31, 32, 33, 64, 1000, 1024])
def test_bad_offsets_of_the_last_group(lib, E):
    """The last group's offsets break the rule, whatever place it has among the
    32 that are looked at together: reported, nothing written."""
    import torch
    T, good = 40, [0] * E + [40]
    c = Case(lib, 200 + E, T, 64, 64, offsets=good)
    for last in (T + 1, 1 << 30, -1, -(1 << 31)):
        c.off = torch.tensor([0] * E + [last], dtype=torch.int32, device="cuda")
        for _ in range(5):
            c.run()
        torch.cuda.synchronize()
        assert lib.workspace_status(c.ws) == lib.ERR_INVALID_ARG
        assert torch.equal(c.guard.t.view(torch.uint8), c.before.view(torch.uint8))
        c.guard.assert_intact()
    c.off = torch.tensor(good, dtype=torch.int32, device="cuda")
    c.run().check("after bad offsets")


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("rpg", [0, 3, 17, 40])
@pytest.mark.parametrize("N", [8, 40, 100, 137])
def test_channels_that_end_inside_a_warp(lib, bf16, rpg, N):
    """Some lanes of a warp have a channel and others none, at the loads of the
    gate, of the residual and of the sums: every epilogue, several chunks."""
    for act in ("none", "gelu"):
        Case(lib, 300 + N + rpg, 77, N, 96, w_tiles=False, bf16=bf16, act=act, rpg=rpg,
             residual=rpg != 17, pad=N % 2).run().check(f"{act} {N} {rpg}")


@pytest.mark.parametrize("rpg", [17, 19, 23, 31, 33, 97])
@pytest.mark.parametrize("N", [144, 132, 137])
def test_gates_that_change_at_odd_rows(lib, N, rpg):
    """A gate that ends inside a chunk of tokens, at an odd place: in bf16 as whole
    pieces of a row, in parts of 4 and by element, with the residual in place."""
    for residual in (False, True):
        c = Case(lib, 500 + N + rpg, 333, N, 160, w_tiles=False, act="silu", rpg=rpg,
                 residual=residual, pad=8 if N == 144 else 4)
        if residual:
            c.Y.copy_(c.R)
            c.R = c.Y
            c.before = c.guard.t.clone()
        c.run().check(f"{N} {rpg} {residual}")


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_pairs_of_ctas_hand_over_their_scales(lib, bf16):
    """A pair's second CTA stores its share of the block scales for the first one's
    MMAs, turn by turn: two products with scales of their own take turns, and
    each result stays bit for bit what it was."""
    import torch
    cases = [Case(lib, 400 + i, 2300, 4100, 1312, w_tiles=False, bf16=bf16, residual=i == 1)
             for i in range(2)]
    first = []
    for c in cases:
        c.run().check("first")
        first.append(c.Y.clone())
    for _ in range(20):
        for c, y in zip(cases, first):
            c.guard.t.copy_(c.before)
            c.run()
            assert torch.equal(c.Y, y)


@pytest.mark.parametrize("K", [32, 1056, 2080])
def test_launches_close_behind_one_another(lib, K):
    """Pairs of CTAs with one turn of scales a tile, or a last turn of one step:
    launch upon launch on the same multiprocessors, each leaving none of its
    signals to the next."""
    import torch
    c = Case(lib, 600 + K, 1900, 4096, K, bf16=False).run().check(str(K))
    first = c.Y.clone()
    for _ in range(5):
        c.guard.t.copy_(c.before)
        for _ in range(40):
            c.run()
        assert torch.equal(c.Y, first)
    assert lib.workspace_status(c.ws) == lib.OK


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("how", ["bf16", "rows", "f32", "gates"])
def test_activations_vanish_far_below_zero(lib, act, how):
    """SiLU and GELU of z from -130 to 10, channel by channel, and of far larger
    ones.  With the product zero z is the bias exactly.  Each x = -v log2 e is off by
    at most two fp32 steps of |x| (one product for SiLU, four for GELU, 2^-24 each,
    so 2^-22 |x| covers both), which is as much in the logarithm of a tail that is
    2^-x, on top of 16 steps for the exponential, the reciprocal and the products."""
    import numpy as np
    import torch
    N = 1024 if how != "rows" else 1022
    bf16 = how != "f32"
    c = Case(lib, 700, 40, N, 64, w_tiles=False, bf16=bf16, act=act, rpg=3 if how == "gates" else 0)
    c.X.codes.zero_()
    if c.gate is not None:
        c.dev["gate"].fill_(1.0)
    z = torch.linspace(-130, 10, N)
    far = torch.tensor([-1e3, -1e4, -1e9, -1e30, -3e38])
    z[5:5 + far.numel()] = far
    c.dev["bias"].copy_(z)
    c.run()
    torch.cuda.synchronize()
    got = c.Y.double().cpu().numpy()
    z = z.numpy().astype(np.float64)
    v = z if act == "silu" else 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    with np.errstate(over="ignore"):
        want = z / (1 + np.exp(-v))
    x = np.maximum(-v * np.log2(np.e), 0)
    # 2^-x below 2^-126 is 0
    tol = np.abs(want) * np.minimum(x * 2.0 ** -22 + 16 * 2.0 ** -24, 1) + np.abs(z) * 2.0 ** -126
    if bf16:
        tol += np.abs(want) * 2.0 ** -8
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    below = z < -130.5
    assert below.sum() == 5 and (got[:, below] == 0).all()


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_a_channel_shut_off_by_its_bias(lib, bf16):
    """A bias of -1e9 ends in 0 behind the activation, not in a share of itself that
    the gate then multiplies; its neighbours stay as they are."""
    import torch
    for act in ("silu", "gelu"):
        c = Case(lib, 710, 50, 80, 128, bf16=bf16, act=act, rpg=20, residual=True)
        c.bias[3], c.bias[64] = -1e9, -1e30
        c.dev["bias"].copy_(torch.from_numpy(c.bias))
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.Y[:, [3, 64]], c.R[:, [3, 64]])
        keep = torch.ones(80, dtype=torch.bool)
        keep[[3, 64]] = False
        d = Case(lib, 710, 50, 80, 128, bf16=bf16, act=act, rpg=20, residual=True).run()
        torch.cuda.synchronize()
        tol = 2.0 ** -7 if bf16 else 2.0 ** -20
        a, b = c.Y[:, keep].double(), d.Y[:, keep].double()
        assert bool(((a - b).abs() <= tol * (a.abs() + 1)).all())


def test_a_product_reads_the_buffers_as_they_are(lib):
    """Operands whose storage was replaced in place, copied or moved through a
    pickle between two products."""
    import copy
    import pickle

    import numpy as np
    import torch

    import matmul_ref as ref
    c = Case(lib, 720, 70, 144, 256, act="silu").run().check("first")
    rng = np.random.default_rng(9)
    c.x = ref.random_matrix(rng, (), 70, 256, False)
    c.X.codes.set_(torch.from_numpy(c.x["codes"]).cuda())
    c.X.scales.data = torch.from_numpy(c.x["scales"]).cuda()
    c.X.tensor_scale = torch.from_numpy(c.x["s"]).cuda()
    c.run().check("other storage")
    keep = c.W
    c.W = pickle.loads(pickle.dumps(keep))
    c.run().check("pickled")
    c.W = copy.copy(keep)
    c.W.codes = torch.zeros_like(keep.codes)
    assert keep.view.codes == keep.codes.data_ptr()
    c.W = copy.deepcopy(keep)
    c.guard.t.copy_(c.before)
    c.run().check("copied")
