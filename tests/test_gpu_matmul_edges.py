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
