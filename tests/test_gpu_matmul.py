"""GPU NVFP4 matrix products (nvfp4kv_matmul, nvfp4kv_grouped_matmul) against
float64 on the same codes and scales: every value within the error of its fp32
sum and one rounding; guard bytes around the output; ragged sizes, strides,
empty groups, rows outside the groups; refusals."""
import numpy as np
import pytest

import matmul_ref as ref

pytestmark = pytest.mark.gpu


def _buffer(lib, m, E=None):
    import torch
    R, C = m["codes"].shape[-2], 2 * m["codes"].shape[-1]
    mode = lib.TILES_2D if m["tiles"] else lib.BLOCKS_1D
    parts = [torch.from_numpy(m[k]).cuda() for k in ("codes", "scales", "s")]
    return lib.MatrixBuffer(R, C, mode, parts=parts) if E is None else \
        lib.GroupedMatrixBuffer(E, R, C, mode, parts=parts)


def _act(lib, act):
    return {"none": lib.ACT_NONE, "gelu": lib.ACT_GELU_TANH, "silu": lib.ACT_SILU}[act]


def _cuda(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(a):
    """float32 values rounded to bf16, and the float64 of them."""
    import torch
    t = torch.from_numpy(a.astype(np.float32)).bfloat16()
    return t, t.float().numpy().astype(np.float64)


def _assert_close(got, y, mag, K, bf16, what):
    tol = ref.tolerance(y, mag, K, bf16)
    err = np.abs(got - y)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), \
        f"{what}: |error| {err[worst]:.3e} at {worst}, allowed {tol[worst]:.3e}, " \
        f"{int((err > tol).sum())} of {err.size} outside"


class Case:
    """One product's operands on the host and the device."""

    def __init__(self, lib, seed, M, N, K, x_tiles=False, w_tiles=True, bf16=True, bias=True,
                 act="none", rpg=0, residual=False, offsets=None, pad=0):
        import torch
        from gpu_util import Guarded
        rng = np.random.default_rng(seed)
        self.lib, self.M, self.N, self.K, self.bf16, self.act = lib, M, N, K, bf16, act
        E = None if offsets is None else len(offsets) - 1
        self.E, self.offsets = E, offsets
        lead = () if E is None else (E,)
        self.x = ref.random_matrix(rng, (), M, K, x_tiles)
        self.w = ref.random_matrix(rng, lead, N, K, w_tiles)
        self.X, self.W = _buffer(lib, self.x), _buffer(lib, self.w, E)
        f = np.float32
        self.bias = rng.standard_normal(lead + (N,)).astype(f) if bias else None
        self.rpg = rpg
        G = 0 if not rpg else (E if E is not None else -(-M // rpg))
        self.gate = rng.standard_normal((G, N)).astype(f) if rpg else None
        dt = torch.bfloat16 if bf16 else torch.float32
        self.guard = Guarded((M, N + pad), dt)
        self.Y = self.guard.t[:, :N]
        self.before = self.guard.t.clone()
        self.R = self.r64 = None
        if residual:
            r = rng.standard_normal((M, N + 2 * pad)).astype(f)
            t, v = _bf16(r) if bf16 else (torch.from_numpy(r), r.astype(np.float64))
            self.R, self.r64 = t.cuda()[:, :N], v[:, :N]
        self.ws = lib.new_matrix_workspace()
        self.dev = dict(bias=_cuda(self.bias), gate=_cuda(self.gate))

    def run(self, stream=None):
        kw = dict(self.dev, activation=_act(self.lib, self.act), residual=self.R, stream=stream)
        if self.E is None:
            self.lib.matmul(self.X, self.W, self.Y, self.ws, rows_per_gate=self.rpg, **kw)
        else:
            if not hasattr(self, "off"):
                self.off = _cuda(np.asarray(self.offsets, np.int32))
            self.lib.grouped_matmul(self.X, self.W, self.off, self.Y, self.ws, **kw)
        return self

    def check(self, what=""):
        import torch
        torch.cuda.synchronize()
        assert self.lib.workspace_status(self.ws) == self.lib.OK
        self.guard.assert_intact(what)
        full = self.guard.t
        assert torch.equal(full[:, self.N:].view(torch.uint8), self.before[:, self.N:].view(torch.uint8)), \
            f"{what}: bytes between the rows of Y changed"
        got = self.Y.float().cpu().numpy().astype(np.float64)
        x = ref.decode(self.x)
        off = [0, self.M] if self.E is None else self.offsets
        for e in range(len(off) - 1):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            g = None
            if self.gate is not None:
                g = self.gate[np.arange(a, b) // self.rpg] if self.E is None else self.gate[e]
            bias = self.bias if self.bias is None or self.E is None else self.bias[e]
            y, mag = ref.reference(x[a:b], ref.decode(self.w, None if self.E is None else e), bias,
                                   self.act, g, None if self.r64 is None else self.r64[a:b])
            _assert_close(got[a:b], y, mag, self.K, self.bf16, f"{what} group {e}")
        for a, b in ((0, off[0]), (off[-1], self.M)):
            assert torch.equal(full[a:b].view(torch.uint8), self.before[a:b].view(torch.uint8)), \
                f"{what}: rows outside the groups changed"
        return self


@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (1, 128, 256), (2, 130, 64), (17, 144, 96),
                                   (32, 256, 512), (33, 1000, 288), (128, 128, 1024),
                                   (129, 384, 2048), (200, 272, 4096), (333, 1001, 1056),
                                   (700, 640, 800)])
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_dense_sizes(lib, M, N, K, bf16):
    tiles = N % 16 == 0
    Case(lib, M * 7 + N + K, M, N, K, w_tiles=tiles, bf16=bf16).run().check(f"{M}x{N}x{K}")


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M", [3, 150])
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_epilogue_parts(lib, act, M, bf16):
    for k, (bias, rpg, residual) in enumerate([(False, 0, False), (True, 1, False),
                                               (False, 7, True), (True, 1000, True)]):
        Case(lib, 40 + k, M, 208, 320, bf16=bf16, act=act, bias=bias, rpg=rpg, residual=residual,
             pad=3 * k).run().check(f"{act} bias {bias} rows_per_gate {rpg} residual {residual}")


@pytest.mark.parametrize("x_tiles,w_tiles", [(False, False), (True, True), (True, False)])
def test_block_shapes(lib, x_tiles, w_tiles):
    Case(lib, 60, 208, 160, 352, x_tiles=x_tiles, w_tiles=w_tiles, bf16=False).run().check()


def test_residual_in_place(lib):
    import torch
    for bf16 in (True, False):
        c = Case(lib, 70, 140, 96, 256, bf16=bf16, residual=True, pad=8, rpg=20)
        c.Y.copy_(c.R)
        c.R = c.Y
        c.before = c.guard.t.clone()
        c.run().check("in place")


@pytest.mark.parametrize("offsets", [[0, 5, 5, 40], [3, 3, 3, 60, 64, 90], [0, 0], [0, 1],
                                     [0, 200, 200, 401, 430], [10] * 9 + [11],
                                     list(range(0, 65)), [0, 700]])
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_grouped(lib, offsets, bf16):
    T = max(offsets[-1] + 13, 16)
    Case(lib, 80 + len(offsets), T, 272, 352, offsets=offsets, bf16=bf16, act="silu", rpg=1,
         residual=True, pad=5).run().check(str(offsets))


@pytest.mark.parametrize("w_tiles", [True, False])
def test_grouped_many_experts(lib, w_tiles):
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 4, 1024) * (rng.random(1024) < 0.3)
    offsets = [0] + np.cumsum(sizes).tolist()
    Case(lib, 90, offsets[-1] + 1, 48, 64, offsets=offsets, w_tiles=w_tiles).run().check()
