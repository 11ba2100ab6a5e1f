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


# ------------------------------------------------------------------ how calls are made

def test_every_tile_width(lib):
    """Sizes at which the cost rule takes each tile width, the widest (a pair of
    CTAs) among them, with rows that end inside tiles."""
    for M, N, K in ((20, 512, 512), (400, 2048, 96), (880, 2048, 2048), (1900, 4100, 544)):
        Case(lib, M + N, M, N, K, w_tiles=False, residual=True, rpg=150, act="gelu",
             pad=4).run().check(f"{M}x{N}x{K}")


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_wide_grouped(lib, bf16):
    """Groups of several wide tiles beside empty and one-row groups."""
    offsets = [7, 7, 400, 401, 1201, 1201, 1590]
    Case(lib, 91, 1600, 2064, 2080, offsets=offsets, bf16=bf16, act="gelu", rpg=1,
         residual=True).run().check(str(offsets))


@pytest.mark.parametrize("rpg", [1, 15, 16, 17, 100])
def test_gate_stretches(lib, rpg):
    Case(lib, 92, 333, 144, 128, rpg=rpg, residual=rpg != 16, bf16=rpg % 2 == 0).run().check(str(rpg))


def test_unaligned_rows(lib):
    """Y and the residual at element alignment only, an odd row stride."""
    import torch
    for bf16 in (True, False):
        c = Case(lib, 93, 50, 33, 64, w_tiles=False, bf16=bf16, pad=6)
        c.Y = c.guard.t[:, 1:34]
        keep = c.guard.t.clone()
        r = torch.randn(50, 71, device="cuda").to(c.Y.dtype)
        c.R = r[:, 3:36]
        c.r64 = c.R.float().cpu().numpy().astype(np.float64)
        c.run()
        torch.cuda.synchronize()
        c.guard.assert_intact()
        assert torch.equal(c.guard.t[:, :1].view(torch.uint8), keep[:, :1].view(torch.uint8))
        assert torch.equal(c.guard.t[:, 34:].view(torch.uint8), keep[:, 34:].view(torch.uint8))
        y, mag = ref.reference(ref.decode(c.x), ref.decode(c.w), c.bias, "none", None, c.r64)
        _assert_close(c.Y.float().cpu().numpy().astype(np.float64), y, mag, 64, bf16, "unaligned")


def test_rows_far_apart(lib):
    """A row stride beyond 2^31 bytes."""
    import torch
    c = Case(lib, 94, 3, 64, 96, bf16=True)
    big = torch.empty(2 * ((1 << 30) + 8) + 64, dtype=torch.bfloat16, device="cuda")
    c.Y = big.as_strided((3, 64), ((1 << 30) + 8, 1))
    c.run()
    torch.cuda.synchronize()
    y, mag = ref.reference(ref.decode(c.x), ref.decode(c.w), c.bias, "none", None, None)
    _assert_close(c.Y.float().cpu().numpy().astype(np.float64), y, mag, 96, True, "far rows")


def test_infinities_and_nan_stay_in_their_places(lib):
    """Residual and gate values that are not finite reach their own outputs only;
    those behind the last group are not read into anything."""
    import torch
    c = Case(lib, 95, 40, 80, 64, bf16=False, residual=True, offsets=[0, 17, 30], rpg=1)
    c.R[3, 5], c.R[29, 79], c.R[35, 1] = float("inf"), float("nan"), float("nan")
    c.dev["gate"][1, 7] = float("-inf")
    c.run()
    torch.cuda.synchronize()
    got = c.Y[:30]
    bad = torch.zeros(30, 80, dtype=torch.bool)
    bad[3, 5] = bad[29, 79] = True
    bad[17:30, 7] = True
    assert torch.equal(~torch.isfinite(got).cpu(), bad)
    assert got[3, 5] == float("inf") and torch.isnan(got[29, 79])


def test_large_activations_inputs(lib):
    """Sums far outside the activations' curved range: SiLU and GELU go to the
    identity and to zero, without a NaN."""
    import torch
    for act in ("silu", "gelu"):
        c = Case(lib, 96, 30, 64, 64, bf16=False, act=act, bias=False)
        c.x["s"][0] = 1e6
        c.X.tensor_scale.fill_(1e6)
        c.run()
        torch.cuda.synchronize()
        z, mag = ref.reference(ref.decode(c.x), ref.decode(c.w), None, "none", None, None)
        got = c.Y.cpu().numpy().astype(np.float64)
        far = np.abs(z) > 100
        assert far.mean() > 0.5 and np.isfinite(got).all()
        want = np.where(z > 0, z, 0.0)
        tol = mag * (64 / 16 + 32) * 2.0 ** -23
        assert (np.abs(got - want)[far] <= tol[far]).all()


def test_repeated_calls_are_bit_identical(lib):
    import torch
    for kw in (dict(M=33, N=272, K=4096), dict(M=1900, N=4112, K=512),
               dict(M=300, N=272, K=512, offsets=[0, 100, 100, 290])):
        c = Case(lib, 97, act="gelu", residual=True, **kw).run()
        torch.cuda.synchronize()
        first = c.Y.clone()
        c.Y.zero_()
        c.run()
        torch.cuda.synchronize()
        a, b = (first, c.Y) if c.E is None else (first[:290], c.Y[:290])
        assert torch.equal(a, b)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(4100, 544), (4096, 512)])
def test_every_run_with_a_residual(lib, bf16, N, K):
    """Three to four tiles a CTA with a residual, many times over: the warp that
    prefetches it takes part in freeing the accumulators."""
    import torch
    c = Case(lib, 103, 1900, N, K, w_tiles=False, residual=True, rpg=150, bf16=bf16, pad=4).run().check()
    first = c.Y.clone()
    for _ in range(30):
        c.guard.t.copy_(c.before)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.Y, first)


def test_streams_and_graphs(lib):
    """A call on another stream than the operands', two captured graphs that
    share a workspace, replayed on new contents of the same buffers."""
    import torch
    c = Case(lib, 98, 70, 144, 256, act="silu", residual=True)
    d = Case(lib, 99, 90, 272, 160, offsets=[0, 40, 90], bf16=False)
    d.ws = c.ws
    d.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c.run(stream=s)
    s.synchronize()
    c.check("other stream")
    graphs = []
    for k in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            k.run()
        graphs.append(g)
    rng = np.random.default_rng(5)
    c.x = ref.random_matrix(rng, (), 70, 256, False)
    c.X.codes.copy_(torch.from_numpy(c.x["codes"]))
    c.X.scales.copy_(torch.from_numpy(c.x["scales"]))
    c.X.tensor_scale.copy_(torch.from_numpy(c.x["s"]))
    d.offsets = [5, 60, 81]
    d.off.copy_(torch.tensor(d.offsets, dtype=torch.int32))
    d.guard.t.copy_(d.before)
    for g in graphs + graphs:
        g.replay()
    c.check("graph")
    d.check("grouped graph with new offsets")
    del graphs


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-1, 2, 3, 9], [0, 2, 3, 41], [4, 3, 2, 1],
                                     [0, 1 << 30, 1 << 30, 1 << 30], [0, 0, 0, -(1 << 31)]])
def test_bad_offsets_are_reported_and_nothing_is_written(lib, offsets):
    import torch
    c = Case(lib, 100, 40, 64, 64, offsets=[0, 0, 0, 40])
    c.off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    c.run()
    torch.cuda.synchronize()
    assert lib.workspace_status(c.ws) == lib.ERR_INVALID_ARG
    assert lib.workspace_status(c.ws) == lib.OK
    assert torch.equal(c.guard.t.view(torch.uint8), c.before.view(torch.uint8))
    c.guard.assert_intact()
    c.off = torch.tensor(c.offsets, dtype=torch.int32, device="cuda")
    c.run().check("after bad offsets")


@pytest.mark.parametrize("M,N", [(20, 256), (1900, 4096)], ids=["one-cta", "pair"])
def test_wait_timeout_is_reported_and_recoverable(lib, M, N):
    """A test word in the workspace makes one scale warp withhold its first
    arrival, so that the waits behind it run out of time: the call must report
    ERR_DEVICE_TIMEOUT and leave the context, and then the workspace, usable."""
    import time

    import torch
    c = Case(lib, 101, M, N, 512)
    torch.cuda.synchronize()
    c.ws.view(torch.int32)[7] = 1              # test_flags
    t0 = time.monotonic()
    c.run()
    diag = c.ws.view(torch.int32)[3:7].cpu().numpy()
    assert lib.workspace_status(c.ws) == lib.ERR_DEVICE_TIMEOUT
    assert time.monotonic() - t0 < 10
    assert 60 <= diag[0] <= 67
    lib.workspace_init(c.ws)
    c.run().check("after the timeout")


def test_a_block_of_the_framework(lib):
    """The products as a transformer block over the cache uses them: the
    chunk's activations quantized, projected to queries, keys and values in
    column ranges of one buffer, keys rotated into the cache, attention over
    it, the output projected onto the residual stream under a gate for each
    frame, then text and video rows through their own weights.  Each product is
    checked against float64 on what it was given."""
    import torch
    T, H, d, C = 96, 2, 128, 256
    rng = np.random.default_rng(8)
    f = np.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()
    ws = lib.new_matrix_workspace()

    def quantized(t, mode):
        q = lib.MatrixBuffer(t.shape[0], t.shape[1], mode)
        lib.quantize_matrix(t.contiguous(), q, ws)
        torch.cuda.synchronize()
        h = q.to_host()
        return q, dict(codes=h["codes"], scales=h["scales"], s=np.array([h["s"]], f),
                       tiles=mode == lib.TILES_2D)

    def checked(Y, x, w, bias, act, gate, res, K, what):
        y, mag = ref.reference(ref.decode(x), ref.decode(w), bias, act, gate, res)
        _assert_close(Y.float().cpu().numpy().astype(np.float64), y, mag, K,
                      Y.dtype == torch.bfloat16, what)

    x = rand(T, C)
    Wq, wq = quantized(rand(3 * H * d, C, scale=C ** -0.5), lib.TILES_2D)
    Wo, wo = quantized(rand(C, H * d, scale=(H * d) ** -0.5), lib.TILES_2D)
    X, xh = quantized(x, lib.BLOCKS_1D)
    bias = rng.standard_normal(3 * H * d).astype(f)
    qkv = torch.empty(T, 3 * H * d, dtype=torch.bfloat16, device="cuda")
    lib.matmul(X, Wq, qkv, ws, bias=_cuda(bias))
    checked(qkv, xh, wq, bias, "none", None, None, C, "projection")

    q, k, v = (qkv[:, i * H * d:(i + 1) * H * d].contiguous().view(T, H, d) for i in range(3))
    cache = lib.KVCache(1, H, T, 1, 0, 1)
    table = lib.RopeTable(3, 4, 8).fill(0)
    cache.append_rope(0, k, v, table)
    O = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda")
    cache.attention(0, lib.rope(q, table), O)

    A, ah = quantized(O.view(T, H * d), lib.BLOCKS_1D)
    gate = rng.standard_normal((3, C)).astype(f)
    stream = x.clone()
    lib.matmul(A, Wo, stream, ws, gate=_cuda(gate), rows_per_gate=32, residual=stream)
    checked(stream, ah, wo, None, "none", gate[np.arange(T) // 32],
            x.float().cpu().numpy().astype(np.float64), H * d, "output projection")

    Wg = lib.GroupedMatrixBuffer(2, 128, C, lib.TILES_2D)
    hosts = []
    for e in range(2):
        m = Wg.expert(e)
        lib.quantize_matrix(rand(128, C, scale=C ** -0.5), m, ws)
        torch.cuda.synchronize()
        h = m.to_host()
        hosts.append(dict(codes=h["codes"], scales=h["scales"], s=np.array([h["s"]], f), tiles=True))
    S, sh = quantized(stream, lib.BLOCKS_1D)
    up = torch.empty(T, 128, device="cuda")
    lib.grouped_matmul(S, Wg, _cuda(np.array([0, 20, T], np.int32)), up, ws,
                       activation=lib.ACT_GELU_TANH)
    for e, (a, b) in enumerate(((0, 20), (20, T))):
        part = dict(sh, codes=sh["codes"][a:b], scales=sh["scales"][a:b])
        checked(up[a:b], part, hosts[e], None, "gelu", None, None, C, f"group {e}")
    assert lib.workspace_status(ws) == lib.OK and cache.check_status() == lib.OK


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_a_nan_stays_with_its_value_through_the_activation(lib, act, bf16):
    """Values share a reciprocal in the activation: a NaN or infinite bias of one
    channel and a NaN scale of one row reach that channel and row only."""
    import torch
    c = Case(lib, 102, 40, 96, 64, bf16=bf16, act=act)
    c.dev["bias"][5], c.dev["bias"][50] = float("nan"), float("inf")
    c.X.scales[7, 1] = 0x7F                      # E4M3 NaN
    c.run()
    torch.cuda.synchronize()
    bad = torch.zeros(40, 96, dtype=torch.bool)
    bad[:, 5] = bad[:, 50] = True
    bad[7] = True
    assert torch.equal(~torch.isfinite(c.Y.float()).cpu(), bad)


def test_first_call_inside_a_capture(lib):
    """A process whose first product is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, sink_window_video_b200 as swv
X, W = swv.MatrixBuffer(300, 64, 1), swv.MatrixBuffer(4096, 64, 2)
X.scales.fill_(0x38); X.tensor_scale.fill_(1); X.codes.fill_(0x22)
W.scales.fill_(0x38); W.tensor_scale.fill_(1); W.codes.fill_(0x22)
Y = torch.zeros(300, 4096, device="cuda")
ws = swv.new_matrix_workspace()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    swv.matmul(X, W, Y, ws)
g.replay()
torch.cuda.synchronize()
assert bool((Y == 64).all()), Y
assert swv.workspace_status(ws) == 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
