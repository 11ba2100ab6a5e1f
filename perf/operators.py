"""Cases of the NVFP4 matrix products: the product of a quantized activation
matrix and a quantized weight matrix with bias, activation, gate and residual,
and the same product grouped by expert.

    Y = R + g * act(s_X s_W X W^T + b)

X [M][K] and W [N][K] are E2M1 codes under E4M3 block scales (16 elements along
k for X; the same, or 16 x 16 tiles, for W) and one FP32 tensor scale each.
"""
import math

import torch

own = False

BLOCKS_1D, TILES_2D = 1, 2
LARGEST = 7040 * 8192 * 2048        # products of the largest listed case

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _dense(name, M, N, K, **kw):
    c = dict(name=name, op="matmul", M=M, N=N, K=K, tiles=True, out="bf16", bias=True, act="none",
             gate=0, residual=False)
    c.update(kw)
    return c


def _grouped(name, T, E, N, K, **kw):
    c = dict(name=name, op="grouped", T=T, E=E, N=N, K=K, tiles=True, out="bf16", bias=True,
             act="none", gate=False, residual=False, skew=1.0, tail=0)
    c.update(kw)
    return c


def listed():
    return [
        # one row: a time embedding or a single token through a projection
        _dense("row", 1, 2048, 2048, act="silu"),
        # a prompt's rows through a text projection, fp32 out
        _dense("prompt", 77, 4096, 4096, out="f32"),
        # sizes that no tile divides, weights in row blocks, any number of columns
        _dense("odd", 333, 1001, 1056, tiles=False, out="f32", act="gelu", residual=True),
        # one latent frame (22 x 40 tokens) through an output projection: gate and residual
        _dense("frame", 880, 2048, 2048, gate=880, residual=True),
        # an 8-frame chunk through the first and the second product of an MLP; the second
        # adds onto an fp32 residual stream under a gate for each frame
        _dense("chunk up", 7040, 8192, 2048, act="gelu"),
        _dense("chunk down", 7040, 2048, 8192, out="f32", gate=880, residual=True),
        # a chunk's rows and a prompt's rows in one sequence, one set of weights for each
        _grouped("joint", 7266, 2, 2048, 2048, skew=40.0, residual=True, gate=True),
        # few rows over many experts, most of them empty: the weights' bytes count
        _grouped("experts few", 48, 64, 2048, 1024, act="silu"),
        # a batch over experts of uneven load, with rows behind the last group
        _grouped("experts up", 8192, 32, 4096, 2048, act="silu", skew=1.4, tail=100),
        _grouped("experts down", 8192, 32, 2048, 4096, out="f32", skew=1.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        tiles = rng.random() < 0.7
        N = _log(rng, 64, 8192)
        N = max(16, N // 16 * 16) if tiles else N
        K = _log(rng, 128, 8192) // 32 * 32
        M = _log(rng, 1, 8192)
        out = rng.choice(["bf16", "f32"])
        act = rng.choice(["none", "gelu", "silu"])
        common = dict(tiles=tiles, out=out, bias=rng.random() < 0.8, act=act,
                      residual=rng.random() < 0.5)
        if M * N * K > LARGEST:
            continue
        if rng.random() < 0.5:
            c = _dense("", M, N, K, gate=rng.choice([0, 0, M, max(1, M // 8), 880]), **common)
        else:
            E = _log(rng, 2, 64)
            if E * N * K > 32 * 4096 * 2048:
                continue
            c = _grouped("", M, E, N, K, gate=rng.random() < 0.3, skew=rng.uniform(1.0, 3.0),
                         tail=rng.choice([0, 0, M // 10]), **common)
        del c["name"]
        return c


# ------------------------------------------------------------------ inputs

def _quantize(x, tiles):
    """NVFP4 codes, block scales and tensor scale of fp32 [..., R, C]: the
    block's (or 16 x 16 tile's) largest magnitude is mapped to 6."""
    lead, (R, C) = x.shape[:-2], x.shape[-2:]
    s = x.abs().amax(dim=(-2, -1)) / 2688.0
    a = x.abs().unflatten(-1, (C // 16, 16)).amax(-1)
    if tiles:
        a = a.unflatten(-2, (R // 16, 16)).amax(-2)
    sb = (a / (6.0 * s[..., None, None])).to(torch.float8_e4m3fn)
    D = sb.float() * s[..., None, None]
    if tiles:
        D = D.repeat_interleave(16, dim=-2)
    q = x.abs() / D.repeat_interleave(16, dim=-1).clamp_min(1e-30)
    code = (x < 0).to(torch.uint8) << 3
    for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += (q > t).to(torch.uint8)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    return codes.contiguous(), sb.view(torch.uint8).contiguous(), s.reshape(lead or (1,)).contiguous()


def _sizes(T, E, skew, tail, g):
    """Rows of each group: T - tail rows over E groups whose shares differ by
    about exp(log(skew) * normal), as device offsets [E + 1] and the largest."""
    w = torch.exp(math.log(max(skew, 1.0)) * torch.randn(E, generator=g, device="cuda"))
    ends = torch.round(torch.cumsum(w.double(), 0) / w.double().sum() * (T - tail))
    off = torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), ends]).to(torch.int32)
    if T - tail < 4 * E:      # few rows: each row's group is drawn
        ids = torch.randint(0, E, (T - tail,), generator=g, device="cuda")
        off[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0).to(torch.int32)
    return off, int((off[1:] - off[:-1]).max())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    grouped = case["op"] == "grouped"
    M, N, K = case["T"] if grouped else case["M"], case["N"], case["K"]
    E = case["E"] if grouped else 0
    dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # activations: channels of different spread, as after a normalisation's weight
    x = randn(M, K) * torch.exp(0.5 * randn(K))
    w = randn(*((E, N, K) if grouped else (N, K))) / math.sqrt(K)
    st = dict(case=case, x=_quantize(x, False), w=_quantize(w, case["tiles"]))
    del x, w
    lead = (E, N) if grouped else (N,)
    st["bias"] = 0.5 * randn(*lead) if case["bias"] else None
    st["gate"] = None
    if case["gate"]:
        st["gate"] = randn(E, N) if grouped else randn(-(-M // case["gate"]), N)
    st["residual"] = randn(M, N).to(dt) if case["residual"] else None
    st["Y"] = randn(M, N).to(dt)
    if grouped:
        st["offsets"], st["most"] = _sizes(M, E, case["skew"], case["tail"], g)
    if own:
        import sink_window_video_b200 as swv
        mode = swv.TILES_2D if case["tiles"] else swv.BLOCKS_1D
        st["X"] = swv.MatrixBuffer(M, K, swv.BLOCKS_1D, parts=st["x"])
        st["W"] = swv.GroupedMatrixBuffer(E, N, K, mode, parts=st["w"]) if grouped else \
            swv.MatrixBuffer(N, K, mode, parts=st["w"])
        st["ws"] = swv.new_matrix_workspace()
        st["act"] = {"none": swv.ACT_NONE, "gelu": swv.ACT_GELU_TANH,
                     "silu": swv.ACT_SILU}[case["act"]]
    return st


# ------------------------------------------------------------------ one pass

def _decode(q, tiles):
    """fp32 values of (codes, block scales, tensor scale)."""
    codes, sb, s = q
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = table[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).int()]
    b = sb.view(torch.float8_e4m3fn).float().repeat_interleave(16, dim=-1)
    if tiles:
        b = b.repeat_interleave(16, dim=-2)
    s = s[:, None, None] if codes.dim() == 3 else s
    return v * (b * s)


def _act(z, act):
    if act == "gelu":
        u = 0.7978845608028654 * (z + 0.044715 * z * z * z)
        return 0.5 * z * (1.0 + torch.tanh(u))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def run(st):
    case = st["case"]
    if own:
        import sink_window_video_b200 as swv
        if case["op"] == "grouped":
            swv.grouped_matmul(st["X"], st["W"], st["offsets"], st["Y"], st["ws"], bias=st["bias"],
                               activation=st["act"], gate=st["gate"], residual=st["residual"])
        else:
            swv.matmul(st["X"], st["W"], st["Y"], st["ws"], bias=st["bias"], activation=st["act"],
                       gate=st["gate"], rows_per_gate=case["gate"], residual=st["residual"])
        return st["Y"]
    x, w, Y = _decode(st["x"], False), _decode(st["w"], case["tiles"]), st["Y"]
    M = x.shape[0]
    rows = torch.arange(M, device="cuda")
    if case["op"] == "grouped":
        # each group's rows in a batch of equal length, the spare places at row 0
        off = st["offsets"].long()
        e = torch.searchsorted(off[1:], rows, right=True).clamp_max(case["E"] - 1)
        at = off[:-1, None] + torch.arange(st["most"], device="cuda")
        z = torch.bmm(x[at.clamp_max(M - 1)], w.transpose(1, 2))
        z = z[e, (rows - off[e]).clamp(0, st["most"] - 1)]
        inside = ((rows >= off[0]) & (rows < off[-1]))[:, None]
    else:
        z, e, inside = x @ w.T, None, None
    if st["bias"] is not None:
        z = z + (st["bias"] if e is None else st["bias"][e])
    z = _act(z, case["act"])
    if st["gate"] is not None:
        z = z * st["gate"][rows // case["gate"] if e is None else e]
    if st["residual"] is not None:
        z = z + st["residual"].float()
    z = z.to(Y.dtype)
    return z if inside is None else torch.where(inside, z, Y)


def work(case):
    grouped = case["op"] == "grouped"
    M, N, K = case["T"] - case["tail"] if grouped else case["M"], case["N"], case["K"]
    size = 2 if case["out"] == "bf16" else 4
    # experts without rows are not read: expected number of those that have some
    E, G = 1, -(-M // case["gate"]) if not grouped and case["gate"] else 1
    if grouped:
        E = case["E"]
        E = E * (1.0 - (1.0 - 1.0 / E) ** M) if M < 4 * E else E
        G = E
    block = 256 if case["tiles"] else 16
    by = M * K * 9 / 16 + E * N * K * (0.5 + 1 / block) + M * N * size
    by += M * N * size * bool(case["residual"])
    by += 4 * N * (E * bool(case["bias"]) + G * bool(case["gate"]))
    return {"bytes": by, "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------ 64 bits

def _exact_matrix(codes, sb, s, tiles):
    """float64 values: E2M1 as (1 + m/2) 2^(e-1), m/2 for e = 0; E4M3 as
    (1 + m/8) 2^(e-7), m/8 2^-6 for e = 0."""
    R, C = codes.shape[0], 2 * codes.shape[1]
    c = torch.empty((R, C), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        q = (codes >> (4 * half)) & 15
        e, m = ((q >> 1) & 3).double(), (q & 1).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
        c[:, half::2] = torch.where(q >= 8, -v, v)
    e, m = ((sb >> 3) & 15).double(), (sb & 7).double()
    b = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    c = c.view(R // 16, 16, C // 16, 16) * b.view(R // 16, 1, C // 16, 1) if tiles else \
        c.view(R, C // 16, 16) * b.view(R, C // 16, 1)
    return c.view(R, C) * s.double()


def exact(case, seed):
    st = prepare(case, seed)
    grouped = case["op"] == "grouped"
    X = _exact_matrix(*st["x"], False)
    Y = st["Y"].double()
    off = st["offsets"].tolist() if grouped else [0, X.shape[0]]
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        W = _exact_matrix(*((p[e] for p in st["w"]) if grouped else st["w"]), case["tiles"])
        z = X[a:b] @ W.T
        if st["bias"] is not None:
            z += st["bias"][e] if grouped else st["bias"]
        if case["act"] == "gelu":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        if st["gate"] is not None:
            z *= st["gate"][e].double() if grouped else \
                st["gate"].double().repeat_interleave(case["gate"], 0)[:b]
        if st["residual"] is not None:
            z += st["residual"][a:b].double()
        Y[a:b] = z
    return Y
