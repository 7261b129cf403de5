"""GPU parity of the operators without a context with the fp64 oracle:
MXFP4 conversion and grouping exactly, products and the combine within bounds
that follow from fp32 accumulation.

Bounds.  A sum of K exact products (bf16 and e2m1 * 2^k products are exact in
fp32) accumulated in fp32 in any order is off by at most (K - 1) ulps of the
magnitude sum; with 2^-23 an addition may also truncate: K * 2^-23 * sum|x w|.
A bf16 result adds half a step, 2^-8 of the value.  GLU: |silu'| <= 1.1, and the
SiLU itself costs at most (2|g| + 8) * 2^-24 (argument scaling, exp, sum,
quotient, product), below 1.3e-5 for |g| <= 100, where exp(-g) leaves fp32."""
import numpy as np
import pytest

from oracle import ops as OO
from tests.harness import log

pytestmark = pytest.mark.gpu

FORMATS = ["bf16-bf16", "bf16-mxfp4", "mxfp4-mxfp4"]


@pytest.fixture(scope="module")
def t():
    import torch
    return torch


@pytest.fixture(scope="module")
def B():
    import routed_expert_execution_moe_amd as B
    return B


def _dev(t, a, dtype=None):
    x = t.from_numpy(np.ascontiguousarray(a)).cuda()
    return x if dtype is None else x.to(dtype)


def _bf16(t, rng, shape, sigma=1.0):
    return _dev(t, (rng.standard_normal(shape) * sigma).astype(np.float32), t.bfloat16)


def _np(x):
    return x.double().cpu().numpy()


class Operand:
    """Rows in bf16 or MXFP4 on the device, and their fp64 values."""

    def __init__(self, t, rng, rows, K, fmt, sigma=1.0, ld=None):
        self.scales = None
        if fmt == "bf16":
            buf = _bf16(t, rng, (rows, ld or K), sigma)
            self.t = buf[:, :K]
            self.v = _np(self.t)
        else:
            c, s = OO.mx_quantize(rng.standard_normal((rows, K)) * sigma)
            self.t, self.scales = _dev(t, c), _dev(t, s)
            self.v = OO.mx_values(c, s)


class Experts:
    def __init__(self, t, rng, E, N, K, fmt, sigma=0.05):
        m = Operand(t, rng, E * N, K, fmt, sigma)
        self.t = m.t.reshape(E, N, -1)
        self.scales = None if m.scales is None else m.scales.reshape(E, N, -1)
        self.v = m.v.reshape(E, N, K)

    def __call__(self, e):
        return self.v[e]


def _close(y, want, bound, bf16, what):
    y = _np(y)
    tol = bound + (2.0 ** -8 * (np.abs(want) + bound) if bf16 else 2.0 ** -24 * np.abs(want))
    bad = ~(np.abs(y - want) <= tol + 1e-36)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), y[bad][:4], want[bad][:4])


def _bound(size, want, K, glu):
    b = K * 2.0 ** -23 * size
    return b + 2e-5 * np.abs(want) if glu else b


# ------------------------------------------------------------------ MXFP4
QUANT = [(1, 32), (1, 2048), (3, 96), (8, 2048), (257, 4128), (1000, 64)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,C", QUANT)
def test_quantize_and_back(t, B, R, C, dtype):
    """Codes, scales and values bit for bit: exponents from subnormal to the
    largest, zero blocks, borders of the grid, infinities and NaN."""
    log(f"quantize {R}x{C} {dtype}")
    rng = np.random.default_rng(R * 7919 + C)
    x = rng.standard_normal((R, C)) * np.exp2(rng.integers(-150, 126, (R, 1)))
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.75])
    pick = rng.random((R, C)) < 0.3
    x = np.where(pick, rng.choice(grid, (R, C)) * rng.choice([-1, 1], (R, C)) * np.exp2(rng.integers(-30, 30, (R, 1))), x)
    x.reshape(R, -1, 32)[rng.random((R, C // 32)) < 0.1] = 0
    x.reshape(R, -1, 32)[rng.random((R, C // 32)) < 0.05] = -0.0
    if R > 2:
        x[1, 7], x[2, 33 % C], x[0, C - 1] = np.inf, np.nan, -np.inf
    with np.errstate(over="ignore"):
        xd = _dev(t, x.astype(np.float32), getattr(t, dtype))
    want_c, want_s = OO.mx_quantize(_np(xd))
    codes = t.full((R, C // 2), 77, dtype=t.uint8, device="cuda")
    scales = t.full((R, C // 32), 77, dtype=t.uint8, device="cuda")
    B.moe_mx_quantize(xd, codes, scales)
    y = t.full((R, C), 3.0, dtype=xd.dtype, device="cuda")
    B.moe_mx_dequantize(codes, scales, y)
    t.cuda.synchronize()
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(_np(y), OO.mx_values(want_c, want_s), equal_nan=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_dequantize_every_code_and_scale(t, B, dtype):
    log(f"dequantize all {dtype}")
    codes = np.tile((np.arange(16) * 17 % 256).astype(np.uint8), (1, 256))  # each block: all 16 codes, both nibbles
    codes = np.concatenate([codes, codes[:, ::-1]])
    scales = np.stack([np.arange(256), np.arange(256)[::-1]]).astype(np.uint8)
    want = OO.mx_values(codes, scales)
    with np.errstate(invalid="ignore"):
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
    for ld in (8192, 8192 + 16, 8192 + 3):  # rows aligned for wide stores, and not
        buf = t.full((2, ld), 5.0, dtype=getattr(t, dtype), device="cuda")
        B.moe_mx_dequantize(_dev(t, codes), _dev(t, scales), buf[:, :8192])
        t.cuda.synchronize()
        assert np.array_equal(_np(buf[:, :8192]), want, equal_nan=True), ld
        assert bool((buf[:, 8192:] == 5).all())
    buf = t.zeros(2 * 8192 + 8, dtype=getattr(t, dtype), device="cuda")
    y = buf[1:1 + 2 * 8192].view(2, 8192)  # element-aligned only
    B.moe_mx_dequantize(_dev(t, codes), _dev(t, scales), y)
    assert np.array_equal(_np(y), want, equal_nan=True)


def test_quantize_strided_rows(t, B):
    log("quantize strided")
    rng = np.random.default_rng(5)
    buf = _bf16(t, rng, (37, 512))
    x = buf[:, 64:64 + 160]
    codes = t.empty((37, 80), dtype=t.uint8, device="cuda")
    scales = t.empty((37, 5), dtype=t.uint8, device="cuda")
    B.moe_mx_quantize(x, codes, scales)
    want = OO.mx_quantize(_np(x))
    assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    with pytest.raises(B.MoertError):
        B.moe_mx_quantize(buf[:, 1:161], codes, scales)  # rows not 16-byte aligned


def test_quantize_past_32_bits(t, B):
    """More than 2^32 bytes of x and of y, more rows than a grid dimension."""
    log("quantize past 32 bits")
    R, C = 70001, 32768
    x = t.zeros((R, C), dtype=t.bfloat16, device="cuda")
    rows = [0, 1, 32767, 65535, 65536, 65537, R - 1]
    rng = np.random.default_rng(9)
    part = _bf16(t, rng, (len(rows), C))
    x[rows] = part
    codes = t.full((R, C // 2), 9, dtype=t.uint8, device="cuda")
    scales = t.full((R, C // 32), 9, dtype=t.uint8, device="cuda")
    B.moe_mx_quantize(x, codes, scales)
    x.fill_(1.0)
    B.moe_mx_dequantize(codes, scales, x)
    want = OO.mx_quantize(_np(part))
    assert np.array_equal(codes[rows].cpu().numpy(), want[0]) and np.array_equal(scales[rows].cpu().numpy(), want[1])
    assert np.array_equal(_np(x[rows]), OO.mx_values(*want))
    rest = t.ones(R, dtype=t.bool, device="cuda")
    rest[rows] = False
    assert int((scales != 127).any(1)[rest].sum()) == 0 and int((x != 0).any(1)[rest].sum()) == 0


# ------------------------------------------------------------------ dense product
GEMM = [  # M, N, K
    (1, 1, 32), (1, 17, 64), (1, 256, 1024), (2, 130, 160), (5, 64, 2080), (16, 48, 96), (17, 33, 128),
    (33, 100, 544), (64, 256, 512), (65, 257, 288), (129, 130, 256), (200, 96, 1056), (256, 512, 128),
    (300, 515, 320), (513, 264, 192),
]


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("out", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,N,K", GEMM)
def test_mx_gemm(t, B, M, N, K, act, out):
    log(f"gemm {M}x{N}x{K} {act} {out}")
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    x, w = Operand(t, rng, M, K, act), Operand(t, rng, N, K, "mxfp4", 0.05)
    y = t.full((M, N), 7.0, dtype=getattr(t, out), device="cuda")
    B.moe_mx_gemm(x.t, w.t, w.scales, y, x_scales=x.scales)
    t.cuda.synchronize()
    want, size = x.v @ w.v.T, np.abs(x.v) @ np.abs(w.v).T
    _close(y, want, _bound(size, want, K, False), out == "bfloat16", (M, N, K))


GEMM_TILES = [  # enough tiles for each of the LDS variants; ends inside steps and scale chunks
    (500, 1100, 544), (500, 1100, 1600), (129, 4100, 2080),      # 64 x 128 tiles, one per CU
    (1500, 1500, 672), (1090, 2050, 2112),                      # 64 x 128 tiles, several per CU
    (1800, 4100, 544), (1793, 4353, 1568), (1900, 4000, 4192),  # 128 x 128 tiles, two per CU
    (4100, 4097, 544), (4353, 3900, 1696), (3850, 4352, 4128),  # and more
    (2050, 4100, 544), (2049, 4353, 1568), (2300, 4000, 4192),  # 256 x 256 tiles (bf16 x MXFP4 128 x 128)
    (3900, 4050, 544), (3841, 4081, 1696), (4090, 3900, 4128),  # 256 x 256 tiles, one for every CU
    # rows of less than 16 scales
    (500, 1100, 480), (1500, 1500, 32), (2050, 4100, 96), (2100, 4000, 416), (4100, 4097, 256), (4200, 4100, 480),
    (3900, 4050, 256), (4000, 4081, 480),
]


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M,N,K", GEMM_TILES)
def test_mx_gemm_tiles(t, B, M, N, K, act):
    log(f"gemm tiles {M}x{N}x{K} {act}")
    rng = np.random.default_rng(M + N + K)
    x, w = Operand(t, rng, M, K, act), Operand(t, rng, N, K, "mxfp4", 0.05)
    if act == "mxfp4":
        x.scales[5, -1] = 255  # the last block of a row: its steps end right behind it
    w.scales[7, -1] = 255
    want = t.from_numpy(x.v).cuda() @ t.from_numpy(w.v).cuda().T
    size = t.from_numpy(np.abs(x.v)).cuda() @ t.from_numpy(np.abs(w.v)).cuda().T
    for out in (t.float32, t.bfloat16):
        y = t.full((M, N + 5), 7.0, dtype=out, device="cuda")
        B.moe_mx_gemm(x.t, w.t, w.scales, y[:, :N], x_scales=x.scales)
        t.cuda.synchronize()
        tol = K * 2.0 ** -23 * size + (2.0 ** -8 * (want.abs() + K * 2.0 ** -23 * size) if out == t.bfloat16 else 2.0 ** -24 * want.abs())
        bad = ~((y[:, :N].double() - want).abs() <= tol)
        nan = t.zeros_like(bad)
        nan[:, 7] = True
        if act == "mxfp4":
            nan[5] = True
        assert bool((y[:, :N].isnan() == nan).all())
        assert not bool((bad & ~nan).any()), t.nonzero(bad & ~nan)[:4].tolist()
        assert bool((y[:, N:] == 7).all())


@pytest.mark.parametrize("M", [3, 150])
def test_mx_gemm_strides_and_alignment(t, B, M):
    """x rows inside a wider buffer; y rows of odd stride at an odd element;
    what lies between them stays as it was."""
    log(f"gemm strides M={M}")
    rng = np.random.default_rng(M)
    N, K = 101, 160
    x, w = Operand(t, rng, M, K, "bf16", ld=K + 40), Operand(t, rng, N, K, "mxfp4", 0.05)
    assert x.t.stride(0) == K + 40
    want, size = x.v @ w.v.T, np.abs(x.v) @ np.abs(w.v).T
    for dt in (t.float32, t.bfloat16):
        buf = t.full((M * (N + 6) + 3,), 7.0, dtype=dt, device="cuda")
        y = t.as_strided(buf, (M, N), (N + 6, 1), 1)
        B.moe_mx_gemm(x.t, w.t, w.scales, y)
        t.cuda.synchronize()
        _close(y, want, _bound(size, want, K, False), dt == t.bfloat16, M)
        keep = t.ones_like(buf, dtype=t.bool)
        t.as_strided(keep, (M, N), (N + 6, 1), 1).fill_(False)
        assert bool((buf[keep] == 7).all())


def test_mx_gemm_special_values(t, B):
    """A NaN scale makes exactly its row or column NaN; infinite x rows stay
    in their rows; extreme scales multiply exactly."""
    log("gemm special")
    rng = np.random.default_rng(2)
    for M in (4, 140):
        N, K = 70, 128
        x, w = Operand(t, rng, M, K, "mxfp4"), Operand(t, rng, N, K, "mxfp4")
        w.t |= 1  # no zero codes: 0 * NaN would hide nothing, but 0 * inf is NaN too
        ws, xs = w.scales.clone(), x.scales.clone()
        ws[3, 1], xs[2, 3] = 255, 255
        y = t.zeros((M, N), device="cuda")
        B.moe_mx_gemm(x.t, w.t, ws, y, x_scales=xs)
        nan = t.zeros((M, N), dtype=t.bool, device="cuda")
        nan[:, 3] = True
        nan[2, :] = True
        assert bool((y.isnan() == nan).all())
        xb = _bf16(t, rng, (M, K))
        xb[1, 5] = float("inf")
        B.moe_mx_gemm(xb, w.t, ws, y)
        assert bool(y[:, 3].isnan().all()) and not bool(y[0, :3].isnan().any())
        assert not bool(y[1, :3].isfinite().any()) and bool(y[2:, 4:].isfinite().all())
        w2, x2 = t.full((N, K // 2), 0x22, dtype=t.uint8, device="cuda"), t.full((M, K // 2), 0x22, dtype=t.uint8, device="cuda")
        s1, s2 = t.full((N, K // 32), 254, dtype=t.uint8, device="cuda"), t.full((M, K // 32), 3, dtype=t.uint8, device="cuda")
        B.moe_mx_gemm(x2, w2, s1, y, x_scales=s2)
        assert bool((y == K * 2.0 ** 3).all())


# ------------------------------------------------------------------ grouping
def _ids(rng, T, k, E, pad=0, wild=False):
    p = 1.0 / (1 + np.arange(E))
    ids = np.argsort(-(np.log(p) + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
    if k > E:
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if pad:
        ids[T - pad:] = -1
    if wild:
        m = rng.random(ids.shape) < 0.2
        ids = np.where(m, rng.choice([-1, -2 ** 31, E, E + 1, 2 ** 31 - 1], ids.shape), ids).astype(np.int32)
    return ids


GROUP = [  # T, k, E
    (1, 1, 1), (1, 8, 128), (8, 8, 128), (7, 3, 1024), (512, 8, 256), (513, 8, 256), (4097, 1, 8), (1000, 6, 60),
    (8192, 8, 256), (3001, 8, 1024), (2048, 2, 1),
]


@pytest.mark.parametrize("T,k,E", GROUP)
def test_group_pairs(t, B, T, k, E):
    rng = np.random.default_rng(T + k + E)
    for case in range(4):
        log(f"group {T}x{k} E={E} case {case}")
        ids = _ids(rng, T, k, E, pad=T // 3 if case == 1 else 0, wild=case == 2)
        if case == 3:
            ids[:] = E // 2 if T % 2 else -1  # one expert, or none at all
        want = OO.group_pairs(ids, E)
        off = t.full((E + 1,), 5, dtype=t.int32, device="cuda")
        perm = t.full((T * k,), 5, dtype=t.int32, device="cuda")
        n = B.moe_group_workspace(T, k, E)
        ws = t.empty(n, dtype=t.uint8, device="cuda") if n else None
        B.moe_group_pairs(_dev(t, ids), E, off, perm, workspace=ws)
        t.cuda.synchronize()
        assert np.array_equal(off.cpu().numpy(), want[0])
        assert np.array_equal(perm.cpu().numpy(), want[1])


def test_group_no_pairs(t, B):
    off = t.full((5,), 9, dtype=t.int32, device="cuda")
    B.moe_group_pairs(t.empty((0, 4), dtype=t.int32, device="cuda"), 4, off, t.empty(0, dtype=t.int32, device="cuda"))
    assert off.tolist() == [0] * 5


# ------------------------------------------------------------------ grouped product
def _grouped(t, B, x, w, off, n_rows, N, out, x_index=None, div=1, y_index=None, n_y=None, glu=False, ld=0):
    cols = N // 2 if glu else N
    buf = t.full((n_y or n_rows, cols + ld), 7.0, dtype=getattr(t, out), device="cuda")
    y = buf[:, :cols]
    idx = [None if i is None else _dev(t, np.asarray(i, np.int32)) for i in (x_index, y_index)]
    B.moe_grouped_gemm(x.t, w.t, _dev(t, np.asarray(off, np.int32)), y, x_scales=x.scales, w_scales=w.scales,
                       x_index=idx[0], x_index_div=div, y_index=idx[1], glu=glu)
    t.cuda.synchronize()
    assert bool((buf[:, cols:] == 7).all())
    return y


GROUPED = [  # T, k, E, N, K
    (1, 1, 1, 2, 32), (1, 8, 16, 64, 128), (1, 2, 8, 1536, 256), (8, 8, 128, 96, 160), (20, 4, 6, 34, 96),
    (64, 8, 16, 130, 192), (100, 3, 5, 258, 64), (300, 4, 8, 300, 320), (520, 2, 3, 512, 128), (700, 1, 2, 66, 544),
    (256, 8, 1000, 32, 32),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K", GROUPED)
def test_grouped_up_and_down(t, B, T, k, E, N, K, fmt):
    """Gate/up with gathered token rows, down with rows scattered to pairs,
    experts without a row among them, padded pairs left out."""
    act, wt = fmt.split("-")
    rng = np.random.default_rng(T * 5 + E + K)
    ids = _ids(rng, T, k, E, pad=T // 5)
    off, perm = OO.group_pairs(ids, E)
    R = T * k
    w = Experts(t, rng, E, N, K, wt)
    x = Operand(t, rng, T, K, act)
    h = Operand(t, rng, R, K, act)
    for out in ("float32", "bfloat16"):
        for glu in (True, False):
            log(f"grouped T={T} k={k} E={E} N={N} K={K} {fmt} {out} glu={glu}")
            want, size = OO.grouped_rows(x.v, w, off, R, N, perm, k, glu)
            y = _grouped(t, B, x, w, off, R, N, out, x_index=perm, div=k, glu=glu, ld=3)
            n = off[-1]
            _close(y[:n], want[:n], _bound(size, want, K, glu)[:n], out == "bfloat16", "up")
            assert bool((y[n:] == 7).all())
        want, size = OO.grouped_rows(h.v, w, off, R, N)
        y = _grouped(t, B, h, w, off, R, N, out, y_index=perm)
        live = perm[:n]
        _close(y[_dev(t, live.astype(np.int64))], want[:n], _bound(size, want, K, False)[:n], out == "bfloat16", "down")
        dead = np.setdiff1d(np.arange(R), live)
        assert bool((y[_dev(t, dead)] == 7).all())


GROUPED_TILES = [  # T, k, E, N, K, glu
    (260, 4, 16, 1538, 544, True), (260, 4, 16, 1538, 544, False), (90, 8, 60, 2050, 1120, False),
    (1500, 2, 5, 2050, 1568, True), (1500, 2, 5, 4098, 544, False), (3001, 3, 6, 1026, 2080, True),
    (1000, 2, 4, 4098, 1568, False), (2000, 2, 4, 4098, 2080, False),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K,glu", GROUPED_TILES)
def test_grouped_tiles(t, B, T, k, E, N, K, glu, fmt):
    """The LDS variants on ragged groups, odd columns, a row of x that no
    position may mix with and positions without a source; compared on the GPU in
    fp64."""
    log(f"grouped tiles T={T} k={k} E={E} N={N} K={K} glu={glu} {fmt}")
    act, wt = fmt.split("-")
    rng = np.random.default_rng(T + N + K)
    ids = _ids(rng, T, k, E, pad=T // 9)
    ids[ids == 1] = 2  # an expert without rows
    off, perm = OO.group_pairs(ids, E)
    R, n = T * k, int(off[-1])
    w, x = Experts(t, rng, E, N, K, wt), Operand(t, rng, T, K, act)
    index = perm.copy()
    index[3:n:41] = -1
    cols = N // 2 if glu else N
    xv = t.from_numpy(x.v).cuda()
    want, size = t.zeros(R, cols, dtype=t.float64, device="cuda"), t.zeros(R, cols, dtype=t.float64, device="cuda")
    for e in range(E):
        p = np.arange(off[e], off[e + 1])
        if len(p):
            a = xv[_dev(t, np.maximum(index[p], 0) // k)] * _dev(t, (index[p] >= 0).astype(np.float64))[:, None]
            we = t.from_numpy(w(e)).cuda()
            z, m = a @ we.T, a.abs() @ we.abs().T
            if glu:
                g, u, mg, mu = z[:, :cols], z[:, cols:], m[:, :cols], m[:, cols:]
                s = g * t.sigmoid(g)
                z, m = s * u, 1.1 * mg * u.abs() + s.abs() * mu + 1e-3 * mg * mu
            want[off[e]:off[e + 1]], size[off[e]:off[e + 1]] = z, m
    tol = K * 2.0 ** -23 * size + (2e-5 * want.abs() if glu else 0)
    for out in ("float32", "bfloat16"):
        y = _grouped(t, B, x, w, off, R, N, out, x_index=index, div=k, glu=glu)
        half = 2.0 ** -8 if out == "bfloat16" else 2.0 ** -24
        bad = ~((y.double() - want).abs() <= tol + half * (want.abs() + tol))
        assert not bool(bad[:n].any()), t.nonzero(bad[:n])[:4].tolist()
        assert bool((y[n:] == 7).all()) and bool((y[3:n:41] == 0).all())


def test_grouped_bf16_k_of_eights(t, B):
    """bf16 products take any K that is a multiple of 8."""
    rng = np.random.default_rng(11)
    for K in (8, 24, 40, 136, 1000):
        for off in ([0, 5, 5, 9], [0, 300, 301, 450]):
            log(f"grouped bf16 K={K} {off}")
            R, N = off[-1], 70
            x, w = Operand(t, rng, R, K, "bf16"), Experts(t, rng, 3, N, K, "bf16")
            want, size = OO.grouped_rows(x.v, w, off, R, N)
            y = _grouped(t, B, x, w, off, R, N, "float32")
            _close(y, want, _bound(size, want, K, False), False, K)
    for K in (8, 40, 72):  # tiles whose only steps end inside
        for R, N in ((700, 1100), (1300, 4100), (3300, 6700)):
            log(f"grouped bf16 tiles K={K} R={R} N={N}")
            off = [0, R // 2, R // 2, R]
            x, w = Operand(t, rng, R, K, "bf16"), Experts(t, rng, 3, N, K, "bf16")
            want, size = OO.grouped_rows(x.v, w, off, R, N)
            _close(_grouped(t, B, x, w, off, R, N, "float32"), want, _bound(size, want, K, False), False, K)


@pytest.mark.parametrize("fmt", FORMATS)
def test_grouped_bad_indices_and_offsets(t, B, fmt):
    """Indices out of range read zeros or write nothing; positions outside
    the offsets, and rows no position names, stay as they were; offsets that do
    not ascend write no row out of range."""
    act, wt = fmt.split("-")
    rng = np.random.default_rng(4)
    for R, E in ((40, 5), (900, 3)):
        log(f"grouped bad indices {fmt} R={R}")
        N, K = 66, 96
        x, w = Operand(t, rng, 20, K, act), Experts(t, rng, E, N, K, wt)
        xi = rng.integers(0, 40, R)
        xi[::7], xi[3::11], xi[5::13] = -1, 40, 2 ** 31 - 1
        xi[6::17] = -2 ** 31
        yi = rng.permutation(R + 5)[:R]
        yi[2::9], yi[4::15], yi[5::19] = -1, R + 5, 2 ** 31 - 1
        off = np.concatenate([[2], np.sort(rng.integers(2, R - 3, E - 1)), [R - 3]])
        want, size = OO.grouped_rows(x.v, w, off, R, N, xi, 2)
        y = _grouped(t, B, x, w, off, R, N, "float32", x_index=xi, div=2, y_index=yi, n_y=R + 5)
        full, tol = np.full((R + 5, N), 7.0), np.zeros((R + 5, N))
        for p in range(2, R - 3):
            if 0 <= yi[p] < R + 5:
                full[yi[p]] = want[p]
                tol[yi[p]] = _bound(size, want, K, False)[p]
        _close(y, full, tol, False, fmt)
        h = Operand(t, rng, R, K, act)
        for bad in ([R] + [0] * E, [-5] + [R + 9] * E, [0, 2 ** 31 - 1] + [-2 ** 31] * (E - 1)):
            y = _grouped(t, B, h, w, bad, R, N, "float32", n_y=R + 64)
            assert bool((y[R:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("glu", [True, False])
def test_grouped_overlapping_offsets(t, B, fmt, glu):
    """Every expert claims all positions, in calls of each variant's size: many
    more tiles than the launch has workgroups.  Rows are unspecified; nothing
    outside the positions' rows is written."""
    act, wt = fmt.split("-")
    rng = np.random.default_rng(14)
    for E, R, N, K in ((1024, 60, 34, 512), (300, 3000, 260, 512), (7, 3000, 4100, 512), (3, 2900, 5000, 512)):
        log(f"grouped overlapping {fmt} E={E} R={R} N={N} glu={glu}")
        x, w = Operand(t, rng, R, K, act), Experts(t, rng, 1, N, K, wt)
        w.t = w.t.expand(E, -1, -1)
        if w.scales is not None:
            w.scales = w.scales.expand(E, -1, -1)
        off = np.tile([0, R], E)[:E + 1]
        y = _grouped(t, B, x, w, off, R, N, "bfloat16", n_y=R + 300, glu=glu)
        assert bool((y[R:] == 7).all())
        y = _grouped(t, B, x, w, [0] + [R] * E, R, N, "bfloat16", n_y=R + 300, glu=glu)  # all of it the first one's
        want, size = OO.grouped_rows(x.v[:50], lambda e: w.v[0], [0, 50], 50, N, glu=glu)
        _close(y[:50], want, _bound(size, want, K, glu), True, E)
        assert bool((y[R:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_grouped_rows_do_not_mix(t, B, fmt):
    """NaN weights of an expert without rows, and NaN rows of x outside the
    positions or of another expert, reach no other row."""
    log(f"grouped rows do not mix {fmt}")
    act, wt = fmt.split("-")
    rng = np.random.default_rng(8)
    for off in ([0, 5, 5, 9, 12], [0, 130, 130, 400, 420]):
        R, N, K = off[-1] + 4, 34, 96
        x, w = Operand(t, rng, R, K, act), Experts(t, rng, 4, N, K, wt)
        want, size = OO.grouped_rows(x.v, w, off, R, N)
        poison = list(range(off[1], off[3])) + list(range(off[-1], R))
        if w.scales is None:
            w.t[1] = float("nan")
        else:
            w.scales[1] = 255
        if x.scales is None:
            x.t[poison] = float("nan")
        else:
            x.scales[poison] = 255
        y = _grouped(t, B, x, w, off, R, N, "float32")
        for lo, hi in ((0, off[1]), (off[3], off[4])):
            _close(y[lo:hi], want[lo:hi], _bound(size, want, K, False)[lo:hi], False, fmt)
        assert bool(y[off[1]:off[3]].isnan().all()) and bool((y[off[-1]:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_grouped_past_32_bits(t, B, fmt):
    """Experts, rows of x (without an index) and rows of y beyond 2^32 bytes."""
    log(f"grouped past 32 bits {fmt}")
    act, wt = fmt.split("-")
    rng = np.random.default_rng(6)
    E, N, K = 3, 64, 64
    w = Experts(t, rng, E, N, K, wt)
    gap = (3 << 30) // w.t.element_size()
    big = t.empty((E - 1) * gap + w.t[0].numel(), dtype=w.t.dtype, device="cuda")
    wide = t.as_strided(big, w.t.shape, (gap, w.t.stride(1), 1))
    wide.copy_(w.t)
    w.t = wide
    for off in ([0, 3, 8, 12], [0, 100, 250, 700]):
        R = off[-1]
        ldy = (5 << 30) // 4 // R
        y = t.as_strided(t.empty(R * ldy, device="cuda"), (R, N), (ldy, 1))
        x = Operand(t, rng, R, K, act)
        if act == "bf16":
            ldx = (5 << 30) // 2 // R // 8 * 8
            xb = t.as_strided(t.empty(R * ldx, dtype=t.bfloat16, device="cuda"), (R, K), (ldx, 1))
            xb.copy_(x.t)
            x.t = xb
        want, size = OO.grouped_rows(x.v, w, off, R, N)
        B.moe_grouped_gemm(x.t, w.t, _dev(t, np.asarray(off, np.int32)), y, x_scales=x.scales, w_scales=w.scales)
        t.cuda.synchronize()
        _close(y, want, _bound(size, want, K, False), False, off)


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("p_dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("y_dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 2048), (8, 8, 2048), (5, 3, 77), (130, 9, 260), (2, 20, 64)])
def test_combine(t, B, T, k, H, p_dtype, y_dtype):
    """fp32 sums over ascending j: off by at most k * 2^-24 of the magnitude
    sum.  Rows of pairs without an expert hold NaN and are not read."""
    log(f"combine {T}x{k}x{H} {p_dtype} {y_dtype}")
    rng = np.random.default_rng(T + k + H)
    p = _dev(t, rng.standard_normal((T * k, H)).astype(np.float32), getattr(t, p_dtype))
    w = _dev(t, rng.standard_normal((T, k)).astype(np.float32))
    E = 6
    ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    ids[0] = -1
    for use in (False, True):
        q = p.clone()
        if use:
            q[_dev(t, np.flatnonzero((ids.reshape(-1) < 0) | (ids.reshape(-1) >= E)))] = float("nan")
        want, size = OO.combine(_np(p), _np(w), ids if use else None, E)
        for pad in (0, 3):
            buf = t.full((T, H + pad), 7.0, dtype=getattr(t, y_dtype), device="cuda")
            qq = t.nn.functional.pad(q, (0, pad))[:, :H]
            B.moe_combine_pairs(qq, w, buf[:, :H], ids=_dev(t, ids) if use else None, n_experts=E)
            t.cuda.synchronize()
            _close(buf[:, :H], want, k * 2.0 ** -24 * size, y_dtype == "bfloat16", (use, pad))
            assert bool((buf[:, H:] == 7).all())


# ------------------------------------------------------------------ together
def _layer(t, B, s, stream=None):
    """Grouping, gate/up, quantisation, down, combine on preallocated buffers."""
    up_x = dict(x_index=s["perm"], x_index_div=s["k"])
    B.moe_group_pairs(s["ids"], s["E"], s["off"], s["perm"], workspace=s["ws"], stream=stream)
    if s["fmt"] == "mxfp4-mxfp4":
        B.moe_mx_quantize(s["x"], s["xc"], s["xsc"], stream=stream)
        B.moe_grouped_gemm(s["xc"], s["wup"], s["off"], s["h"], x_scales=s["xsc"], w_scales=s["sup"], glu=True,
                           stream=stream, **up_x)
        B.moe_mx_quantize(s["h"], s["hc"], s["hsc"], stream=stream)
        B.moe_grouped_gemm(s["hc"], s["wdn"], s["off"], s["p"], x_scales=s["hsc"], w_scales=s["sdn"],
                           y_index=s["perm"], stream=stream)
    else:
        B.moe_grouped_gemm(s["x"], s["wup"], s["off"], s["h"], w_scales=s["sup"], glu=True, stream=stream, **up_x)
        B.moe_grouped_gemm(s["h"], s["wdn"], s["off"], s["p"], w_scales=s["sdn"], y_index=s["perm"], stream=stream)
    B.moe_combine_pairs(s["p"], s["w"], s["y"], ids=s["ids"], n_experts=s["E"], stream=stream)


def _state(t, B, fmt, T, k, E, H, I, seed):
    import workload as W
    wl = W.Workload("ops-layer", 1, E, k, H, I, "bf16" if fmt == "bf16-bf16" else "mxfp4", "bf16", 1, 1, 1, 1, T, seed,
                    w_sigma=0.1)
    stride = W.slot_stride(wl)
    bank = np.zeros(E * stride + 256, np.uint8)
    W.fill_banks(wl, bank.ctypes.data, 0, E)
    rng = np.random.default_rng(seed)
    dev = _dev(t, bank)
    s = dict(fmt=fmt, k=k, E=E, bank=bank, stride=stride, wl=wl)
    s["sup"] = s["sdn"] = None
    u8 = t.uint8
    if wl.w_dtype == "bf16":
        b = dev.view(t.bfloat16)
        s["wup"] = t.as_strided(b, (E, 2 * I, H), (stride // 2, H, 1))
        s["wdn"] = t.as_strided(b, (E, H, I), (stride // 2, I, 1), 2 * I * H)
    else:
        sc = 3 * H * I // 2
        s["wup"] = t.as_strided(dev, (E, 2 * I, H // 2), (stride, H // 2, 1))
        s["wdn"] = t.as_strided(dev, (E, H, I // 2), (stride, I // 2, 1), I * H)
        s["sup"] = t.as_strided(dev, (E, 2 * I, H // 32), (stride, H // 32, 1), sc)
        s["sdn"] = t.as_strided(dev, (E, H, I // 32), (stride, I // 32, 1), sc + 2 * I * H // 32)
    ids = _ids(rng, T, k, E, pad=T // 6)
    R = T * k
    s["np_ids"] = ids
    s["ids"], s["x"] = _dev(t, ids), _bf16(t, rng, (T, H))
    s["w"] = _dev(t, rng.random((T, k)).astype(np.float32))

    def e(shape, dt):
        return t.zeros(shape, dtype=dt, device="cuda")
    s["off"], s["perm"] = e(E + 1, t.int32), e(R, t.int32)
    s["ws"] = e(max(1, B.moe_group_workspace(T, k, E)), u8)
    s["xc"], s["xsc"] = e((T, H // 2), u8), e((T, H // 32), u8)
    s["h"], s["hc"], s["hsc"] = e((R, I), t.bfloat16), e((R, I // 2), u8), e((R, I // 32), u8)
    s["p"], s["y"] = e((R, H), t.float32), e((T, H), t.bfloat16)
    return s


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 8, 64, 128), (9, 4, 16, 256, 192), (700, 8, 32, 128, 64)])
def test_layer_over_resident_banks(t, B, fmt, T, k, E, H, I):
    """A routed FFN out of expert banks in device memory, in the layout the
    framework streams them in, against the layer oracle's expert arithmetic.
    The intermediate is rounded to bf16 (2^-8 of it) and, in the 4-bit form, x
    and h are taken as the oracle's quantiser rounds what the GPU held."""
    from oracle import expert as OX
    log(f"layer {fmt} T={T} E={E}")
    s = _state(t, B, fmt, T, k, E, H, I, 77 + T)
    _layer(t, B, s)
    t.cuda.synchronize()
    wl, st = s["wl"], s["stride"]
    ws = [OX.expert_weights(s["bank"][e * st:(e + 1) * st], wl.w_dtype, H, I) for e in range(E)]
    off, perm = OO.group_pairs(s["np_ids"], E)
    four = fmt == "mxfp4-mxfp4"
    x = _np(s["x"])
    x = OO.mx_values(*OO.mx_quantize(x)) if four else x
    h, hs = OO.grouped_rows(x, lambda e: np.concatenate(ws[e][:2]), off, T * k, 2 * I, perm, k, True)
    n = off[-1]
    _close(s["h"][:n], h[:n], _bound(hs, h, H, True)[:n], True, "h")
    hg = _np(s["h"])
    hg = OO.mx_values(*OO.mx_quantize(hg)) if four else hg
    rows, rs = OO.grouped_rows(hg, lambda e: ws[e][2], off, T * k, H)
    p, ps = np.zeros((T * k, H)), np.zeros((T * k, H))
    p[perm[:n]], ps[perm[:n]] = rows[:n], rs[:n]
    want, size = OO.combine(p, _np(s["w"]), s["np_ids"], E)
    _, err = OO.combine(I * 2.0 ** -23 * ps, _np(s["w"]), s["np_ids"], E)
    _close(s["y"], want, err + k * 2.0 ** -24 * size, True, "y")


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_streams_and_graph(t, B, fmt):
    """The same layer on side streams with other inputs at once, then captured
    and replayed between eager calls, with inputs changed in place: bit-equal to
    the eager result every time."""
    log(f"layer graph {fmt}")
    states = [_state(t, B, fmt, T, 4, 16, 128, 64, 5 + T) for T in (1, 40, 1200)]
    eager = []
    for s in states:
        _layer(t, B, s)
        t.cuda.synchronize()
        eager.append(s["y"].clone())
        s["y"].zero_()
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in states]
    for _ in range(3):
        for s, st in zip(states, streams):
            _layer(t, B, s, stream=st)
    t.cuda.synchronize()
    for s, want in zip(states, eager):
        assert t.equal(s["y"], want)
    for s in states:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            _layer(t, B, s)
        other = s["x"].flip(0).contiguous()
        for turn in range(4):
            s["x"], keep = s["x"].copy_(other) if turn % 2 else s["x"], s["x"].clone()
            s["y"].fill_(3)
            g.replay()
            t.cuda.synchronize()
            got = s["y"].clone()
            s["y"].zero_()
            _layer(t, B, s)
            t.cuda.synchronize()
            assert t.equal(s["y"], got), turn
            s["x"].copy_(keep)
            t.cuda.synchronize()


# ------------------------------------------------------------------ the SiLU's range
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R", [3, 300])
def test_glu_far_gates(t, B, R, fmt):
    """silu(gate) * up where exp(-gate) leaves fp32 and up is large enough that the
    product does not vanish.  The sums are exact (two terms of few bits), so the
    error is the SiLU's: exp(-|g|/2) (1.5 |g| / 2 + 2) * 2^-24 and used squared,
    reciprocal, sum and four products under 12 * 2^-24; subnormal results one step."""
    log(f"glu far gates {fmt} R={R}")
    act, wt = fmt.split("-")
    half, K = 128 * 33, 64
    gates = [(-64, -24), (-64, -8), (-96, 0), (-96, -8), (-64, -64), (-96, -64), (-8, -4), (64, 24), (96, 32), (0, 0)]
    ups = [1.0, -2.0 ** 60, 2.0 ** 100, 1.5 * 2.0 ** 126]
    g = np.array([gates[n % len(gates)] for n in range(half)], np.float64)
    u = np.array([ups[n // len(gates) % len(ups)] for n in range(half)])
    wide = (g.sum(1) > 0) & (np.abs(u) > 2.0 ** 100)
    u[wide] = 1.0  # the product would leave fp32
    w, x = np.zeros((2 * half, K)), np.zeros((R, K))
    w[:half, :2], w[half:, 0], x[:, :2] = g, u, 1.0
    if wt == "bf16":
        wd, wsc = _dev(t, w.astype(np.float32), t.bfloat16)[None], None
    else:
        c, s = OO.mx_quantize(w)
        assert np.array_equal(OO.mx_values(c, s), w)
        wd, wsc = _dev(t, c)[None], _dev(t, s)[None]
    if act == "bf16":
        xd, xs = _dev(t, x.astype(np.float32), t.bfloat16), None
    else:
        xd, xs = (_dev(t, a) for a in OO.mx_quantize(x))
    z = g.sum(1)
    want = z / (1 + np.exp(-z)) * u
    for out in (t.float32, t.bfloat16):
        y = t.full((R, half), 7.0, dtype=out, device="cuda")
        B.moe_grouped_gemm(xd, wd, _dev(t, np.array([0, R], np.int32)), y, x_scales=xs, w_scales=wsc, glu=True)
        t.cuda.synchronize()
        step = 2.0 ** -8 if out == t.bfloat16 else 2.0 ** -24
        tiny = 2.0 ** -133 if out == t.bfloat16 else 2.0 ** -148
        tol = ((1.5 * np.abs(z) + 16) * 2.0 ** -24 + step) * np.abs(want) + tiny
        got = _np(y)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), z[np.argwhere(bad)[:3, 1]],
                               got[bad][:3], np.broadcast_to(want, bad.shape)[bad][:3])


def test_glu_infinite_up(t, B):
    """An infinite up keeps its row's sign through a gate whose exp(-gate) overflows."""
    log("glu infinite up")
    for R, half in ((3, 70), (300, 128 * 33)):
        w = t.zeros((1, 2 * half, 32), dtype=t.bfloat16, device="cuda")
        w[0, :half, 0], w[0, half:, 0] = -100.0, float("inf")
        w[0, half + 1, 0] = -float("inf")
        x = t.zeros((R, 32), dtype=t.bfloat16, device="cuda")
        x[:, 0] = 1
        y = t.empty((R, half), device="cuda")
        B.moe_grouped_gemm(x, w, _dev(t, np.array([0, R], np.int32)), y, glu=True)
        t.cuda.synchronize()
        want = t.full((R, half), -float("inf"), device="cuda")
        want[:, 1] = float("inf")
        assert t.equal(y, want)


# ------------------------------------------------------------------ the ends of the formats' ranges
@pytest.mark.parametrize("M,N", [(4, 70), (600, 4100)])
def test_mx_gemm_bf16_extremes(t, B, M, N):
    """Subnormal rows of x and weights count in full; a weight is taken as the bf16
    value nearest to it, so magnitudes from 2^128 on, which no conversion of finite
    numbers gives, are infinite.  K equal powers of two: the sums are exact."""
    log(f"gemm bf16 extremes M={M}")
    K = 64
    for xv, code, value, scale in ((2.0 ** -130, 2, 1.0, 254), (2.0 ** -133, 2, 1.0, 254), (2.0 ** 120, 1, .5, 0),
                                   (2.0 ** 120, 7, 6.0, 0), (2.0 ** -100, 7, 6.0, 252), (2.0 ** -100, 5, 3.0, 253),
                                   (2.0 ** -100, 6, 4.0, 253), (2.0 ** -100, 6, 4.0, 254)):
        w = t.full((N, K // 2), code * 17, dtype=t.uint8, device="cuda")
        s = t.full((N, K // 32), scale, dtype=t.uint8, device="cuda")
        x = _dev(t, np.full((M, K), xv, np.float32), t.bfloat16)
        y = t.zeros((M, N), device="cuda")
        B.moe_mx_gemm(x, w, s, y)
        big = value * 2.0 ** (scale - 127)
        assert bool((y == (K * xv * big if big < 2.0 ** 128 else float("inf"))).all()), (xv, code, scale)


# ------------------------------------------------------------------ every variant
GROUPED_VARIANTS = [  # T, k, E, N, K, glu
    (60, 1, 1, 2090, 544, False), (75, 2, 3, 1000, 1120, False),   # 32 x 32 blocks
    (180, 1, 1, 2040, 544, False), (150, 2, 2, 1000, 1120, False),  # 64 x 64 blocks
    (150, 2, 4, 4340, 2080, True), (150, 2, 4, 4340, 4128, True),   # GLU 64 x 256 tiles, scales of more than one chunk
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K,glu", GROUPED_VARIANTS)
def test_grouped_variants(t, B, T, k, E, N, K, glu, fmt):
    """Sizes for the variants that no other test's sizes lead to."""
    test_grouped_tiles(t, B, T, k, E, N, K, glu, fmt)


# ------------------------------------------------------------------ large calls
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad", [0, 64])
def test_quantize_large(t, B, dtype, pad):
    """Inputs of 128 MiB are read past the caches: as many bytes as that and one
    row less, contiguous and with gaps, against the oracle in some rows and the
    same rows converted in small calls."""
    dt = getattr(t, dtype)
    C = 2048
    R = (128 << 20) // (C * dt.itemsize)
    log(f"quantize large {dtype} {R}x{C} pad {pad}")
    g = t.Generator(device="cuda").manual_seed(21)
    buf = t.randn(R, C + pad, generator=g, device="cuda")
    buf *= t.exp2(t.randint(-140, 120, (R, 1), generator=g, device="cuda").float())
    buf[7, 5], buf[R - 1, C - 1], buf[11, 64:96] = float("inf"), float("nan"), 0.0
    x = buf.to(dt)[:, :C]
    rows = [0, 7, 11, R // 2, R - 2, R - 1]
    want = OO.mx_quantize(_np(x[rows]))
    for n in (R, R - 1):
        codes = t.full((n, C // 2), 77, dtype=t.uint8, device="cuda")
        scales = t.full((n, C // 32), 77, dtype=t.uint8, device="cuda")
        B.moe_mx_quantize(x[:n], codes, scales)
        for i in range(0, n, 4096):
            m = min(4096, n - i)
            c = t.empty((m, C // 2), dtype=t.uint8, device="cuda")
            s = t.empty((m, C // 32), dtype=t.uint8, device="cuda")
            B.moe_mx_quantize(x[i:i + m], c, s)
            assert t.equal(codes[i:i + m], c) and t.equal(scales[i:i + m], s)
        live = [r for r in rows if r < n]
        assert np.array_equal(codes[live].cpu().numpy(), want[0][:len(live)])
        assert np.array_equal(scales[live].cpu().numpy(), want[1][:len(live)])


@pytest.mark.parametrize("T,k,E", [(1 << 17, 8, 256), (1 << 21, 8, 1024)])
def test_group_pairs_large(t, B, T, k, E):
    """2^20 pairs, and the 2^24 that a call may have."""
    log(f"group large {T}x{k} E={E}")
    rng = np.random.default_rng(k + E)
    flat = rng.integers(-1, E + 1, T * k).astype(np.int32)
    key = np.where((flat < 0) | (flat >= E), E, flat).astype(np.int16)
    order = np.argsort(key, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]).astype(np.int32)
    order[off[-1]:] = -1
    offsets = t.full((E + 1,), 5, dtype=t.int32, device="cuda")
    perm = t.full((T * k,), 5, dtype=t.int32, device="cuda")
    ws = t.empty(B.moe_group_workspace(T, k, E), dtype=t.uint8, device="cuda")
    B.moe_group_pairs(_dev(t, flat.reshape(T, k)), E, offsets, perm, workspace=ws)
    t.cuda.synchronize()
    assert np.array_equal(offsets.cpu().numpy(), off)
    assert np.array_equal(perm.cpu().numpy(), order)


@pytest.mark.parametrize("T,k,H", [(300001, 2, 36), (300001, 1, 7), (9, 3, 1 << 28)])
def test_combine_large(t, B, T, k, H):
    """More tokens than the grid's second dimension has rows of workgroups, and
    rows of p past 2^32 bytes; powers of two, so every sum is exact."""
    log(f"combine large {T}x{k}x{H}")
    p = t.ones((T * k, H), dtype=t.bfloat16, device="cuda")
    p *= t.arange(1, T * k + 1, device="cuda").remainder(61).to(t.bfloat16)[:, None]
    w = t.full((T, k), 0.5, device="cuda")
    y = t.full((T, H), 7.0, dtype=t.float32, device="cuda")
    B.moe_combine_pairs(p, w, y)
    want = 0.5 * t.arange(1, T * k + 1, device="cuda").remainder(61).view(T, k).sum(1).float()
    assert bool((y == want[:, None]).all())


@pytest.mark.parametrize("fmt,M,N,K", [("mxfp4-mxfp4", 64, 4096, 1024), ("mxfp4-mxfp4", 256, 1024, 2080),
                                       ("bf16-mxfp4", 128, 6000, 1024), ("bf16-mxfp4", 64, 16384, 512)])
def test_one_expert_is_the_dense_product(t, B, fmt, M, N, K):
    """One group takes the variant of the dense product of its size, so the sums are
    formed in the same order and every bit agrees; sizes on the rule's borders."""
    log(f"one expert {fmt} {M}x{N}x{K}")
    act, wt = fmt.split("-")
    rng = np.random.default_rng(M + N + K)
    x, w = Operand(t, rng, M, K, act), Experts(t, rng, 1, N, K, wt)
    y = t.zeros((M, N), device="cuda")
    B.moe_mx_gemm(x.t, w.t[0], w.scales[0], y, x_scales=x.scales)
    assert t.equal(_grouped(t, B, x, w, [0, M], M, N, "float32"), y)
