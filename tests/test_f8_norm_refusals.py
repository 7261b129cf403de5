"""Arguments that the F8 operators and the norms refuse (CPU only: every call here
fails its checks before anything is enqueued), their exports, and the oracle's
e4m3 rounding against the code table."""
import ctypes
import subprocess
import sys

import numpy as np
import pytest
import torch

import routed_expert_execution_moe_amd as B
from oracle import ops as OO
from routed_expert_execution_moe_amd.binding import CombineNormArgs, GroupedArgs, MOE_EINVAL, MOE_EUNSUPPORTED, MoeConfig
from tests.conftest import ROOT

A = 1 << 20  # stands for an aligned device address that no call gets to use
F32, BF16, MX, F8 = B.MOE_F32, B.MOE_BF16, B.MOE_MXFP4, B.MOE_F8


def test_exports():
    for n in ("moe_f8_quantize", "moe_f8_dequantize", "moe_f8_gemm", "moe_norm", "moe_combine_norm"):
        assert hasattr(B.lib(), n) and hasattr(B, n)


def _quantize(**kw):
    a = dict(x=A, dtype=F32, n=1, rows=4, cols=64, ld=64, stride=0, block=1, codes=A, scales=A)
    a.update(kw)
    return B.lib().moe_f8_quantize(*a.values(), None)


def _dequantize(**kw):
    a = dict(codes=A, scales=A, n=1, rows=4, cols=64, block=1, x=A, dtype=F32, ld=64, stride=0)
    a.update(kw)
    return B.lib().moe_f8_dequantize(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=MX), MOE_EUNSUPPORTED), (dict(dtype=F8), MOE_EUNSUPPORTED), (dict(dtype=-1), MOE_EUNSUPPORTED),
    (dict(rows=-1), MOE_EINVAL), (dict(n=-1), MOE_EINVAL), (dict(cols=0), MOE_EINVAL), (dict(cols=24), MOE_EINVAL),
    (dict(cols=-16), MOE_EINVAL), (dict(cols=(1 << 30) + 16, ld=1 << 31), MOE_EINVAL),
    (dict(block=0), MOE_EINVAL), (dict(block=64), MOE_EINVAL), (dict(block=1, n=2), MOE_EINVAL),
    (dict(ld=63), MOE_EINVAL), (dict(ld=1 << 41), MOE_EINVAL), (dict(block=128, n=2, stride=-4), MOE_EINVAL),
    (dict(rows=1 << 40), MOE_EINVAL), (dict(rows=(1 << 62)), MOE_EINVAL),
    (dict(x=None), MOE_EINVAL), (dict(codes=None), MOE_EINVAL), (dict(scales=None), MOE_EINVAL),
    (dict(x=A + 2), MOE_EINVAL), (dict(x=A + 1, dtype=BF16), MOE_EINVAL), (dict(codes=A + 8), MOE_EINVAL),
    (dict(scales=A + 2), MOE_EINVAL),
    (dict(rows=0, x=None, codes=None, scales=None), 0), (dict(block=128, n=0, x=None), 0),
])
def test_conversion_refusals(kw, status):
    if kw.get("rows") == 1 << 40:
        kw = dict(kw, cols=256, ld=256)  # two blocks a row: past 2^40 of them
    for call in (_quantize, _dequantize):
        assert call(**kw) == status
        if status:
            assert call.__name__[1:] in B.moe_last_error()


def test_dequantize_matrices_that_overlap():
    """y of matrices less than a row apart; x may repeat one matrix, so the other direction takes it."""
    for stride in (0, 48):
        assert _dequantize(block=128, n=2, stride=stride) == MOE_EINVAL and "overlap" in B.moe_last_error()


def _gemm(**kw):
    a = dict(x=A, xs=A, ldx=64, w=A, ws=A, y=A, y_dtype=F32, ldy=16, M=4, N=16, K=64)
    a.update(kw)
    return B.lib().moe_f8_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(y_dtype=F8), MOE_EUNSUPPORTED), (dict(y_dtype=MX), MOE_EUNSUPPORTED), (dict(M=-1), MOE_EINVAL),
    (dict(N=0), MOE_EINVAL), (dict(K=0, ldx=0), MOE_EINVAL), (dict(K=72, ldx=80), MOE_EINVAL),
    (dict(ldx=48), MOE_EINVAL), (dict(ldx=72), MOE_EINVAL), (dict(ldx=1 << 41), MOE_EINVAL), (dict(ldy=15), MOE_EINVAL),
    (dict(ldy=1 << 62), MOE_EINVAL), (dict(x=A + 8), MOE_EINVAL), (dict(w=A + 4), MOE_EINVAL), (dict(xs=A + 2), MOE_EINVAL),
    (dict(ws=A + 1), MOE_EINVAL), (dict(y=A + 2), MOE_EINVAL), (dict(x=None), MOE_EINVAL), (dict(xs=None), MOE_EINVAL),
    (dict(w=None), MOE_EINVAL), (dict(ws=None), MOE_EINVAL), (dict(y=None), MOE_EINVAL),
    (dict(N=1 << 20, K=2048, ldx=2048, ldy=1 << 20), MOE_EINVAL),  # 2^31 bytes of codes
    (dict(K=(1 << 30) + 16, ldx=(1 << 30) + 16, N=1, M=1), MOE_EINVAL),
    (dict(M=(1 << 31) - 1), MOE_EINVAL),
    (dict(M=0, x=None, xs=None, w=None, ws=None, y=None), 0),
])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


def _grouped(**kw):
    a = dict(n_experts=4, n_rows=8, N=32, K=64, x_dtype=F8, w_dtype=F8, y_dtype=F32, glu=0, x=A, x_scales=A, ldx=64,
             n_x=8, x_index_div=1, x_index=None, w=A, w_scales=A, w_stride=2048, ws_stride=4, offsets=A, y=A, ldy=32,
             n_y=8, reserved=0, y_index=None)
    a.update(kw)
    return B.lib().moe_grouped_gemm(ctypes.byref(GroupedArgs(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(w_dtype=BF16), MOE_EUNSUPPORTED), (dict(w_dtype=MX), MOE_EUNSUPPORTED), (dict(x_dtype=BF16), MOE_EUNSUPPORTED),
    (dict(x_dtype=MX), MOE_EUNSUPPORTED), (dict(y_dtype=F8), MOE_EUNSUPPORTED), (dict(K=72, ldx=80), MOE_EINVAL),
    (dict(ldx=72), MOE_EINVAL), (dict(x_scales=None), MOE_EINVAL), (dict(w_scales=None), MOE_EINVAL),
    (dict(x_scales=A + 2), MOE_EINVAL), (dict(w_scales=A + 2), MOE_EINVAL), (dict(ws_stride=6), MOE_EINVAL),
    (dict(ws_stride=-4), MOE_EINVAL), (dict(w_stride=8), MOE_EINVAL), (dict(glu=1, N=33), MOE_EINVAL),
    (dict(x_index=A, n_x=1 << 25), MOE_EINVAL),  # 2^31 bytes of indexed rows
    (dict(N=1 << 25, ldy=1 << 25), MOE_EINVAL),  # 2^31 bytes per expert
    (dict(n_rows=0, x=None, w=None, y=None, offsets=None), 0),
])
def test_grouped_refusals(kw, status):
    assert _grouped(**kw) == status


def test_other_calls_keep_refusing_f8():
    """The type belongs to the operators that name it."""
    assert B.lib().moe_mx_gemm(A, F8, A, 64, A, A, A, F32, 16, 4, 16, 64, None) == MOE_EUNSUPPORTED
    assert B.lib().moe_mx_quantize(A, F8, 4, 64, 64, A, A, None) == MOE_EUNSUPPORTED
    assert B.lib().moe_combine_pairs(A, F8, 64, A, None, 0, 2, 2, 64, A, F32, 64, None) == MOE_EUNSUPPORTED
    cfg = MoeConfig(48, 128, 8, 2048, 768, F8, BF16, 100, 100, 8, 1, 1, 0, 0, 0, 0, 0)
    assert B.lib().moe_expert_bytes(ctypes.byref(cfg)) == 0


def _norm(**kw):
    a = dict(x=A + 4096, x_dtype=BF16, ldx=64, weight=A, weight_dtype=BF16, eps=1e-6, T=4, H=64, y=A, y_dtype=BF16, ys=None, ldy=64)
    a.update(kw)
    return B.lib().moe_norm(*a.values(), None)


_LEAVING = [  # rows that leave a norm, and its constants
    (dict(H=0), MOE_EINVAL), (dict(H=32769, ld=40000), MOE_EINVAL), (dict(T=-1), MOE_EINVAL), (dict(T=(1 << 40) + 1), MOE_EINVAL),
    (dict(eps=0.0), MOE_EINVAL), (dict(eps=-1e-6), MOE_EINVAL), (dict(eps=1e-40), MOE_EINVAL),
    (dict(eps=float("nan")), MOE_EINVAL), (dict(eps=float("inf")), MOE_EINVAL),
    (dict(weight_dtype=F8), MOE_EUNSUPPORTED), (dict(weight_dtype=MX), MOE_EUNSUPPORTED), (dict(y_dtype=MX), MOE_EUNSUPPORTED),
    (dict(y=None), MOE_EINVAL), (dict(ys=A), MOE_EINVAL), (dict(y_dtype=F8), MOE_EINVAL), (dict(ldy=63), MOE_EINVAL),
    (dict(ldy=1 << 41), MOE_EINVAL), (dict(y_dtype=F8, ys=A, H=40, ld=64), MOE_EINVAL), (dict(y_dtype=F8, ys=A, ldy=72), MOE_EINVAL),
    (dict(y_dtype=F8, ys=A, y=A + 8), MOE_EINVAL), (dict(y_dtype=F8, ys=A + 2), MOE_EINVAL), (dict(y=A + 1), MOE_EINVAL),
    (dict(y=A + 2, y_dtype=F32), MOE_EINVAL), (dict(weight=A + 1), MOE_EINVAL), (dict(weight=A + 2, weight_dtype=F32), MOE_EINVAL),
]


@pytest.mark.parametrize("kw,status", _LEAVING + [
    (dict(weight=None), MOE_EINVAL), (dict(x=None), MOE_EINVAL), (dict(x_dtype=F8), MOE_EUNSUPPORTED), (dict(x_dtype=MX), MOE_EUNSUPPORTED),
    (dict(ldx=63), MOE_EINVAL), (dict(ldx=1 << 41), MOE_EINVAL), (dict(x=A + 1), MOE_EINVAL),
    (dict(x=A, x_dtype=F32), MOE_EINVAL), (dict(x=A, ldx=72), MOE_EINVAL), (dict(x=A, y_dtype=F8, ys=A + 64), MOE_EINVAL), (dict(T=0, x=None, y=None, weight=None), 0),
])
def test_norm_refusals(kw, status):
    kw = dict(kw)
    if "ld" in kw:
        kw["ldx"] = kw["ldy"] = kw.pop("ld")
    assert _norm(**kw) == status


def _combine_norm(**kw):
    a = dict(p=A + 8192, w=A, ids=None, residual=A + 4096, out=A + 16384, post_weight=A, gate=A, weight=A, y=A, y_scales=None, ldp=64, ldres=64,
             ldout=64, ldg=0, ldy=64, T=4, k=2, H=64, n_experts=0, gate_cols=64, p_dtype=F32, residual_dtype=BF16,
             out_dtype=BF16, post_dtype=BF16, gate_dtype=F32, weight_dtype=BF16, y_dtype=BF16, reserved=0, scale=1.0, eps=1e-6)
    a.update(kw)
    return B.lib().moe_combine_norm(ctypes.byref(CombineNormArgs(**a)), None)


@pytest.mark.parametrize("kw,status", _LEAVING + [
    (dict(weight=None), MOE_EINVAL), (dict(weight=None, y=None, ys=A), MOE_EINVAL), (dict(reserved=1), MOE_EINVAL),
    (dict(p_dtype=F8), MOE_EUNSUPPORTED), (dict(residual_dtype=MX), MOE_EUNSUPPORTED), (dict(out_dtype=F8), MOE_EUNSUPPORTED),
    (dict(post_dtype=7), MOE_EUNSUPPORTED), (dict(gate_dtype=F8), MOE_EUNSUPPORTED),
    (dict(k=0), MOE_EINVAL), (dict(k=(1 << 30) + 1), MOE_EINVAL), (dict(T=1 << 40, k=2), MOE_EINVAL), (dict(w=None), MOE_EINVAL),
    (dict(ids=A, n_experts=0), MOE_EINVAL), (dict(scale=float("nan")), MOE_EINVAL), (dict(scale=float("inf")), MOE_EINVAL),
    (dict(gate_cols=2), MOE_EINVAL), (dict(gate_cols=0), MOE_EINVAL), (dict(gate=None), MOE_EINVAL), (dict(ldg=-1), MOE_EINVAL),
    (dict(ldg=1 << 41), MOE_EINVAL), (dict(p=None), MOE_EINVAL), (dict(residual=None), MOE_EINVAL), (dict(out=None), MOE_EINVAL),
    (dict(ldp=63), MOE_EINVAL), (dict(ldres=63), MOE_EINVAL), (dict(ldout=63), MOE_EINVAL), (dict(ldres=1 << 41), MOE_EINVAL),
    (dict(out=A + 4096, ldout=72), MOE_EINVAL), (dict(out=A + 4096, out_dtype=F32), MOE_EINVAL),
    (dict(p=A + 2), MOE_EINVAL), (dict(residual=A + 1), MOE_EINVAL), (dict(out=A + 1), MOE_EINVAL), (dict(w=A + 2), MOE_EINVAL),
    (dict(ids=A + 2, n_experts=4), MOE_EINVAL), (dict(post_weight=A + 1), MOE_EINVAL), (dict(gate=A + 2), MOE_EINVAL),
    (dict(y=A + 16384), MOE_EINVAL), (dict(y=A + 4096), MOE_EINVAL), (dict(y=A + 8192, y_dtype=F32), MOE_EINVAL),
    (dict(T=0, p=None, residual=None, out=None), 0),
])
def test_combine_norm_refusals(kw, status):
    kw = dict(kw)
    if "ld" in kw:
        kw["ldp"] = kw["ldres"] = kw["ldout"] = kw["ldy"] = kw.pop("ld")
        kw["gate_cols"] = kw["H"]
    if kw.get("H") == 0:
        kw["gate_cols"] = 1
    if "ys" in kw:
        kw["y_scales"] = kw.pop("ys")
    assert _combine_norm(**kw) == status


def test_combine_norm_null_args():
    assert B.lib().moe_combine_norm(None, None) == MOE_EINVAL


def _refused(call, *args, **kw):
    with pytest.raises(B.MoertError) as e:
        call(*args, **kw)
    assert e.value.status == MOE_EINVAL
    return str(e.value)


def test_binding_refusals():
    """Shapes, element types, strides and devices that only the binding sees."""
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    x = torch.zeros(4, 144, dtype=bf)
    codes, scales = torch.zeros(4, 144, dtype=f8), torch.zeros(4, 2)
    assert "GPU" in _refused(B.moe_f8_quantize, x, codes, scales)
    assert "GPU" in _refused(B.moe_f8_quantize, x, codes, scales[:1], block_rows=128)
    assert "GPU" in _refused(B.moe_f8_quantize, x[None], codes[None], scales[None, :1], block_rows=128)
    _refused(B.moe_f8_quantize, x[None], codes[None], scales[None])  # a stack with scales per row
    _refused(B.moe_f8_quantize, x, codes, scales, block_rows=64)
    _refused(B.moe_f8_quantize, x.half(), codes, scales)
    _refused(B.moe_f8_quantize, x, codes.view(torch.uint8), scales)
    _refused(B.moe_f8_quantize, x, codes.view(torch.uint8).view(torch.float8_e4m3fnuz), scales)
    _refused(B.moe_f8_quantize, x, codes[:3], scales)
    _refused(B.moe_f8_quantize, x, codes, scales[:, :1])
    _refused(B.moe_f8_quantize, x, codes, scales.double())
    _refused(B.moe_f8_quantize, x[:, :136], codes[:, :136], scales)
    _refused(B.moe_f8_quantize, x.t(), codes.t(), scales)
    _refused(B.moe_f8_dequantize, codes, scales[:3], x)
    w, ws, y, xs = torch.zeros(6, 144, dtype=f8), torch.zeros(1, 2), torch.zeros(4, 6), scales
    assert "GPU" in _refused(B.moe_f8_gemm, codes, xs, w, ws, y)
    _refused(B.moe_f8_gemm, x, xs, w, ws, y)
    _refused(B.moe_f8_gemm, codes, xs[:, :1], w, ws, y)
    _refused(B.moe_f8_gemm, codes, xs, w[:, :128], ws, y)
    _refused(B.moe_f8_gemm, codes, xs, w, torch.zeros(6, 2), y)
    _refused(B.moe_f8_gemm, codes, xs, w, ws, y[:, :5])
    _refused(B.moe_f8_gemm, codes, xs, w, ws, y[:3])
    we, wes = torch.zeros(8, 6, 144, dtype=f8), torch.zeros(8, 1, 2)
    off, yg, perm = torch.zeros(9, dtype=torch.int32), torch.zeros(8, 6), torch.zeros(8, dtype=torch.int32)
    args = dict(x_scales=xs, w_scales=wes, x_index=perm)
    assert "GPU" in _refused(B.moe_grouped_gemm, codes, we, off, yg, **args)
    _refused(B.moe_grouped_gemm, codes, we, off, yg, **{**args, "x_scales": None})
    _refused(B.moe_grouped_gemm, codes, we, off, yg, **{**args, "w_scales": None})
    _refused(B.moe_grouped_gemm, codes, we, off, yg[:, :3], glu=True, **args)  # gate and up need rows of scales each
    assert "GPU" in _refused(B.moe_grouped_gemm, codes, we, off, yg[:, :3].contiguous(), glu=True, **{**args, "w_scales": torch.zeros(8, 2, 2)})
    _refused(B.moe_grouped_gemm, codes, we.view(torch.uint8), off, yg, **args)
    _refused(B.moe_grouped_gemm, codes, we.float(), off, yg, **args)
    _refused(B.moe_grouped_gemm, x, we, off, yg, x_index=perm)  # bf16 rows, 8-bit weights
    wt = torch.zeros(144, dtype=bf)
    assert "GPU" in _refused(B.moe_norm, x, wt, x.clone())
    assert "GPU" in _refused(B.moe_norm, x, wt, codes, y_scales=scales)
    _refused(B.moe_norm, x, wt, codes)
    _refused(B.moe_norm, x, wt, x.clone(), y_scales=scales)
    _refused(B.moe_norm, x, wt, codes, y_scales=scales[:, :1])
    _refused(B.moe_norm, x, wt[:143], x.clone())
    _refused(B.moe_norm, x, wt, x[:3].clone())
    _refused(B.moe_norm, x, wt, x.half())
    p, cw, res = torch.zeros(8, 144), torch.zeros(4, 2), x.clone()
    assert "GPU" in _refused(B.moe_combine_norm, p, cw, x, res)
    assert "GPU" in _refused(B.moe_combine_norm, p[:4], None, x, x)
    assert "GPU" in _refused(B.moe_combine_norm, p, cw, x, res, gate=torch.zeros(4, 1), weight=wt, y=codes, y_scales=scales, post_weight=wt)
    _refused(B.moe_combine_norm, p, None, x, res)
    _refused(B.moe_combine_norm, p[:7], cw, x, res)
    _refused(B.moe_combine_norm, p, cw[:3], x, res)
    _refused(B.moe_combine_norm, p, cw, x, res[:, :143])
    _refused(B.moe_combine_norm, p, cw, x, res, weight=wt)
    _refused(B.moe_combine_norm, p, cw, x, res, y=codes, y_scales=scales)
    _refused(B.moe_combine_norm, p, cw, x, res, y_scales=scales)
    _refused(B.moe_combine_norm, p, cw, x, res, gate=torch.zeros(3, 1))
    _refused(B.moe_combine_norm, p, cw, x, res, gate=torch.zeros(4, 2))
    _refused(B.moe_combine_norm, p, cw, x, res, gate=torch.zeros(144))
    _refused(B.moe_combine_norm, p, cw, x, res, post_weight=wt[:100])
    _refused(B.moe_combine_norm, p, cw, x, res, scale=1e300)
    _refused(B.moe_combine_norm, p, cw, x, res, scale="1")
    _refused(B.moe_combine_norm, p, cw, x, res, ids=torch.zeros(4, 2, dtype=torch.int32))
    _refused(B.moe_combine_norm, p, cw, x, res, ids=torch.zeros(4, 2, dtype=torch.int64), n_experts=4)


def test_oracle_e4m3():
    """Every code's value comes back, midpoints take the even code, and torch's own conversion agrees."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, OO.E4M3, equal_nan=True)
    mags = OO.E4M3[:127]
    assert np.array_equal(OO.f8_codes(mags), np.arange(127)) and np.array_equal(OO.f8_codes(-mags[1:]), np.arange(129, 255))
    mid = (mags[1:] + mags[:-1]) / 2
    assert (OO.f8_codes(mid) % 2 == 0).all()
    rng = np.random.default_rng(1)
    q = (rng.standard_normal(20000) * np.exp2(rng.integers(-12, 7, 20000))).clip(-448, 448).astype(np.float32)
    q[:126] = mid.astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OO.f8_codes(q.astype(np.float64)), want)
    c, s = OO.f8_quantize(np.array([[448.0] + [0.0] * 15, [np.inf] + [1.0] * 15, [0.0] * 16, [-1e-45] * 16]))
    assert s[0, 0] == 1 and c[0, 0] == 126 and np.isnan(s[1, 0]) and not c[1].any()
    assert s[2, 0] == np.float32(2.0 ** -126) and s[3, 0] == np.float32(2.0 ** -126) and not (c[2:] & 127).any()


def test_gpu_sizes_reach_every_f8_variant():
    """The rule that picks an F8 product's kernel, on the sizes of the GPU tests: every kernel has one."""
    from tests import test_gpu_f8 as G
    f = B.lib().moert_f8_variant
    f.argtypes, f.restype = [ctypes.c_int] * 6, ctypes.c_int
    names = ["small16", "small32", "small64", "deep", "shared", "half", "big"]
    assert f(0, 0, 0, 8, 64, 64) == -1
    got = set()
    for y_f32 in (0, 1):
        calls = [(0, 1, M, N, K) for M, N, K in G.GEMM + G.GEMM_TILES]
        calls += [(glu, E, T * min(k, E), N, K) for T, k, E, N, K in G.GROUPED for glu in (0, 1)]
        calls += [(int(glu), E, T * k, N, K) for T, k, E, N, K, glu in G.GROUPED_TILES + G.GROUPED_VARIANTS]
        for glu, *c in calls:
            n = names[f(y_f32, glu, *c)]
            got.add((None if n.startswith("small") else y_f32, glu, n))  # the few-row kernels write either type
    want = {(y, glu, n) for glu in (0, 1) for y, n in [(None, "small16"), (None, "small32"), (None, "small64"), (0, "shared"),
                                                       (0, "half"), (0, "big"), (1, "shared"), (1, "half")]}
    assert got == want, (sorted(want - got), sorted(got - want))


def test_few_rows_take_the_few_row_kernel_at_any_width():
    """One matrix's 8 rows or fewer, whose products keep all of their bits, also past 32,768 columns (a vocabulary)."""
    f = B.lib().moert_f8_variant
    f.argtypes, f.restype = [ctypes.c_int] * 6, ctypes.c_int
    for M in range(1, 9):
        for N in (2, 4096, 32768, 32770, 36864, 65536, 152064, 1 << 20):
            for K in (128, 1024, 4096):
                for y_f32 in (0, 1):
                    for glu in (0, 1):
                        assert f(y_f32, glu, 1, M, N, K) == 0, (M, N, K, y_f32, glu)


def test_norm_refuses_rows_that_overlap():
    """y must be x itself or apart from it: also by less than the whole, and in another type."""
    x = A + 4096  # 4 rows of 64 bf16, 128 bytes each
    for kw in (dict(y=x + 128), dict(y=x - 128), dict(y=x + 2), dict(y=x + 510), dict(y=x - 510), dict(y=x, ldy=128, ldx=64),
               dict(y=x + 16, y_dtype=F8, ys=A), dict(y=x + 256, y_dtype=F32), dict(ldx=160, ldy=160, y=x + 126),
               dict(ldx=160, ldy=160, y=x + 194), dict(ldx=160, ldy=160, y=x + 320 * 2 + 194), dict(T=1, y=x + 126)):
        assert _norm(**kw) == MOE_EINVAL and "memory of its own" in B.moe_last_error(), kw


def test_combine_norm_refuses_rows_that_overlap():
    """out over p with several rows a token is read by other workgroups while it is written; y and out have no part of p,
    residual and each other."""
    p, res, out, y = A + 8192, A + 4096, A + 16384, A
    for kw in (dict(out=p, out_dtype=F32), dict(out=p), dict(out=p + 256, out_dtype=F32), dict(out=p + 1792), dict(out=p - 384),
               dict(k=1, out=p), dict(k=1, out=p, out_dtype=F32, ldout=72), dict(k=1, out=p + 256, out_dtype=F32),
               dict(out=res + 128), dict(out=res - 128), dict(out=res, ldout=72), dict(out=res + 2, ldout=64),
               dict(weight=None, y=None, out=p, out_dtype=F32), dict(weight=None, y=None, out=res + 128)):
        assert _combine_norm(**kw) == MOE_EINVAL and "out must be" in B.moe_last_error(), kw
    for kw in (dict(y=out + 128), dict(y=out - 510), dict(y=res + 128), dict(y=p + 1792), dict(y=p + 2040),
               dict(y=out, y_dtype=F8, y_scales=A), dict(y=out + 64, ldy=160, ldout=160), dict(ldy=1 << 40, y=res - 128)):
        assert _combine_norm(**kw) == MOE_EINVAL and "y must have" in B.moe_last_error(), kw


def test_dequantize_matrices_that_share_rows():
    """Matrices at least a row apart whose later rows meet the next matrix's."""
    for kw in (dict(n=2, stride=64), dict(n=2, stride=64 * 3 + 63), dict(n=3, ld=128, stride=64), dict(n=2, ld=100, stride=130),
               dict(n=1 << 20, ld=1 << 20, stride=1 << 20), dict(n=2, rows=1 << 38, ld=1 << 40, stride=1 << 40)):
        assert _dequantize(block=128, **kw) == MOE_EINVAL and "overlap" in B.moe_last_error(), kw


def test_import_with_a_torch_without_gpu_support():
    """Such a torch lacks the two names that a call looks its device and stream up with; nothing but a call needs them."""
    code = """
import torch
del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
import routed_expert_execution_moe_amd as B, routed_expert_execution_moe_amd.build
try:
    B.moe_norm(torch.zeros(2, 8), torch.zeros(8), torch.zeros(2, 8))
except B.MoertError as e:
    print("refused:", e)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and "refused:" in r.stdout and "GPU" in r.stdout, r.stderr
