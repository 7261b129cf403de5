"""Arguments that the operators without a context refuse (CPU only: every
call here fails its checks before anything is enqueued), the workspace sizes,
and the oracle's MXFP4 quantiser against the code table."""
import ctypes

import numpy as np
import pytest
import torch

import routed_expert_execution_moe_amd as B
from oracle import ops as OO
from routed_expert_execution_moe_amd.binding import GroupedArgs, MOE_EINVAL, MOE_EUNSUPPORTED

A = 1 << 20  # stands for an aligned device address that no call gets to use
F32, BF16, MX = B.MOE_F32, B.MOE_BF16, B.MOE_MXFP4


@pytest.mark.parametrize("args,status", [
    ((A, MX, 4, 64, 64, A, A), MOE_EUNSUPPORTED),
    ((A, 7, 4, 64, 64, A, A), MOE_EUNSUPPORTED),
    ((A, F32, -1, 64, 64, A, A), MOE_EINVAL),
    ((A, F32, 4, 48, 64, A, A), MOE_EINVAL),
    ((A, F32, 4, 0, 64, A, A), MOE_EINVAL),
    ((A, F32, 4, 64, 32, A, A), MOE_EINVAL),
    ((A, F32, 4, 64, 66, A, A), MOE_EINVAL),
    ((A, BF16, 4, 64, 68, A, A), MOE_EINVAL),
    ((A, BF16, 4, 64, 1 << 41, A, A), MOE_EINVAL),
    ((A + 8, F32, 4, 64, 64, A, A), MOE_EINVAL),
    ((A, F32, 4, 64, 64, A + 4, A), MOE_EINVAL),
    ((None, F32, 4, 64, 64, A, A), MOE_EINVAL),
    ((A, F32, 4, 64, 64, None, A), MOE_EINVAL),
    ((A, F32, 4, 64, 64, A, None), MOE_EINVAL),
    ((None, F32, 0, 64, 64, None, None), 0),  # no rows: nothing to do
])
def test_quantize_refusals(args, status):
    assert B.lib().moe_mx_quantize(*args, None) == status
    if status:
        assert "moe_mx_quantize" in B.moe_last_error()


@pytest.mark.parametrize("args,status", [
    ((A, A, 4, 64, A, MX, 64), MOE_EUNSUPPORTED),
    ((A, A, 4, 40, A, F32, 64), MOE_EINVAL),
    ((A, A, 4, 64, A, F32, 63), MOE_EINVAL),
    ((A, A, 4, 64, A + 2, F32, 64), MOE_EINVAL),
    ((A, A, 4, 64, A + 1, BF16, 64), MOE_EINVAL),
    ((A, None, 4, 64, A, F32, 64), MOE_EINVAL),
    ((A, A, -4, 64, A, F32, 64), MOE_EINVAL),
    ((None, None, 0, 64, None, F32, 64), 0),
])
def test_dequantize_refusals(args, status):
    assert B.lib().moe_mx_dequantize(*args, None) == status


def _gemm(**kw):
    a = dict(x=A, x_dtype=BF16, xs=None, ldx=64, w=A, ws=A, y=A, y_dtype=F32, ldy=16, M=4, N=16, K=64)
    a.update(kw)
    return B.lib().moe_mx_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x_dtype=F32), MOE_EUNSUPPORTED),
    (dict(y_dtype=MX), MOE_EUNSUPPORTED),
    (dict(M=-1), MOE_EINVAL),
    (dict(N=0), MOE_EINVAL),
    (dict(K=48, ldx=48), MOE_EINVAL),
    (dict(K=0, ldx=0), MOE_EINVAL),
    (dict(ldx=56), MOE_EINVAL),
    (dict(ldx=65), MOE_EINVAL),
    (dict(ldx=1 << 62), MOE_EINVAL),
    (dict(ldy=15), MOE_EINVAL),
    (dict(xs=A), MOE_EINVAL),
    (dict(x_dtype=MX), MOE_EINVAL),                    # scales missing
    (dict(x_dtype=MX, xs=A, ldx=128), MOE_EINVAL),     # strided codes
    (dict(x=A + 8), MOE_EINVAL),
    (dict(w=A + 4), MOE_EINVAL),
    (dict(y=A + 2), MOE_EINVAL),
    (dict(x=None), MOE_EINVAL),
    (dict(ws=None), MOE_EINVAL),
    (dict(y=None), MOE_EINVAL),
    (dict(N=1 << 20, K=4096, ldx=4096, ldy=1 << 20), MOE_EINVAL),  # 2^31 bytes of codes
    (dict(M=(1 << 31) - 1), MOE_EINVAL),
    (dict(M=0, x=None, w=None, y=None), 0),
])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


def _grouped(**kw):
    a = dict(n_experts=4, n_rows=8, N=32, K=64, x_dtype=BF16, w_dtype=BF16, y_dtype=F32, glu=0, x=A,
             x_scales=None, ldx=64, n_x=8, x_index_div=1, x_index=None, w=A, w_scales=None, w_stride=4096,
             ws_stride=0, offsets=A, y=A, ldy=32, n_y=8, reserved=0, y_index=None)
    a.update(kw)
    return B.lib().moe_grouped_gemm(ctypes.byref(GroupedArgs(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), MOE_EINVAL),
    (dict(n_experts=1025), MOE_EINVAL),
    (dict(n_rows=-1), MOE_EINVAL),
    (dict(reserved=1), MOE_EINVAL),
    (dict(x_index_div=0), MOE_EINVAL),
    (dict(x_dtype=F32), MOE_EUNSUPPORTED),
    (dict(w_dtype=F32), MOE_EUNSUPPORTED),
    (dict(x_dtype=MX, x_scales=A), MOE_EUNSUPPORTED),  # bf16 weights
    (dict(glu=2), MOE_EINVAL),
    (dict(glu=1, N=33), MOE_EINVAL),
    (dict(K=60, ldx=64), MOE_EINVAL),
    (dict(w_dtype=MX, w_scales=A, K=40, ldx=40), MOE_EINVAL),
    (dict(w_dtype=MX), MOE_EINVAL),
    (dict(w_scales=A), MOE_EINVAL),
    (dict(w_stride=8), MOE_EINVAL),
    (dict(w_stride=-16), MOE_EINVAL),
    (dict(ws_stride=-1), MOE_EINVAL),
    (dict(offsets=None), MOE_EINVAL),
    (dict(offsets=A + 2), MOE_EINVAL),
    (dict(x_index=A + 1), MOE_EINVAL),
    (dict(n_x=7), MOE_EINVAL),
    (dict(n_x=0, x_index=A), MOE_EINVAL),
    (dict(n_y=7), MOE_EINVAL),
    (dict(ldy=31), MOE_EINVAL),
    (dict(ldy=15, glu=1), MOE_EINVAL),
    (dict(x_index=A, n_x=1 << 24), MOE_EINVAL),        # 2^31 bytes of indexed rows
    (dict(N=1 << 24, ldy=1 << 24), MOE_EINVAL),        # 2^31 bytes per expert
    (dict(n_rows=(1 << 31) - 1, n_x=(1 << 31) - 1, n_y=(1 << 31) - 1), MOE_EINVAL),
    # more workgroups than one launch may have
    (dict(n_rows=(1 << 31) - 8192, n_x=(1 << 31) - 1, n_y=(1 << 31) - 1, N=16384, ldy=16384), MOE_EINVAL),
    (dict(n_rows=0, x=None, w=None, y=None, offsets=None), 0),
])
def test_grouped_refusals(kw, status):
    assert _grouped(**kw) == status


def test_grouped_null_args():
    assert B.lib().moe_grouped_gemm(None, None) == MOE_EINVAL


def test_group_refusals_and_workspace():
    f = B.lib().moe_group_pairs
    assert B.moe_group_workspace(8, 8, 128) == 0
    assert B.moe_group_workspace(0, 8, 128) == 0
    big = B.moe_group_workspace(8192, 8, 256)
    assert 0 < big <= 4 * 256 * (8192 * 8 // 256)
    for bad in ((-1, 8, 128), (8, 0, 128), (8, 8, 0), (8, 8, 1025), (1 << 28, 8, 4), ((1 << 24) + 1, 1, 4)):
        assert B.moe_group_workspace(*bad) == 0
        assert f(A, *bad, A, A, A, 1 << 40, None) == MOE_EINVAL
    assert f(None, 8, 8, 128, A, A, None, 0, None) == MOE_EINVAL
    assert f(A, 8, 8, 128, None, A, None, 0, None) == MOE_EINVAL
    assert f(A, 8, 8, 128, A, None, None, 0, None) == MOE_EINVAL
    assert f(A + 2, 8, 8, 128, A, A, None, 0, None) == MOE_EINVAL
    assert f(A, 8192, 8, 256, A, A, None, 0, None) == MOE_EINVAL
    assert f(A, 8192, 8, 256, A, A, A, big - 1, None) == MOE_EINVAL
    assert f(A, 8192, 8, 256, A, A, A + 2, big, None) == MOE_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(p_dtype=MX), MOE_EUNSUPPORTED), (dict(y_dtype=9), MOE_EUNSUPPORTED), (dict(T=-1), MOE_EINVAL),
    (dict(k=0), MOE_EINVAL), (dict(k=(1 << 30) + 1), MOE_EINVAL), (dict(k=(1 << 31) - 1), MOE_EINVAL), (dict(H=0), MOE_EINVAL), (dict(ldp=63), MOE_EINVAL), (dict(ldy=63), MOE_EINVAL),
    (dict(ids=A, E=0), MOE_EINVAL), (dict(ids=A + 1), MOE_EINVAL), (dict(p=A + 2), MOE_EINVAL),
    (dict(H=(1 << 30) + 1, ldp=1 << 31, ldy=1 << 31), MOE_EINVAL), (dict(w=None), MOE_EINVAL), (dict(w=A + 2), MOE_EINVAL), (dict(T=0, p=None), 0),
])
def test_combine_refusals(kw, status):
    a = dict(p=A, p_dtype=F32, ldp=64, w=A, ids=None, E=4, T=2, k=2, H=64, y=A, y_dtype=F32, ldy=64)
    a.update(kw)
    assert B.lib().moe_combine_pairs(*a.values(), None) == status


def _refused(call, *args, **kw):
    with pytest.raises(B.MoertError) as e:
        call(*args, **kw)
    assert e.value.status == MOE_EINVAL
    return str(e.value)


def test_binding_refusals():
    """Shapes, element types, strides and devices that only the binding sees."""
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    x = torch.zeros(4, 64, dtype=bf)
    codes, scales = torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8)
    assert "GPU" in _refused(B.moe_mx_quantize, x, codes, scales)  # all fits, but the tensors are on the host
    _refused(B.moe_mx_quantize, x.half(), codes, scales)
    _refused(B.moe_mx_quantize, x[:, :40], codes, scales)
    _refused(B.moe_mx_quantize, x, codes[:3], scales)
    _refused(B.moe_mx_quantize, x, codes.int(), scales)
    _refused(B.moe_mx_quantize, x, torch.zeros(4, 64, dtype=u8)[:, ::2], scales)
    _refused(B.moe_mx_quantize, torch.zeros(4, 128, dtype=bf)[:, ::2], codes, scales)
    _refused(B.moe_mx_quantize, x[0], codes, scales)
    _refused(B.moe_mx_dequantize, codes, scales[:, :1], x)
    w, ws, y = torch.zeros(6, 32, dtype=u8), torch.zeros(6, 2, dtype=u8), torch.zeros(4, 6)
    assert "GPU" in _refused(B.moe_mx_gemm, x, w, ws, y)
    assert "GPU" in _refused(B.moe_mx_gemm, codes, w, ws, y, x_scales=scales)
    _refused(B.moe_mx_gemm, x.float(), w, ws, y)
    _refused(B.moe_mx_gemm, x, w, ws, y[:, :5])
    _refused(B.moe_mx_gemm, x, w[:5], ws, y)
    _refused(B.moe_mx_gemm, codes, w, ws, y, x_scales=scales[:3])
    ids, off, perm = torch.zeros(4, 2, dtype=i32), torch.zeros(9, dtype=i32), torch.zeros(8, dtype=i32)
    assert "GPU" in _refused(B.moe_group_pairs, ids, 8, off, perm)
    _refused(B.moe_group_pairs, ids.long(), 8, off, perm)
    _refused(B.moe_group_pairs, ids, 7, off, perm)
    _refused(B.moe_group_pairs, ids, 8, off, perm[:7])
    we, yg = torch.zeros(8, 6, 64, dtype=bf), torch.zeros(8, 6)
    assert "GPU" in _refused(B.moe_grouped_gemm, x, we, off, yg, x_index=perm, x_index_div=2)
    _refused(B.moe_grouped_gemm, x, we, off, yg[:, :3], x_index=perm, x_index_div=2)
    _refused(B.moe_grouped_gemm, x, we, off[:8], yg, x_index=perm)
    _refused(B.moe_grouped_gemm, x, we, off, yg, x_index=perm, y_index=perm[:7])
    _refused(B.moe_grouped_gemm, x, we[:, ::2], off, yg[:, :3], x_index=perm)
    _refused(B.moe_grouped_gemm, x, we[..., :32], off, yg, x_index=perm)
    _refused(B.moe_grouped_gemm, x, we, off, yg, x_index=perm, x_index_div=(1 << 32) + 2)
    _refused(B.moe_grouped_gemm, x, we, off, yg, x_index=perm.long())
    p, cw, cy = torch.zeros(8, 6), torch.zeros(4, 2), torch.zeros(4, 6)
    assert "GPU" in _refused(B.moe_combine_pairs, p, cw, cy)
    _refused(B.moe_combine_pairs, p[:7], cw, cy)
    _refused(B.moe_combine_pairs, p, cw.double(), cy)
    _refused(B.moe_combine_pairs, p, cw, cy[:, :5])
    _refused(B.moe_combine_pairs, p, cw, cy, ids=ids[:3])
    _refused(B.moe_combine_pairs, p, cw, cy, ids=ids, n_experts=1 << 32)


def test_oracle_quantiser():
    """Every grid value comes back, borders take the even code, and the error
    stays within half a step: 1 at most where the magnitude is 4..6 (8 saturates)."""
    from oracle.expert import e2m1_value
    row = np.zeros((1, 32))
    row[0, :16] = [e2m1_value(c) for c in range(16)]
    codes, scales = OO.mx_quantize(row)
    assert scales[0, 0] == 127 and np.array_equal(OO.mx_values(codes, scales), row)
    assert (codes[0, 4] & 15) == 0  # -0 is code 0
    row[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert np.array_equal(OO.mx_values(*OO.mx_quantize(row))[0, :8], [6, 0, 1, 1, 2, 2, 4, 4])
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 256)) * np.exp2(rng.integers(-140, 120, (50, 1)))
    x[0, :32] = 0
    v = OO.mx_values(*OO.mx_quantize(x))
    blocks, err = np.abs(x).reshape(50, 8, 32), np.abs(v - x).reshape(50, 8, 32)
    top = np.maximum(np.exp2(np.floor(np.log2(np.maximum(blocks.max(-1, keepdims=True), 1e-300)))), 2.0 ** -125)
    step = np.where(blocks < top / 2, top / 8, np.where(blocks < top, top / 4, top / 2))
    assert np.all(err <= np.where(blocks >= 1.5 * top, blocks - 1.5 * top + step / 2, step / 2))
    x[1, 5], x[2, 40] = np.inf, np.nan
    codes, scales = OO.mx_quantize(x)
    assert scales[1, 0] == 255 and scales[2, 1] == 255 and not codes[1, :16].any() and scales[1, 1] != 255


@pytest.mark.parametrize("N,K,status", [(1, (1 << 31) - 32, MOE_EINVAL), (2, (1 << 31) - 896, MOE_EINVAL),
                                        (1, (1 << 30) + 32, MOE_EINVAL)])
def test_products_refuse_k_past_the_kernels_cursor(N, K, status):
    """The few-row kernel's waves step through K by 1,024 in 32 bits.  One or two
    rows of 4-bit weights stay below 2^31 bytes with a K that such a cursor would pass."""
    for x in (dict(x_dtype=BF16, ldx=K), dict(x_dtype=MX, xs=A, ldx=K)):
        assert _gemm(N=N, K=K, M=1, ldy=N, **x) == status
        assert "2^30" in B.moe_last_error()
    for x in (dict(x_dtype=BF16), dict(x_dtype=MX, x_scales=A)):
        assert _grouped(N=N, K=K, n_rows=1, ldx=K, w_dtype=MX, w_scales=A, w_stride=K, ldy=N, **x) == status
        assert "2^30" in B.moe_last_error()


def test_combine_refuses_more_workgroups_than_a_launch_has():
    """A column a thread (p off the four-column alignment): 2^24 workgroups of 256
    at H = 2^30, one too many."""
    f = B.lib().moe_combine_pairs
    H = 1 << 30
    assert f(A + 4, F32, H, A, None, 0, 1, 1, H, A, F32, H, None) == MOE_EINVAL
    assert "workgroups" in B.moe_last_error()


def test_gpu_sizes_reach_every_product_variant():
    """The rule that picks a product's kernel, on the sizes of the GPU tests: every
    kernel of every pair of types has one."""
    from tests import test_gpu_ops as G
    f = B.lib().moert_product_variant
    f.argtypes, f.restype = [ctypes.c_int] * 7, ctypes.c_int
    types = {"bf16-bf16": (BF16, BF16), "bf16-mxfp4": (BF16, MX), "mxfp4-mxfp4": (MX, MX)}
    names = ["small16", "small32", "small64", "deep", "shared", "half", "big"]
    assert f(BF16, BF16, 0, 0, 8, 64, 64) == -1
    got = set()
    for fmt in G.FORMATS:
        calls = [(glu, E, T * k, N, K) for T, k, E, N, K in G.GROUPED for glu in (0, 1)]
        calls += [(int(glu), E, T * k, N, K) for T, k, E, N, K, glu in G.GROUPED_TILES + G.GROUPED_VARIANTS]
        if fmt != "bf16-bf16":
            calls += [(0, 1, M, N, K) for M, N, K in G.GEMM + G.GEMM_TILES]
        got |= {(fmt, c[0], names[f(*types[fmt], *c)]) for c in calls}
    want = set()
    for fmt in G.FORMATS:
        w4 = fmt == "bf16-mxfp4"
        want |= {(fmt, 0, n) for n in names if not (w4 and n == "deep")}
        want |= {(fmt, 1, n) for n in ("small16", "small32", "small64", "shared" if w4 else "deep", "big")}
    assert got == want, (sorted(want - got), sorted(got - want))
