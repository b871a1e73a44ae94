"""Host-side refusals of dsa_norm_q8, dsa_gemm_q8 and dsa_cache_append: decided before anything reaches the GPU."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa

P = ctypes.c_void_p
INVALID, UNSUPPORTED, OK = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_OK


def norm(n=4, dim=256, x=P(4096), x_ld=256, residual=None, residual_ld=0, gamma=P(4096), eps=1e-6, total=None, sum_ld=0,
         out=P(4096), scale=P(4096)):
    return dsa._lib.dsa_norm_q8(n, dim, x, x_ld, residual, residual_ld, gamma, eps, total, sum_ld, out, scale, None)


def gemm(m=4, n=256, k=256, groups=1, a=P(4096), a_ld=None, a_scale=P(4096), a_scale_ld=None, w=P(4096), w_scale=P(4096),
         fmt=dsa.DSA_BF16, out=P(4096), out_ld=None, out_scale=None):
    return dsa._lib.dsa_gemm_q8(m, n, k, groups, a, groups * k if a_ld is None else a_ld, a_scale,
                                groups * -(-k // 128) if a_scale_ld is None else a_scale_ld, w, w_scale, fmt, out,
                                groups * n if out_ld is None else out_ld, out_scale, None, None)


def append(batch=2, cu=P(4096), start=P(4096), n=4, x=P(4096), x_ld=512, norm=1, gamma=P(4096), eps=1e-6, rope=(64, 1e4),
           pool=(4096, None, 4, 256, 512, dsa.DSA_BF16), bt=(4096, 2, 4)):
    r, p, t = dsa.DsaRope(*rope), dsa.DsaPool(*pool), dsa.DsaBlockTable(*bt)
    return dsa._lib.dsa_cache_append(batch, cu, start, n, x, x_ld, norm, gamma, eps, ctypes.byref(r), ctypes.byref(p),
                                     ctypes.byref(t), None, None)


@pytest.mark.parametrize("want,args", [
    (OK, dict(n=0)), (INVALID, dict(n=-1)), (INVALID, dict(dim=0)), (UNSUPPORTED, dict(dim=250)),
    (UNSUPPORTED, dict(dim=16400)), (INVALID, dict(x=None)), (INVALID, dict(x=P(4104))), (INVALID, dict(x_ld=250)),
    (INVALID, dict(x_ld=248)), (INVALID, dict(residual=P(4096), residual_ld=128)), (INVALID, dict(residual=P(4098), residual_ld=256)),
    (INVALID, dict(total=P(4096), sum_ld=0)), (INVALID, dict(gamma=P(4100))), (INVALID, dict(eps=0.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))), (INVALID, dict(out=None)),
    (INVALID, dict(out=P(4100))), (INVALID, dict(scale=None)), (INVALID, dict(scale=P(4098)))])
def test_norm_refusals(want, args):
    assert norm(**args) == want


@pytest.mark.parametrize("want,args", [
    (OK, dict(m=0)), (INVALID, dict(m=-1)), (INVALID, dict(n=0)), (INVALID, dict(k=0)), (INVALID, dict(groups=0)),
    (UNSUPPORTED, dict(k=264)), (UNSUPPORTED, dict(n=1 << 21, k=1 << 19)), (INVALID, dict(a=None)), (INVALID, dict(a=P(4104))),
    (INVALID, dict(w=P(4104))), (INVALID, dict(a_scale=None)), (INVALID, dict(w_scale=None)), (INVALID, dict(a_scale=P(4098))),
    (INVALID, dict(a_ld=255)), (INVALID, dict(a_ld=240)), (INVALID, dict(a_ld=264)), (INVALID, dict(a_scale_ld=1)),
    (INVALID, dict(out=None)), (INVALID, dict(out=P(4097))), (INVALID, dict(out_ld=255)), (INVALID, dict(groups=2, a_ld=256)),
    (INVALID, dict(fmt=dsa.DSA_FP4_BLOCK)), (INVALID, dict(fmt=dsa.DSA_FP8_E4M3)), (INVALID, dict(fmt=dsa.DSA_FP32, out=P(4098))),
    (UNSUPPORTED, dict(a_ld=1 << 40)), (UNSUPPORTED, dict(out_ld=1 << 38))])
def test_gemm_refusals(want, args):
    assert gemm(**args) == want


@pytest.mark.parametrize("want,args", [
    (OK, dict(n=0)), (OK, dict(batch=0)), (INVALID, dict(n=-1)), (INVALID, dict(batch=-1)), (INVALID, dict(cu=None)),
    (INVALID, dict(start=None)), (INVALID, dict(x=None)), (INVALID, dict(x=P(4104))), (INVALID, dict(x_ld=504)),
    (INVALID, dict(x_ld=516)), (INVALID, dict(eps=0.0)), (INVALID, dict(gamma=P(4098))), (INVALID, dict(rope=(63, 1e4))),
    (INVALID, dict(rope=(-2, 1e4))), (INVALID, dict(rope=(64, 0.0))), (UNSUPPORTED, dict(rope=(128, 1e4))),
    (INVALID, dict(bt=(4096, 1, 4))), (INVALID, dict(bt=(None, 2, 4))), (INVALID, dict(pool=(4096, None, 4, 256, 512, 1))),
    (UNSUPPORTED, dict(pool=(4096, None, 4, 256, 256, 0))), (UNSUPPORTED, dict(pool=(4096, 4096, 4, 256, 128, 3), x_ld=128))])
def test_append_refusals(want, args):
    assert append(**args) == want


def test_plans_host_only():
    assert dsa.dsa_gemm_q8_plan(1, 512, 4096)[1] == 16
    for m in (1, 16, 17, 64, 65, 300, 1000, 8192):
        for n, k, g in ((64, 16, 1), (1024, 4096, 8), (32768, 4096, 1), (520, 1040, 3)):
            feat, rows, share = dsa.dsa_gemm_q8_plan(m, n, k, g)
            assert feat % 128 == 0 and rows in (16, 32, 64, 128, 256) and 1 <= share <= 8
    with pytest.raises(dsa.DsaError):
        dsa.dsa_gemm_q8_plan(0, 64, 64)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_gemm_q8_plan(4, 64, 72)


def test_stalled_hook_limits_host_only():
    f = dsa._lib.dsa_debug_gemm_q8_stalled
    args = [4, 256, 256, 1, P(4096), 256, P(4096), 2, P(4096), P(4096), dsa.DSA_BF16, P(4096), 256, None]
    assert f(*args, 0, None, None) == INVALID and f(*args, 2000000001, None, None) == INVALID
    args[0] = 0
    assert f(*args, 5, None, None) == OK


def _cpu_norm(**over):
    n, d = 4, 256
    args = dict(x=torch.zeros((n, d), dtype=torch.bfloat16), gamma=torch.ones(d), eps=1e-6, out=torch.zeros((n, d), dtype=torch.uint8),
                out_scale=torch.zeros((n, 2)))
    args.update(over)
    return lambda: dsa.dsa_norm_q8(**args)


def _cpu_gemm(**over):
    args = dict(a=torch.zeros((4, 2, 256), dtype=torch.uint8), a_scale=torch.ones((4, 2, 2)), w=torch.zeros((2, 130, 256), dtype=torch.uint8),
                w_scale=torch.ones((2, 2, 2)), out=torch.zeros((4, 2, 130)))
    args.update(over)
    return lambda: dsa.dsa_gemm_q8(**args)


def _cpu_append(**over):
    args = dict(cu_new=torch.zeros(3, dtype=torch.int32), start_pos=torch.zeros(2, dtype=torch.int32),
                x=torch.zeros((4, 64), dtype=torch.bfloat16), rope_cfg=dsa.rope(64), pool_=dsa.DsaPool(4096, None, 4, 256, 64, 0),
                bt=dsa.DsaBlockTable(4096, 2, 4))
    args.update(over)
    return lambda: dsa.dsa_cache_append(**args)


@pytest.mark.parametrize("call", [
    _cpu_norm(),                                                       # not on the current device
    _cpu_norm(x=torch.zeros((4, 256))), _cpu_norm(x=torch.zeros((256, 4), dtype=torch.bfloat16).t()),
    _cpu_norm(x=torch.zeros(256, dtype=torch.bfloat16)), _cpu_norm(gamma=torch.ones(128)), _cpu_norm(gamma=torch.ones(256).double()),
    _cpu_norm(out=torch.zeros((4, 512), dtype=torch.uint8)[:, ::2]), _cpu_norm(out_scale=torch.zeros((4, 3))),
    _cpu_norm(residual=torch.zeros((3, 256), dtype=torch.bfloat16)), _cpu_norm(sum_out=torch.zeros((4, 256))),
    _cpu_gemm(), _cpu_gemm(a=torch.zeros((4, 512), dtype=torch.uint8)), _cpu_gemm(a=torch.zeros((4, 256, 2), dtype=torch.uint8).transpose(1, 2)),
    _cpu_gemm(a=torch.zeros((4, 2, 256), dtype=torch.int32)), _cpu_gemm(a_scale=torch.ones((4, 2, 1))), _cpu_gemm(w=torch.zeros((130, 256), dtype=torch.uint8)),
    _cpu_gemm(w=torch.zeros((2, 256, 130), dtype=torch.uint8).transpose(1, 2)), _cpu_gemm(w_scale=torch.ones((2, 2, 2)).double()),
    _cpu_gemm(w_scale=torch.ones((2, 1, 2))), _cpu_gemm(out=torch.zeros((4, 2, 130), dtype=torch.float16)),
    _cpu_gemm(out=torch.zeros((4, 2, 130), dtype=torch.uint8)), _cpu_gemm(out=torch.zeros((4, 130, 2)).transpose(1, 2)),
    _cpu_append(), _cpu_append(x=torch.zeros((4, 64))), _cpu_append(x=torch.zeros((4, 128), dtype=torch.bfloat16)),
    _cpu_append(cu_new=torch.zeros(2, dtype=torch.int32)), _cpu_append(cu_new=torch.zeros(3, dtype=torch.int64)),
    _cpu_append(start_pos=torch.zeros(4, dtype=torch.int32)[::2]), _cpu_append(rms_gamma=torch.ones(32))])
def test_tensors_that_the_call_cannot_see_are_refused(call):
    with pytest.raises(dsa.DsaError) as e:
        call()
    assert e.value.code == INVALID
