"""Host-side checks of the MXFP4 calls and of the step gradients: the numpy
definition against the format's own values, and every refusal before a launch."""
import ctypes

import numpy as np
import pytest

import mx_reference as mx


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import routing_grouped_gemm_gb300 as m
    return m


def test_reference_rounds_to_nearest_even():
    a = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2500001, 4.999, 7.9, -0.75, -5.0])
    assert mx.round_e2m1(a).tolist() == [0, 1, 1, 2, 2, 4, 4, 0.5, 4, 6, -1, -4]


def test_reference_scales():
    x = np.zeros((9, 32))
    x[1, 3] = 4.0                  # floor(log2 4) - 2 = 0
    x[2, 0] = 7.99                 # saturates: same scale as 4
    x[3, 0] = 8.0
    x[4, 31] = 2.0 ** -140         # below the smallest scale
    x[5, 5] = np.finfo(np.float32).max
    x[6, 0], x[7, 0] = np.nan, np.inf
    x[8] = -1e-3
    v, b = mx.quantize(x)
    assert b[:, 0].tolist() == [0, 127, 127, 128, 0, 252, 255, 255, 115]
    assert v[1, 3] == 4 and v[2, 0] == 6 and v[3, 0] == 8 and v[4, 31] == 0
    assert np.isnan(v[6]).all() and np.isnan(v[7]).all()
    ok = [0, 1, 2, 3, 4, 5, 8]
    assert np.array_equal(mx.values(mx.pack(v[ok], b[ok]), b[ok]), v[ok])


def _cfg(moe, **kw):
    base = dict(T=64, D=128, H_local=64, E=8, k=2, dtype=moe.MOE_BF16)
    base.update(kw)
    return moe.Config(**base)


def test_quantize_refusals(moe):
    lib, bad, ok = moe._lib, moe.MOE_ERR_INVALID_ARG, moe.MOE_OK
    n0 = moe.kernel_launches()
    q = lib.moe_quantize_rows_mxfp4
    d = lib.moe_dequantize_rows_mxfp4
    assert q(256, moe.MOE_BF16, 4, 48, 256, 256, None) == bad       # not whole blocks
    assert q(256, moe.MOE_BF16, 4, 0, 256, 256, None) == bad
    assert q(256, moe.MOE_BF16, -1, 64, 256, 256, None) == bad
    assert q(256, 7, 4, 64, 256, 256, None) == bad                  # no such type
    assert q(None, moe.MOE_F32, 4, 64, 256, 256, None) == bad
    assert q(264, moe.MOE_F32, 4, 64, 256, 256, None) == bad        # misaligned
    assert q(256, moe.MOE_F32, 4, 64, 256, 264, None) == bad
    assert q(256, moe.MOE_F32, 1 << 62, 64, 256, 256, None) == bad  # rows * cols overflows
    assert q(None, moe.MOE_F32, 0, 64, None, None, None) == ok      # nothing to do
    assert d(256, 256, 4, 33, 256, moe.MOE_F32, None) == bad
    assert d(256, 256, 4, 64, 256, 2, None) == bad
    assert d(256, None, 4, 64, 256, moe.MOE_F32, None) == bad
    assert d(256, 256, 4, 64, 258, moe.MOE_BF16, None) == bad
    assert d(None, None, 0, 64, None, moe.MOE_BF16, None) == ok
    assert moe.kernel_launches() == n0


@pytest.mark.parametrize("over", [dict(dtype=0), dict(D=136), dict(H_local=72)])
def test_mxfp4_unsupported_configs(moe, over):
    cfg = _cfg(moe, **over)
    assert moe.validate_config(cfg) == moe.MOE_OK
    c, p = ctypes.byref(cfg.c()), 256
    n = moe.layer_workspace_size(cfg)
    lib, un = moe._lib, moe.MOE_ERR_UNSUPPORTED
    n0 = moe.kernel_launches()
    assert lib.moe_permute_mxfp4(c, *[p] * 8, p, n, None) == un
    assert lib.moe_grouped_swiglu_mxfp4(c, *[p] * 13, p, n, None) == un
    assert lib.moe_layer_forward_mxfp4(c, p, p, None, *[p] * 7, p, n, None) == un
    assert moe.kernel_launches() == n0


def test_mxfp4_bad_tensors_and_workspaces(moe):
    cfg = _cfg(moe)
    c, p = ctypes.byref(cfg.c()), 256
    n = moe.layer_workspace_size(cfg)
    lib, bad, wserr = moe._lib, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE
    n0 = moe.kernel_launches()
    assert lib.moe_permute_mxfp4(c, *[p] * 8, None, n, None) == wserr
    assert lib.moe_permute_mxfp4(c, *[p] * 8, p, 256, None) == wserr
    assert lib.moe_permute_mxfp4(c, *[p] * 8, p + 16, n, None) == wserr
    for i in range(8):                        # each tensor NULL in turn
        a = [p] * 8
        a[i] = None
        assert lib.moe_permute_mxfp4(c, *a, p, n, None) == bad, i
    for i in range(13):
        a = [p] * 13
        a[i] = None
        assert lib.moe_grouped_swiglu_mxfp4(c, *a, p, n, None) == bad, i
        if i not in (2, 3):                   # the int32 arrays need no 16 bytes
            a[i] = p + 8
            assert lib.moe_grouped_swiglu_mxfp4(c, *a, p, n, None) == bad, i
    assert lib.moe_layer_forward_mxfp4(c, p, p, None, *[p] * 7, p, n - 1, None) == wserr
    for i in range(7):
        a = [p] * 7
        a[i] = p + 8
        assert lib.moe_layer_forward_mxfp4(c, p, p, None, *a, p, n, None) == bad, i
    assert moe.kernel_launches() == n0


def test_step_gradient_refusals(moe):
    cfg = _cfg(moe)
    c, p = ctypes.byref(cfg.c()), 256
    n = moe.workspace_size(cfg)
    lib, bad = moe._lib, moe.MOE_ERR_INVALID_ARG
    n0 = moe.kernel_launches()
    for i in range(6):
        a = [p] * 6
        a[i] = None
        assert lib.moe_unpermute_combine_backward(c, *a, p, n, None) == bad, i
    assert lib.moe_unpermute_combine_backward(c, *[p] * 6, None, n, None) == moe.MOE_ERR_WORKSPACE
    assert lib.moe_permute_backward(c, p, 5, p, p, p, n, None) == bad
    assert lib.moe_permute_backward(c, p + 8, moe.MOE_F32, p, p, p, n, None) == bad
    assert lib.moe_permute_backward(c, p, moe.MOE_F32, None, p, p, n, None) == bad
    assert lib.moe_permute_backward(c, p, moe.MOE_F32, p, None, p, n, None) == bad
    assert lib.moe_permute_backward(c, p, moe.MOE_F32, p, p, p, n - 1, None) == moe.MOE_ERR_WORKSPACE
    f32 = _cfg(moe, dtype=moe.MOE_F32)
    assert lib.moe_permute_backward(ctypes.byref(f32.c()), p, moe.MOE_BF16, p, p, p, 1 << 30,
                                    None) == moe.MOE_ERR_UNSUPPORTED
    empty = ctypes.byref(_cfg(moe, T=0).c())
    assert lib.moe_permute_backward(empty, None, moe.MOE_F32, None, None, p, n, None) == moe.MOE_OK
    assert lib.moe_unpermute_combine_backward(empty, *[None] * 6, p, n, None) == moe.MOE_OK
    assert moe.kernel_launches() == n0
