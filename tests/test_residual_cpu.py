"""Refusals of the norms around a block, before anything is launched (no GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import routing_grouped_gemm_gb300 as m
    return m


def _rc(moe, **kw):
    return moe.ResidualConfig(**(dict(T=4, D=64) | kw))


@pytest.mark.parametrize("bad,unsupported", [
    (dict(T=-1), False), (dict(D=12), False), (dict(D=0), False), (dict(D=32776), True), (dict(dtype=2), False),
    (dict(gate=4), False), (dict(gate=-1), False), (dict(eps=0.0), False), (dict(eps=float("nan")), False),
    (dict(eps=float("inf")), False), (dict(res_scale=float("inf")), False), (dict(branch_scale=float("nan")), False),
    (dict(p_drop=-0.1), False), (dict(p_drop=1.0), False), (dict(p_drop=0.999999), False),
    (dict(p_drop=float("nan")), False), (dict(p_drop=float("inf")), False),
])
def test_bad_configs(moe, bad, unsupported):
    rc = _rc(moe, **bad)
    assert moe.residual_workspace_size(rc) == -1
    st = moe._lib.moe_residual_norm(ctypes.byref(rc.c()), 16, 16, None, None, 16, None, 16, 16, None)
    assert st == (moe.MOE_ERR_UNSUPPORTED if unsupported else moe.MOE_ERR_INVALID_ARG)
    with pytest.raises(moe.MoeError):
        moe.alloc_residual_workspace(rc)


def test_workspace_size(moe):
    assert moe.residual_workspace_size(_rc(moe, T=0)) == 0
    for T, D in ((1, 8), (4096, 2048), (16384, 32768)):
        n = moe.residual_workspace_size(_rc(moe, T=T, D=D))
        assert n % 256 == 0 and n >= 8 * D


# resid, y, post, gate, pre, rng, resid_out, norm_out
@pytest.mark.parametrize("over,rc", [
    (dict(resid=None), {}), (dict(resid=8), {}), (dict(y=8), {}), (dict(y=None), {}), (dict(resid_out=None), {}),
    (dict(resid_out=24), {}), (dict(norm_out=None), {}), (dict(pre=None), {}), (dict(norm_out=8), {}),
    (dict(post=8), {}), (dict(gate=16), {}), ({}, dict(gate=1)), (dict(gate=8), dict(gate=1)), ({}, dict(p_drop=0.5)),
    (dict(rng=4), dict(p_drop=0.5)), (dict(y=None, resid_out=None, post=16), {}),
    (dict(y=None, resid_out=None, gate=16), dict(gate=1)), (dict(y=None, resid_out=None, rng=16), dict(p_drop=0.5)),
    (dict(y=None, resid_out=None, pre=None, norm_out=None), {}),
])
def test_forward_refusals(moe, over, rc):
    a = dict(resid=16, y=16, post=None, gate=None, pre=16, rng=None, resid_out=16, norm_out=16) | over
    before = moe.kernel_launches()
    assert moe._lib.moe_residual_norm(ctypes.byref(_rc(moe, **rc).c()), *a.values(), None) == moe.MOE_ERR_INVALID_ARG
    assert moe.kernel_launches() == before


@pytest.mark.parametrize("over,rc,status", [
    (dict(s=None), {}, 1), (dict(s=8), {}, 1), (dict(y=None), {}, 1), (dict(dy=None), {}, 1), (dict(dresid=None), {}, 1),
    (dict(dn=None), {}, 1), (dict(pre=None), {}, 1), (dict(dpre=None), {}, 1), (dict(dpre=24), {}, 1),
    (dict(post=16), {}, 1), (dict(dpost=16), {}, 1), (dict(dgate=16), {}, 1), (dict(gate=16), dict(gate=2), 1),
    (dict(dso=8), {}, 1), (dict(dso=None, dn=None, pre=None, dpre=None), {}, 1), ({}, dict(p_drop=0.5), 1),
    (dict(ws=None), {}, 7), (dict(ws=128), {}, 7), (dict(n=100), {}, 7),
])
def test_backward_refusals(moe, over, rc, status):
    a = dict(s=16, y=16, post=None, gate=None, pre=16, rng=None, dso=16, dn=16, dresid=16, dy=16, dpost=None,
             dgate=None, dpre=16, ws=256, n=1 << 20) | over
    before = moe.kernel_launches()
    assert moe._lib.moe_residual_norm_backward(ctypes.byref(_rc(moe, **rc).c()), *a.values(), None) == status
    assert moe.kernel_launches() == before


def test_combine_refusals(moe):
    cfg = moe.Config(T=4, D=64, H_local=64, E=8, k=2)
    n = moe.workspace_size(cfg)
    base = dict(y_perm=16, row_of=16, topk_w=16, resid=16, post=None, gate=None, pre=16, rng=None, y_out=None,
                resid_out=16, norm_out=16, ws=256, n=n)
    for over, rc, status in ((dict(y_perm=None), {}, 1), (dict(row_of=None), {}, 1), (dict(topk_w=8), {}, 1),
                             (dict(resid=None), {}, 1), (dict(resid_out=None), {}, 1), (dict(y_out=8), {}, 1),
                             (dict(norm_out=None), {}, 1), (dict(gate=16), {}, 1), ({}, dict(gate=1), 1),
                             ({}, dict(p_drop=0.5), 1), ({}, dict(T=5), 1), ({}, dict(D=128), 1), ({}, dict(dtype=0), 1),
                             (dict(ws=None), {}, 7), (dict(ws=64), {}, 7), (dict(n=n - 1), {}, 7)):
        st = moe._lib.moe_combine_residual_norm(cfg.ref()[0], ctypes.byref(_rc(moe, **rc).c()), *(base | over).values(), None)
        assert st == status, (over, rc)


def test_missing_tensors_are_named(moe):
    rc = _rc(moe)
    cfg = moe.Config(T=4, D=64, H_local=64, E=8, k=2)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="resid is required"):
        moe.moe_residual_norm(rc, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="ws is required"):
        moe.moe_combine_residual_norm(cfg, rc, *[None] * 11, None)
    with pytest.raises(ValueError, match="ws is on cpu"):
        moe.moe_residual_norm_backward(rc, *[None] * 13, ws)
    with pytest.raises(ValueError, match="no kind of gate"):
        moe.moe_residual_norm_backward(rc, *[None] * 11, torch.zeros(64), None, ws)


# ---------------------------------------------------------------------------
# the layer for a few tokens
# ---------------------------------------------------------------------------

def test_few_refusals(moe):
    cfg = moe.Config(T=4, D=64, H_local=64, E=8, k=2)
    n = moe.layer_few_workspace_size(cfg)
    assert n % 256 == 0 and n > 256
    base = dict(x=16, wg=16, bias=None, w1=16, w3=16, w2=16, out=16, ws=256, n=n)
    before = moe.kernel_launches()

    def call(c, **over):
        return moe._lib.moe_layer_forward_few(c.ref()[0], *(base | over).values(), None)
    for over, status in ((dict(x=None), 1), (dict(wg=8), 1), (dict(bias=8), 1), (dict(w1=None), 1), (dict(w3=8), 1),
                         (dict(w2=None), 1), (dict(out=None), 1), (dict(ws=None), 7), (dict(ws=128), 7), (dict(n=n - 1), 7)):
        assert call(cfg, **over) == status, over
    many = moe.Config(T=33, D=64, H_local=64, E=8, k=2)
    assert moe.layer_few_workspace_size(many) == -1
    assert call(many) == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError):
        moe.alloc_workspace(many, few=True)
    assert call(moe.Config(T=4, D=12, H_local=64, E=8, k=2)) == moe.MOE_ERR_INVALID_ARG
    assert call(moe.Config(T=0, D=64, H_local=64, E=8, k=2), x=None, out=None) == moe.MOE_OK
    assert moe.kernel_launches() == before
    with pytest.raises(ValueError, match="ws is required"):
        moe.moe_layer_forward_few(cfg, *[None] * 7, None)


def test_a_changed_config_is_taken(moe):
    rc = moe.ResidualConfig(T=4, D=64)
    assert rc.ref()[0].contents.eps == pytest.approx(1e-6) and rc.ref()[4] is None and rc.ref() is rc.ref()
    rc.eps, rc.gate, rc.T = 0.5, moe.MOE_GATE_TOKEN, 7
    c, rows, gain, dt, gate = rc.ref()
    assert (c.contents.eps, c.contents.gate, c.contents.T, rows) == (0.5, moe.MOE_GATE_TOKEN, 7, (7, 64))
    assert gate == ((7,), torch.float32) and gain == (64,) and dt is torch.bfloat16
