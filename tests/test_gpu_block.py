"""A training step of a block around the layer, as the calls would be used together: norm, layer, norm with
dropout and residual sum, and back through all three, against automatic differentiation in 64 bits."""
import pytest
import torch

import residual_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _rms(x, gain, eps):
    return x / torch.sqrt(x.square().mean(1, keepdim=True) + eps) * gain


def test_training_step_of_a_block(moe):
    T, D, H, E, k, p = 192, 128, 64, 4, 2, 0.25
    g = torch.Generator(device="cuda").manual_seed(5)

    def n(*s, scale=1.0):
        return (scale * torch.randn(s, generator=g, device="cuda")).bfloat16()
    resid, pre, post, after, gate = n(T, D, scale=2), 1 + n(D, scale=0.2), 1 + n(D, scale=0.2), 1 + n(D, scale=0.2), n(D)
    wg, w1, w3, w2 = n(E, D, scale=0.2), n(E, H, D, scale=0.1), n(E, H, D, scale=0.1), n(E, D, H, scale=0.1)
    ds, dn = n(T, D), n(T, D)
    rng = torch.tensor([11, 3], device="cuda")
    cfg = moe.Config(T=T, D=D, H_local=H, E=E, k=k, renorm=1, align_m=64)
    rc0 = moe.ResidualConfig(T=T, D=D)
    rc = moe.ResidualConfig(T=T, D=D, gate=moe.MOE_GATE_CHANNEL, branch_scale=0.5, p_drop=p)
    x, y, s, o = (torch.empty_like(resid) for _ in range(4))
    ws = moe.alloc_workspace(cfg, train=True)
    moe.moe_residual_norm(rc0, resid, None, None, None, pre, None, None, x)
    moe.moe_layer_forward_train(cfg, x, wg, None, w1, w3, w2, y, ws)
    moe.moe_residual_norm(rc, resid, y, post, gate, after, rng, s, o)
    f = [torch.empty(D, device="cuda") for _ in range(4)]
    dsum, dy, dx, dresid = (torch.empty_like(resid) for _ in range(4))
    dwg, dw1, dw3, dw2 = (torch.empty(w.shape, device="cuda") for w in (wg, w1, w3, w2))
    rws = moe.alloc_residual_workspace(rc)
    moe.moe_residual_norm_backward(rc, s, y, post, gate, after, rng, ds, dn, dsum, dy, f[0], f[1], f[2], rws)
    moe.moe_layer_backward(cfg, x, wg, w1, w3, w2, dy, dx, dwg, None, dw1, dw3, dw2, ws)
    # the first norm's gradient takes the residual's as what flows past it
    moe.moe_residual_norm_backward(rc0, resid, None, None, None, pre, None, dsum, dx, dresid, None, None, None, f[3], rws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK

    leaves = {m: v.double().cpu().requires_grad_() for m, v in dict(resid=resid, pre=pre, post=post, after=after,
                                                                    gate=gate, wg=wg, w1=w1, w3=w3, w2=w2).items()}
    v = leaves
    xr = _rms(v["resid"], v["pre"], 1e-6)
    key = xr @ v["wg"].T
    # the experts that the kernels chose, from the x that they had (a choice within rounding has no single answer)
    idx = torch.topk(x.double().cpu() @ wg.double().cpu().T, k, dim=1).indices
    prob = torch.softmax(torch.gather(key, 1, idx), dim=1)
    yr = torch.zeros(T, D, dtype=torch.float64)
    for j in range(k):
        e = idx[:, j]
        gt = torch.einsum("thd,td->th", v["w1"][e], xr)
        h = gt * torch.sigmoid(gt) * torch.einsum("thd,td->th", v["w3"][e], xr)
        yr = yr + prob[:, j:j + 1] * torch.einsum("tdh,th->td", v["w2"][e], h)
    sr = v["resid"] + 0.5 * v["gate"] * ref.keep(T, D, p, (11, 3)) * _rms(yr, v["post"], 1e-6)
    orf = _rms(sr, v["after"], 1e-6)
    ((sr * ds.double().cpu()).sum() + (orf * dn.double().cpu()).sum()).backward()

    def close(got, want, name, tol):
        got, want = got.double().cpu(), want.detach()
        err = (got - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert err <= tol, f"{name}: {err}"
    # Every bf16 tensor on the way (x, h, y and its fp16 rows, s; backwards dsum, dy, the layer's dh and dg | du, dx)
    # is off by at most 2^-8 of itself, evenly spread: 2^-8 / sqrt 3 = 0.0023 RMS.  Forward, four of them meet in s
    # and o; backward, up to ten in a gradient: sqrt(4) and sqrt(10) of it, and half as much again for the factors
    # that the two norms' means take from rows that are off themselves.
    for got, want, name in ((s, sr, "s"), (o, orf, "o")):
        close(got, want, name, 1.5 * 4 ** 0.5 * 0.0023)
    for got, m in ((dresid, "resid"), (f[3], "pre"), (f[0], "post"), (f[1], "gate"), (f[2], "after"), (dwg, "wg"),
                   (dw1, "w1"), (dw3, "w3"), (dw2, "w2")):
        close(got, v[m].grad, m, 1.5 * 10 ** 0.5 * 0.0023)
