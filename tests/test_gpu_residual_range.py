"""The norms around a block where fp32 could spoil a result: rows far from one, rows of zeros at a tiny eps,
infinities where a form does not look.

Bounds as in test_gpu_residual_norm: what fp32 may add (residual_reference derives it, relative to the terms, so it
holds at any scale) plus half a step of the output's type.
"""
import pytest
import torch

from test_gpu_residual_norm import (GATES, _case, _check_forward, _check_gradient, _forward, _gradient, _keep,
                                    moe)  # noqa: F401

pytestmark = pytest.mark.gpu

# a row per warp with one and with two vectors a lane, per CTA with one and with two, without a ring
SHAPES = [(37, 136), (21, 392), (9, 1048), (5, 4104), (3, 8200)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["channel", "token", "element"])
@pytest.mark.parametrize("scale", [1e13, 1e15, 1e17])
@pytest.mark.parametrize("T,D", SHAPES)
def test_gradient_of_large_rows(moe, T, D, scale, gate, dtype):
    """Rows of `scale`, whose squares' sum (at most 8200 e34) fp32 holds.  dnorm_out has the same scale and leans
    towards s, so that every term of ds is about one."""
    rc, t, n = _case(moe, T, D, dtype, gate, res_scale=0.7)
    s = n(T, D, to=torch.float32)
    t["pre"] = t["pre"].abs()
    t["resid"], t["y"] = (scale * s).to(rc.torch_dtype), n(T, D, scale=scale)
    dn = (scale * (n(T, D, to=torch.float32) + s)).to(rc.torch_dtype)
    for dso in (n(T, D), None):
        _check_gradient(rc, t, gate, dso, dn, _gradient(moe, rc, t, gate, dso, dn))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["channel", "token", "element"])
@pytest.mark.parametrize("T,D", SHAPES)
def test_gradient_of_rows_of_zeros_and_small_rows_at_a_tiny_eps(moe, T, D, gate, dtype):
    rc, t, n = _case(moe, T, D, dtype, gate, eps=1e-30)
    t["resid"][0] = t["y"][0] = 0
    t["resid"][1] *= 1e-14
    t["y"][1] *= 1e-14
    dn = n(T, D)
    for dso in (n(T, D), None):
        _check_gradient(rc, t, gate, dso, dn, _gradient(moe, rc, t, gate, dso, dn))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("T,D", SHAPES)
def test_gradient_without_the_next_norm_does_not_look_at_s(moe, T, D, gate, dtype):
    """Without pre_gain ds is dresid_out, whatever s holds (a residual that overflowed, say)."""
    rc, t, n = _case(moe, T, D, dtype, gate, pre=False, p=0.2)
    dso = n(T, D)
    want = _gradient(moe, rc, t, gate, dso, None)
    _check_gradient(rc, t, gate, dso, None, want)
    t["resid"][0, 3], t["resid"][1, D - 1], t["resid"][2] = float("inf"), float("nan"), 3e38
    got = _gradient(moe, rc, t, gate, dso, None)
    assert all(want[k] is None or torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("T,D", SHAPES)
def test_gradient_without_the_branch_norm_keeps_y_out_of_dy(moe, T, D, gate, pre, dtype):
    """Without post_gain dy = gate u does not depend on y: an infinity there reaches the gate's gradient alone."""
    rc, t, n = _case(moe, T, D, dtype, gate, post=False, pre=pre)
    dso, dn = n(T, D), n(T, D) if pre else None
    want = _gradient(moe, rc, t, gate, dso, dn)
    _check_gradient(rc, t, gate, dso, dn, want)
    t["y"][1, 5], t["y"][2, D - 2] = float("inf"), float("nan")
    got = _gradient(moe, rc, t, gate, dso, dn)
    for k in want:
        if want[k] is None:
            continue
        same = torch.ones_like(want[k], dtype=torch.bool)
        if k == "dgate":
            same[(..., [5, D - 2]) if gate == "channel" else [1, 2] if gate == "token" else ([1, 2], [5, D - 2])] = False
            assert not got[k][~same].isfinite().any()
        assert torch.equal(got[k][same], want[k][same]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("T,D", [(5, 72), (2500, 72), (5, 1048), (1300, 1048), (3, 8200)])
def test_a_dropped_element_adds_nothing(moe, T, D, post, dtype):
    """Infinities and NaN in dropped places -- of a gate for every element, and of y where it has no norm -- change
    nothing, forward (few rows and many take different kernels) and gradient."""
    rc, t, n = _case(moe, T, D, dtype, "element", post=post, p=0.5)
    dso, dn = n(T, D), n(T, D)
    want, dwant = _forward(moe, rc, t), _gradient(moe, rc, t, "element", dso, dn)
    gone = (_keep(rc, t) == 0).cuda()
    for name, bad in (("gate", float("inf")), ("gate", float("nan")), ("y", float("inf")), ("y", float("nan"))):
        if name == "y" and post:
            continue
        u = dict(t, **{name: t[name].masked_fill(gone, bad)})
        got, dgot = _forward(moe, rc, u), _gradient(moe, rc, u, "element", dso, dn)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(dwant[k] is None or torch.equal(dgot[k], dwant[k]) for k in dwant)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("T,D", [(5, 72), (2500, 72), (5, 1048), (1300, 1048), (3, 8200)])
def test_a_dropped_element_under_an_infinite_shared_gate(moe, T, D, gate, dtype):
    rc, t, n = _case(moe, T, D, dtype, gate, p=0.5, pre=False)
    gone = (_keep(rc, t) == 0).cuda()
    t["gate"][2] = float("inf")
    r, _ = _forward(moe, rc, t)
    assert torch.equal(r[gone], t["resid"][gone])
    there = ~gone[:, 2] if gate == "channel" else ~gone[2]
    assert not (r[:, 2] if gate == "channel" else r[2])[there].isfinite().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_dropped_element(moe, dtype):
    rc, t, n = _case(moe, 9, 264, dtype, "element", p=0.5)
    cfg = moe.Config(T=9, D=264, H_local=64, E=1, k=1, align_m=1, dtype=rc.dtype)
    yp = n(9, 264, to=torch.float16 if dtype == "bf16" else torch.float32)
    row, w = torch.arange(9, device="cuda").int()[:, None].contiguous(), torch.ones(9, 1, device="cuda")
    ws = moe.alloc_workspace(cfg)

    def call(gate):
        out = [torch.empty_like(t["resid"]) for _ in range(3)]
        moe.moe_combine_residual_norm(cfg, rc, yp, row, w, t["resid"], t["post"], gate, t["pre"], t["rng"], *out, ws)
        return out
    got = call(t["gate"].masked_fill((_keep(rc, t) == 0).cuda(), float("inf")))
    assert all(torch.equal(a, b) for a, b in zip(got, call(t["gate"])))


def test_the_most_rows(moe):
    """2^31 - 1 rows, as many as a config can say: the norm alone and its gradient."""
    T, D = 2 ** 31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("two tensors of 34 GB")
    rc = moe.ResidualConfig(T=T, D=D)
    g = torch.Generator(device="cuda").manual_seed(5)
    s, d = (torch.zeros(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pre = torch.randn(D, generator=g, device="cuda").bfloat16()
    rows = [slice(0, 40), slice(1 << 30, (1 << 30) + 40), slice(T - 41, T)]
    for r in rows:
        s[r].normal_(generator=g)
        d[r].normal_(generator=g)
    few = [torch.cat([v[r] for r in rows]) for v in (s, d)]
    small = moe.ResidualConfig(T=len(few[0]), D=D)
    t = dict(resid=few[0], y=None, post=None, gate=None, pre=pre, rng=None)
    dpre = torch.empty(D, device="cuda")
    moe.moe_residual_norm_backward(rc, s, None, None, None, pre, None, None, d, d, None, None, None, dpre,
                                   moe.alloc_residual_workspace(rc))
    got = dict(dresid=torch.cat([d[r] for r in rows]), dy=None, dpost_gain=None, dgate=None, dpre_gain=dpre)
    _check_gradient(small, t, "none", None, few[1], got)
    moe.moe_residual_norm(rc, s, None, None, None, pre, None, None, d)
    _check_forward(small, t, "none", None, torch.cat([d[r] for r in rows]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["channel", "element"])
@pytest.mark.parametrize("T,D", [(11003, 72), (7001, 392), (5003, 520), (1501, 4104), (331, 12296)])
def test_gradient_in_place_over_many_rows(moe, T, D, gate, dtype):
    """dresid over dnorm_out and dy over dresid_out, with later rows on their way while one is stored."""
    rc, t, n = _case(moe, T, D, dtype, gate, p=0.1)
    dso, dn = n(T, D), n(T, D)
    want, got = _gradient(moe, rc, t, gate, dso, dn), _gradient(moe, rc, t, gate, dso, dn, in_place=True)
    assert all(torch.equal(got[k], want[k]) for k in want)
