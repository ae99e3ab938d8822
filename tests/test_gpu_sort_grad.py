"""Gradients of the permute and combine steps against 64 bits and differences.

Bounds: dy_perm and dx are one rounding of an fp32 result (half a step of the
type: bf16 2^-8, fp32 2^-24; dx's sum of k terms adds k 2^-24 of their
magnitudes, dy's product 2^-24); dtopk_w is an fp32 sum of D products, within
2^-20 of the sum of their magnitudes for D <= 2^13 (a lane adds at most D / 32
terms in a row, then 5 more)."""
import numpy as np
import pytest
import torch

import moe_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _case(moe, T, D, E, k, bf16, **kw):
    cfg = moe.Config(T=T, D=D, H_local=64, E=E, k=k, dtype=moe.MOE_BF16 if bf16 else moe.MOE_F32, **kw)
    g = torch.Generator(device="cuda").manual_seed(T * 7 + D)
    ra = moe.rows_alloc(cfg)
    idx = torch.from_numpy(moe_inputs.random_topk_idx(T, E, k, seed=T)).cuda().int()
    i32 = dict(dtype=torch.int32, device="cuda")
    lay = [torch.empty(n, **i32) for n in ((E,), (cfg.e_local + 1,), (T, k), (ra,))]
    ws = moe.alloc_workspace(cfg)
    moe.moe_permute_index(cfg, idx, *lay, ws)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (cfg, ws, lay[2], r(T, D).to(cfg.torch_dtype), r(ra, D).to(cfg.y_dtype),
            torch.rand((T, k), generator=g, device="cuda"), r(ra, D))


CASES = [
    (1, 8, 4, 1, True, {}), (1, 2048, 64, 6, True, {}), (300, 128, 8, 2, False, {}),
    (257, 1000, 12, 5, True, dict(align_m=1)), (257, 1000, 12, 5, False, dict(align_m=1)),
    (64, 136, 16, 9, True, dict(e_first=3, E_local=6)), (64, 136, 40, 32, False, dict(e_first=30, E_local=10)),
    (40, 264, 8, 3, True, dict(layout=1, capacity=9)),        # capacity drops some slots
    (33, 64, 8, 2, True, dict(e_first=8, E_local=0)),         # no expert here: zeros
]


@pytest.mark.parametrize("T,D,E,k,bf16,kw", CASES)
def test_gradients(moe, T, D, E, k, bf16, kw):
    cfg, ws, row_of, dout, y, w, dxp = _case(moe, T, D, E, k, bf16, **kw)
    moe.moe_get_device_status(ws)                             # clears the capacity flag
    ra = y.shape[0]
    dy = torch.full((ra, D), 77.0, dtype=cfg.torch_dtype, device="cuda")
    dw = torch.full((T, k), 77.0, device="cuda")
    moe.moe_unpermute_combine_backward(cfg, dout, y, row_of, w, dy, dw, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    ro, g, yv, wv = row_of.cpu().numpy(), _f64(dout), _f64(y), _f64(w)
    rdy, rdw, mag = np.full((ra, D), 77.0), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if ro[t, j] >= 0:
                rdy[ro[t, j]] = wv[t, j] * g[t]
                rdw[t, j] = g[t] @ yv[ro[t, j]]
                mag[t, j] = np.abs(g[t]) @ np.abs(yv[ro[t, j]])
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    assert (np.abs(_f64(dy) - rdy) <= (half + 2.0 ** -24) * np.abs(rdy) * (1 + 2.0 ** -8) + 1e-38).all()
    assert (np.abs(_f64(dw) - rdw) <= 2.0 ** -20 * mag).all()
    for dt in ([torch.float32, torch.bfloat16] if bf16 else [torch.float32]):
        p = dxp.to(dt)
        dx = torch.full((T, D), 77.0, dtype=cfg.torch_dtype, device="cuda")
        moe.moe_permute_backward(cfg, p, row_of, dx, ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_OK
        pv, ref, m = _f64(p), np.zeros((T, D)), np.zeros((T, D))
        for t in range(T):
            for j in range(k):
                if ro[t, j] >= 0:
                    ref[t] += pv[ro[t, j]]
                    m[t] += np.abs(pv[ro[t, j]])
        assert (np.abs(_f64(dx) - ref) <= half * np.abs(ref) + (k + 1) * 2.0 ** -24 * m).all()


def test_gradients_are_the_forwards(moe):
    """L = <dout, combine(y * (1 + m))> of the fp32 steps by central differences: the
    forward is linear in y and in w, so a difference is exact but for fp32 rounding
    (2^-20 of the magnitudes) over the step."""
    T, D, E, k = 37, 64, 6, 3
    cfg, ws, row_of, dout, y, w, dxp = _case(moe, T, D, E, k, False)
    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    moe.moe_unpermute_combine_backward(cfg, dout, y, row_of, w, dy, dw, ws)
    g = torch.Generator(device="cuda").manual_seed(1)

    def loss(yy, ww):
        out = torch.empty((T, D), device="cuda")
        moe.moe_unpermute_combine(cfg, yy, row_of, ww, out, ws)
        return float((out.double() * dout.double()).sum())
    vy, vw = torch.randn(y.shape, generator=g, device="cuda"), torch.randn(w.shape, generator=g, device="cuda")
    there = torch.zeros(y.shape[0], dtype=torch.bool, device="cuda")
    there[row_of.long().flatten()] = True
    mag = float((dout.abs().double().unsqueeze(1) * (y.abs() + vy.abs())[row_of.long()].double()
                 * (w.abs() + vw.abs()).double().unsqueeze(-1)).sum())
    by_y = (loss(y + vy, w) - loss(y - vy, w)) / 2
    by_w = (loss(y, w + vw) - loss(y, w - vw)) / 2
    assert abs(by_y - float((dy.double() * vy.double())[there].sum())) <= 2.0 ** -18 * mag
    assert abs(by_w - float((dw.double() * vw.double()).sum())) <= 2.0 ** -18 * mag
    # permute: <dx_perm, permute(v)> = <dx, v>
    v = torch.randn((T, D), generator=g, device="cuda")
    dx = torch.empty((T, D), device="cuda")
    moe.moe_permute_backward(cfg, dxp, row_of, dx, ws)
    left = float((dxp[row_of.long()].double() * v.double().unsqueeze(1)).sum())
    m = float((dxp[row_of.long()].abs().double() * v.abs().double().unsqueeze(1)).sum())
    assert abs(left - float((dx.double() * v.double()).sum())) <= 2.0 ** -20 * m


def test_bad_rows_are_flagged_and_skipped(moe):
    cfg, ws, row_of, dout, y, w, dxp = _case(moe, 16, 64, 4, 2, True)
    want_dx = torch.empty((16, 64), dtype=torch.bfloat16, device="cuda")
    good = row_of.clone()
    good[3, 0], good[5, 1] = -1, -1
    bad = row_of.clone()
    bad[3, 0], bad[5, 1] = y.shape[0], -2
    outs = []
    for ro in (good, bad):
        dy, dw, dx = torch.zeros_like(y, dtype=torch.bfloat16), torch.empty_like(w), torch.empty_like(want_dx)
        moe.moe_unpermute_combine_backward(cfg, dout, y, ro, w, dy, dw, ws)
        st = moe.moe_get_device_status(ws)
        moe.moe_permute_backward(cfg, dxp, ro, dx, ws)
        assert st == moe.moe_get_device_status(ws) == (moe.MOE_OK if ro is good else moe.MOE_ERR_BAD_ROUTING)
        outs.append((dy, dw, dx))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_sort_and_back_with_gradients_together(moe):
    """A run as a training step makes it: dispatch, the caller's own experts in
    between (here y = a x per expert), combine, and both gradients; captured too."""
    T, D, E, k = 130, 256, 8, 2
    cfg, ws, _, dout, _, w, _ = _case(moe, T, D, E, k, False)
    ra = moe.rows_alloc(cfg)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, D), generator=g, device="cuda")
    idx = torch.from_numpy(moe_inputs.random_topk_idx(T, E, k, seed=9)).cuda().int()
    i32 = dict(dtype=torch.int32, device="cuda")
    tpe, seg, row_of, tor = [torch.empty(n, **i32) for n in ((E,), (E + 1,), (T, k), (ra,))]
    xp, dy = torch.zeros((ra, D), device="cuda"), torch.zeros((ra, D), device="cuda")
    out, dw, dx = torch.empty((T, D), device="cuda"), torch.empty((T, k), device="cuda"), torch.empty((T, D), device="cuda")
    a = torch.randn(E, generator=g, device="cuda")
    rows = torch.arange(ra, device="cuda")

    def step():
        moe.moe_permute(cfg, x, idx, tpe, seg, row_of, tor, xp, ws)
        scale = a[(torch.searchsorted(seg[1:], rows, right=True)).clamp(max=E - 1)].unsqueeze(1)
        y = (xp * scale).contiguous()
        moe.moe_unpermute_combine(cfg, y, row_of, w, out, ws)
        moe.moe_unpermute_combine_backward(cfg, dout, y, row_of, w, dy, dw, ws)
        moe.moe_permute_backward(cfg, (dy * scale).contiguous(), row_of, dx, ws)
    step()
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    c = (w * a[idx.long()]).double()
    want_dx = c.sum(1, keepdim=True) * dout.double()
    # sums of k terms of two fp32 products each: (k + 3) roundings of 2^-24 of the magnitudes
    bound = (k + 3) * 2.0 ** -24 * c.abs().sum(1, keepdim=True)
    assert ((dx.double() - want_dx).abs() <= bound * dout.abs().double()).all()
    assert ((out.double() - c.sum(1, keepdim=True) * x.double()).abs() <= bound * x.abs().double()).all()
    dots = a[idx.long()].double() * (dout.double() * x.double()).sum(1, keepdim=True)
    mags = a[idx.long()].abs().double() * (dout.double() * x.double()).abs().sum(1, keepdim=True)
    assert ((dw.double() - dots).abs() <= 2.0 ** -20 * mags).all()
    first = [t.clone() for t in (out, dw, dx, dy)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t in (out, dw, dx):
        t.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(first, (out, dw, dx, dy)):
        assert torch.equal(p, q)
