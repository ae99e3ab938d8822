"""SiLU far below zero in the MXFP4 grouped call, where 1 + e^-g leaves fp32's range.

g = w1 x and u = w3 x are exact here: two products of e2m1 values each.  With u = 2^100 the
result g e^g / (1 + e^g) u is an ordinary number down to g = -100, and so is y.  e^g = 2^(g / ln 2)
in fp32 has the exponent's rounding, at most 2^-17 of 144 absolute, and a few 2^-23 beside it: 2^-15
in all; below 2^-126 e^g has whole steps of 2^-149 and so has its product with g:
|u| (|g| + 2) 2^-149 more.  The stored value lies between the
quantised ends of that interval (mx_reference.py), y is its product with w2 as in
test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

import mx_reference as mx
from test_gpu_mxfp4 import _between, _dev, _f64, _np, moe  # noqa: F401

pytestmark = pytest.mark.gpu

G = [-100.0, -96.0, -90.0, -88.0, -84.0, -80.0, -72.0, -48.0, 88.0, 96.0]
U = 2.0 ** 100


def test_silu_of_large_gates(moe):  # noqa: F811
    rows, D, H = 3, 64, 32 * len(G)
    x = np.zeros((rows, D))
    x[:, [0, 32]] = 1.0
    w1, w3, w2 = np.zeros((H, D)), np.zeros((H, D)), np.zeros((D, H))
    for i, g in enumerate(G):                                  # a block of hidden units each
        w1[32 * i:32 * i + 32, 0] = np.copysign(96.0 if g != -48 and g != -72 else 64.0, g)
        w1[32 * i:32 * i + 32, 32] = g - w1[32 * i, 0]
        w3[32 * i:32 * i + 32, 0] = U if g < 0 else 2.0
        # output i sums block i, brought near 1
        w2[i, 32 * i:32 * i + 32] = 2.0 ** -np.round(np.log2(32 * abs(g) * np.exp(min(g, 0)) * w3[32 * i, 0]))
    cfg = moe.Config(T=rows, D=D, H_local=H, E=1, k=1, align_m=1)
    assert moe.rows_alloc(cfg) == rows
    ops = []
    for a in (x, w1, w3, w2):
        v, b = mx.quantize(a)
        assert np.array_equal(v, a)                            # the format holds them
        ops.append((torch.from_numpy(mx.pack(v, b)).cuda(), torch.from_numpy(b).cuda()))
    (xq, xs), w = ops[0], [(q[None].contiguous(), s[None].contiguous()) for q, s in ops[1:]]
    hq = torch.empty((rows, H // 2), dtype=torch.uint8, device="cuda")
    hs = torch.empty((rows, H // 32), dtype=torch.uint8, device="cuda")
    y = torch.empty((rows, D), dtype=torch.float16, device="cuda")
    ws = moe.alloc_workspace(cfg)
    moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, _dev([0, rows]), _dev([rows]), *w[0], *w[1], *w[2], hq, hs, y, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    g, u = x @ w1.T, x @ w3.T
    assert np.array_equal(g[0, ::32], G)
    ref = g * np.exp(np.minimum(g, 0)) / (1 + np.exp(-np.abs(g))) * u
    d = 2.0 ** -15 * np.abs(ref) + np.abs(u) * (np.abs(g) + 2) * 2.0 ** -149
    h = mx.values(_np(hq), _np(hs))
    top, dt = np.abs(ref).reshape(rows, -1, 32), d.reshape(rows, -1, 32)
    ok = _between(h, ref - d, ref + d, np.maximum(top - dt, 0).max(-1), (top + dt).max(-1))
    assert ok.all(), f"h of gates {sorted(set(g[~ok]))}: {sorted(set(h[~ok]))} for {sorted(set(ref[~ok]))}"
    ry = h @ w2.T
    dy = 2.0 ** -20 * (np.abs(h) @ np.abs(w2).T)
    dy = dy + 2.0 ** -11 * (np.abs(ry) + dy) + 2.0 ** -25
    assert (np.abs(_f64(y) - ry) <= dy).all()
