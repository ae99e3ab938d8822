"""MXFP4 rows, dispatch, grouped SwiGLU and layer on the GPU against 64 bits.

Codes and scales are exact functions of their input and are compared as such.
The products run on exactly the values that the codes stand for.  Bounds, from
the arithmetic:
  * a product's fp32 sum is within 2^-20 of the sum of the magnitudes of its
    terms (at most 2^7 MMAs of K = 64 each, whose truncated additions lose at
    most a few 2^-24 each);
  * h = SiLU(g) u in fp32 inherits 1.1 dg |u| + |SiLU(g)| du (|SiLU'| <= 1.1)
    and 2^-20 |h| of the fast exponential and division; it is then a value of
    its block's grid, so the stored value lies between the quantised ends of
    that interval, under the scale of either end of the block's maximum;
  * y, from the h that is stored, is one product plus one fp16 rounding
    (2^-11 of the value, 2^-25 below the normal range).
"""
import numpy as np
import pytest
import torch

import moe_inputs
import mx_reference as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _np(t):
    return t.detach().cpu().numpy()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _spread(shape, seed, span=12):
    """Normal values whose blocks of 32 have scales of their own, so that a scale
    taken for another row or block shows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    e = torch.randint(-span // 2, span // 2 + 1, (*shape[:-1], shape[-1] // 32, 1), generator=g, device="cuda")
    return (x.view(*shape[:-1], shape[-1] // 32, 32) * torch.exp2(e.float())).view(shape)


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------

def _edge_rows(cols):
    x = np.zeros((12, cols), np.float32)
    x[1] = 1e-30
    x[2, ::2] = -0.0
    x[3, : min(cols, 32)] = np.linspace(-8, 8, min(cols, 32))
    x[4, 0], x[4, 1:9] = 6.0, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25]  # every tie, scale 1
    x[5, 0] = np.nan
    x[6, -1] = np.inf
    x[7, 1] = -np.inf
    x[8] = 2.0 ** -126
    x[8, 0] = 2.0 ** -120
    x[9] = 3.0e38
    x[10] = 2.0 ** -133            # subnormal (exact in bf16)
    x[11, 0], x[11, 1] = 7.9, 0.26
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (12, 64), (37, 2048), (300, 1056), (5, 7168), (1, 2048)])
def test_rows_exact(moe, dtype, rows, cols):
    x = _spread((rows, cols), rows + cols, 40)
    if rows >= 12:
        x[:12] = torch.from_numpy(_edge_rows(cols)).cuda()
    x = x.to(dtype)
    q = torch.full((rows, cols // 2), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, cols // 32), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows_mxfp4(x, q, s)
    v, b = mx.quantize(_f64(x))
    assert np.array_equal(_np(s), b)
    got = mx.values(_np(q), _np(s))
    assert np.array_equal(got, v, equal_nan=True)
    assert (_np(q).reshape(rows, -1, 16)[b == 255] == 0).all()     # a NaN block's codes
    for out in (torch.bfloat16, torch.float32):
        back = torch.full((rows, cols), 7.0, dtype=out, device="cuda")
        moe.moe_dequantize_rows_mxfp4(q, s, back)
        assert np.array_equal(_f64(back), v, equal_nan=True)


def test_every_byte_and_scale_reads_back(moe):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)     # 512 values a row
    scale = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1).repeat(1, 16)
    out = torch.empty((256, 512), device="cuda")
    moe.moe_dequantize_rows_mxfp4(codes, scale, out)
    want = mx.values(_np(codes), _np(scale))
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)                             # 253 and 254 pass the fp32 range
    assert np.array_equal(_np(out), want, equal_nan=True)


def test_rows_in_more_dimensions_and_none(moe):
    w = _spread((3, 5, 96), 1)
    q, s = moe.quantize_weights_mxfp4(w)
    assert q.shape == (3, 5, 48) and s.shape == (3, 5, 3)
    assert np.array_equal(mx.values(_np(q), _np(s)), mx.quantize(_f64(w))[0])
    empty = torch.empty((0, 64), device="cuda")
    q, s = moe.quantize_weights_mxfp4(empty)
    moe.moe_dequantize_rows_mxfp4(q, s, empty)
    with pytest.raises(ValueError):
        moe.quantize_weights_mxfp4(torch.zeros((4, 48), device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_quantize_rows_mxfp4(w[:, :, ::2], q, s)
    with pytest.raises(ValueError):
        moe.moe_quantize_rows_mxfp4(w.half(), q, s)


# ---------------------------------------------------------------------------
# dispatch
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,k,D,align,e_first,E_local,masked", [
    (700, 16, 4, 512, 128, 0, 16, False), (333, 5, 2, 352, 1, 1, 3, False), (1, 8, 8, 32, 128, 0, 8, False),
    (40, 8, 3, 1056, 64, 0, 8, True), (20000, 256, 2, 64, 128, 0, 256, False), (50, 4, 1, 64, 128, 4, 0, False),
    (5000, 256, 2, 64, 128, 0, 256, False), (5000, 256, 2, 64, 1, 200, 56, False), (0, 8, 2, 64, 128, 0, 8, False)])
def test_dispatch(moe, T, E, k, D, align, e_first, E_local, masked):
    idx = _dev(moe_inputs.random_topk_idx(T, E, k, seed=T))
    x = _spread((T, D), T).to(torch.bfloat16)
    cfg = moe.Config(T=T, D=D, H_local=64, E=E, k=k, align_m=align, e_first=e_first, E_local=E_local,
                     layout=moe.MOE_LAYOUT_MASKED if masked else moe.MOE_LAYOUT_CONTIGUOUS, capacity=T)
    ra, ws = moe.rows_alloc(cfg), moe.alloc_workspace(cfg)

    def layout():
        return [torch.full(n, -7, dtype=torch.int32, device="cuda") for n in ((E,), (E_local + 1,), (T, k), (ra,))]
    a, b = layout(), layout()
    xq = torch.full((ra, D // 2), 0xAA, dtype=torch.uint8, device="cuda")
    xs = torch.full((ra, D // 32), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_permute_mxfp4(cfg, x, idx, *a, xq, xs, ws)
    moe.moe_permute_index(cfg, idx, *b, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    tor = _np(a[3])
    held = tor >= 0
    v, sc = mx.quantize(_f64(x))
    assert np.array_equal(_np(xs)[held], sc[tor[held]])
    assert np.array_equal(mx.values(_np(xq)[held], _np(xs)[held]), v[tor[held]])
    assert (_np(xq)[~held] == 0xAA).all() and (_np(xs)[~held] == 0xAA).all()


@pytest.mark.parametrize("T,E,k,cap", [(60, 8, 3, 9), (3000, 256, 4, 32), (5000, 16, 2, 0)])
def test_rows_past_the_capacity_are_dropped(moe, T, E, k, cap):
    """Masked layout: an expert's first `capacity` tokens are kept, the rest have no
    row, the status says so, and the layer is still its steps."""
    D, H = 128, 64
    cfg, x, wg, w = _layer(moe, T, D, H, E, k, seed=T, layout=1, capacity=cap)
    ra, ws = moe.rows_alloc(cfg), moe.alloc_workspace(cfg, layer=True)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
    moe.moe_route_topk(cfg, x, wg, None, None, idx, tw, ws)
    lay = [torch.full(n, -7, dtype=torch.int32, device="cuda") for n in ((E,), (E + 1,), (T, k), (ra,))]
    want = [torch.empty_like(t) for t in lay]
    xq = torch.full((ra, D // 2), 0xAA, dtype=torch.uint8, device="cuda")
    xs = torch.full((ra, D // 32), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_permute_mxfp4(cfg, x, idx, *lay, xq, xs, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_CAPACITY
    moe.moe_permute_index(cfg, idx, *want, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_CAPACITY
    for p, q in zip(lay, want):
        assert torch.equal(p, q)
    tor = _np(lay[3])
    held = tor >= 0
    assert held.sum() == np.minimum(_np(lay[0]), cap).sum() < T * k
    v, sc = mx.quantize(_f64(x))
    assert np.array_equal(_np(xs)[held], sc[tor[held]])
    assert np.array_equal(mx.values(_np(xq)[held], _np(xs)[held]), v[tor[held]])
    assert (_np(xq)[~held] == 0xAA).all() and (_np(xs)[~held] == 0xAA).all()
    hq, hs = torch.empty((ra, H // 2), dtype=torch.uint8, device="cuda"), torch.empty((ra, H // 32), dtype=torch.uint8, device="cuda")
    y, steps, out = torch.empty((ra, D), dtype=torch.float16, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, lay[1], lay[0], *w[0], *w[1], *w[2], hq, hs, y, ws)
    moe.moe_unpermute_combine(cfg, y, lay[2], tw, steps, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_CAPACITY
    assert torch.equal(out, steps)


# ---------------------------------------------------------------------------
# grouped SwiGLU
# ---------------------------------------------------------------------------

def _segments(counts, align):
    seg = np.zeros(len(counts) + 1, np.int64)
    for i, c in enumerate(counts):
        seg[i + 1] = seg[i] + -(-c // align) * align
    return seg


def _between(got, lo, hi, top_lo, top_hi):
    """got lies between the quantised ends, under the block scale of either end of the maximum."""
    ok = np.zeros(got.shape, bool)
    for top in (top_lo, top_hi):
        e = mx.exponents(np.repeat(top, 32, axis=-1))
        ok |= (got >= mx.with_exponents(lo, e)) & (got <= mx.with_exponents(hi, e))
    return ok


def _hidden(x, w1, w3):
    """SiLU(x w1^T) * (x w3^T) in 64 bits and how far the fp32 result may be from it."""
    g, u = x @ w1.T, x @ w3.T
    dg, du = (2.0 ** -20 * (np.abs(x) @ np.abs(v).T) for v in (w1, w3))
    with np.errstate(over="ignore"):
        sil = g / (1 + np.exp(-g))
    h = sil * u
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(sil) * du + 2.0 ** -20 * np.abs(h) + 1e-37


def _check_grouped(seg, counts, xv, w1v, w3v, w2v, hv, y):
    for i, c in enumerate(counts):
        r = slice(int(seg[i]), int(seg[i]) + c)
        if c == 0:
            continue
        x, h, yy = xv[r], hv[r], y[r]
        ref, dh = _hidden(x, w1v[i], w3v[i])
        blk = np.abs(ref).reshape(c, -1, 32)
        d = dh.reshape(c, -1, 32)
        ok = _between(h, ref - dh, ref + dh, np.maximum(blk - d, 0).max(-1), (blk + d).max(-1))
        assert ok.all(), f"expert {i}: {(~ok).sum()} of {ok.size} values of h"
        ry = h @ w2v[i].T
        dy = 2.0 ** -20 * (np.abs(h) @ np.abs(w2v[i]).T)
        dy = dy + 2.0 ** -11 * (np.abs(ry) + dy) + 2.0 ** -25
        bad = np.abs(yy - ry) > dy
        assert not bad.any(), f"expert {i}: {bad.sum()} of {bad.size} values of y"


def _grouped_case(moe, counts, D, H, align, seed, tail_rows=0, span=12):
    """Quantised operands, poisoned outputs and the call's arguments."""
    E = len(counts)
    seg = _segments(counts, align)
    rows = int(seg[-1]) + tail_rows
    T = sum(counts)
    # a config with exactly enough rows: k = 1, rows_alloc = T + E (align - 1) >= rows
    cfg = moe.Config(T=T, D=D, H_local=H, E=E, k=1, align_m=align)
    ra = moe.rows_alloc(cfg)
    assert ra >= rows
    xq, xs = moe.quantize_weights_mxfp4(_spread((ra, D), seed, span))
    # 2^-6: with the weights at D^-1/2 alone, spread scales make |y| pass fp16's range
    w = [moe.quantize_weights_mxfp4(_spread(s, seed + 1 + j, span) * D ** -0.5 * 2.0 ** -6)
         for j, s in enumerate([(E, H, D), (E, H, D), (E, D, H)])]
    out = dict(hq=torch.full((ra, H // 2), 0xAA, dtype=torch.uint8, device="cuda"),
               hs=torch.full((ra, H // 32), 0xAA, dtype=torch.uint8, device="cuda"),
               y=torch.full((ra, D), float("nan"), dtype=torch.float16, device="cuda"))
    return cfg, seg, xq, xs, w, out


def _call(moe, cfg, seg, counts, xq, xs, w, out, ws):
    moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, _dev(seg), _dev(np.array(counts)), *w[0], *w[1], *w[2],
                                 out["hq"], out["hs"], out["y"], ws)


def _held(seg, counts, n):
    m = np.zeros(n, bool)
    for i, c in enumerate(counts):
        m[int(seg[i]):int(seg[i]) + c] = True
    return m


ALL = [1, 15, 16, 17, 31, 33, 0, 64, 65, 96, 127, 128, 129, 0, 255, 256, 257, 300]


@pytest.mark.parametrize("counts,D,H,align", [
    ([5], 32, 32, 1),                 # one block each way
    ([1], 256, 96, 128),              # one row, whole K block and tile
    ([3, 0, 130], 64, 64, 128),
    ([200, 7, 64], 512, 256, 128),    # scale rows of 8-byte units
    ([200, 7, 64], 384, 128, 1),      # of 4-byte units, segments at any row
    ([150, 9, 33], 1056, 416, 1),     # of single bytes
    ([140, 2], 2048, 1408, 128),      # sizes of the fine-grained layer
    (ALL, 320, 192, 128),
    (ALL, 320, 224, 1),
    # averages that take the tile of 208 tokens: tiles full, one row over, one row
    ([416, 0, 417, 385, 400, 350], 288, 160, 128),
    ([208, 209, 160, 63, 1, 320], 768, 128, 1),
    # few rows on average (tiles of 32), one expert with several tiles
    ([0, 1, 100, 0, 32, 33, 2, 0, 0, 1, 0, 16, 0, 0, 3, 0, 0, 5], 224, 288, 64),
])
def test_grouped(moe, counts, D, H, align):
    cfg, seg, xq, xs, w, out = _grouped_case(moe, counts, D, H, align, D + H)
    ws = moe.alloc_workspace(cfg)
    _call(moe, cfg, seg, counts, xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    held = _held(seg, counts, len(xq))
    hv = np.zeros((len(xq), H))
    hv[held] = mx.values(_np(out["hq"])[held], _np(out["hs"])[held])
    y = _f64(out["y"])
    _check_grouped(seg, counts, mx.values(_np(xq), _np(xs)),
                   *[mx.values(_np(q), _np(s)) for q, s in w], hv, y)
    # rows that hold no token are left as they were
    assert (_np(out["hq"])[~held] == 0xAA).all() and (_np(out["hs"])[~held] == 0xAA).all()
    assert np.isnan(y[~held]).all()


def test_grouped_shard_takes_its_experts_counts(moe):
    """e_first > 0: counts are read at the expert's global index."""
    counts, e_first, E = [40, 0, 131], 3, 9
    cfg, seg, xq, xs, w, out = _grouped_case(moe, counts, 288, 160, 128, 5)
    cfg = moe.Config(T=cfg.T, D=288, H_local=160, E=E, k=1, e_first=e_first, E_local=3, align_m=128)
    tpe = np.full(E, 9999)
    tpe[e_first:e_first + 3] = counts
    ws = moe.alloc_workspace(cfg)
    moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, _dev(seg), _dev(tpe), *w[0], *w[1], *w[2], out["hq"], out["hs"],
                                 out["y"], ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    held = _held(seg, counts, len(xq))
    hv = np.zeros((len(xq), 160))
    hv[held] = mx.values(_np(out["hq"])[held], _np(out["hs"])[held])
    _check_grouped(seg, counts, mx.values(_np(xq), _np(xs)), *[mx.values(_np(q), _np(s)) for q, s in w], hv,
                   _f64(out["y"]))
    assert np.isnan(_f64(out["y"])[~held]).all()


def test_grouped_nan_rows_stay_in_their_rows(moe):
    """A token with a NaN block gives NaN rows; garbage in padding rows (NaN scales) reaches none."""
    counts, D, H = [20, 70], 288, 96
    cfg, seg, xq, xs, w, out = _grouped_case(moe, counts, D, H, 128, 8)
    held = _held(seg, counts, len(xq))
    xs[torch.from_numpy(~held).cuda()] = 255
    xs[3, 1] = 255
    xs[128 + 69, 0] = 255
    ws = moe.alloc_workspace(cfg)
    _call(moe, cfg, seg, counts, xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    y = _f64(out["y"])
    nan = np.zeros(len(xq), bool)
    nan[[3, 128 + 69]] = True
    assert np.isnan(y[nan]).all()
    assert (_np(out["hs"])[nan] == 255).all() and (_np(out["hq"])[nan] == 0).all()
    assert np.isfinite(y[held & ~nan]).all()


def test_grouped_flags(moe):
    # an output beyond fp16's range
    cfg, seg, xq, xs, w, out = _grouped_case(moe, [4], 64, 32, 128, 3)
    w[2][1].fill_(127 + 40)
    ws = moe.alloc_workspace(cfg)
    _call(moe, cfg, seg, [4], xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_UNSUPPORTED
    # offsets outside the buffers: flagged, the segment skipped, the other one done
    cfg, seg, xq, xs, w, out = _grouped_case(moe, [4, 6], 64, 32, 128, 3)
    ws = moe.alloc_workspace(cfg)
    bad = seg.copy()
    bad[2] = moe.rows_alloc(cfg) + 1
    _call(moe, cfg, bad, [4, 6], xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BAD_ROUTING
    y = _f64(out["y"])
    assert np.isfinite(y[:4]).all() and np.isnan(y[4:]).all()


def test_grouped_scales_on_16_bytes(moe):
    """Scales whose arrays start on 16 bytes and not on 32: the same bits."""
    counts = [40, 0, 7, 161]
    cfg, seg, xq, xs, w, out = _grouped_case(moe, counts, 1024, 1024, 16, 5)
    ws = moe.alloc_workspace(cfg)
    _call(moe, cfg, seg, counts, xq, xs, w, out, ws)
    want = {k: v.clone() for k, v in out.items()}

    def moved(t):
        b = torch.empty(t.numel() + 16, dtype=torch.uint8, device="cuda")[16:].view(t.shape)
        return b.copy_(t)
    out["hs"] = moved(torch.full_like(out["hs"], 0xAA))
    _call(moe, cfg, seg, counts, xq, moved(xs), [(q, moved(s)) for q, s in w], out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    for k in out:
        assert torch.equal(out[k].view(torch.uint8), want[k].view(torch.uint8)), k


def test_grouped_many_experts(moe):
    """1024 experts, the largest table, most of them empty."""
    E, D, H = 1024, 64, 32
    counts = [0] * E
    for e, c in ((0, 3), (511, 129), (900, 1), (1023, 20)):
        counts[e] = c
    cfg, seg, xq, xs, w, out = _grouped_case(moe, counts, D, H, 16, 2)
    ws = moe.alloc_workspace(cfg)
    _call(moe, cfg, seg, counts, xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    held = _held(seg, counts, len(xq))
    hv = np.zeros((len(xq), H))
    hv[held] = mx.values(_np(out["hq"])[held], _np(out["hs"])[held])
    _check_grouped(seg, counts, mx.values(_np(xq), _np(xs)), *[mx.values(_np(q), _np(s)) for q, s in w], hv,
                   _f64(out["y"]))


# ---------------------------------------------------------------------------
# the calls together
# ---------------------------------------------------------------------------

def _layer(moe, T, D, H, E, k, seed=0, **kw):
    cfg = moe.Config(T=T, D=D, H_local=H, E=E, k=k, renorm=1, **kw)
    x = _spread((T, D), seed, 4).to(torch.bfloat16)
    wg = (0.02 * torch.randn((E, D), device="cuda", generator=torch.Generator("cuda").manual_seed(seed))).bfloat16()
    el = cfg.e_local
    w = [moe.quantize_weights_mxfp4(0.05 * _spread(s, seed + 1 + j, 4))
         for j, s in enumerate([(el, H, D), (el, H, D), (el, D, H)])]
    return cfg, x, wg, w


def _by_steps(moe, cfg, x, wg, w):
    T, k, ra, el = cfg.T, cfg.k, moe.rows_alloc(cfg), cfg.e_local
    i32 = dict(dtype=torch.int32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    idx, tw = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    lay = [torch.empty(n, **i32) for n in ((cfg.E,), (el + 1,), (T, k), (ra,))]
    xq, xs = torch.empty((ra, cfg.D // 2), **u8), torch.empty((ra, cfg.D // 32), **u8)
    hq, hs = torch.empty((ra, cfg.H_local // 2), **u8), torch.empty((ra, cfg.H_local // 32), **u8)
    y = torch.empty((ra, cfg.D), dtype=torch.float16, device="cuda")
    out = torch.empty((T, cfg.D), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(cfg)
    moe.moe_route_topk(cfg, x, wg, None, None, idx, tw, ws)
    moe.moe_permute_mxfp4(cfg, x, idx, *lay, xq, xs, ws)
    moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, lay[1], lay[0], *w[0], *w[1], *w[2], hq, hs, y, ws)
    moe.moe_unpermute_combine(cfg, y, lay[2], tw, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    return out, idx, tw


@pytest.mark.parametrize("T,D,H,E,k,kw", [
    (1, 2048, 1408, 64, 6, {}), (300, 256, 96, 8, 2, {}), (77, 352, 160, 12, 5, dict(align_m=1)),
    (64, 512, 256, 16, 4, dict(layout=1, capacity=64)), (129, 256, 128, 16, 3, dict(e_first=5, E_local=7)),
    (40, 64, 64, 8, 2, dict(e_first=8, E_local=0))])
def test_layer_is_its_steps(moe, T, D, H, E, k, kw):
    cfg, x, wg, w = _layer(moe, T, D, H, E, k, **kw)
    want, idx, tw = _by_steps(moe, cfg, x, wg, w)
    ws = moe.alloc_workspace(cfg, layer=True)
    out = torch.full((T, D), 9.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):                                   # the workspace is left usable
        moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], out, ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_OK
        assert torch.equal(out, want)
    # and its value, per token in 64 bits: h may round to either side of a tie that
    # its fp32 error reaches (the spread between the quantised ends); y adds its sum's
    # and its fp16 rounding, out half a bf16 step
    xv = mx.quantize(_f64(x))[0]
    wv = [mx.values(_np(q), _np(s)) for q, s in w]
    idx, tw = _np(idx), _np(tw).astype(np.float64)
    ref, bound = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j in range(k):
            i = idx[t, j] - cfg.e_first
            if not 0 <= i < cfg.e_local:
                continue
            h, dh = _hidden(xv[t:t + 1], wv[0][i], wv[1][i])
            q = mx.quantize(h)[0]
            top, d = np.abs(h).reshape(1, -1, 32), dh.reshape(1, -1, 32)
            spread = np.zeros_like(q)
            for end in (np.maximum(top - d, 0).max(-1), (top + d).max(-1)):
                e = mx.exponents(np.repeat(end, 32, axis=-1))
                for v in (h - dh, h + dh):
                    spread = np.maximum(spread, np.abs(mx.with_exponents(v, e) - q))
            y = wv[2][i] @ q[0]
            dy = np.abs(wv[2][i]) @ (spread[0] + 2.0 ** -20 * np.abs(q[0]))
            dy += 2.0 ** -11 * (np.abs(y) + dy) + 2.0 ** -25
            ref[t] += tw[t, j] * y
            bound[t] += tw[t, j] * (dy + (k + 1) * 2.0 ** -24 * np.abs(y))
    bound += 2.0 ** -8 * (np.abs(ref) + bound)
    assert (np.abs(_f64(out) - ref) <= bound).all()


def test_layer_without_tokens(moe):
    cfg, x, wg, w = _layer(moe, 0, 64, 64, 4, 2)
    ws = moe.alloc_workspace(cfg, layer=True)
    moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], torch.empty_like(x), ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK


def test_streams_graphs_and_repeats(moe):
    """On a side stream, captured and replayed, and run again: the same bits."""
    cfg, x, wg, w = _layer(moe, 200, 512, 192, 8, 2, seed=4)
    want, _, _ = _by_steps(moe, cfg, x, wg, w)
    ws = moe.alloc_workspace(cfg, layer=True)
    out = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], out, ws)
    for seed in (5, 6):
        x.copy_(_spread(tuple(x.shape), seed, 4))
        want, _, _ = _by_steps(moe, cfg, x, wg, w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # two workspaces on two streams at once
    outs, wss = [torch.zeros_like(x) for _ in range(2)], [moe.alloc_workspace(cfg, layer=True) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, k in zip(streams, outs, wss):
            moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], o, k, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
