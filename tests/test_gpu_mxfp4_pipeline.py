"""The MXFP4 grouped kernel where each CTA pair takes several tiles, against 64 bits.

A pair walks tile after tile with its accumulators, operand ring, scale groups and scale
buffers running on across them.  Every case has more than two tiles per pair in both GEMMs
and more K blocks (of 256) per tile than operand stages and than the scale groups in shared
memory hold; the segments are such that the launch takes tiles of at most 32, 144 or 208
tokens.  Products in 64 bits on the GPU; bounds as in test_gpu_mxfp4.py."""
import math

import pytest
import torch

from test_gpu_mxfp4 import _call, _grouped_case, _held, moe  # noqa: F401

pytestmark = pytest.mark.gpu

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
PAIRS = 76


def _values(q, s):
    grid = torch.tensor(GRID, dtype=torch.float64, device=q.device)
    c = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    v = torch.where(c >= 8, -grid[c & 7], grid[c & 7])
    scale = torch.ldexp(torch.ones_like(s, dtype=torch.float64), s.long() - 127)
    return v * scale.repeat_interleave(32, -1)


def _on_grid(x, top):
    """x rounded to the e2m1 values under the scale of a block whose largest magnitude is top."""
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full_like(top, -127).int()).clamp(min=-127)
    scale = torch.ldexp(torch.ones_like(top), e).unsqueeze(-1)
    a = x.unflatten(-1, (-1, 32)) / scale
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    down, up = torch.searchsorted(mid, a.abs()), torch.searchsorted(mid, a.abs(), right=True)
    return (torch.copysign(grid[torch.where(down % 2 == 0, down, up)], a) * scale).flatten(-2)


def _check_expert(x, w1, w3, w2, h, y):
    """Truth per value of h and of y (the bounds of test_gpu_mxfp4.py)."""
    g, u = x @ w1.T, x @ w3.T
    dg, du = 2.0 ** -20 * (x.abs() @ w1.abs().T), 2.0 ** -20 * (x.abs() @ w3.abs().T)
    sil = g * torch.sigmoid(g)
    ref = sil * u
    dh = 1.1 * dg * (u.abs() + du) + sil.abs() * du + 2.0 ** -20 * ref.abs() + 1e-37
    blk, d = ref.abs().unflatten(-1, (-1, 32)), dh.unflatten(-1, (-1, 32))
    ok = torch.zeros_like(h, dtype=torch.bool)
    for top in ((blk - d).clamp(min=0).amax(-1), (blk + d).amax(-1)):
        ok |= (h >= _on_grid(ref - dh, top)) & (h <= _on_grid(ref + dh, top))
    ry = h @ w2.T
    dy = 2.0 ** -20 * (h.abs() @ w2.abs().T)
    dy = dy + 2.0 ** -11 * (ry.abs() + dy) + 2.0 ** -25
    return ok, (y.double() - ry).abs() <= dy


def _tokens(bn, E, seed):
    """Segments whose average makes the launch take tiles of bn tokens, odd lengths, one empty
    and one of several tiles."""
    g = torch.Generator().manual_seed(seed)
    lo, hi = {32: (9, 29), 144: (100, 138), 208: (155, 195)}[bn]
    c = torch.randint(lo, hi, (E,), generator=g).tolist()
    c[1], c[3] = 0, 2 * bn + 1
    return c


def _tile_rule(rows):
    rows += math.sqrt(rows)
    n = lambda b: max(1, math.ceil(rows / b))  # noqa: E731
    return 32 if n(32) == n(208) else 144 if n(144) == n(208) else 208


def _run(moe, counts, D, H, align, seed):
    cfg, seg, xq, xs, w, out = _grouped_case(moe, counts, D, H, align, seed, span=8)
    ws = moe.alloc_workspace(cfg)
    _call(moe, cfg, seg, counts, xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    for i, c in enumerate(counts):
        if c == 0:
            continue
        r = slice(int(seg[i]), int(seg[i]) + c)
        ok_h, ok_y = _check_expert(_values(xq[r], xs[r]), *[_values(q[i], s[i]) for q, s in w],
                                   _values(out["hq"][r], out["hs"][r]), out["y"][r])
        assert bool(ok_h.all()), f"expert {i}: {int((~ok_h).sum())} of {ok_h.numel()} values of h"
        assert bool(ok_y.all()), f"expert {i}: {int((~ok_y).sum())} of {ok_y.numel()} values of y"
    held = torch.from_numpy(_held(seg, counts, len(xq))).cuda()
    assert (out["hq"][~held] == 0xAA).all() and (out["hs"][~held] == 0xAA).all()
    assert torch.isnan(out["y"][~held]).all()
    # the same bits again, into buffers that hold the first call's
    first = {k: v.clone() for k, v in out.items()}
    for _ in range(3):
        _call(moe, cfg, seg, counts, xq, xs, w, out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    for k, v in out.items():
        assert torch.equal(v.view(torch.uint8), first[k].view(torch.uint8)), k


@pytest.mark.parametrize("bn,E,D,H,align", [
    (32, 12, 4352, 2336, 128),    # 17 and 10 K blocks; h's scale rows of 73 bytes
    (32, 16, 2336, 4352, 1),
    (144, 20, 2304, 2080, 16),    # 9 K blocks each way; h's scale rows of 65 bytes
    (144, 20, 2080, 2304, 1),
    (208, 20, 2304, 2016, 1),     # h's scale rows of 63 bytes
    (208, 16, 4096, 2560, 128),   # 16 and 10 K blocks, scale rows on 16 bytes
])
def test_pairs_take_several_tiles(moe, bn, E, D, H, align):  # noqa: F811
    counts = _tokens(bn, E, D + H)
    assert _tile_rule(sum(counts) / E) == bn
    tiles = sum(-(-c // bn) for c in counts)
    assert tiles * -(-H // 128) > 2 * PAIRS and tiles * -(-D // 256) > 2 * PAIRS
    _run(moe, counts, D, H, align, bn + D)


@pytest.mark.parametrize("bn,E", [(32, 256), (144, 90), (208, 90)])
def test_accumulators_change_hands(moe, bn, E):  # noqa: F811
    """GEMM1 tiles of one K block: their products take less than their epilogues, and both
    accumulators wait for it at every tile."""
    counts = _tokens(bn, E, E + bn)
    assert _tile_rule(sum(counts) / E) == bn
    tiles = sum(-(-c // bn) for c in counts)
    assert tiles * 4 > 4 * PAIRS and tiles > PAIRS
    _run(moe, counts, 256, 512, 1, bn)
