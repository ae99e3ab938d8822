"""The norms around a block in 64 bits, by their formulas, with bounds on what fp32 arithmetic may
add to each output (tests only)."""
import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32 at 1


def philox(i, offset, seed):
    """Philox4x32, ten rounds, for counters (i, offset) under the key seed: uint64 array [n, 4]."""
    u64, low, w = np.uint64, np.uint64(0xffffffff), np.uint64(32)
    i = np.asarray(i, u64)
    c = [i & low, i >> w, np.full_like(i, offset & 0xffffffff), np.full_like(i, offset >> 32)]
    k0, k1 = seed & 0xffffffff, seed >> 32
    for _ in range(10):
        p, q = c[0] * u64(0xD2511F53), c[2] * u64(0xCD9E8D57)
        c = [(q >> w) ^ c[1] ^ u64(k0), q & low, (p >> w) ^ c[3] ^ u64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return np.stack(c, 1)


def keep(T, D, p, rng):
    """The dropout's factors [T, D] in fp64."""
    cut = round(p * 65536)
    if cut == 0:
        return torch.ones(T, D, dtype=torch.float64)
    seed, offset = (int(v) & (1 << 64) - 1 for v in rng)
    w = philox(np.arange(T * D // 8), offset, seed)
    half = np.stack([w & np.uint64(0xffff), w >> np.uint64(16)], 2).reshape(T, D)
    return torch.from_numpy((half >= cut).astype(np.float64)) * 65536 / (65536 - cut)


def _rms(x, eps):
    return 1 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)


def _wide(gate, kind):
    if gate is None:
        return 1.0
    return gate[:, None] if kind == "token" else gate


def forward(rc, kind, resid, y, post, gate, pre, kp):
    """(s, n) in the inputs' precision; differentiable."""
    s = resid
    if y is not None:
        v = y if post is None else y * _rms(y, rc.eps) * post
        s = rc.res_scale * resid + rc.branch_scale * _wide(gate, kind) * (kp * v)
    return s, None if pre is None else s * _rms(s, rc.eps) * pre


def forward_bounds(rc, kind, resid, y, post, gate, pre, kp, y_err=0.0):
    """What fp32 may add to s and n.  A row sum of D products is a chain of at most 32 terms per thread
    and ten steps of a tree: 43 U relative, half of it on the rsqrt factor, which itself is within 2 steps;
    with the eight products and sums of an element, 64 U of the terms' magnitudes covers both.

    y_err: how far the y that the kernel has may be off, element by element (a weighted sum whose terms
    cancel is off by more than 64 U of itself).  v = y r1 post moves by y_err r1 post and, through r1, by
    at most v mean(y_err |y|) / (mean(y^2) + eps); the gate, dropout and scale multiply both."""
    s, n = forward(rc, kind, resid, y, post, gate, pre, kp)
    mag = s.abs()
    if y is not None:
        v = y if post is None else y * _rms(y, rc.eps) * post
        mag = (rc.res_scale * resid).abs() + (rc.branch_scale * _wide(gate, kind) * (kp * v)).abs()
        if torch.is_tensor(y_err):
            dv = y_err
            if post is not None:
                r1 = _rms(y, rc.eps)
                dv = (y_err * r1 * post).abs() + v.abs() * (y_err * y.abs()).mean(1, keepdim=True) * r1 ** 2
            mag = mag + (rc.branch_scale * _wide(gate, kind) * (kp * dv)).abs() / (64 * U)
    r2 = _rms(s, rc.eps)
    # an error of s moves r2 too: by at most its own row mean against s
    shift = (mag * s.abs()).mean(1, keepdim=True) * r2 * r2
    return 64 * U * mag, None if pre is None else 64 * U * r2 * pre.abs() * (mag + s.abs() * (1 + shift))


def gradient(rc, kind, s, y, post, gate, pre, kp, dso, dn):
    """Every gradient by the formulas, and what fp32 may add to each: 256 U of the magnitudes that are
    summed, and for a sum over rows the length of its chains on top."""
    T = s.shape[0]
    out, tol = {}, {}
    ds = torch.zeros_like(s) if dso is None else dso
    dsa = ds.abs()
    if pre is not None:
        r2 = _rms(s, rc.eps)
        g = dn * pre
        ds = ds + r2 * (g - s * r2 ** 2 * (g * s).mean(1, keepdim=True))
        dsa = dsa + r2 * (g.abs() + s.abs() * r2 ** 2 * (g * s).abs().mean(1, keepdim=True))
        out["dpre_gain"] = (dn * s * r2).sum(0)
        tol["dpre_gain"] = (256 + T) * U * (dn * s * r2).abs().sum(0)
    if y is None:
        out["dresid"], tol["dresid"] = ds, 256 * U * dsa
        return out, tol
    out["dresid"], tol["dresid"] = rc.res_scale * ds, 256 * U * abs(rc.res_scale) * dsa
    r1 = torch.ones_like(s[:, :1]) if post is None else _rms(y, rc.eps)
    po = torch.ones_like(s[:1]) if post is None else post
    u, ua = rc.branch_scale * kp * ds, abs(rc.branch_scale) * kp * dsa
    gt = _wide(gate, kind)
    ga = gt if isinstance(gt, float) else gt.abs()
    dg, dga = u * y * r1 * po, ua * (y * r1 * po).abs()
    if kind == "channel":
        out["dgate"], tol["dgate"] = dg.sum(0), (256 + T) * U * dga.sum(0)
    elif kind == "token":
        out["dgate"], tol["dgate"] = dg.sum(1), 512 * U * dga.sum(1)
    elif kind == "element":
        out["dgate"], tol["dgate"] = dg, 256 * U * dga
    dv, dva = u * gt, ua * ga
    if post is None:
        out["dy"], tol["dy"] = dv, 256 * U * dva
        return out, tol
    out["dpost_gain"] = (dv * y * r1).sum(0)
    tol["dpost_gain"] = (256 + T) * U * (dva * (y * r1).abs()).sum(0)
    out["dy"] = r1 * (dv * post - y * r1 ** 2 * (dv * post * y).mean(1, keepdim=True))
    tol["dy"] = 256 * U * r1 * (dva * post.abs() + y.abs() * r1 ** 2 * (dva * (post * y).abs()).mean(1, keepdim=True))
    return out, tol
