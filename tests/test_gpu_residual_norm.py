"""moe_residual_norm, moe_combine_residual_norm and the gradient against their formulas in 64 bits.

Tolerances: what fp32 may add (residual_reference derives it) plus half a step of the output's type.
"""
import pytest
import torch

import residual_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


GATES = {"none": 0, "channel": 1, "token": 2, "element": 3}


def _case(moe, T, D, dtype, gate="none", post=True, branch=True, pre=True, p=0.0, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * T + D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def n(*s, scale=1.0, to=dt):
        return (scale * torch.randn(s, generator=g, device="cuda")).to(to)
    rc = moe.ResidualConfig(T=T, D=D, dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32,
                            gate=GATES[gate], p_drop=p, **kw)
    t = dict(resid=n(T, D, scale=3.0), y=n(T, D) if branch else None, post=n(D) if post and branch else None,
             gate=None, pre=n(D) if pre else None, rng=None)
    if gate == "channel":
        t["gate"] = n(D)
    elif gate == "token":
        t["gate"] = n(T, to=torch.float32)
    elif gate == "element":
        t["gate"] = n(T, D)
    if p:
        t["rng"] = torch.tensor([0x0123456789abcdef, -(1 << 40) + seed], device="cuda")
    return rc, t, n


def _wide(t):
    return {k: None if v is None else v.double().cpu() for k, v in t.items() if k != "rng"}


def _keep(rc, t):
    return ref.keep(rc.T, rc.D, rc.p_drop, t["rng"].tolist() if t["rng"] is not None else (0, 0))


def _close(got, want, tol, name):
    """Within tol and half a step of got's type."""
    want = want.cpu()
    step = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    bound = tol.cpu() + step * (want.abs() + tol.cpu()) + 1e-37
    worst = ((got.double().cpu() - want).abs() / bound).max().item() if want.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst} of its bound"


def _forward(moe, rc, t, in_place=False):
    r = None if t["y"] is None else (t["resid"].clone() if in_place else torch.full_like(t["resid"], float("nan")))
    y = t["y"].clone() if in_place and t["y"] is not None else t["y"]
    n = None if t["pre"] is None else (y if in_place and y is not None else torch.full_like(t["resid"], float("nan")))
    moe.moe_residual_norm(rc, r if in_place and r is not None else t["resid"], y, t["post"], t["gate"], t["pre"],
                          t["rng"], r, n)
    return r, n


def _check_forward(rc, t, gate, r, n, y=None, y_err=0.0):
    w = _wide(t)
    if y is not None:
        w["y"] = y
    kp = _keep(rc, t)
    s_ref, n_ref = ref.forward(rc, gate, w["resid"], w["y"], w["post"], w["gate"], w["pre"], kp)
    s_tol, n_tol = ref.forward_bounds(rc, gate, w["resid"], w["y"], w["post"], w["gate"], w["pre"], kp, y_err)
    if r is not None:
        _close(r, s_ref, s_tol, "resid_out")
    if n is not None:
        _close(n, n_ref, n_tol, "norm_out")


SIZES = [(1, 8), (1, 2048), (3, 264), (5, 7168), (2, 8200), (700, 64), (2, 32768), (1300, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_forward(moe, T, D, dtype):
    rc, t, _ = _case(moe, T, D, dtype, "channel", res_scale=0.7, branch_scale=-1.3)
    _check_forward(rc, t, "channel", *_forward(moe, rc, t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_forward_forms(moe, dtype, gate, post, pre):
    rc, t, _ = _case(moe, 37, 520, dtype, gate, post=post, pre=pre, p=0.3, eps=1e-5)
    _check_forward(rc, t, gate, *_forward(moe, rc, t))
    _check_forward(rc, t, gate, *_forward(moe, rc, t, in_place=True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_norm(moe, dtype):
    rc, t, _ = _case(moe, 33, 1048, dtype, branch=False, post=False)
    _check_forward(rc, t, "none", *_forward(moe, rc, t))


def test_no_tokens(moe):
    rc, t, n = _case(moe, 0, 64, "bf16", "channel")
    r, o = _forward(moe, rc, t)
    d = {k: torch.full((64,), 7.0, device="cuda") for k in ("dpost_gain", "dgate", "dpre_gain")}
    moe.moe_residual_norm_backward(rc, r, t["y"], t["post"], t["gate"], t["pre"], None, r, r, o, r, **d,
                                   ws=moe.alloc_residual_workspace(rc))
    assert all((v == 0).all() for v in d.values())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_rows(moe, dtype):
    """A row of zeros, one that cancels to zero, one below eps, NaN and infinities: each stays in its row."""
    rc, t, _ = _case(moe, 6, 256, dtype)
    t["y"][0] = 0
    t["resid"][0] = 0
    t["post"] = t["post"] * 0 + 1
    t["y"][1] = 1
    t["resid"][1] = -1
    t["y"][2] *= 1e-6
    t["resid"][2] *= 1e-6
    t["y"][3, 5] = float("nan")
    t["resid"][4, 7] = float("inf")
    r, n = _forward(moe, rc, t)
    assert (r[0] == 0).all() and (n[0] == 0).all()
    assert r[1].float().abs().max() < 1e-5  # 1 rsqrt(1 + 1e-6) - 1
    assert r[3].isnan().all() and n[3].isnan().all()
    assert torch.isinf(r[4, 7]) and r[4].float().isinf().sum() == 1
    assert n[4, 7].isnan() and (n[4, :7] == 0).all()
    rows = [2, 5]
    sub = {k: (v[rows] if v is not None and v.dim() == 2 else v) for k, v in t.items()}
    rc2 = moe.ResidualConfig(T=2, D=256, dtype=rc.dtype)
    _check_forward(rc2, sub, "none", r[rows], n[rows])


def test_dropout_pinned(moe):
    """The published answer of Philox4x32-10 for the zero counter and key, and the share that stays."""
    assert [hex(int(v)) for v in ref.philox([0], 0, 0)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    T, D = 64, 4096
    rc = moe.ResidualConfig(T=T, D=D, dtype=moe.MOE_F32, p_drop=0.25)
    z, one = torch.zeros(T, D, device="cuda"), torch.ones(T, D, device="cuda")
    rng = torch.tensor([5, 9], device="cuda")
    r = torch.empty_like(z)
    moe.moe_residual_norm(rc, z, one, None, None, None, rng, r, None)
    assert torch.equal(r.cpu().double(), ref.keep(T, D, 0.25, (5, 9)).float().double())
    # 2^18 draws: six standard deviations are 6 sqrt(.25 .75 / 2^18) = 0.0051
    assert abs((r == 0).double().mean().item() - 0.25) < 0.0051
    other = torch.empty_like(z)
    for seed, offset in ((6, 9), (5, 10), (5 + (1 << 32), 9)):
        moe.moe_residual_norm(rc, z, one, None, None, None, torch.tensor([seed, offset], device="cuda"), other, None)
        assert not torch.equal(other, r)


# ---------------------------------------------------------------------------
# behind the combine
# ---------------------------------------------------------------------------

def _rows(moe, T, D, dtype, E, k, n, drop_all=False, e_first=0, e_local=-1):
    cfg = moe.Config(T=T, D=D, H_local=64, E=E, k=k, align_m=64, e_first=e_first, E_local=e_local,
                     dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32)
    ra = moe.rows_alloc(cfg)
    gen = torch.Generator().manual_seed(T + D)
    row = torch.randperm(ra, generator=gen)[:T * k].view(T, k).int() if ra >= T * k else \
        torch.randint(-1, max(ra, 1), (T, k), generator=gen).int()
    row[torch.rand(T, k, generator=gen) < 0.2] = -1
    row[0] = -1
    if drop_all:
        row[:] = -1
    w = torch.rand(T, k, generator=gen)
    y = n(ra, D, to=torch.float16 if dtype == "bf16" else torch.float32)
    y[torch.isin(torch.arange(ra), row.flatten(), invert=True).cuda()] = float("nan")  # rows of no token are not read
    return cfg, y, row.cuda(), w.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,E,k,gate", [(1, 2048, 8, 2, "channel"), (130, 264, 20, 3, "token"),
                                          (17, 7168, 16, 8, "none"), (9, 64, 40, 32, "element"), (3, 16392, 4, 4, "none")])
def test_combine(moe, dtype, T, D, E, k, gate):
    rc, t, n = _case(moe, T, D, dtype, gate, p=0.1)
    cfg, yp, row, w = _rows(moe, T, D, dtype, E, k, n)
    t["y"] = None
    ws = moe.alloc_workspace(cfg)
    outs = [torch.full_like(t["resid"], float("nan")) for _ in range(3)]
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, t["resid"], t["post"], t["gate"], t["pre"], t["rng"], *outs, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    at = row.long().clamp(min=0).cpu()
    part = torch.where((row >= 0).cpu()[..., None], w.double().cpu()[..., None] * yp.double().cpu()[at], 0.0)
    y = part.sum(1)
    y_err = 2 * k * ref.U * part.abs().sum(1)  # k products and k sums
    _close(outs[0], y, y_err, "y_out")
    _check_forward(rc, t, gate, outs[1], outs[2], y, y_err)
    # in place; y_out left out, and the unfused combine's rows
    r3, n3 = t["resid"].clone(), torch.empty_like(outs[0])
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, r3, t["post"], t["gate"], t["pre"], t["rng"], None, r3, n3, ws)
    assert torch.equal(r3, outs[1]) and torch.equal(n3, outs[2])
    y2, r2, n2 = (torch.empty_like(outs[0]) for _ in range(3))
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, t["resid"], t["post"], t["gate"], t["pre"], t["rng"], None, r2, n2, ws)
    assert torch.equal(r2, outs[1]) and torch.equal(n2, outs[2])
    moe.moe_unpermute_combine(cfg, yp, row, w, y2, ws)
    assert torch.equal(y2, outs[0])


def test_combine_no_local_expert(moe):
    rc, t, n = _case(moe, 5, 128, "bf16")
    cfg, yp, row, w = _rows(moe, 5, 128, "bf16", 8, 2, n, drop_all=True)
    t["y"] = None
    ws = moe.alloc_workspace(cfg)
    y, r, o = (torch.empty_like(t["resid"]) for _ in range(3))
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, t["resid"], t["post"], None, t["pre"], None, y, r, o, ws)
    assert (y == 0).all() and torch.equal(r, t["resid"])


def test_combine_bad_row_is_flagged(moe):
    rc, t, n = _case(moe, 4, 128, "bf16")
    cfg, yp, row, w = _rows(moe, 4, 128, "bf16", 8, 2, n)
    row[1, 0], row[2, 1] = moe.rows_alloc(cfg), -2
    ws = moe.alloc_workspace(cfg)
    outs = [torch.empty_like(t["resid"]) for _ in range(3)]
    args = (t["resid"], t["post"], None, t["pre"], None)
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, *args, *outs, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BAD_ROUTING
    row[1, 0] = row[2, 1] = -1
    want = [torch.empty_like(t["resid"]) for _ in range(3)]
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, *args, *want, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def _gradient(moe, rc, t, gate, dso, dn, in_place=False, ws=None):
    nan = float("nan")
    f32 = dict(device="cuda", dtype=torch.float32)
    d = dict(dresid=torch.full_like(t["resid"], nan), dy=None, dpost_gain=None, dgate=None, dpre_gain=None)
    if t["y"] is not None:
        d["dy"] = torch.full_like(t["resid"], nan)
    if in_place:
        dso, dn = dso.clone(), dn.clone()
        d["dresid"], d["dy"] = dn, dso
    if t["post"] is not None:
        d["dpost_gain"] = torch.full((rc.D,), nan, **f32)
    if t["pre"] is not None:
        d["dpre_gain"] = torch.full((rc.D,), nan, **f32)
    if t["gate"] is not None:
        d["dgate"] = torch.full_like(t["gate"], nan, dtype=None if gate == "element" else torch.float32)
    moe.moe_residual_norm_backward(rc, t["resid"], t["y"], t["post"], t["gate"], t["pre"], t["rng"], dso, dn, **d,
                                   ws=moe.alloc_residual_workspace(rc) if ws is None else ws)
    return d


def _check_gradient(rc, t, gate, dso, dn, d):
    w = _wide(t)
    want, tol = ref.gradient(rc, gate, w["resid"], w["y"], w["post"], w["gate"], w["pre"], _keep(rc, t),
                             None if dso is None else dso.double().cpu(), None if dn is None else dn.double().cpu())
    assert {k for k, v in d.items() if v is not None} == set(want)
    for k in want:
        _close(d[k], want[k], tol[k], k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_gradient(moe, T, D, dtype):
    rc, t, n = _case(moe, T, D, dtype, "channel", res_scale=0.7, branch_scale=-1.3)
    dso, dn = n(T, D), n(T, D)
    _check_gradient(rc, t, "channel", dso, dn, _gradient(moe, rc, t, "channel", dso, dn))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_gradient_forms(moe, dtype, gate, post, pre):
    rc, t, n = _case(moe, 37, 520, dtype, gate, post=post, pre=pre, p=0.3, eps=1e-5)
    dso, dn = n(37, 520), n(37, 520) if pre else None
    d = _gradient(moe, rc, t, gate, dso, dn)
    _check_gradient(rc, t, gate, dso, dn, d)
    if pre:
        e = _gradient(moe, rc, t, gate, dso, dn, in_place=True)
        assert all(d[k] is None or torch.equal(d[k], e[k]) for k in d)
        d = _gradient(moe, rc, t, gate, None, dn)
        _check_gradient(rc, t, gate, None, dn, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_first_norm(moe, dtype):
    rc, t, n = _case(moe, 700, 136, dtype, branch=False, post=False)
    for dso in (n(700, 136), None):
        dn = n(700, 136)
        _check_gradient(rc, t, "none", dso, dn, _gradient(moe, rc, t, "none", dso, dn))


@pytest.mark.parametrize("gate", list(GATES))
def test_gradient_against_differences(moe, gate):
    """The forward's change along a direction, by central differences in 64 bits, against the gradient's
    product with it.  Half a step h: rounding 1e-16 / h and the third derivative's h^2 stay below 1e-6 of the
    sum of the products' magnitudes, and so does fp32 (256 U = 1.5e-5 at most)."""
    T, D = 6, 72
    rc, t, n = _case(moe, T, D, "f32", gate, p=0.2)
    w, kp = _wide(t), _keep(rc, t)
    dso, dn = n(T, D), n(T, D)
    names = [k for k in ("resid", "y", "post", "gate", "pre") if w[k] is not None]
    s, _ = ref.forward(rc, gate, *(w[k] for k in ("resid", "y", "post", "gate", "pre")), kp)
    d = _gradient(moe, rc, dict(t, resid=s.float().cuda()), gate, dso, dn)

    def loss(x):
        s, o = ref.forward(rc, gate, *(x[k] for k in ("resid", "y", "post", "gate", "pre")), kp)
        return (s * dso.double().cpu() + o * dn.double().cpu()).sum()
    grads = dict(resid="dresid", y="dy", post="dpost_gain", gate="dgate", pre="dpre_gain")
    gen = torch.Generator().manual_seed(3)
    for k in names:
        way, h = torch.randn(w[k].shape, generator=gen, dtype=torch.float64), 1e-5
        change = (loss(dict(w, **{k: w[k] + h * way})) - loss(dict(w, **{k: w[k] - h * way}))) / (2 * h)
        prod = d[grads[k]].double().cpu() * way
        assert abs(change - prod.sum()) <= 2e-5 * prod.abs().sum() + 1e-8, k


def test_gradient_bitwise_reproducible_and_leaves_the_workspace_to_others(moe):
    rc, t, n = _case(moe, 999, 1048, "bf16", "channel", p=0.1)
    dso, dn = n(999, 1048), n(999, 1048)
    ws = moe.alloc_residual_workspace(rc)
    a = _gradient(moe, rc, t, "channel", dso, dn, ws=ws)
    ws.fill_(255)
    b = _gradient(moe, rc, t, "channel", dso, dn, ws=ws)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_captured_and_replayed_with_new_random_numbers(moe):
    rc, t, n = _case(moe, 64, 512, "bf16", "channel", p=0.5)
    dso, dn = n(64, 512), n(64, 512)
    r, o = torch.empty_like(t["resid"]), torch.empty_like(t["resid"])
    ws = moe.alloc_residual_workspace(rc)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        _gradient(moe, rc, t, "channel", dso, dn, ws=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            moe.moe_residual_norm(rc, t["resid"], t["y"], t["post"], t["gate"], t["pre"], t["rng"], r, o)
            d = _gradient(moe, rc, t, "channel", dso, dn, ws=ws)
    for i in range(3):
        t["rng"][1] = i
        t["y"].copy_(n(64, 512))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _check_forward(rc, t, "channel", r, o)
        _check_gradient(rc, t, "channel", dso, dn, d)


def test_side_stream(moe):
    rc, t, n = _case(moe, 300, 2048, "bf16", "token")
    dso, dn = n(300, 2048), n(300, 2048)
    want = _forward(moe, rc, t), _gradient(moe, rc, t, "token", dso, dn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _forward(moe, rc, t), _gradient(moe, rc, t, "token", dso, dn)
    side.synchronize()
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1], want[0][1])
    assert all(want[1][k] is None or torch.equal(got[1][k], want[1][k]) for k in want[1])


# rows enough for several a CTA (or a warp), in every shape of the kernels, with the last rows ragged
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(11003, 72), (7001, 264), (5003, 520), (4999, 1000), (2003, 1032), (1501, 2056), (1301, 4104),
                                 (701, 8192), (331, 12296), (309, 16400), (8195, 1608)])
def test_many_rows(moe, T, D, dtype):
    for gate, p in (("channel", 0.1), ("element", 0.0)):
        rc, t, n = _case(moe, T, D, dtype, gate, p=p)
        _check_forward(rc, t, gate, *_forward(moe, rc, t, in_place=gate == "element"))
        dso, dn = n(T, D), n(T, D)
        _check_gradient(rc, t, gate, dso, dn, _gradient(moe, rc, t, gate, dso, dn))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,E,k,gate,pre", [(3001, 520, 8, 2, "channel", True), (1999, 2048, 16, 6, "token", True),
                                              (1400, 4104, 12, 3, "element", True), (2500, 1032, 8, 4, "none", False),
                                              (1203, 1048, 40, 32, "channel", True)])
def test_combine_many_rows(moe, dtype, T, D, E, k, gate, pre):
    rc, t, n = _case(moe, T, D, dtype, gate, p=0.1 if k < 4 else 0.0, pre=pre)
    cfg, yp, row, w = _rows(moe, T, D, dtype, E, k, n)
    t["y"] = None
    row[T // 2, 0], row[T - 1, k - 1] = moe.rows_alloc(cfg), -7  # flagged, and left out
    ws = moe.alloc_workspace(cfg)
    y, r, o = (torch.full_like(t["resid"], float("nan")) for _ in range(3))
    o = o if pre else None
    moe.moe_combine_residual_norm(cfg, rc, yp, row, w, t["resid"], t["post"], t["gate"], t["pre"], t["rng"], y, r, o, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BAD_ROUTING
    row[T // 2, 0] = row[T - 1, k - 1] = -1
    at = row.long().clamp(min=0)
    want, size = torch.zeros(T, D, dtype=torch.float64, device="cuda"), torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for j in range(k):
        part = torch.where((row[:, j] >= 0)[:, None], w[:, j, None].double() * yp[at[:, j]].double(), 0.0)
        want += part
        size += part.abs()
    y_err = 2 * k * ref.U * size.cpu()
    _close(y, want, y_err, "y_out")
    _check_forward(rc, t, gate, r, o, want.cpu(), y_err)
