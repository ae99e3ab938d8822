"""moe_layer_forward_few against the layer in 64 bits.

Keys of different experts that lie within rounding of each other have no single answer, so tokens whose
choice is that close are drawn anew before anything runs."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _choose(c, key):
    """(chosen experts in order, how far the choice is from another one) by the rules of moe_route_topk."""
    idx, gaps = [], []
    for row in key.tolist():
        among, gap = range(c.E), float("inf")
        if c.n_group > 1:
            n, m = c.E // c.n_group, c.k // c.topk_group
            score = [sum(sorted(row[q * n:q * n + n], reverse=True)[:m]) for q in range(c.n_group)]
            order = sorted(range(c.n_group), key=lambda q: (-score[q], q))
            if c.topk_group < c.n_group:
                gap = score[order[c.topk_group - 1]] - score[order[c.topk_group]]
            among = [e for e in among if e // n in order[:c.topk_group]]
        order = sorted(among, key=lambda e: (-row[e], e))
        if c.k < len(order):
            gap = min(gap, row[order[c.k - 1]] - row[order[c.k]])
        idx.append(order[:c.k])
        gaps.append(gap)
    return torch.tensor(idx), torch.tensor(gaps)


def _inputs(moe, c, seed=0, bias=True, hot=None):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * c.T + c.D)
    dt = c.torch_dtype

    def n(*s, scale=1.0, to=dt):
        return (scale * torch.randn(s, generator=g, device="cuda")).to(to)
    t = dict(wg=n(c.E, c.D, scale=c.D ** -0.5), bias=n(c.E, scale=0.1, to=torch.float32) if bias else None,
             w1=n(c.e_local, c.H_local, c.D, scale=c.D ** -0.5), w3=n(c.e_local, c.H_local, c.D, scale=c.D ** -0.5),
             w2=n(c.e_local, c.D, c.H_local, scale=c.H_local ** -0.5))
    if hot is not None:
        t["bias"][hot] += 30.0
    x = n(c.T, c.D)
    for _ in range(50):
        close = _choose(c, _keys(dict(t, x=x)))[1] < 1e-4
        if not close.any():
            break
        x[close.cuda()] = n(int(close.sum()), c.D)
    else:
        raise AssertionError("no clear choice found")
    return dict(t, x=x)


def _keys(t):
    key = t["x"].double() @ t["wg"].double().T
    return (key if t["bias"] is None else key + t["bias"].double()).cpu()


def _reference(c, t, moe):
    """out in 64 bits and what the kernel's roundings may add: fp32 sums of n terms are off by n U of the terms'
    magnitudes, h by half a step of its type, silu' <= 1.1, and a weight by the keys' errors (twice the largest:
    numerator and sum) and 32 U of exp and division."""
    key = _keys(t)
    idx, _ = _choose(c, key)
    p = torch.softmax(key, 1) if c.score == moe.MOE_SCORE_SOFTMAX else torch.sigmoid(key)
    w = torch.gather(p, 1, idx)
    if c.renorm:
        w = w / w.sum(1, keepdim=True)
    kerr = (c.D + 8) * U * (t["x"].double().abs() @ t["wg"].double().abs().T).max().item() + 8 * U * key.abs().max().item()
    werr = 2 * kerr + 32 * U
    step = 2.0 ** -8 if c.torch_dtype == torch.bfloat16 else U
    out = torch.zeros(c.T, c.D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for i in range(c.e_local):
        at, slot = torch.nonzero(idx == c.e_first + i, as_tuple=True)
        if len(at) == 0:
            continue
        w1, w3, w2 = (t[k][i].double() for k in ("w1", "w3", "w2"))
        x = t["x"][at.cuda()].double()
        gate, up = x @ w1.T, x @ w3.T
        dg, du = (c.D + 8) * U * (x.abs() @ w1.abs().T), (c.D + 8) * U * (x.abs() @ w3.abs().T)
        h = gate * torch.sigmoid(gate) * up
        dh = 1.1 * dg * (up.abs() + du) + (gate * torch.sigmoid(gate)).abs() * du + (16 * U + step) * h.abs()
        wt = w[at, slot].cuda()[:, None]
        a = at.cuda()
        out[a] += wt * (h @ w2.T)
        tol[a] += wt * (dh @ w2.abs().T + (c.H_local + c.k + 64 + werr / U) * U * (h.abs() @ w2.abs().T))
    return out, tol + step * (out.abs() + tol) + 1e-37


def _call(moe, c, t, ws=None, **kw):
    ws = moe.alloc_workspace(c, few=True) if ws is None else ws
    out = torch.full((c.T, c.D), float("nan"), dtype=c.torch_dtype, device="cuda")
    before = moe.kernel_launches()
    moe.moe_layer_forward_few(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], out, ws, **kw)
    launched = moe.kernel_launches() - before
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    return out, launched


def _check(moe, c, t, out):
    want, tol = _reference(c, t, moe)
    err = (out.double() - want).abs()
    worst = (err / tol).max().item()
    assert worst <= 1.0, f"{worst} of the bound"
    # That bound adds every h's error up in full.  They are independent: relative errors of h spread evenly over a
    # step (at most 2^-8 either way: a deviation of 2^-8 / sqrt 3) move out by 2^-8 / sqrt 3 = 0.0023 of its RMS, and
    # 1e-2 is over four such deviations at the least favourable place of h in its binade.  out's own rounding, up to
    # 2^-8 of the value (0.02 of the RMS for a value of five), comes on top: it is taken off first.
    rms = want.square().mean().sqrt().item()
    if rms > 0:
        bf16 = c.torch_dtype == torch.bfloat16
        beyond = (err - 2.0 ** -8 * want.abs()).max().item() if bf16 else err.max().item()
        assert beyond <= (1e-2 if bf16 else 1e-4) * rms


CASES = [
    dict(T=1, D=2048, H_local=1408, E=64, k=6, renorm=1),
    dict(T=1, D=8, H_local=8, E=1, k=1),
    dict(T=1, D=24, H_local=8, E=3, k=2, score=1),
    dict(T=2, D=1048, H_local=424, E=20, k=3, score=1, renorm=1),
    dict(T=7, D=520, H_local=72, E=130, k=8, renorm=1),
    dict(T=8, D=256, H_local=512, E=16, k=4, n_group=4, topk_group=2, score=1, renorm=1),
    dict(T=9, D=4104, H_local=136, E=5, k=5),
    dict(T=16, D=640, H_local=1032, E=256, k=8, n_group=8, topk_group=4),
    dict(T=31, D=136, H_local=264, E=2, k=2, renorm=1),
    dict(T=32, D=264, H_local=40, E=1024, k=32, renorm=1),
    dict(T=32, D=8, H_local=2048, E=4, k=1),
    dict(T=32, D=520, H_local=264, E=32, k=32),
    dict(T=3, D=4608, H_local=4104, E=3, k=1, score=1),
    dict(T=32, D=1048, H_local=424, E=20, k=3, e_first=3, E_local=13, score=1, renorm=1),
]


@pytest.mark.parametrize("dtype", [1, 0], ids=["bf16", "f32"])
@pytest.mark.parametrize("kw", CASES, ids=lambda kw: f"T{kw['T']}D{kw['D']}H{kw['H_local']}E{kw['E']}k{kw['k']}")
def test_layer(moe, kw, dtype):
    c = moe.Config(dtype=dtype, **kw)
    t = _inputs(moe, c, bias=kw["T"] % 2 == 0)
    out, launched = _call(moe, c, t)
    assert launched == 1
    _check(moe, c, t, out)


@pytest.mark.parametrize("T", range(1, 33))
def test_every_number_of_tokens(moe, T):
    c = moe.Config(T=T, D=128, H_local=136, E=8, k=2, renorm=1)
    t = _inputs(moe, c, seed=T)
    _check(moe, c, t, _call(moe, c, t)[0])


@pytest.mark.parametrize("T", [8, 9, 25, 32])
def test_every_token_on_one_expert(moe, T):
    c = moe.Config(T=T, D=512, H_local=264, E=8, k=1)
    t = _inputs(moe, c, hot=5)
    _check(moe, c, t, _call(moe, c, t)[0])


@pytest.mark.parametrize("dtype", [1, 0], ids=["bf16", "f32"])
def test_no_local_expert(moe, dtype):
    for kw in (dict(e_first=3, E_local=0), dict(e_first=0, E_local=3)):
        c = moe.Config(T=5, D=136, H_local=64, E=8, k=1, dtype=dtype, **kw)
        t = _inputs(moe, c, hot=6)
        assert (_call(moe, c, t)[0] == 0).all()


def test_no_tokens(moe):
    c = moe.Config(T=0, D=64, H_local=64, E=8, k=2)
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 64, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_forward_few(c, z, w[0, :8].contiguous(), None, w, w, w, z, moe.alloc_workspace(c, few=True))


def test_shards_add_up(moe):
    full = moe.Config(T=6, D=264, H_local=128, E=12, k=4, dtype=0, renorm=1)
    t = _inputs(moe, full)
    want, _ = _reference(full, t, moe)
    got = torch.zeros_like(want)
    for e0, el in ((0, 5), (5, 7)):
        for h0 in (0, 64):
            c = moe.Config(T=6, D=264, H_local=64, E=12, k=4, dtype=0, renorm=1, e_first=e0, E_local=el)
            part = dict(t, w1=t["w1"][e0:e0 + el, h0:h0 + 64].contiguous(), w3=t["w3"][e0:e0 + el, h0:h0 + 64].contiguous(),
                        w2=t["w2"][e0:e0 + el, :, h0:h0 + 64].contiguous())
            got += _call(moe, c, part)[0].double()
    assert (got - want).abs().max() <= 1e-5 * want.square().mean().sqrt()


def test_agrees_with_the_layer(moe):
    c = moe.Config(T=16, D=512, H_local=256, E=32, k=4, renorm=1)
    t = _inputs(moe, c)
    out = torch.empty_like(t["x"])
    ws = moe.alloc_workspace(c, layer=True)
    moe.moe_layer_forward(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], out, ws)
    got, _ = _call(moe, c, t)
    # each side rounds out once, at most 2^-8 of the value: together a whole step, 2^-7; the layer's h and y_perm,
    # rounded where this call's are not, add less than 1e-2 of the RMS (see _check)
    a, b = got.float(), out.float()
    assert ((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 1e-2 * b.square().mean().sqrt()).all()


def test_workspace_reused_for_fewer_tokens_and_left_dirty(moe):
    """One workspace for the largest batch serves every smaller one; what a call leaves behind is not read."""
    big = moe.Config(T=32, D=264, H_local=136, E=16, k=4, renorm=1)
    ws = moe.alloc_workspace(big, few=True)
    head = 256 + -(-4 * (64 + -(-264 // 16)) // 256) * 256  # status and counters
    for T in (32, 1, 9, 32, 3):
        c = moe.Config(T=T, D=264, H_local=136, E=16, k=4, renorm=1)
        t = _inputs(moe, c, seed=T)
        fresh, _ = _call(moe, c, t)
        assert torch.equal(_call(moe, c, t, ws)[0], fresh)
        assert (ws[:head] == 0).all()
        ws[head:] = 255


def test_workspace_shared_by_configs_of_the_same_width(moe):
    cfgs = [moe.Config(T=T, D=264, H_local=H, E=E, k=k, renorm=1, dtype=dt)
            for T, H, E, k, dt in ((32, 264, 64, 8, 0), (5, 72, 3, 3, 1), (16, 520, 100, 2, 1), (1, 8, 8, 8, 0))]
    n = max(moe.layer_few_workspace_size(c) for c in cfgs)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for c in cfgs + cfgs[::-1]:
        t = _inputs(moe, c)
        assert torch.equal(_call(moe, c, t, ws)[0], _call(moe, c, t)[0])


def test_in_place(moe):
    """out may be x: every CTA has read x before any writes."""
    c = moe.Config(T=7, D=520, H_local=136, E=8, k=2, renorm=1)
    t = _inputs(moe, c)
    want, ws = _call(moe, c, t)[0], moe.alloc_workspace(c, few=True)
    moe.moe_layer_forward_few(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], t["x"], ws)
    assert torch.equal(t["x"], want)


def test_two_streams_with_a_workspace_each(moe):
    """Two calls at once: each grid needs the whole device, so they take turns."""
    c = moe.Config(T=8, D=1032, H_local=520, E=16, k=4, renorm=1)
    t = [_inputs(moe, c, seed=i) for i in range(2)]
    want = [_call(moe, c, v)[0] for v in t]
    ws, out = [moe.alloc_workspace(c, few=True) for _ in t], [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in t]
    torch.cuda.synchronize()
    for _ in range(20):
        for v, w, o, s in zip(t, ws, out, streams):
            moe.moe_layer_forward_few(c, v["x"], v["wg"], v["bias"], v["w1"], v["w3"], v["w2"], o, w, stream=s)
    torch.cuda.synchronize()
    for w, o, e in zip(ws, out, want):
        assert moe.moe_get_device_status(w) == moe.MOE_OK and torch.equal(o, e)


def test_another_device_or_the_host(moe, monkeypatch):
    """A workspace that is not on the current device is refused before any launch (the current device is made
    to look like another one)."""
    c = moe.Config(T=4, D=64, H_local=64, E=8, k=2)
    t = _inputs(moe, c)
    rc = moe.ResidualConfig(T=4, D=64)
    ws, rws = moe.alloc_workspace(c, few=True), moe.alloc_residual_workspace(rc)
    x, g = t["x"], t["x"][0].contiguous()
    y = torch.zeros(moe.rows_alloc(c), 64, dtype=torch.float16, device="cuda")
    row, w, f = (torch.zeros(4, 2, dtype=d, device="cuda") for d in (torch.int32, torch.float32, torch.float32))
    sw, f = moe.alloc_workspace(c), torch.empty(64, device="cuda")

    def calls(ws, rws, sw, x):
        return (lambda: moe.moe_layer_forward_few(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], t["x"], ws),
                lambda: moe.moe_residual_norm(rc, x, None, None, None, g, None, None, x),
                lambda: moe.moe_combine_residual_norm(c, rc, y, row, w, t["x"], None, None, g, None, None, t["x"], t["x"], sw),
                lambda: moe.moe_residual_norm_backward(rc, t["x"], None, None, None, g, None, None, t["x"], t["x"], None,
                                                       None, None, f, rws))
    before, real = moe.kernel_launches(), torch.cuda.current_device()
    for call in calls(ws.cpu(), rws.cpu(), sw.cpu(), x.cpu()):
        with pytest.raises(ValueError, match="on cpu|CUDA tensor"):
            call()
    monkeypatch.setattr(moe, "_device", lambda: real + 1)
    for call in calls(ws, rws, sw, x):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert moe.kernel_launches() == before


def test_bitwise_reproducible(moe):
    c = moe.Config(T=12, D=2056, H_local=512, E=32, k=4, renorm=1)
    t, ws = _inputs(moe, c), None
    ws = moe.alloc_workspace(c, few=True)
    first = _call(moe, c, t, ws)[0]
    for _ in range(10):
        assert torch.equal(_call(moe, c, t, ws)[0], first)


def test_three_launches(moe, monkeypatch):
    """Where the grid cannot be resident at once its stages are launched one by one: the same results."""
    for kw in CASES[:6]:
        for dtype in (0, 1):
            c = moe.Config(dtype=dtype, **kw)
            t = _inputs(moe, c)
            monkeypatch.delenv("MOE_FEW_LAUNCHES", raising=False)
            one, n1 = _call(moe, c, t)
            monkeypatch.setenv("MOE_FEW_LAUNCHES", "3")
            three, n3 = _call(moe, c, t)
            assert (n1, n3) == (1, 3) and torch.equal(one, three)


def test_nan_and_infinity_stay_in_their_token(moe):
    c = moe.Config(T=4, D=264, H_local=72, E=8, k=2, renorm=1)
    t = _inputs(moe, c)
    clean = {k: v for k, v in t.items()} | dict(x=t["x"][[0, 2, 3]].contiguous())
    t["x"][1, 3] = float("nan")
    ws = moe.alloc_workspace(c, few=True)
    out = torch.empty_like(t["x"])
    moe.moe_layer_forward_few(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BAD_ROUTING
    assert out[1].isnan().all()
    _check(moe, moe.Config(T=3, D=264, H_local=72, E=8, k=2, renorm=1), clean, out[[0, 2, 3]])


def test_captured_replayed_and_on_a_side_stream(moe):
    c = moe.Config(T=5, D=512, H_local=256, E=16, k=4, renorm=1)
    t = _inputs(moe, c)
    ws, out = moe.alloc_workspace(c, few=True), torch.empty_like(t["x"])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        def call():
            moe.moe_layer_forward_few(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], out, ws)
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
            t["x"].copy_(out)  # a step feeds the next
            call()
    for seed in range(3):
        new = _inputs(moe, c, seed=seed)
        with torch.cuda.stream(stream):
            t["x"].copy_(new["x"])
            graph.replay()
        stream.synchronize()
        twice = dict(t, x=_call(moe, c, dict(t, x=new["x"]))[0])
        assert torch.equal(out, _call(moe, c, twice)[0])
    assert moe.moe_get_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("barrier", [0, 1])
def test_a_barrier_that_is_never_met_is_reported(moe, barrier):
    """A count planted in the workspace that cannot be reached: the waits give up after a second, the call
    reports it, and the next call is right again."""
    c = moe.Config(T=3, D=512, H_local=256, E=16, k=4, renorm=1)
    t = _inputs(moe, c)
    ws = moe.alloc_workspace(c, few=True)
    want = _call(moe, c, t, ws)[0]
    bars = ws[256:256 + 12].view(torch.int32)
    bars[barrier] = -(1 << 30)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    moe.moe_layer_forward_few(c, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], torch.empty_like(want), ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_TIMEOUT
    assert 0.9 < time.perf_counter() - t0 < 30
    assert (ws[:256 + 4 * (64 + 32)] == 0).all()
    assert torch.equal(_call(moe, c, t, ws)[0], want)


def test_a_decode_step_between_its_norms(moe):
    """Norm, layer and norm as a step of decoding runs them, against the same in 64 bits."""
    T, D = 4, 512
    c = moe.Config(T=T, D=D, H_local=256, E=16, k=4, renorm=1)
    t = _inputs(moe, c, bias=False)
    g = torch.Generator(device="cuda").manual_seed(1)
    resid, pre, post, after = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, D), (D,), (D,), (D,)))
    rc = moe.ResidualConfig(T=T, D=D, branch_scale=0.5)
    x, y, r, n = (torch.empty_like(resid) for _ in range(4))
    moe.moe_residual_norm(rc, resid, None, None, None, pre, None, None, x)
    ws = moe.alloc_workspace(c, few=True)
    moe.moe_layer_forward_few(c, x, t["wg"], None, t["w1"], t["w3"], t["w2"], y, ws)
    moe.moe_residual_norm(rc, resid, y, post, None, after, None, r, n)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK

    def rms(v, gain):
        v = v.double()
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * gain.double()
    _check(moe, c, dict(t, x=x), y)
    assert torch.allclose(x.double(), rms(resid, pre), rtol=2 ** -8 * 1.01, atol=1e-30)
    s = resid.double() + 0.5 * rms(y, post)
    assert ((r.double() - s).abs() <= 2 ** -8 * s.abs() + 2 ** -18 * (resid.double().abs() + 1)).all()
    assert ((n.double() - rms(s, after)).abs() <= 2 ** -8 * rms(s, after).abs() + 2 ** -16).all()


# rows of 1, 2, 3, 4, 5, 8 and 9 steps of 256 bytes: fewer than all warps share the short ones
@pytest.mark.parametrize("dtype", [1, 0], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,H", [(128, 1152), (136, 1032), (264, 1024), (392, 640), (520, 512), (640, 264), (1024, 136), (1160, 120)])
def test_rows_of_every_length(moe, D, H, dtype):
    f = 1 if dtype else 2  # the same bytes in fp32
    for T, E, k in ((1, 9, 7), (13, 6, 3), (30, 3, 2)):
        c = moe.Config(T=T, D=D // f // 8 * 8, H_local=H // f // 8 * 8, E=E, k=k, dtype=dtype, renorm=1)
        t = _inputs(moe, c)
        _check(moe, c, t, _call(moe, c, t)[0])
