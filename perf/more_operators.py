"""Measured cases of the layer for a few tokens and of the norms around a block.

Four kinds of pass, each in a plain form (elementary torch operations, fp32)
and through this package's entry points:

  few       the whole layer for at most 32 tokens, from the router to the
            weighted sum of the chosen experts;
  norm      the end of a block and the norm in front of the next one: the
            branch's output normalised, dropped out, gated, scaled and added
            to the scaled residual, and the norm of that sum;
  combine   the same with the branch's output still in the experts' rows: the
            weighted sum over a token's rows comes first;
  gradient  the gradient of `norm`: of the residual, the branch, both norms'
            gains and the gate.
"""
import math

import numpy
import torch

own = False

FEW_TOKENS = 32
BACKWARD_KEYS = ("dresid", "dy", "dpost_gain", "dgate", "dpre_gain")


def listed():
    return [
        # one token of a decode step through the fine-grained layer: latency and weight streaming
        dict(name="few-one-token", kind="few", T=1, D=2048, H=1408, E=64, k=6, e_first=0, E_local=64,
             dtype="bf16", score="softmax", renorm=1, bias=False, n_group=0, topk_group=0),
        # a handful of sequences decoded together, or the drafted tokens of one
        dict(name="few-eight-tokens", kind="few", T=8, D=2048, H=1408, E=64, k=6, e_first=0, E_local=64,
             dtype="bf16", score="softmax", renorm=1, bias=False, n_group=0, topk_group=0),
        # 256 large experts, group-limited routing by biased sigmoid scores, a decode batch of 16
        dict(name="few-256-large", kind="few", T=16, D=7168, H=2048, E=256, k=8, e_first=0, E_local=256,
             dtype="bf16", score="sigmoid", renorm=1, bias=True, n_group=8, topk_group=4),
        # odd sizes and a shard that holds only some of the experts, as many tokens as the call takes
        dict(name="few-odd-shard", kind="few", T=32, D=1048, H=424, E=20, k=3, e_first=3, E_local=13,
             dtype="bf16", score="sigmoid", renorm=1, bias=True, n_group=0, topk_group=0),
        # the smallest layer, fp32 throughout: latency
        dict(name="few-tiny-f32", kind="few", T=4, D=128, H=256, E=8, k=2, e_first=0, E_local=8,
             dtype="f32", score="softmax", renorm=0, bias=False, n_group=0, topk_group=0),
        # one token between two blocks: latency
        dict(name="norm-one-token", kind="norm", T=1, D=7168, dtype="bf16", branch=True, post=True, gate="channel",
             p_drop=0.0),
        # a prefill chunk's residual stream between two blocks, both norms and a learned gate per channel
        dict(name="norm-prefill", kind="norm", T=16384, D=4096, dtype="bf16", branch=True, post=True, gate="channel",
             p_drop=0.0),
        # a decode batch behind the experts
        dict(name="combine-decode", kind="combine", T=128, D=7168, E=256, k=8, e_first=0, E_local=256, align_m=128,
             dtype="bf16", post=True, gate="none", p_drop=0.0),
        # the fine-grained layer's batch behind the experts, a gate per token
        dict(name="combine-fine-grained", kind="combine", T=4096, D=2048, E=64, k=6, e_first=0, E_local=64,
             align_m=128, dtype="bf16", post=True, gate="token", p_drop=0.0),
        # a training step of the fine-grained layer with dropout on the branch
        dict(name="gradient-dropout", kind="gradient", T=4096, D=2048, dtype="bf16", branch=True, post=True,
             gate="channel", p_drop=0.1),
        # wide rows of a long batch
        dict(name="gradient-wide", kind="gradient", T=8192, D=7168, dtype="bf16", branch=True, post=True,
             gate="channel", p_drop=0.0),
        # odd sizes in fp32, a gate for every element
        dict(name="gradient-odd-f32", kind="gradient", T=777, D=1048, dtype="f32", branch=True, post=True,
             gate="element", p_drop=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["few", "few", "few", "norm", "combine", "gradient", "gradient"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind != "few":
        D = 8 * _log_int(rng, 8, 1024)
        T = _log_int(rng, 1, min(16384, (1 << 26) // D))
        c = dict(kind=kind, T=T, D=D, dtype=dtype, post=rng.random() < 0.7,
                 gate=rng.choice(["none", "channel", "token", "element"]), p_drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
        if kind != "combine":
            c["branch"] = rng.random() < 0.85
            if not c["branch"]:
                c.update(post=False, gate="none", p_drop=0.0)
            return c
        E = _log_int(rng, 1, 256)
        first = rng.randint(0, E // 2) if rng.random() < 0.3 else 0
        return c | dict(T=min(T, 8192), E=E, k=rng.randint(1, min(E, 8)), e_first=first,
                        E_local=rng.randint(1, E - first) if first else E, align_m=rng.choice([1, 64, 128]))
    E = _log_int(rng, 2, 256)
    k = rng.randint(1, min(E, 8))
    e_first, E_local = 0, E
    if rng.random() < 0.3:
        e_first = rng.randint(0, E // 2)
        E_local = rng.randint(1, E - e_first)
    n_group = topk_group = 0
    if E % 4 == 0 and E >= 16 and k % 2 == 0 and rng.random() < 0.3:
        n_group, topk_group = 4, 2
        k = min(k, E // 2)
    D, H = 8 * _log_int(rng, 8, 896), 8 * _log_int(rng, 4, 256)
    # all experts' weights take no more than the largest listed case's
    while E_local * D * H > 256 * 7168 * 2048 * (1 if dtype == "bf16" else 0.5):
        H = max(8, H // 16 * 8)
    return dict(kind=kind, T=rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, FEW_TOKENS)]), D=D, H=H, E=E, k=k,
                e_first=e_first, E_local=E_local, dtype=dtype, score=rng.choice(["softmax", "sigmoid"]),
                renorm=rng.randint(0, 1), bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _normal(g, shape, dtype, scale=1.0):
    """Normal values, made in pieces: a layer's weights in fp32 would not fit beside themselves."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        p = flat[i:i + (1 << 28)]
        p.copy_(torch.randn(p.shape, generator=g, device="cuda").mul_(scale))
    return out


def _stream(g, T, D, dtype):
    """A residual stream: rows of different size and a few outlier channels."""
    x = torch.randn((T, D), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))
    x *= 1.0 + 15.0 * (torch.rand((1, D), generator=g, device="cuda") < 0.01)
    return x.to(dtype)


def _gap(v, n):
    """How far the n-th largest lies above the next one, by rows."""
    if n >= v.shape[1]:
        return torch.full_like(v[:, 0], math.inf)
    top = torch.topk(v, n + 1, dim=1).values
    return top[:, n - 1] - top[:, n]


def _unclear(c, key):
    """Tokens whose choice of experts hangs on a difference within rounding: it has no single answer."""
    if c["n_group"] > 1:
        by = key.unflatten(1, (c["n_group"], -1))
        score = torch.topk(by, c["k"] // c["topk_group"], dim=2).values.sum(2)
        close = _gap(score, c["topk_group"]) < 1e-3
        kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, torch.topk(score, c["topk_group"]).indices, True)
        return close | (_gap(by.masked_fill(~kept.unsqueeze(2), -1e30).flatten(1), c["k"]) < 1e-3)
    return _gap(key, c["k"]) < 1e-3


def _prepare_few(c, g):
    dt, T, D, H, E, El = _dtype(c), c["T"], c["D"], c["H"], c["E"], c["E_local"]
    s = dict(case=c)
    s["wg"] = _normal(g, (E, D), dt, 1.0 / math.sqrt(D))
    s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if c["bias"] else None
    x = torch.randn((T, D), generator=g, device="cuda").to(dt)
    for _ in range(20):
        key = x.double() @ s["wg"].double().T + (0 if s["bias"] is None else s["bias"].double())
        bad = _unclear(c, key).unsqueeze(1)
        x = torch.where(bad, torch.randn((T, D), generator=g, device="cuda").to(dt), x)
    s["x"] = x
    s["w1"] = _normal(g, (El, H, D), dt, 1.0 / math.sqrt(D))
    s["w3"] = _normal(g, (El, H, D), dt, 1.0 / math.sqrt(D))
    s["w2"] = _normal(g, (El, D, H), dt, 1.0 / math.sqrt(H))
    return s


def _prepare_rows(c, g):
    """The experts' rows of a routed batch, their places and weights."""
    T, k, El = c["T"], c["k"], c["E_local"]
    score, idx = torch.topk(torch.randn((T, c["E"]), generator=g, device="cuda"), k, dim=1)
    e = idx.reshape(-1) - c["e_first"]
    e = torch.where((e >= 0) & (e < El), e, torch.full_like(e, El))
    order = torch.argsort(e, stable=True)
    count = torch.bincount(e, minlength=El + 1)
    rank = torch.empty_like(e)
    rank[order] = torch.arange(T * k, device=e.device) - (torch.cumsum(count, 0) - count)[e[order]]
    a = c["align_m"]
    size = (count[:El] + a - 1) // a * a
    start = torch.cumsum(size, 0) - size
    row = torch.where(e < El, start[e.clamp(max=El - 1)] + rank, torch.full_like(e, -1))
    rows = T * min(k, El) + El * (a - 1)
    y = _normal(g, (rows, c["D"]), torch.float16 if c["dtype"] == "bf16" else torch.float32)
    return dict(row_of=row.view(T, k).int(), topk_w=torch.softmax(score, dim=1).contiguous(), y_perm=y)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["kind"] == "few":
        return _prepare_few(c, g)
    dt, T, D = _dtype(c), c["T"], c["D"]
    s = dict(case=c, eps=1e-6, res_scale=1.0, branch_scale=0.22, resid=_stream(g, T, D, dt), y=None, post=None,
             gate=None, rng=None)
    s["pre"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    if c["kind"] == "combine":
        s.update(_prepare_rows(c, g))
    elif c["branch"]:
        s["y"] = _normal(g, (T, D), dt)
    if c["post"]:
        s["post"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    if c["gate"] == "channel":
        s["gate"] = torch.randn(D, generator=g, device="cuda").to(dt)
    elif c["gate"] == "token":
        s["gate"] = torch.sigmoid(torch.randn(T, generator=g, device="cuda"))
    elif c["gate"] == "element":
        s["gate"] = torch.sigmoid(torch.randn((T, D), generator=g, device="cuda")).to(dt)
    if c["p_drop"]:
        s["rng"] = torch.randint(1 << 40, (2,), generator=g, device="cuda")  # seed, offset
    if c["kind"] == "gradient":
        s["dresid_out"], s["dnorm_out"] = _normal(g, (T, D), dt), _normal(g, (T, D), dt)
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------

def _plain_route(s):
    """Chosen experts and their weights."""
    c = s["case"]
    key = s["x"].double() @ s["wg"].double().T  # in 64 bits: values next to a border
    if s["bias"] is not None:
        key = key + s["bias"].double()
    open_ = key
    if c["n_group"] > 1:
        by = key.unflatten(1, (c["n_group"], -1))
        score = torch.sort(by, dim=2, descending=True).values[..., :c["k"] // c["topk_group"]].sum(2)
        best = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        open_ = torch.where(kept.unsqueeze(2), by, torch.full_like(by, -math.inf)).flatten(1)
    idx = torch.sort(open_, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-key))
    else:
        p = torch.exp(key - key.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, w.float()


def _plain_few(s):
    c = s["case"]
    idx, w = _plain_route(s)
    x = s["x"].float().unsqueeze(2)
    out = torch.zeros((c["T"], c["D"]), device=x.device)
    for j in range(c["k"]):
        e = idx[:, j] - c["e_first"]
        here = (e >= 0) & (e < c["E_local"])
        e = e.clamp(0, c["E_local"] - 1)
        gate = torch.bmm(s["w1"][e].float(), x)
        h = gate / (1 + torch.exp(-gate)) * torch.bmm(s["w3"][e].float(), x)
        y = torch.bmm(s["w2"][e].float(), h).squeeze(2)
        out += torch.where(here, w[:, j], torch.zeros_like(w[:, j])).unsqueeze(1) * y
    return out.to(s["x"].dtype)


def _words(rng, n):
    """Philox4x32 of ten rounds (Salmon and others, "Parallel random numbers: as easy as 1, 2, 3", 2011) for the
    counters (i, offset), i < n, under the key seed: [n, 4] words."""
    low = 0xffffffff
    i = torch.arange(n, device=rng.device)
    seed, offset = rng[0], rng[1]
    c0, c1 = i & low, i >> 32
    c2, c3 = (offset & low).expand(n), ((offset >> 32) & low).expand(n)
    k0, k1 = seed & low, (seed >> 32) & low

    def product(a, b):  # high and low word of a 64-bit product, in halves of b
        t = a * (b >> 16) + ((a * (b & 0xffff)) >> 16)
        return t >> 16, (a * b) & low

    for _ in range(10):
        h0, l0 = product(0xd2511f53, c0)
        h1, l1 = product(0xcd9e8d57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9e3779b9) & low, (k1 + 0xbb67ae85) & low
    return torch.stack([c0, c1, c2, c3], dim=1)


def _plain_keep(s):
    """1 / (1 - p) for an element that stays and 0 for one that is dropped, p in steps of 2^-16: eight elements to
    a counter, a half word each, the low half first."""
    c = s["case"]
    if not c["p_drop"]:
        return 1.0
    cut = round(c["p_drop"] * 65536)
    w = _words(s["rng"], c["T"] * c["D"] // 8)
    u = torch.stack([w & 0xffff, w >> 16], dim=2).view(c["T"], c["D"])
    return torch.where(u >= cut, 65536.0 / (65536 - cut), 0.0)


def _rate(x, eps):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)


def _gate(s):
    if s["gate"] is None:
        return 1.0
    g = s["gate"].float()
    return g.unsqueeze(1) if s["case"]["gate"] == "token" else g


def _plain_norm(s):
    c, dt = s["case"], s["resid"].dtype
    r, out = s["resid"].float(), {}
    y = None
    if c["kind"] == "combine":
        row = s["row_of"].long()
        y = torch.zeros_like(r)
        for j in range(c["k"]):
            there = (row[:, j] >= 0).unsqueeze(1)
            y += torch.where(there, s["topk_w"][:, j:j + 1] * s["y_perm"][row[:, j].clamp(min=0)].float(), 0.0)
        out["y"] = y.to(dt)
    elif c["branch"]:
        y = s["y"].float()
    if y is not None:
        v = y if s["post"] is None else y * _rate(y, s["eps"]) * s["post"].float()
        r = s["res_scale"] * r + s["branch_scale"] * _gate(s) * (_plain_keep(s) * v)
        out["resid"] = r.to(dt)
    out["norm"] = (r * _rate(r, s["eps"]) * s["pre"].float()).to(dt)
    return out


def _plain_gradient(s):
    c, dt = s["case"], s["resid"].dtype
    x, dn, gain = s["resid"].float(), s["dnorm_out"].float(), s["pre"].float()
    rate = _rate(x, s["eps"])
    g = dn * gain
    dx = s["dresid_out"].float() + rate * (g - x * rate * rate * (g * x).mean(1, keepdim=True))
    out = dict.fromkeys(BACKWARD_KEYS)
    out["dpre_gain"] = (dn * x * rate).sum(0)
    if not c["branch"]:
        return out | dict(dresid=dx.to(dt))
    out["dresid"] = (s["res_scale"] * dx).to(dt)
    y = s["y"].float()
    rate = _rate(y, s["eps"]) if c["post"] else None
    v = y if rate is None else y * rate * s["post"].float()
    keep = _plain_keep(s)
    db = s["branch_scale"] * dx * keep
    if c["gate"] != "none":
        dg = db * v
        out["dgate"] = dg.sum(0) if c["gate"] == "channel" else dg.sum(1) if c["gate"] == "token" else dg.to(dt)
    dv = db * _gate(s)
    if rate is not None:
        out["dpost_gain"] = (dv * y * rate).sum(0)
        g = dv * s["post"].float()
        dv = rate * (g - y * rate * rate * (g * y).mean(1, keepdim=True))
    out["dy"] = dv.to(dt)
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_few(s):
    import routing_grouped_gemm_gb300 as moe
    if "own" not in s:
        c = s["case"]
        cfg = moe.Config(T=c["T"], D=c["D"], H_local=c["H"], E=c["E"], k=c["k"], e_first=c["e_first"],
                         E_local=c["E_local"], dtype=moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_F32,
                         score=moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                         renorm=c["renorm"], n_group=c["n_group"], topk_group=c["topk_group"])
        s["own"] = cfg, moe.alloc_workspace(cfg, few=True), torch.empty_like(s["x"])
    cfg, ws, out = s["own"]
    moe.moe_layer_forward_few(cfg, s["x"], s["wg"], s["bias"], s["w1"], s["w3"], s["w2"], out, ws)
    return out


def _own_residual_config(s):
    import routing_grouped_gemm_gb300 as moe
    c = s["case"]
    gate = dict(none=moe.MOE_GATE_NONE, channel=moe.MOE_GATE_CHANNEL, token=moe.MOE_GATE_TOKEN,
                element=moe.MOE_GATE_ELEMENT)[c["gate"]]
    return moe, moe.ResidualConfig(T=c["T"], D=c["D"], dtype=moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_F32,
                                   gate=gate, eps=s["eps"], res_scale=s["res_scale"],
                                   branch_scale=s["branch_scale"], p_drop=c["p_drop"])


def _own_norm(s):
    c = s["case"]
    if "own" not in s:
        moe, rc = _own_residual_config(s)
        cfg = ws = y = None
        if c["kind"] == "combine":
            cfg = moe.Config(T=c["T"], D=c["D"], H_local=64, E=c["E"], k=c["k"], e_first=c["e_first"],
                             E_local=c["E_local"], dtype=rc.dtype, align_m=c["align_m"])
            ws, y = moe.alloc_workspace(cfg), torch.empty_like(s["resid"])
        has = c["kind"] == "combine" or c["branch"]
        s["own"] = moe, rc, cfg, ws, y, torch.empty_like(s["resid"]) if has else None, torch.empty_like(s["resid"])
    moe, rc, cfg, ws, y, r, n = s["own"]
    if c["kind"] == "combine":
        moe.moe_combine_residual_norm(cfg, rc, s["y_perm"], s["row_of"], s["topk_w"], s["resid"], s["post"],
                                      s["gate"], s["pre"], s["rng"], y, r, n, ws)
        return dict(y=y, resid=r, norm=n)
    moe.moe_residual_norm(rc, s["resid"], s["y"], s["post"], s["gate"], s["pre"], s["rng"], r, n)
    return dict(resid=r, norm=n) if r is not None else dict(norm=n)


def _own_gradient(s):
    if "own" not in s:
        moe, rc = _own_residual_config(s)
        c, new = s["case"], lambda *n: torch.empty(n, device="cuda")
        b = dict(dresid=torch.empty_like(s["resid"]), dy=torch.empty_like(s["y"]) if c["branch"] else None,
                 dpost_gain=new(c["D"]) if c["post"] else None, dgate=None, dpre_gain=new(c["D"]))
        if c["gate"] != "none":
            b["dgate"] = torch.empty_like(s["gate"], dtype=_dtype(c) if c["gate"] == "element" else torch.float32)
        s["own"] = moe, rc, b, moe.alloc_residual_workspace(rc)
    moe, rc, b, ws = s["own"]
    moe.moe_residual_norm_backward(rc, s["resid"], s["y"], s["post"], s["gate"], s["pre"], s["rng"], s["dresid_out"],
                                   s["dnorm_out"], b["dresid"], b["dy"], b["dpost_gain"], b["dgate"], b["dpre_gain"],
                                   ws)
    return b


def run(state):
    kind = state["case"]["kind"]
    if kind == "few":
        return (_own_few if own else _plain_few)(state)
    if kind == "gradient":
        return (_own_gradient if own else _plain_gradient)(state)
    return (_own_norm if own else _plain_norm)(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    T, D, b = c["T"], c["D"], 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "few":
        H, E = c["H"], c["E"]
        touched = c["E_local"] * (1 - (1 - c["k"] / E) ** T)  # experts with a token, evenly loaded
        return dict(bytes=touched * 3 * D * H * b + E * D * b + 2 * T * D * b,
                    flops=6 * T * c["k"] * c["E_local"] / E * D * H + 2 * T * E * D)
    gate = dict(none=0, channel=D * b, token=4 * T, element=T * D * b)[c["gate"]]
    gains = D * b * (1 + c["post"])
    if c["kind"] == "combine":
        slots = T * c["k"] * c["E_local"] / c["E"]
        # the experts' rows and the residual in; the branch, the sum and its norm out
        return dict(bytes=slots * D * b + 8 * T * c["k"] + 4 * T * D * b + gate + gains, flops=2 * slots * D)
    if c["kind"] == "norm":
        return dict(bytes=T * D * b * (4 if c["branch"] else 2) + gate + gains, flops=0)
    # the sum, the branch and two gradients in; two gradients out
    dgate = dict(none=0, channel=4 * D, token=4 * T, element=T * D * b)[c["gate"]]
    return dict(bytes=T * D * b * (6 if c["branch"] else 4) + gate + dgate + gains + 4 * D * (1 + c["post"]), flops=0)


def _exact_few(s):
    c = s["case"]
    x = s["x"].double().cpu()
    key = x @ s["wg"].double().cpu().T
    if s["bias"] is not None:
        key = key + s["bias"].double().cpu()
    if c["score"] == "sigmoid":
        p = torch.sigmoid(key)
    else:
        p = torch.softmax(key, dim=1)
    chosen, k = [], c["k"]
    for t in range(c["T"]):
        row = key[t].tolist()
        among = range(c["E"])
        if c["n_group"] > 1:
            n, m = c["E"] // c["n_group"], k // c["topk_group"]
            score = [sum(sorted(row[q * n:q * n + n], reverse=True)[:m]) for q in range(c["n_group"])]
            best = sorted(range(c["n_group"]), key=lambda q: (-score[q], q))[:c["topk_group"]]
            among = [e for e in among if e // n in best]
        chosen.append(sorted(among, key=lambda e: (-row[e], e))[:k])
    out = torch.zeros((c["T"], c["D"]), dtype=torch.float64, device="cuda")
    for e in range(c["e_first"], c["e_first"] + c["E_local"]):
        ts = [t for t in range(c["T"]) if e in chosen[t]]
        if not ts:
            continue
        i = e - c["e_first"]
        w = [p[t, e] / (sum(p[t, q] for q in chosen[t]) if c["renorm"] else 1) for t in ts]
        xe = s["x"][ts].double()
        gate = xe @ s["w1"][i].double().T
        h = gate * torch.sigmoid(gate) * (xe @ s["w3"][i].double().T)
        out[ts] += torch.stack(w).to(out.device).unsqueeze(1) * (h @ s["w2"][i].double().T)
    return out


def _exact_keep(s):
    """The dropout's factors, by 64-bit unsigned products on the host."""
    c = s["case"]
    n = c["T"] * c["D"] // 8
    seed, offset = (int(v) & (1 << 64) - 1 for v in s["rng"].tolist())
    u64, low = numpy.uint64, numpy.uint64(0xffffffff)
    i = numpy.arange(n, dtype=u64)
    ctr = [i & low, i >> u64(32), numpy.full(n, offset & 0xffffffff, u64), numpy.full(n, offset >> 32, u64)]
    key = [seed & 0xffffffff, seed >> 32]
    for _ in range(10):
        a, b = ctr[0] * u64(0xd2511f53), ctr[2] * u64(0xcd9e8d57)
        ctr = [(b >> u64(32)) ^ ctr[1] ^ u64(key[0]), b & low, (a >> u64(32)) ^ ctr[3] ^ u64(key[1]), a & low]
        key = [(key[0] + 0x9e3779b9) % (1 << 32), (key[1] + 0xbb67ae85) % (1 << 32)]
    half = numpy.stack([h for w in ctr for h in (w & u64(0xffff), w >> u64(16))], axis=1)
    cut = round(c["p_drop"] * 65536)
    keep = torch.from_numpy((half >= u64(cut)).reshape(c["T"], c["D"])).cuda()
    return keep.double() * 65536 / (65536 - cut)


def _exact_norm_of(x, gain, eps):
    return x / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + eps) * gain


def _exact_branch(s, y, post, gate):
    """What a branch adds to the residual."""
    c = s["case"]
    if post is not None:
        y = _exact_norm_of(y, post, s["eps"])
    if c["p_drop"]:
        y = y * _exact_keep(s)
    if gate is not None:
        y = y * (gate[:, None] if c["gate"] == "token" else gate)
    return s["branch_scale"] * y


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == "few":
        return _exact_few(s)
    wide = {n: None if s[n] is None else s[n].double() for n in ("resid", "y", "post", "gate", "pre")}
    r, y, post, gate, pre = wide.values()
    if c["kind"] != "gradient":
        out = {}
        if c["kind"] == "combine":
            y = torch.zeros_like(r)
            for j in range(c["k"]):
                t = torch.nonzero(s["row_of"][:, j] >= 0).squeeze(1)
                y[t] += s["topk_w"][t, j].double()[:, None] * s["y_perm"][s["row_of"][t, j].long()].double()
            out["y"] = y
        if y is not None:
            r = s["res_scale"] * r + _exact_branch(s, y, post, gate)
            out["resid"] = r
        out["norm"] = _exact_norm_of(r, pre, s["eps"])
        return out
    # by differentiation: the norm behind the sum, then the branch under the sum's gradient
    leaf = [v.requires_grad_() for v in (r, pre)]
    dr, dpre = torch.autograd.grad(_exact_norm_of(r, pre, s["eps"]), leaf, s["dnorm_out"].double())
    ds = s["dresid_out"].double() + dr
    out = dict.fromkeys(BACKWARD_KEYS)
    out["dpre_gain"] = dpre
    if y is None:
        return out | dict(dresid=ds)
    out["dresid"] = s["res_scale"] * ds
    leaf = {n: v.requires_grad_() for n, v in (("dy", y), ("dpost_gain", post), ("dgate", gate)) if v is not None}
    grad = torch.autograd.grad(_exact_branch(s, y, post, gate), list(leaf.values()), ds)
    return out | dict(zip(leaf, grad))
