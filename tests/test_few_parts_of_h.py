"""moe_layer_forward_few keeps h of a bf16 layer to 16 significant bits, as the sum of two bf16.

The rows of x are short here, so that the first product's fp32 sums add next to nothing, and h's own rounding is what
the bound leaves room for: 2^-16 of each h (half a step of bf16, 2^-8, of the rest that the first bf16 left, itself at
most 2^-8 of h).  out's rounding, 2^-8 of the value, hides an h in one bf16 wherever out is not small against its
terms; some of the elements always are, and that they give it away is checked on the host.
"""
import pytest
import torch

U = 2.0 ** -24

# tokens, experts, choices: entries of one to four pairs, whole and not, in rings for 1, 2, 3 and 4 rows of an entry
CASES = [(1, 4, 2), (2, 1, 1), (2, 5, 3), (3, 1, 1), (3, 3, 2), (4, 1, 1), (5, 1, 1), (7, 2, 1), (9, 3, 2), (13, 8, 5), (32, 2, 1)]
SHAPES = [(8, 264), (24, 1048), (64, 136)]


def _case(T, E, k, D, H):
    g = torch.Generator().manual_seed(100 * T + E + D)
    x, wg, w1, w3, w2 = (torch.randn(*s, generator=g) * f for s, f in (
        ((T, D), 1.0), ((E, D), 0.0), ((E, H, D), D ** -0.5), ((E, H, D), D ** -0.5), ((E, D, H), H ** -0.5)))
    bias = torch.arange(E, 0, -1).float()  # every key is its expert's bias: no near ties
    return dict(x=x.bfloat16(), wg=wg.bfloat16(), bias=bias, w1=w1.bfloat16(), w3=w3.bfloat16(), w2=w2.bfloat16())


def _layer(t, k, one_bf16=False):
    """(out in 64 bits, what the kernel's roundings may add to it before its own), experts 0 .. k - 1 for every
    token with the softmax of their biases."""
    D, H = t["x"].shape[1], t["w1"].shape[1]
    w = torch.softmax(t["bias"].double(), 0)
    x = t["x"].double()
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(k):
        w1, w3, w2 = (t[n][e].double() for n in ("w1", "w3", "w2"))
        gate, up = x @ w1.T, x @ w3.T
        silu = gate * torch.sigmoid(gate)
        h = silu * up
        # fp32 sums of D products; silu' <= 1.1; 16 U for exp, division and the product
        dg, du = (D + 8) * U * (x.abs() @ w1.abs().T), (D + 8) * U * (x.abs() @ w3.abs().T)
        dh = 1.1 * dg * (up.abs() + du) + silu.abs() * du + (16 * U + 2.0 ** -16) * h.abs()
        if one_bf16:
            h = h.bfloat16().double()
        out += w[e] * (h @ w2.T)
        # the second product's sum, the weights (exp, division) and the sum over experts
        tol += w[e] * (dh @ w2.abs().T + (H + k + 64) * U * (h.abs() @ w2.abs().T))
    return out, tol


def _worst(out, want, tol):
    return ((out.double() - want).abs() / (tol + 2.0 ** -8 * (want.abs() + tol))).max().item()


# elements of out enough for some to be small
@pytest.mark.parametrize("T,E,k,D,H", [c + s for c in CASES for s in SHAPES if c[0] * s[0] >= 64])
def test_one_bf16_would_show(T, E, k, D, H):
    t = _case(T, E, k, D, H)
    want, tol = _layer(t, k)
    assert _worst(want.bfloat16(), want, tol) <= 1.0
    assert _worst(_layer(t, k, one_bf16=True)[0].bfloat16(), want, tol) > 1.5


@pytest.mark.gpu
@pytest.mark.parametrize("D,H", SHAPES)
@pytest.mark.parametrize("T,E,k", CASES)
def test_two_parts_of_h(T, E, k, D, H):
    import routing_grouped_gemm_gb300 as moe
    t = _case(T, E, k, D, H)
    c = moe.Config(T=T, D=D, H_local=H, E=E, k=k)
    ws, out = moe.alloc_workspace(c, few=True), torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_forward_few(c, *(t[n].cuda() for n in ("x", "wg", "bias", "w1", "w3", "w2")), out, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    want, tol = _layer(t, k)
    worst = _worst(out.cpu(), want, tol)
    assert worst <= 1.0, f"{worst} of the bound"
