"""moe_layer_forward_few where an expert's values leave the ordinary range."""
import pytest
import torch

from test_gpu_few import _call, _inputs, _keys, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [1, 0], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 4, 9])
def test_infinite_weights_of_the_second_product(moe, T, dtype):
    """An infinity in w2 makes its element of out infinite, with the sign of its hidden unit, for the tokens of that
    expert and no others (h of a bf16 layer is a sum of two: the second's product must not turn it into NaN)."""
    c = moe.Config(T=T, D=264, H_local=136, E=4, k=1, dtype=dtype)
    t = _inputs(moe, c, hot=2 if T < 9 else None)
    t["w2"][:] = t["w2"].abs()  # no other term of an infinite sum is infinite
    want, _ = _call(moe, c, t)
    at, unit = [3, 17, 200], [5, 130, 66]
    t["w2"][2, at, unit] = float("inf")
    got, _ = _call(moe, c, t)
    here = (_keys(t).argmax(1) == 2).cuda()
    assert here.any()
    x = t["x"].double()
    h = torch.nn.functional.silu(x @ t["w1"][2].double().T) * (x @ t["w3"][2].double().T)
    same = torch.ones_like(got, dtype=torch.bool)
    for d, u in zip(at, unit):
        assert (got[here, d].double() == h[here, u].sign() * float("inf")).all()
        same[here, d] = False
    assert torch.equal(got[same], want[same])


def test_h_next_to_the_largest_bf16(moe):
    """h = 3.2e38 (bf16 ends at 3.39e38) keeps its second part: unit 0's h takes 16 bits, unit 1's is the bf16 next
    to it, and w2 takes their difference.  Every product here is exact but silu(1.8e19) = 1.8e19."""
    c = moe.Config(T=1, D=8, H_local=8, E=1, k=1)
    z = torch.zeros(1, 8, 8, dtype=torch.bfloat16, device="cuda")
    x = z[0, :1].clone()
    x[0, 0] = 1
    gate = 249 * 2.0 ** 56   # eight bits
    up = 251 * 2.0 ** 56
    h = gate * up            # 62499 2^112 = 3.2e38: sixteen
    first = torch.tensor(h, dtype=torch.float64).to(torch.bfloat16).double().item()
    assert 3.0e38 < first < 3.39e38 and first != h
    # unit 1: 2^63 times first 2^-63
    w1, w3, w2 = z.clone(), z.clone(), z.clone()
    w1[0, 0, 0], w3[0, 0, 0] = gate, up
    w1[0, 1, 0], w3[0, 1, 0] = 2.0 ** 63, first / 2.0 ** 63
    w2[0, 0, 0], w2[0, 0, 1] = 2.0 ** -112, -(2.0 ** -112)
    out, _ = _call(moe, c, dict(x=x, wg=z[0, :1].clone(), bias=None, w1=w1, w3=w3, w2=w2))
    assert out[0, 0].item() == (h - first) * 2.0 ** -112
    assert (out[0, 1:] == 0).all()


def test_one_workspace_for_layers_of_different_width(moe):
    """What one width leaves in the workspace is not taken for another one's counters."""
    cfgs = [moe.Config(T=T, D=D, H_local=H, E=8, k=2, renorm=1, dtype=dt)
            for T, D, H, dt in ((4, 4104, 2048, 1), (9, 264, 2048, 1), (3, 8, 4096, 0), (32, 1048, 1032, 1), (1, 2056, 4104, 1))]
    ws = torch.zeros(max(moe.layer_few_workspace_size(c) for c in cfgs), dtype=torch.uint8, device="cuda")
    t = [_inputs(moe, c) for c in cfgs]
    want = [_call(moe, c, v)[0] for c, v in zip(cfgs, t)]
    for i in (1, 0, 2, 3, 4, 0, 4, 2, 1, 3):
        assert torch.equal(_call(moe, cfgs[i], t[i], ws)[0], want[i]), cfgs[i]
