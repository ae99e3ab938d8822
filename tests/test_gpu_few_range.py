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
