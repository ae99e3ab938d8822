"""Weights quantised on a side stream: the results are that stream's memory, not a block that the
current stream has freed and still works on."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _owner(t):
    """Stream that the allocator keeps t's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


@pytest.mark.parametrize("name", ["quantize_weights_mxfp4", "quantize_weights_fp8"])
def test_results_belong_to_the_stream(moe, name):
    quantize = getattr(moe, name)
    w = torch.randn((4, 96, 256), device="cuda").to(torch.bfloat16)
    want = quantize(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = quantize(w, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
        assert _owner(a) == side.cuda_stream
        assert _owner(b) == torch.cuda.current_stream().cuda_stream
