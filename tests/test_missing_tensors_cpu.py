"""A tensor that is not given is named in a ValueError, as by every other call."""
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import routing_grouped_gemm_gb300 as m
    return m


def test_missing_tensors(moe):
    cfg = moe.Config(T=4, D=64, H_local=64, E=8, k=2)
    ws = torch.zeros(moe.workspace_size(cfg), dtype=torch.uint8)
    with pytest.raises(ValueError, match="src is required"):
        moe.moe_quantize_rows_mxfp4(None, None, None)
    with pytest.raises(ValueError, match="dst is required"):
        moe.moe_dequantize_rows_mxfp4(None, None, None)
    with pytest.raises(ValueError, match="w is required"):
        moe.quantize_weights_mxfp4(None)
    with pytest.raises(ValueError, match="rows of a multiple of 32|CUDA tensor"):
        moe.quantize_weights_mxfp4(torch.zeros(()))
    with pytest.raises(ValueError, match="dx_perm is required"):
        moe.moe_permute_backward(cfg, None, None, None, ws)
    with pytest.raises(ValueError, match="dout is required"):
        moe.moe_unpermute_combine_backward(cfg, None, None, None, None, None, None, ws)
    with pytest.raises(ValueError, match="x is required"):
        moe.moe_permute_mxfp4(cfg, None, None, None, None, None, None, None, None, ws)
