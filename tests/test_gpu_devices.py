"""A call whose workspace or rows are not on the current device is refused before any launch: its
kernels would run on a device that does not hold them.  (The current device is made to look like
another one; there need be only one.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _calls(moe, ws):
    T, D, H, E, k = 4, 64, 64, 8, 2
    cfg = moe.Config(T=T, D=D, H_local=H, E=E, k=k)
    ra = moe.rows_alloc(cfg)

    def z(dtype, *s):
        return torch.zeros(s, dtype=dtype, device="cuda")
    u8, i32, bf, f32, f16 = torch.uint8, torch.int32, torch.bfloat16, torch.float32, torch.float16
    w = [z(u8, E, H, D // 2), z(u8, E, H, D // 32)] * 2 + [z(u8, E, D, H // 2), z(u8, E, D, H // 32)]
    idx, tpe, seg, row, tor = z(i32, T, k), z(i32, E), z(i32, E + 1), z(i32, T, k), z(i32, ra)
    xq, xs, hq, hs = z(u8, ra, D // 2), z(u8, ra, D // 32), z(u8, ra, H // 2), z(u8, ra, H // 32)
    x, wg, y, tw = z(bf, T, D), z(bf, E, D), z(f16, ra, D), z(f32, T, k)
    return {
        "permute": lambda: moe.moe_permute_mxfp4(cfg, x, idx, tpe, seg, row, tor, xq, xs, ws),
        "grouped": lambda: moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, seg, tpe, *w, hq, hs, y, ws),
        "layer": lambda: moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w, x, ws),
        "combine backward": lambda: moe.moe_unpermute_combine_backward(cfg, x, y, row, tw, z(bf, ra, D), tw, ws),
        "permute backward": lambda: moe.moe_permute_backward(cfg, z(bf, ra, D), row, x, ws),
        "rows": lambda: moe.moe_quantize_rows_mxfp4(x, z(u8, T, D // 2), z(u8, T, D // 32)),
        "rows back": lambda: moe.moe_dequantize_rows_mxfp4(z(u8, T, D // 2), z(u8, T, D // 32), x),
    }


def test_another_device(moe, monkeypatch):
    n = moe.workspace_size(moe.Config(T=4, D=64, H_local=64, E=8, k=2))
    calls = _calls(moe, torch.zeros(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    before, real = moe.kernel_launches(), torch.cuda.current_device()
    monkeypatch.setattr(moe, "_device", lambda: real + 1)
    for name, call in calls.items():
        with pytest.raises(ValueError, match="current device"):
            call()
    assert moe.kernel_launches() == before


def test_workspace_on_the_host_or_missing(moe):
    n = moe.layer_workspace_size(moe.Config(T=4, D=64, H_local=64, E=8, k=2))
    before = moe.kernel_launches()
    for ws, match in ((torch.zeros(n, dtype=torch.uint8), "ws is on cpu"), (None, "ws is required")):
        for name, call in _calls(moe, ws).items():
            if not name.startswith("rows"):
                with pytest.raises(ValueError, match=match):
                    call()
    assert moe.kernel_launches() == before
