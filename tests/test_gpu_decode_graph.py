"""Decode steps captured into a graph: norm, layer for a few tokens and norm, block after block on one workspace."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,H,E,k", [(1, 512, 256, 16, 4), (5, 1048, 424, 20, 3), (32, 256, 2048, 8, 2)])
@pytest.mark.parametrize("dtype", [1, 0], ids=["bf16", "f32"])
def test_blocks_in_one_graph(T, D, H, E, k, dtype):
    import routing_grouped_gemm_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(T)
    c = moe.Config(T=T, D=D, H_local=H, E=E, k=k, renorm=1, dtype=dtype)
    dt = c.torch_dtype

    def n(*s, scale=1.0):
        return (scale * torch.randn(s, generator=g, device="cuda")).to(dt)
    blocks = [dict(wg=n(E, D, scale=D ** -0.5), w1=n(E, H, D, scale=D ** -0.5), w3=n(E, H, D, scale=D ** -0.5),
                   w2=n(E, D, H, scale=H ** -0.5), post=1 + n(D, scale=0.1), pre=1 + n(D, scale=0.1), gate=n(D))
              for _ in range(3)]
    rc0 = moe.ResidualConfig(T=T, D=D, dtype=dtype)
    rc = moe.ResidualConfig(T=T, D=D, dtype=dtype, gate=moe.MOE_GATE_CHANNEL, branch_scale=0.5, p_drop=0.1)
    resid, x, y = (torch.zeros(T, D, dtype=dt, device="cuda") for _ in range(3))
    rng = torch.tensor([3, 0], device="cuda")
    ws = moe.alloc_workspace(c, few=True)

    def step():
        moe.moe_residual_norm(rc0, resid, None, None, None, blocks[0]["pre"], None, None, x)
        for i, b in enumerate(blocks):
            moe.moe_layer_forward_few(c, x, b["wg"], None, b["w1"], b["w3"], b["w2"], y, ws)
            moe.moe_residual_norm(rc, resid, y, b["post"], b["gate"], blocks[(i + 1) % 3]["pre"], rng, resid, x)
    stream = torch.cuda.Stream()
    starts = [n(T, D, scale=2.0) for _ in range(4)]
    want = []
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for i, s in enumerate(starts):
            resid.copy_(s)
            rng[1] = i
            step()
            want.append((resid.clone(), x.clone()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for i in (2, 0, 3, 1, 2):
            resid.copy_(starts[i])
            rng[1] = i
            graph.replay()
            stream.synchronize()
            assert torch.equal(resid, want[i][0]) and torch.equal(x, want[i][1])
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    assert all(v.isfinite().all() for w in want for v in w)
