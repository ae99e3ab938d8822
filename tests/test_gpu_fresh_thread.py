"""Calls made first thing on a thread that has made no CUDA call: the same bits as on the main thread."""
import threading

import pytest
import torch

import test_gpu_mxfp4 as mxfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_gb300 as m
    assert torch.cuda.is_available()
    return m


def _on_a_thread(call, *outs):
    """call() here, then on a new thread, on cleared outputs each time; the outputs are compared."""
    for o in outs:
        o.zero_()
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join(60)
    torch.cuda.synchronize()
    assert not errors
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.uint8), w.view(torch.uint8))


def _bf16(moe, seed=2):
    T, D, H, E, k = 300, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16)  # noqa: E731
    cfg = moe.Config(T=T, D=D, H_local=H, E=E, k=k, renorm=1)
    return cfg, r(T, D), r(E, D), r(E, H, D), r(E, H, D), r(E, D, H)


def test_mxfp4_grouped(moe):
    counts = [40, 0, 300, 7]
    cfg, seg, xq, xs, w, out = mxfp4._grouped_case(moe, counts, 256, 96, 16, 4)
    ws = moe.alloc_workspace(cfg)
    seg, tpe = mxfp4._dev(seg), mxfp4._dev(counts)
    _on_a_thread(lambda: moe.moe_grouped_swiglu_mxfp4(cfg, xq, xs, seg, tpe, *w[0], *w[1], *w[2], out["hq"],
                                                      out["hs"], out["y"], ws), *out.values())
    assert moe.moe_get_device_status(ws) == moe.MOE_OK


def test_mxfp4_layer(moe):
    cfg, x, wg, w = mxfp4._layer(moe, 100, 256, 96, 8, 2)
    ws, out = moe.alloc_workspace(cfg, layer=True), torch.empty_like(x)
    _on_a_thread(lambda: moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], out, ws), out)


def test_bf16_layer(moe):
    cfg, x, wg, w1, w3, w2 = _bf16(moe)
    ws, out = moe.alloc_workspace(cfg, layer=True), torch.empty_like(x)
    _on_a_thread(lambda: moe.moe_layer_forward(cfg, x, wg, None, w1, w3, w2, out, ws), out)


def test_captured_on_the_thread(moe):
    cfg, x, wg, w1, w3, w2 = _bf16(moe)
    ws, out = moe.alloc_workspace(cfg, layer=True), torch.empty_like(x)
    moe.moe_layer_forward(cfg, x, wg, None, w1, w3, w2, out, ws)
    want, graph, errors = out.clone(), torch.cuda.CUDAGraph(), []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def work():
        try:
            moe.moe_layer_forward(cfg, x, wg, None, w1, w3, w2, out, ws, stream=side)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    out.zero_()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        t = threading.Thread(target=work)
        t.start()
        t.join(60)
    assert not errors
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
