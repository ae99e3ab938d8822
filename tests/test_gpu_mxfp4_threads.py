"""MXFP4 layers of different sizes called from several threads at once, each on a stream and a
workspace of its own: the bits of the same calls one after another."""
import threading

import pytest
import torch

from test_gpu_mxfp4 import _layer, moe  # noqa: F401

pytestmark = pytest.mark.gpu


def test_layers_from_threads(moe):  # noqa: F811
    cases = [(64, 256, 128, 4, 2), (200, 320, 96, 40, 3), (33, 256, 256, 300, 2), (500, 128, 64, 16, 4)]
    layers = [_layer(moe, *c, seed=i) for i, c in enumerate(cases)]
    wss = [moe.alloc_workspace(cfg, layer=True) for cfg, *_ in layers]

    def call(i, out, stream=None):
        cfg, x, wg, w = layers[i]
        moe.moe_layer_forward_mxfp4(cfg, x, wg, None, *w[0], *w[1], *w[2], out, wss[i], stream=stream)
    want = [torch.empty_like(x) for _, x, *_ in layers]
    for i, o in enumerate(want):
        call(i, o)
        assert moe.moe_get_device_status(wss[i]) == moe.MOE_OK
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[torch.zeros_like(o) for _ in range(20)] for o in want]
    torch.cuda.synchronize()
    errors, go = [], threading.Barrier(len(layers))

    def work(i):
        try:
            go.wait(30)
            for o in outs[i]:
                call(i, o, streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(layers))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not errors
    for i, o in enumerate(want):
        assert moe.moe_get_device_status(wss[i]) == moe.MOE_OK
        assert all(torch.equal(o, got) for got in outs[i])
