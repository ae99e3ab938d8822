"""dx of the layer's backward where rows end inside a warp's columns and where they do not.

The dispatch's backward takes 128 columns of a row at a time: D = 256 is whole, 64, 192 and
320 leave half of a warp without columns.  k = 20 is more than the lanes that are left.  With renormalised weights the router's part of dx
is formed from wg in the kernel, without it is read.  Measure and bound as in
test_gpu_backward.py."""
import numpy as np
import pytest

from test_gpu_backward import GRAD_TOL, _errs, _f64, _oracle, _run, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("D", [64, 192, 256, 320])
def test_dx_of_ragged_and_whole_rows(moe, D, renorm):  # noqa: F811
    k = 20
    cfg, ws, _, grads, inputs = _run(moe, 70, D, 64, 24, k, "softmax", renorm, seed=D)
    ref = _oracle(inputs, k, "softmax", renorm)
    assert np.array_equal(moe.layer_views(cfg, ws)["topk_idx"].cpu().numpy(), ref["topk_idx"])
    rms, mx = _errs(_f64(grads["dx"]), ref["dx"])
    assert rms < GRAD_TOL and mx < GRAD_TOL, f"rms ratio {rms:.2e}, max ratio {mx:.2e}"
    tail = _errs(_f64(grads["dx"])[:, -64:], ref["dx"][:, -64:])   # the last lanes' columns by themselves
    assert tail[0] < GRAD_TOL
