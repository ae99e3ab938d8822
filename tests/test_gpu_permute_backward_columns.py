"""moe_permute_backward where a warp takes several runs of a row's columns.

From 487 tokens on a row is split over four warps, 512 bytes each at a time: rows of more than
2048 bytes (of dx) make each warp go round, here four or five times and with a ragged end; k = 12
has more rows than stay in registers over the columns.  Bound as in test_gpu_sort_grad.py."""
import numpy as np
import pytest
import torch

from test_gpu_sort_grad import _case, _f64, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16,D", [(True, 4104), (False, 2056)])
@pytest.mark.parametrize("k,kw", [(3, {}), (12, dict(align_m=1)), (5, dict(e_first=4, E_local=9))])
def test_rows_of_several_column_runs(moe, bf16, D, k, kw):  # noqa: F811
    T, E = 1301, 16
    cfg, ws, row_of, _, _, _, dxp = _case(moe, T, D, E, k, bf16, **kw)
    ro = row_of.cpu().numpy()
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    for dt in ([torch.float32, torch.bfloat16] if bf16 else [torch.float32]):
        p = dxp.to(dt)
        dx = torch.full((T, D), 77.0, dtype=cfg.torch_dtype, device="cuda")
        moe.moe_permute_backward(cfg, p, row_of, dx, ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_OK
        pv, ref, m = _f64(p), np.zeros((T, D)), np.zeros((T, D))
        for j in range(k):
            t = np.nonzero(ro[:, j] >= 0)[0]
            ref[t] += pv[ro[t, j]]
            m[t] += np.abs(pv[ro[t, j]])
        assert (np.abs(_f64(dx) - ref) <= half * np.abs(ref) + (k + 1) * 2.0 ** -24 * m).all()
