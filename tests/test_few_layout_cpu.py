"""moe_layer_forward_few lays nothing out: the config's layout, align_m and capacity play no part (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import routing_grouped_gemm_gb300 as m
    return m


@pytest.mark.parametrize("kw", [dict(align_m=0), dict(align_m=1 << 20), dict(align_m=-5), dict(layout=1, capacity=-1),
                                dict(layout=1, capacity=2 ** 31 - 1), dict(layout=9)])
def test_any_layout_is_taken(moe, kw):
    base = dict(T=0, D=64, H_local=64, E=8, k=2)
    assert moe._lib.moe_layer_forward_few(moe.Config(**base, **kw).ref()[0], *[None] * 7, 256, 1 << 30, None) == moe.MOE_OK
    base["T"] = 32
    assert moe.layer_few_workspace_size(moe.Config(**base, **kw)) == moe.layer_few_workspace_size(moe.Config(**base))


def test_other_fields_are_still_checked(moe):
    for kw in (dict(T=-1), dict(D=12), dict(k=9), dict(E_local=9), dict(dtype=5), dict(n_group=3)):
        c = moe.Config(**(dict(T=4, D=64, H_local=64, E=8, k=2) | kw))
        assert moe.layer_few_workspace_size(c) == -1
    assert moe._lib.moe_layer_few_workspace_size(None) == -1
    assert moe._lib.moe_layer_forward_few(None, *[None] * 7, 256, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG
