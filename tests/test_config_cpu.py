"""Config keeps the C struct of its values: never that of values it had before."""
import copy
import dataclasses
import pickle

import pytest


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import routing_grouped_gemm_gb300 as m
    return m


def _holds(moe, cfg, T):
    p, rows = cfg.ref()
    return p.contents.T == T and rows == T * 2 + 8 * 127 and moe.rows_alloc(cfg) == rows


def _cfg(moe, T):
    return moe.Config(T=T, D=64, H_local=64, E=8, k=2)


def test_kept_until_a_value_changes(moe):
    cfg = _cfg(moe, 10)
    first = cfg.ref()
    assert cfg.ref() is first and _holds(moe, cfg, 10)
    cfg.T = 33
    assert _holds(moe, cfg, 33)
    assert first[0].contents.T == 10             # who holds the old one keeps the old values


def test_a_value_set_while_the_struct_is_built(moe, monkeypatch):
    """As from another thread, between the reading of the values and the keeping of the struct."""
    cfg = _cfg(moe, 10)
    real = moe.Config.c

    def c(self):
        out = real(self)
        monkeypatch.setattr(moe.Config, "c", real)
        self.T = 20
        return out
    monkeypatch.setattr(moe.Config, "c", c)
    assert cfg.ref()[0].contents.T == 10         # that call began before
    assert _holds(moe, cfg, 20)


def test_copies_have_their_own(moe):
    cfg = _cfg(moe, 10)
    cfg.ref()
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), dataclasses.replace(cfg)):
        assert other == cfg and _holds(moe, other, 10)
        other.T = 11
        assert _holds(moe, other, 11) and _holds(moe, cfg, 10)
