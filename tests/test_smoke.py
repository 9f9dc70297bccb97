"""The entry point's own smoke check (one small forward and backward on
cuda:0, compared with the oracle) runs as a GPU test too."""
import pytest

pytestmark = pytest.mark.gpu


def test_graft_entry_smoke():
    import __graft_entry__
    __graft_entry__.smoke()


def test_smoke_takes_the_operators_around_the_norm(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    called = []
    for name in ("cake_sandwich_fwd", "cake_sandwich_bwd", "cake_clip_grad_norm", "cake_embedding_fwd",
                 "cake_embedding_bwd"):
        def call(*a, _name=name, _f=getattr(cake, name), **kw):
            called.append(_name)
            return _f(*a, **kw)
        monkeypatch.setattr(cake, name, call)
    __graft_entry__.smoke()
    assert len(set(called)) == 5
