"""The package's names are the binding's, also after one is replaced there."""
import importlib

import pytest

pkg = pytest.importorskip("combine_moe_route_amd")
binding = pytest.importorskip("combine_moe_route_amd.binding")


def test_every_name_is_the_bindings():
    for name in pkg._API:
        assert getattr(pkg, name) is getattr(binding, name), name
        assert getattr(pkg, name) is getattr(binding, name), name
    with pytest.raises(AttributeError):
        pkg.no_such_name


def test_a_replacement_is_seen_and_taken_back(monkeypatch):
    real = pkg.moe_combine                           # looked up before
    with monkeypatch.context() as m:
        m.setattr(binding, "moe_combine", len)
        assert pkg.moe_combine is len                # and kept while it stands
        assert pkg.moe_combine is len
    assert pkg.moe_combine is real and binding.moe_combine is real


def test_first_looked_up_while_replaced(monkeypatch):
    real = binding.status_string
    vars(pkg).pop("status_string", None)
    with monkeypatch.context() as m:
        m.setattr(binding, "status_string", len)
        assert pkg.status_string is len
    assert pkg.status_string is real


def test_a_removed_name_is_missed(monkeypatch):
    assert pkg.moe_combine_recv is binding.moe_combine_recv
    with monkeypatch.context() as m:
        m.delattr(binding, "moe_combine_recv")
        with pytest.raises(AttributeError):
            pkg.moe_combine_recv
    assert pkg.moe_combine_recv is binding.moe_combine_recv


def test_the_packages_own_replacement_stands(monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(pkg, "moe_combine", len)
        m.setattr(binding, "moe_combine", max)
        assert pkg.moe_combine is len
    assert pkg.moe_combine is binding.moe_combine


def test_loading_the_binding_again():
    held = dict(vars(binding))
    try:
        old = pkg.moe_dispatch
        importlib.reload(binding)
        assert binding.moe_dispatch is not old
        assert pkg.moe_dispatch is binding.moe_dispatch
        assert pkg.MoeRouteError is binding.MoeRouteError
    finally:                                         # other tests hold the first classes
        pkg._forget(pkg._API, vars(binding))
        vars(binding).update(held)
    assert pkg.moe_dispatch is old
