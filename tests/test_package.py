"""The package's names are those of its binding, at every access."""
import pytest

import top_kv_routing_b200 as msa
from top_kv_routing_b200 import abi


@pytest.mark.parametrize("name", ["msa_paged_append", "msa_sparse_decode", "MSA_OK", "loaded_libraries"])
def test_what_is_replaced_in_the_binding_is_replaced_in_the_package(name, monkeypatch):
    before = getattr(abi, name)
    assert getattr(msa, name) is before  # (used once)
    other = object()
    monkeypatch.setattr(abi, name, other)
    assert getattr(msa, name) is other
    monkeypatch.undo()
    assert getattr(msa, name) is before


def test_names_that_the_binding_lacks():
    with pytest.raises(AttributeError):
        msa.msa_no_such_call
