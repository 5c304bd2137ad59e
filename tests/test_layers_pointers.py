"""Pointers that a kernel would read, refused on the host where they are missing or off
their type's alignment (include/kda_layers.h); no GPU."""
import pytest

from gated_delta_rule_46_gb300 import kda
from test_layers_abi import A, _append, _attend, _decode, _linear, _prefill

INV = kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(table=None, P=0), dict(table=None, P=0, kc=None, vc=None)])
def test_a_table_is_read_even_if_the_cache_has_no_pages(kw):
    """Ids are looked up before they are compared with the number of pages."""
    assert _attend(**kw) == INV
