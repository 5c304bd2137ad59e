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


@pytest.mark.parametrize("call,names", [
    (_linear, ["status"]),
    (_prefill, ["ld", "cu", "status"]),
    (_decode, ["ld", "slots", "status"]),
    (_append, ["table", "start", "cu", "status"]),
    (_attend, ["table", "lens", "lse", "status"]),
])
def test_four_byte_values_off_their_alignment(call, names):
    """Their loads, and the status word's atomic, would be misaligned addresses on the device."""
    for name in names:
        for off in (1, 2, 3):
            assert call(**{name: A + off}) == INV, (name, off)
