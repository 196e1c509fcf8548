"""Refusals of bsa_prefix_attn_slots: those of bsa_prefix_attn, and its own (CPU only: nothing is
launched)."""
import pytest

from test_paged_abi import ARG, ATTN, FAKE, OK, SHAPE, UNSUPPORTED, WORKSPACE


def call(lib, slots, num_slots, **kw):
    a = dict(ATTN, **kw)
    at = list(a).index("o")
    values = list(a.values())
    return lib.bsa_prefix_attn_slots(*values[:at], slots, num_slots, *values[at:])


@pytest.mark.parametrize("slots,num_slots,change,code", [
    (FAKE, -1, {}, ARG), (None, -1, {}, ARG), (FAKE, 4, {}, WORKSPACE), (FAKE, 0, {}, WORKSPACE),
    (None, 0, {}, WORKSPACE), (FAKE, 4, dict(q=None), ARG), (FAKE, 4, dict(T=5), SHAPE),
    (FAKE, 4, dict(d=96), UNSUPPORTED), (FAKE, 0, dict(T=0, B=0), OK),
])
def test_prefix_attn_slots_refusals(bsa_lib, slots, num_slots, change, code):
    assert call(bsa_lib, slots, num_slots, **change) == code
