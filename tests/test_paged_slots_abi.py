"""Refusals of bsa_prefix_attn_slots: those of bsa_prefix_attn, and its own (CPU only: nothing is
launched)."""
import pytest
import torch

import block_sparse_attention_summaries_b200 as bsa
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


def test_workspace_of_a_type_that_is_not_attended(bsa_lib):
    """The query refuses the types that the call refuses."""
    sizes = (4, 4, 8, 2, 128, 64, 8, 100)
    assert bsa.prefix_attn_workspace_bytes(torch.bfloat16, *sizes) > 0
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError):
            bsa.prefix_attn_workspace_bytes(dtype, *sizes)
