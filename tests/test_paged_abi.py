"""Refusals of the paged serving calls: host-side argument checks of bsa_page_tables,
bsa_paged_append and bsa_prefix_attn, and of their binding (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch

import block_sparse_attention_summaries_b200 as bsa

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call fails validation or has no work
ODD = ctypes.c_void_p(0x1002)
OK, ARG, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 7


def with_(base, **kw):
    a = dict(base, **kw)
    return list(a.values())


TABLES = dict(B=4, page=64, lens=FAKE, new_lens=FAKE, table=FAKE, ld=16, ring=FAKE, num_pages=64,
              free_in=FAKE, lens_out=FAKE, free_out=FAKE, cu_new=FAKE, slots=FAKE, positions=None,
              max_tokens=64, pos_offset=0, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), ARG), (dict(page=0), ARG), (dict(max_tokens=-1), ARG), (dict(ld=-1), ARG),
    (dict(num_pages=0), ARG), (dict(lens=None), ARG), (dict(new_lens=None), ARG),
    (dict(table=None), ARG), (dict(ring=None), ARG), (dict(free_in=None), ARG),
    (dict(lens_out=None), ARG), (dict(free_out=None), ARG), (dict(cu_new=None), ARG),
    (dict(slots=None), ARG), (dict(pos_offset=-1), ARG), (dict(pos_offset=2**31 - 64), ARG),
    (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(B=8193), UNSUPPORTED), (dict(num_pages=2**25), UNSUPPORTED),
    (dict(ld=2**25), UNSUPPORTED), (dict(max_tokens=2**31 - 1), UNSUPPORTED),
])
def test_page_tables_refusals(bsa_lib, change, code):
    assert bsa_lib.bsa_page_tables(*with_(TABLES, **change)) == code


APPEND = dict(k=FAKE, v=FAKE, dt=1, T=8, Hk=2, d=128, ks=256, vs=256, slots=FAKE, page=64,
              num_pages=16, kp=FAKE, vp=FAKE, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(kp=None), ARG),
    (dict(vp=None), ARG), (dict(T=-1), ARG), (dict(Hk=0), ARG), (dict(num_pages=0), ARG),
    (dict(kp=ODD), ARG), (dict(k=ctypes.c_void_p(0x1001)), ARG), (dict(dt=2), DTYPE),
    (dict(ks=255), SHAPE), (dict(vs=0), SHAPE), (dict(d=96), UNSUPPORTED),
    (dict(page=100), UNSUPPORTED), (dict(num_pages=2**25), UNSUPPORTED), (dict(T=0), OK),
])
def test_paged_append_refusals(bsa_lib, change, code):
    assert bsa_lib.bsa_paged_append(*with_(APPEND, **change)) == code


ATTN = dict(q=FAKE, q_stride=1024, k=FAKE, v=FAKE, dt=1, T=4, B=4, Hq=8, Hk=2, d=128, page=64,
            num_pages=64, table=FAKE, ld=8, lens=FAKE, ptable=FAKE, prefix=100, cu_q=None, max_q=1,
            o=FAKE, lse=None, status=None, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(o=None), ARG),
    (dict(lens=None), ARG), (dict(table=None), ARG), (dict(ptable=None), ARG),
    (dict(T=-1), ARG), (dict(B=-1), ARG), (dict(prefix=-1), ARG), (dict(max_q=0), ARG),
    (dict(num_pages=0), ARG), (dict(q=ODD), ARG), (dict(k=ODD), ARG), (dict(o=ODD), ARG),
    (dict(q_stride=1025), ARG), (dict(dt=3), DTYPE), (dict(Hq=7), SHAPE),
    (dict(q_stride=512), SHAPE), (dict(T=5), SHAPE), (dict(max_q=2), SHAPE),
    (dict(cu_q=FAKE, max_q=5), SHAPE), (dict(Hq=24), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(page=20), UNSUPPORTED), (dict(num_pages=2**24), UNSUPPORTED),
    (dict(ld=2**25), UNSUPPORTED), (dict(), WORKSPACE), (dict(ws=None), WORKSPACE),
    (dict(T=0, B=0), OK), (dict(T=4, B=0, cu_q=FAKE), OK), (dict(T=0, B=3, cu_q=FAKE), OK),
])
def test_prefix_attn_refusals(bsa_lib, change, code):
    assert bsa_lib.bsa_prefix_attn(*with_(ATTN, **change)) == code


def test_prefix_attn_workspace(bsa_lib):
    q = bsa_lib.bsa_prefix_attn_workspace_bytes
    base = [1, 64, 64, 32, 8, 128, 64, 16, 32768, 1]
    n = q(*base)
    assert n > 0 and q(*base) == n
    for at, value in [(0, 7), (1, -1), (3, 30), (5, 96), (6, 24), (9, 0)]:
        bad = list(base)
        bad[at] = value
        assert q(*bad) == 0
    args = dict(ATTN, T=64, B=64, Hq=32, Hk=8, q_stride=4096, ld=16, prefix=32768, ws_bytes=n - 1)
    assert bsa_lib.bsa_prefix_attn(*args.values()) == WORKSPACE
    args = dict(args, ws=ctypes.c_void_p(0x1008), ws_bytes=n)
    assert bsa_lib.bsa_prefix_attn(*args.values()) == ARG


def test_binding_refuses(bsa_lib):
    """Shapes, types and strides that the binding turns away before the C call (CPU tensors are
    refused too: there is no fallback)."""
    k = torch.zeros(3, 2, 64)
    pages = torch.zeros(4, 2, 16, 64)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        bsa.paged_append(k, k, slots, pages, pages)  # CPU
    with pytest.raises(ValueError):
        bsa.paged_append(k.transpose(0, 1), k, slots, pages, pages)  # heads not contiguous
    with pytest.raises(ValueError):
        bsa.paged_append(k, k, slots[:2], pages, pages)
    with pytest.raises(ValueError):
        bsa.paged_append(k, k.bfloat16(), slots, pages, pages)
    q = torch.zeros(3, 4, 64)
    table = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bsa.prefix_attn(q, pages, pages, table[:2], slots, None, 0)
    with pytest.raises(ValueError):
        bsa.prefix_attn(q, pages, pages, table, slots, table[0], 33)  # 2 pages of 16 < 33
    with pytest.raises(ValueError):
        bsa.prefix_attn(q, pages, pages[:, :1], table, slots, None, 0)
    with pytest.raises(ValueError):
        bsa.prefix_attn(q.bfloat16(), pages, pages, table, slots, None, 0)
    with pytest.raises(ValueError):
        bsa.page_tables(slots, slots, table[:2], slots, slots[:2], 16, 8)
