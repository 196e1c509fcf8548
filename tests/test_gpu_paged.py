"""GPU parity of the paged serving operators: page tables, paged append and shared-prefix attention
against plain implementations (whole numbers in Python, attention in float64).

Tolerances of the attention (derived, per output element; u = 2^-24, W = sum_j w_j |v_j| with the
exact softmax weights w):
* a score is a sum of d products and a few scalings in float32, each off by at most u relative, and
  the tensor cores may cut instead of round (2 u): |ds| <= 2 (d + 8) u S, S = max_j sum |q k_j| /
  sqrt(d); the exponential adds 2^-22 |.| and the rounding of its argument u |s log2 e|.  So each
  weight is off by a factor of at most 1 + e, e = 2 (d + 8) u S + 4 u S + 2^-21, and the
  normalised sum by 2 e plus the rounding of a sum of n terms, 2 (n + 16) u;
* bf16: the weights are rounded to bf16 for the product with V (half a step, 2^-8 relative), and
  the output once more (2^-8 |o|).
lse: e + (n + 16) 2 u + 4 u |lse|.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_summaries_b200 as bsa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib(bsa_lib):
    return bsa_lib


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


# -------------------------------------------------------------------------------------------
# attention
# -------------------------------------------------------------------------------------------


class Batch:
    """A paged cache whose every unused place holds NaN, and requests on it."""

    def __init__(self, seed, dtype, heads, kv_heads, d, page, prefix, nq, lens, decode=False,
                 pad_tokens=0, spare_ld=0, q_scale=1.0, strided=False):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.dtype, self.heads, self.kv_heads, self.d, self.page = dtype, heads, kv_heads, d, page
        self.prefix, self.nq, self.lens_list = prefix, list(nq), list(lens)
        B = len(lens)
        pp = -(-prefix // page)
        held = [-(-n // page) for n in lens]
        pool = pp + sum(held) + 3
        ids = rng.permutation(pool)
        nan = float("nan")
        self.k = torch.full((pool, kv_heads, page, d), nan, device=DEV, dtype=dtype)
        self.v = torch.full((pool, kv_heads, page, d), nan, device=DEV, dtype=dtype)
        ld = max(held + [0]) + spare_ld
        table = np.full((B, ld), 2**31 - 1, np.int32)  # entries past the last page mean nothing
        self.own_ids, at = [], pp
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            self.own_ids.append(ids[at:at + h])
            at += h
        self.prefix_ids = ids[:pp]
        for pages, n in [(self.prefix_ids, prefix)] + list(zip(self.own_ids, lens)):
            for i, p in enumerate(pages):
                m = min(page, n - i * page)
                for x in (self.k, self.v):
                    x[int(p), :, :m] = torch.randn(kv_heads, m, d, device=DEV, generator=gen).to(
                        dtype)
        T = sum(nq) + pad_tokens
        if strided:  # a slice of a fused projection
            wide = torch.randn(T, (heads + 2 * kv_heads) * d, device=DEV, generator=gen)
            self.q = (wide * q_scale).to(dtype)[:, :heads * d].view(T, heads, d)
        else:
            self.q = (torch.randn(T, heads, d, device=DEV, generator=gen) * q_scale).to(dtype)
        self.table, self.lens = i32(table.reshape(B, ld)), i32(lens)
        self.prefix_table = i32(self.prefix_ids)
        self.cu_list = [0] + list(np.cumsum(nq))
        self.cu = None if decode else i32(self.cu_list)
        self.max_q = max(list(nq) + [1])

    def run(self, **kw):
        kw = dict(dict(cu_q=self.cu, max_q=self.max_q), **kw)
        return bsa.prefix_attn(self.q, self.k, self.v, self.table, self.lens, self.prefix_table,
                               self.prefix, **kw)

    def rows(self, pages, ids, n, h):
        ids = torch.as_tensor(np.asarray(ids, dtype=np.int64), device=DEV)
        return pages[ids, h].reshape(-1, self.d)[:n].double()

    def check(self, o, lse, requests=None, hidden=()):
        """Against float64; ``hidden``: (request or -1 for the prefix, page) that take no part."""
        G, d, page = self.heads // self.kv_heads, self.d, self.page
        for b in (range(len(self.nq)) if requests is None else requests):
            nq, n, c0 = self.nq[b], self.lens_list[b], self.cu_list[b]
            if nq == 0:
                continue
            drop = torch.zeros(self.prefix + n, dtype=torch.bool, device=DEV)
            for who, c in hidden:
                if who == -1:
                    drop[c * page:min((c + 1) * page, self.prefix)] = True
                elif who == b:
                    drop[self.prefix + c * page:self.prefix + min((c + 1) * page, n)] = True
            last = self.prefix + n - nq + torch.arange(nq, device=DEV).repeat_interleave(G)
            for h in range(self.kv_heads):
                k = torch.cat([self.rows(self.k, self.prefix_ids, self.prefix, h),
                               self.rows(self.k, self.own_ids[b], n, h)])
                v = torch.cat([self.rows(self.v, self.prefix_ids, self.prefix, h),
                               self.rows(self.v, self.own_ids[b], n, h)])
                q = self.q[c0:c0 + nq, h * G:(h + 1) * G].double().reshape(nq * G, d)
                s = q @ k.T / math.sqrt(d)
                big = (q.abs() @ k.abs().T / math.sqrt(d))
                j = torch.arange(len(k), device=DEV)[None]
                see = ((j < self.prefix) | (j <= last[:, None])) & ~drop[None]
                got_o = o[c0:c0 + nq, h * G:(h + 1) * G].double().reshape(nq * G, d)
                got_l = lse[c0:c0 + nq, h * G:(h + 1) * G].double().reshape(-1)
                none = ~see.any(1) if len(k) else torch.ones(nq * G, dtype=torch.bool, device=DEV)
                assert (got_o[none] == 0).all() and (got_l[none] == -math.inf).all(), (b, h)
                if none.all():
                    continue
                keep = ~none
                s = s.masked_fill(~see, -math.inf)[keep]
                S = torch.where(see, big, 0.0)[keep].amax(1)
                want_l = torch.logsumexp(s, 1)
                w = torch.exp(s - want_l[:, None])
                v = torch.where(drop[:, None], 0.0, v)
                want_o, W = w @ v, w @ v.abs()
                e = 2 * (d + 8) * U * S + 4 * U * S + 2.0 ** -21
                n_terms = 2 * (len(k) + 16) * U
                tol = (2 * e + n_terms)[:, None] * W
                if self.dtype == BF16:
                    tol = tol + 2.0 ** -8 * W * 1.01 + 2.0 ** -8 * want_o.abs()
                else:
                    tol = tol + U * want_o.abs()
                err = (got_o[keep] - want_o).abs()
                assert torch.isfinite(got_o).all(), (b, h)
                assert (err <= tol).all(), (b, h, float((err / tol).max()))
                errl = (got_l[keep] - want_l).abs()
                assert (errl <= e + n_terms + 4 * U * want_l.abs()).all(), (b, h)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (4, 2), (4, 1), (16, 2)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode(dtype, d, heads, kv_heads, page):
    m = Batch(1, dtype, heads, kv_heads, d, page, 200, [1] * 7, [1, 64, 65, 130, 16, 17, 300],
              decode=True)
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 63, 64, 127, 128, 129, 1000, 4096, 5001])
def test_prefix_lengths(dtype, prefix):
    m = Batch(2, dtype, 8, 2, 128, 32, prefix, [1] * 5, [1, 2, 31, 33, 70], decode=True,
              spare_ld=2, q_scale=2.0)
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 2, 33, 70])
def test_batch_sizes(dtype, page, B):
    rng = np.random.default_rng(B)
    m = Batch(3, dtype, 8, 2, 64, page, 333, [1] * B, list(rng.integers(0, 200, B)), decode=True)
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,heads,kv_heads,page", [(128, 8, 2, 64), (64, 4, 4, 16), (128, 8, 1, 128),
                                                   (64, 16, 8, 32)])
@pytest.mark.parametrize("nq,lens", [
    ([1, 5, 0, 8, 3], [1, 9, 4, 8, 300]),           # drafted tokens; a request without new ones
    ([40, 1, 129, 64], [40, 77, 129, 500]),         # prompts beside decode
    ([300], [300]), ([257, 2], [700, 2]),
    ([5, 7], [3, 0]),                               # more new tokens than own ones: rows with none
])
@pytest.mark.parametrize("prefix", [0, 150, 700])
def test_ragged(dtype, d, heads, kv_heads, page, nq, lens, prefix):
    m = Batch(4, dtype, heads, kv_heads, d, page, prefix, nq, lens, pad_tokens=3, strided=True)
    T = m.q.shape[0]
    o = torch.full((T, heads, d), 7.0, device=DEV, dtype=dtype)
    lse = torch.full((T, heads), 7.0, device=DEV)
    m.run(o=o, lse=lse)
    m.check(o, lse)
    assert (o[sum(nq):] == 7).all() and (lse[sum(nq):] == 7).all()  # rows behind the last sequence


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_to_see(dtype):
    m = Batch(5, dtype, 4, 2, 64, 16, 0, [1, 1, 1], [0, 3, 0], decode=True)
    o, lse = m.run()
    m.check(o, lse)
    m = Batch(5, dtype, 4, 2, 64, 16, 0, [1, 1], [0, 0], decode=True)  # a table of no columns
    o, lse = m.run()
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [1, 40])
def test_long_own_tokens(dtype, nq):
    """One request owns nearly all keys: its pieces are spread, the others' are short."""
    m = Batch(6, dtype, 8, 2, 128, 64, 70, [nq, 1, 1], [9000, 1, 64])
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(dtype, d):
    """Scores of several hundred: all weight on few keys, no overflow."""
    m = Batch(7, dtype, 8, 2, d, 32, 900, [1, 1, 20], [10, 400, 100], q_scale=60.0)
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [[1, 1, 1], [20, 1, 9]])
def test_pages_outside_the_pool_take_no_part(dtype, nq):
    m = Batch(8, dtype, 8, 2, 128, 32, 300, nq, [100, 70, 90])
    m.prefix_table[3] = -1
    m.prefix_table[9] = 2**31 - 1  # the last, partly filled page
    m.table[0, 1] = m.k.shape[0]
    m.table[2, 0] = -7
    for ids, at in ((m.prefix_ids, 3), (m.prefix_ids, 9), (m.own_ids[0], 1), (m.own_ids[2], 0)):
        ids[at] = 0  # the reference reads some page and drops it
    m.check(*m.run(), hidden=[(-1, 3), (-1, 9), (0, 1), (2, 0)])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nonfinite_rows_stay_where_they_are(dtype):
    """A NaN in one request's own values or queries reaches that request alone."""
    m = Batch(9, dtype, 8, 2, 128, 32, 260, [1] * 6, [40, 41, 42, 43, 44, 45], decode=True)
    m.v[int(m.own_ids[2][0]), :, 5] = float("inf")
    m.k[int(m.own_ids[4][1]), :, 3] = float("nan")
    m.q[1] = float("nan")
    o, lse = m.run()
    m.check(o, lse, requests=[0, 3, 5])
    assert not torch.isfinite(o[2]).any() and torch.isnan(o[4]).all() and torch.isnan(o[1]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,n,at,prefix", [(6, 50, 46, 200), (30, 90, 70, 0), (100, 300, 250, 130),
                                            (400, 400, 37, 5), (400, 700, 690, 300)])
def test_nonfinite_values_reach_only_rows_that_see_them(dtype, d, nq, n, at, prefix):
    """An infinity and a NaN in V at own position `at`: earlier rows are as without them, later ones
    hold them in the columns concerned and are as without them in the others."""
    m = Batch(16, dtype, 8, 2, d, 16, prefix, [1, nq, 2], [9, n, 30])
    clean, clean_lse = m.run()
    page, off = int(m.own_ids[1][at // 16]), at % 16
    m.v[page, 0, off, 3] = float("inf")
    m.v[page, 1, off, d - 1] = float("nan")
    if at + 1 < n - 1:  # a second one, seen by fewer rows
        page, off = int(m.own_ids[1][(at + 1) // 16]), (at + 1) % 16
        m.v[page, 0, off, 20] = float("-inf")
    o, lse = m.run()
    assert torch.equal(lse, clean_lse)
    t = torch.arange(o.shape[0], device=DEV)[:, None, None]
    pos = torch.where((t >= 1) & (t < 1 + nq), n - nq + t - 1, -1)  # own position, request 1
    h = torch.arange(8, device=DEV)[None, :, None]
    c = torch.arange(d, device=DEV)[None, None, :]
    inf = (pos >= at) & (h < 4) & (c == 3)
    nan = (pos >= at) & (h >= 4) & (c == d - 1)
    neg = (pos >= at + 1) & (h < 4) & (c == 20) & (at + 1 < n - 1)
    assert (o[inf] == float("inf")).all() and torch.isnan(o[nan]).all()
    assert (o[neg] == float("-inf")).all()
    rest = ~(inf | nan | neg)
    assert inf.any() and torch.equal(o[rest], clean[rest])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tokens_beyond_max_q_are_left(dtype):
    m = Batch(10, dtype, 8, 2, 64, 16, 50, [3, 9, 2], [30, 40, 2])
    o = torch.full(m.q.shape, 7.0, device=DEV, dtype=dtype)
    lse = torch.full(m.q.shape[:2], 7.0, device=DEV)
    m.run(o=o, lse=lse, max_q=4)
    m.check(o, lse, requests=[0, 2])
    assert (o[3 + 4:3 + 9] == 7).all() and (o[3:3 + 4] != 7).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [[2, 1], [70, 3], [200, 1]])
def test_tokens_before_the_first_request_are_left(dtype, nq):
    """cu_q may start behind the first token, as a slice of a longer batch does."""
    m = Batch(14, dtype, 8, 2, 64, 16, 90, nq, [300, 20], pad_tokens=5)
    q = m.q.clone()
    m.q[5:] = q[:-5]
    m.cu = m.cu + 5
    o = torch.full(m.q.shape, 7.0, device=DEV, dtype=dtype)
    lse = torch.full(m.q.shape[:2], 7.0, device=DEV)
    m.run(o=o, lse=lse)
    assert (o[:5] == 7).all() and (lse[:5] == 7).all()
    m.q = m.q[5:]
    m.check(o[5:], lse[5:])


@pytest.mark.parametrize("B,n,ld", [(1, 1, 1), (2, 17, 2), (9, 40, 3), (30, 64, 4), (60, 16, 1)])
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 8, 64), (32, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_small_calls(dtype, B, n, ld, heads, kv_heads, d):
    """Small enough for one launch, up to and past the border; twice."""
    m = Batch(15, dtype, heads, kv_heads, d, 16, 100, [1] * B, [1 + (n + i) % n for i in range(B)],
              decode=True, spare_ld=ld)
    for _ in range(2):
        m.check(*m.run())


def test_repeats_bit_for_bit():
    m = Batch(11, BF16, 32, 8, 128, 64, 5000, [1] * 40, list(range(1, 41)), decode=True)
    a, la = m.run()
    for _ in range(3):
        b, lb = m.run()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_batch_does_not_change_a_request():
    """The pool's other requests and their lengths do not move a row beyond its tolerance."""
    m = Batch(12, BF16, 8, 2, 128, 64, 700, [1] * 90, [(37 * i) % 500 + 1 for i in range(90)],
              decode=True)
    m.check(*m.run(), requests=[0, 1, 31, 32, 63, 64, 88, 89])


def test_no_lse_and_given_workspace():
    m = Batch(13, BF16, 8, 2, 128, 64, 700, [1] * 9, [50] * 9, decode=True)
    need = bsa.prefix_attn_workspace_bytes(BF16, 9, 9, 8, 2, 128, 64, m.table.shape[1], 700)
    ws = torch.full((need,), 255, device=DEV, dtype=torch.uint8)  # NaN bit patterns
    m.check(*m.run(ws=ws))
    with pytest.raises(bsa.BsaError):
        m.run(ws=ws[:need - 16])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_head_of_any_stride(dtype):
    """[heads, T, d] seen as [T, heads, d] with one head: the stride of the heads says nothing."""
    m = Batch(14, dtype, 1, 1, 64, 16, 100, [1, 3, 20], [5, 30, 40])
    q = m.q.as_strided(m.q.shape, (m.d, len(m.q) * m.d, 1))
    assert q.stride(1) != m.d
    m.q = q
    m.check(*m.run())
    slots = torch.arange(len(q), device=DEV, dtype=torch.int32)
    k, v = (torch.zeros(2, 1, 16, 64, device=DEV, dtype=dtype) for _ in range(2))
    bsa.paged_append(q, q, slots, k, v)
    assert torch.equal(k.view(-1, 64)[:len(q)], q[:, 0]) and torch.equal(k, v)


# -------------------------------------------------------------------------------------------
# page tables
# -------------------------------------------------------------------------------------------


def plain_tables(lens, new, table, ring, free, page, max_tokens, off):
    """The definition of bsa_page_tables, one request at a time."""
    table, ring = table.copy(), ring.copy()
    N, ld = len(ring), table.shape[1]
    head, avail = int(free[0]), int(free[1])
    bits, taken, freed, out, cu = 0, 0, 0, [], [0]
    need = 0
    slots, pos = [], []
    before = table.copy()
    for b in range(len(lens)):
        l, n = int(lens[b]), int(new[b])
        if min(l, n) < 0 or max(l, n) > ld * page:
            bits |= 2
            out.append(l)
            cu.append(cu[-1])
            continue
        have, want = -(-l // page), -(-n // page)
        grow, add = max(0, want - have), max(0, n - l)
        need += grow
        cu.append(cu[-1] + add)
        if grow and need > avail:
            bits |= 1
            out.append(l)
            slots += [-1] * add
            pos += [-1] * add
            continue
        for c in range(have, want):
            table[b, c] = ring[(head + taken) % N]
            taken += 1
        for c in range(want, have):
            if avail + freed < N:
                ring[(head + avail + freed) % N] = before[b, c]
                freed += 1
            else:
                bits |= 4
        out.append(n)
        for p in range(l, n):
            i = int(table[b, p // page])
            bad = i < 0 or i >= N
            bits |= 16 if bad and len(slots) < max_tokens else 0  # looked up for a token's slot
            slots.append(-1 if bad else i * page + p % page)
            pos.append(off + p)
    if cu[-1] > max_tokens:
        bits |= 8
    pad = max(0, max_tokens - len(slots))
    return (out, [(head + taken) % N, avail - taken + freed], cu,
            (slots + [-1] * pad)[:max_tokens], (pos + [-1] * pad)[:max_tokens], table, ring, bits)


def make_tables(rng, B, page, ld, spare):
    lens = rng.integers(0, ld * page + 1, B)
    held = -(-lens // page)
    N = int(held.sum()) + spare
    ids = rng.permutation(N).astype(np.int32)
    table = np.full((B, ld), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    ring = np.full(N, -1, np.int32)
    head = int(rng.integers(0, N))
    ring[(head + np.arange(spare)) % N] = ids[at:]
    return lens.astype(np.int32), table, ring, np.array([head, spare], np.int32)


def check_tables(lens, new, table, ring, free, page, max_tokens, off=0, in_place=False,
                 into_new=False):
    want = plain_tables(lens, new, table, ring, free, page, max_tokens, off)
    g = [i32(x) for x in (lens, new, table, ring, free)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(lens_out=g[1] if into_new else g[0], free_out=g[4]) if in_place else {}
    got = bsa.page_tables(*g, page, max_tokens, pos_offset=off, status=status, **kw)
    got = [x.cpu().numpy().tolist() for x in got]
    for a, b, name in zip(got, want, ["lens", "free", "cu", "slots", "positions"]):
        assert a == list(np.asarray(b).tolist()), name
    assert np.array_equal(g[2].cpu().numpy(), want[5])
    assert np.array_equal(g[3].cpu().numpy(), want[6])
    assert int(status) == want[7]
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 300, 1025, 2500])
def test_page_tables(B, page, in_place):
    rng = np.random.default_rng(B * page)
    ld = 5
    lens, table, ring, free = make_tables(rng, B, page, ld, 3 * B + 7)
    new = rng.integers(0, ld * page + 1, B).astype(np.int32)
    keep = rng.random(B) < 0.5  # half of them grow by one token or not at all
    new[keep] = np.minimum(lens + rng.integers(0, 2, B), ld * page)[keep]
    total = int(np.maximum(new - lens, 0).sum())
    check_tables(lens, new, table, ring, free, page, total + 5, off=77, in_place=in_place)


@pytest.mark.parametrize("B", [5000, 8192])
def test_page_tables_most_requests(B):
    rng = np.random.default_rng(B)
    lens, table, ring, free = make_tables(rng, B, 16, 3, 2 * B)
    new = rng.integers(0, 49, B).astype(np.int32)
    check_tables(lens, new, table, ring, free, 16, int(np.maximum(new - lens, 0).sum()) + 3)


@pytest.mark.parametrize("spare", [0, 1, 3, 10])
def test_page_tables_exhausted(spare):
    rng = np.random.default_rng(spare)
    lens, table, ring, free = make_tables(rng, 40, 16, 6, spare)
    new = np.minimum(lens + rng.integers(0, 60, 40), 96).astype(np.int32)
    new[::7] = 0
    want = check_tables(lens, new, table, ring, free, 16, 2000)
    assert want[7] & 1


def test_page_tables_bad_states():
    rng = np.random.default_rng(4)
    lens, table, ring, free = make_tables(rng, 12, 16, 4, 30)
    new = lens.copy()
    new[2], new[3], new[4] = -1, 65, 2**31 - 1  # impossible lengths
    lens[6] = -5
    new[7], new[8] = 64, 64
    check_tables(lens, new, table, ring, free, 16, 300)
    # a page id outside the pool in a partly filled page; too few places for the new tokens
    lens[9], new[9] = 17, 30
    table[9, 1] = 10**6
    assert check_tables(lens, new, table, ring, free, 16, 300)[7] & 16
    assert check_tables(lens, new, table, ring, free, 16, 10)[7] & 8
    # a ring that claims to be full has no room for what is freed
    full = np.array([5, len(ring)], np.int32)
    want = check_tables(lens, np.zeros_like(new), table, ring, full, 16, 10)
    assert want[7] & 4


@pytest.mark.parametrize("B", [3, 1500])
def test_page_tables_into_the_new_lengths(B):
    """lens_out = new_lens; the refused requests read their old length there."""
    rng = np.random.default_rng(B)
    lens, table, ring, free = make_tables(rng, B, 32, 4, B // 2)
    new = rng.integers(0, 129, B).astype(np.int32)
    new[B // 2] = 1000
    check_tables(lens, new, table, ring, free, 32, 5000, in_place=True, into_new=True)


def test_page_tables_without_tokens():
    """No places for tokens: the tables still move."""
    rng = np.random.default_rng(1)
    lens, table, ring, free = make_tables(rng, 9, 16, 3, 20)
    new = np.minimum(lens + 3, 48).astype(np.int32)
    assert check_tables(lens, new, table, ring, free, 16, 0)[7] == 8


def test_page_tables_no_requests():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    lens, free, cu, slots, pos = bsa.page_tables(e, e, e.view(0, 4), i32([1, 2, 0]), i32([1, 2]),
                                                 16, 5)
    assert free.tolist() == [1, 2] and cu.tolist() == [0] and slots.tolist() == [-1] * 5


@pytest.mark.parametrize("max_tokens", [128, 1000, 300000])
def test_page_tables_no_requests_many_places(max_tokens):
    """Places for whole warps of tokens, after a step whose sums are still in shared memory."""
    rng = np.random.default_rng(2)
    lens, table, ring, free = make_tables(rng, 300, 16, 40, 20000)
    new = (lens + 300).astype(np.int32)
    check_tables(lens, new, table, ring, free, 16, 300 * 300)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    _, free, cu, slots, pos = bsa.page_tables(e, e, e.view(0, 4), i32([1, 2, 0]), i32([1, 2]), 16,
                                              max_tokens)
    assert free.tolist() == [1, 2] and cu.tolist() == [0]
    assert bool((slots == -1).all()) and bool((pos == -1).all())


# -------------------------------------------------------------------------------------------
# paged append
# -------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["dense", "fused", "odd"])
@pytest.mark.parametrize("T,page", [(1, 16), (7, 32), (300, 64), (2049, 128)])
def test_paged_append(dtype, d, layout, T, page):
    rng = np.random.default_rng(T)
    Hk = 3
    if layout == "dense":
        k, v = (torch.randn(T, Hk, d, device=DEV).to(dtype) for _ in range(2))
    else:
        # a fused projection; "odd": rows that start at any element
        shift = 0 if layout == "fused" else 3
        wide = torch.randn(T, 5 * d + 2 * Hk * d + shift + (1 if shift else 0), device=DEV)
        wide = wide.to(dtype)
        a = 5 * d + shift
        k = wide[:, a:a + Hk * d].view(T, Hk, d) if T == 1 or not shift else \
            wide[:, a:a + Hk * d].unflatten(1, (Hk, d))
        v = wide[:, a + Hk * d:a + 2 * Hk * d].unflatten(1, (Hk, d))
    pool = T // page + 5
    slots = rng.permutation(pool * page)[:T].astype(np.int32)
    if T > 5:
        slots[[1, 4]] = -1
        slots[5] = pool * page  # outside the pool
    kp, vp = (torch.randn(pool, Hk, page, d, device=DEV).to(dtype) for _ in range(2))
    want_k, want_v = kp.clone(), vp.clone()
    for t, s in enumerate(slots):
        if 0 <= s < pool * page:
            want_k[s // page, :, s % page] = k[t]
            want_v[s // page, :, s % page] = v[t]
    bsa.paged_append(k, v, i32(slots), kp, vp)
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


# -------------------------------------------------------------------------------------------
# the operators together
# -------------------------------------------------------------------------------------------


class Server:
    """Requests behind a shared prefix, served with the three operators; a dense copy of every
    request's keys and values beside it."""

    def __init__(self, dtype=BF16, B=6, heads=8, kv_heads=2, d=64, page=16, prefix=100, ld=8,
                 pool=60):
        self.dtype, self.heads, self.kv_heads, self.d, self.page = dtype, heads, kv_heads, d, page
        self.prefix, self.B = prefix, B
        self.gen = torch.Generator(device=DEV).manual_seed(3)
        pp = -(-prefix // page)
        self.k = torch.full((pool, kv_heads, page, d), float("nan"), device=DEV, dtype=dtype)
        self.v = self.k.clone()
        self.prefix_table = torch.arange(pool - pp, pool, device=DEV, dtype=torch.int32)
        self.pk, self.pv = self.randn(prefix, kv_heads, d), self.randn(prefix, kv_heads, d)
        at = torch.arange(prefix, device=DEV, dtype=torch.int32) + (pool - pp) * page
        bsa.paged_append(self.pk, self.pv, at, self.k, self.v)
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.table = torch.full((B, ld), -1, dtype=torch.int32, device=DEV)
        self.ring = torch.arange(pool, device=DEV, dtype=torch.int32)
        self.free = i32([0, pool - pp])
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.own = [(self.randn(0, kv_heads, d), self.randn(0, kv_heads, d)) for _ in range(B)]

    def randn(self, *shape):
        return torch.randn(*shape, device=DEV, generator=self.gen).to(self.dtype)

    def step(self, q, k, v, new_lens, max_tokens, max_q):
        _, _, cu, slots, _ = bsa.page_tables(self.lens, new_lens, self.table, self.ring, self.free,
                                             self.page, max_tokens, pos_offset=self.prefix,
                                             lens_out=self.lens, free_out=self.free,
                                             status=self.status)
        bsa.paged_append(k, v, slots, self.k, self.v)
        return bsa.prefix_attn(q, self.k, self.v, self.table, self.lens, self.prefix_table,
                               self.prefix, cu_q=cu, max_q=max_q)

    def record(self, b, k, v):
        self.own[b] = (torch.cat([self.own[b][0], k]), torch.cat([self.own[b][1], v]))

    def want(self, b, q):
        """float64 attention of the last len(q) tokens of request b."""
        G, d = self.heads // self.kv_heads, self.d
        k = torch.cat([self.pk, self.own[b][0]]).double()
        v = torch.cat([self.pv, self.own[b][1]]).double()
        nq = q.shape[0]
        x = torch.einsum("ikgd,jkd->ikgj", q.double().view(nq, self.kv_heads, G, d), k) / d ** 0.5
        last = len(k) - nq + torch.arange(nq, device=DEV)
        x = x.masked_fill((torch.arange(len(k), device=DEV) > last[:, None])[:, None, None],
                          -math.inf)
        p = torch.softmax(x, -1)
        o = torch.einsum("ikgj,jkd->ikgd", p, v).reshape(nq, self.heads, d)
        W = torch.einsum("ikgj,jkd->ikgd", p, v.abs()).reshape(nq, self.heads, d)
        # bf16 weights and output (2^-8 each) beside float32 sums (under 2^-14 here: |s| < 2^4,
        # a few hundred terms)
        if self.dtype == F32:
            return o, 2.0 ** -14 * W
        return o, 2.0 ** -8 * (1.01 * W + o.abs()) + 2.0 ** -14 * W


def run_script(s, script, run):
    """script: list of {request: tokens to add, or None to finish it}."""
    for moves in script:
        before = s.lens.cpu().numpy()
        new = before.copy()
        for b, n in moves.items():
            new[b] = 0 if n is None else before[b] + n
        add = [max(0, int(n - o)) for o, n in zip(before, new)]
        T = sum(add)
        q, k, v = s.randn(T, s.heads, s.d), s.randn(T, s.kv_heads, s.d), s.randn(T, s.kv_heads, s.d)
        o, lse = run(q, k, v, i32(new), T, max(add + [1]))
        at = 0
        for b, n in enumerate(add):
            if moves.get(b, 0) is None:
                s.own[b] = (s.randn(0, s.kv_heads, s.d), s.randn(0, s.kv_heads, s.d))
            if n:
                s.record(b, k[at:at + n], v[at:at + n])
                want, tol = s.want(b, q[at:at + n])
                err = (o[at:at + n].double() - want).abs()
                assert (err <= tol).all(), (moves, b, float((err / tol).max()))
            at += n
        assert int(s.status) == 0


SCRIPT = ([{0: 37, 1: 1, 2: 16, 3: 50}] + [{b: 1 for b in range(4)}] * 3 +
          [{0: None, 4: 64, 1: 5, 2: 1}, {1: 1, 2: 1, 3: 1, 4: 1}] +
          [{1: None, 2: None}, {0: 20, 5: 33, 3: 1}] + [{0: 1, 3: 1, 4: 1, 5: 1}] * 4)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_serving_steps(dtype):
    s = Server(dtype=dtype)
    run_script(s, SCRIPT, s.step)


def test_serving_steps_on_another_stream():
    s = Server()
    st = torch.cuda.Stream()

    def run(*a):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            r = s.step(*a)
        torch.cuda.current_stream().wait_stream(st)
        return r

    run_script(s, SCRIPT, run)


def test_captured_decode_steps():
    """One captured tick, replayed: lengths, pages and positions advance on the device."""
    s = Server(prefix=333, pool=80)
    run_script(s, SCRIPT[:1], s.step)
    live = [0, 1, 2, 3]
    one = i32([1 if b in live else 0 for b in range(s.B)])
    q, k, v = s.randn(4, s.heads, s.d), s.randn(4, s.kv_heads, s.d), s.randn(4, s.kv_heads, s.d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = s.step(q, k, v, s.lens + one, 4, 1)
    for _ in range(20):
        q.copy_(s.randn(4, s.heads, s.d))
        k.copy_(s.randn(4, s.kv_heads, s.d))
        v.copy_(s.randn(4, s.kv_heads, s.d))
        g.replay()
        for i, b in enumerate(live):
            s.record(b, k[i:i + 1], v[i:i + 1])
            want, tol = s.want(b, q[i:i + 1])
            assert ((o[i:i + 1].double() - want).abs() <= tol).all()
    assert int(s.status) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_captured_long_batches(dtype, decode):
    """A captured call with many key pieces, replayed on other lengths, queries and cache contents."""
    nq = [1] * 40 if decode else [3, 200, 1, 1, 90]
    lens = [(53 * i) % 400 + 1 for i in range(40)] if decode else [40, 260, 5, 1, 90]
    m = Batch(17, dtype, 8, 2, 128, 32, 6000, nq, lens, decode=decode, spare_ld=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = m.run()
    for step in range(3):
        g.replay()
        m.check(o, lse, requests=[0, 1, 4])
        m.q.copy_(torch.randn_like(m.q))
        m.v.nan_to_num_().mul_(0.5)
        m.lens_list = [max(q, n - 7 * (step + 1)) for q, n in zip(nq, lens)]
        m.lens.copy_(i32(m.lens_list))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_long_prompt_among_many(dtype):
    """A prompt beside 300 requests of one token: row tiles go by the tokens there are."""
    nq = [1] * 150 + [700] + [1] * 150
    m = Batch(18, dtype, 4, 2, 64, 16, 90, nq, [n + 10 for n in nq])
    m.check(*m.run(), requests=[0, 149, 150, 151, 300])


def test_far_pages():
    """Pages behind the first 2^31 elements of the pool, in all three operators."""
    P, Hk, page, d = 270_000, 1, 64, 128  # 2.2e9 elements
    k = torch.empty(P, Hk, page, d, device=DEV, dtype=BF16)
    v = torch.empty(P, Hk, page, d, device=DEV, dtype=BF16)
    pk, pv = (torch.randn(130, Hk, d, device=DEV).to(BF16) for _ in range(2))
    ids = i32([P - 1, 5, P - 3])
    at = (ids.long()[torch.arange(130, device=DEV) // 64] * 64
          + torch.arange(130, device=DEV) % 64).int()
    bsa.paged_append(pk, pv, at, k, v)
    assert torch.equal(k[P - 1, 0, :], pk[:64, 0]) and torch.equal(v[P - 3, 0, :2], pv[128:, 0])
    ring = torch.arange(P - 1, -1, -1, device=DEV, dtype=torch.int32)
    table = torch.zeros(2, 2, device=DEV, dtype=torch.int32)
    lens, free, cu, slots, pos = bsa.page_tables(i32([0, 0]), i32([70, 3]), table, ring,
                                                 i32([2, P - 2]), page, 80)
    assert table.tolist()[0] == [P - 3, P - 4] and slots[69] == (P - 4) * 64 + 5
    for dtype, T in ((BF16, 1), (BF16, 30)):  # few rows; 128-row tiles
        q = torch.randn(T, 8, d, device=DEV).to(dtype)
        o, _ = bsa.prefix_attn(q, k, v, torch.zeros(T, 0, device=DEV, dtype=torch.int32),
                               torch.zeros(T, device=DEV, dtype=torch.int32), ids, 130)
        x = torch.einsum("thd,nd->thn", q.double(), pk[:, 0].double()) / d ** 0.5
        p = torch.softmax(x, -1)
        want, W = (torch.einsum("thn,nd->thd", p, y.double()) for y in (pv[:, 0], pv[:, 0].abs()))
        assert ((o.double() - want).abs() <= 2.0 ** -8 * (1.01 * W + want.abs())
                + 2.0 ** -14 * W).all()


def test_two_streams_at_once():
    """Two batches on two streams, each with its own workspace from the allocator."""
    ms = [Batch(20 + i, BF16, 8, 2, 128, 64, 3000, [1] * 20, [100 + i] * 20, decode=True)
          for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    out = [[], []]
    for _ in range(10):
        for i, m in enumerate(ms):
            with torch.cuda.stream(streams[i]):
                out[i].append(m.run())
    torch.cuda.synchronize()
    for m, got in zip(ms, out):
        m.check(*got[0], requests=[0, 19])
        assert all(torch.equal(got[0][0], o) and torch.equal(got[0][1], lse) for o, lse in got)
