"""Every kernel of the shared-prefix attention against float64, by name: each case says which
kernels it is to launch, read from a captured graph, so that a changed rule cannot leave one
untested.  Tolerances: those of test_gpu_paged.Batch.check."""
import re

import numpy as np
import pytest
import torch
from cuda.bindings import driver

import block_sparse_attention_summaries_b200 as bsa
from test_gpu_paged import BF16, DEV, F32, SCRIPT, Batch, Server, run_script

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(bsa_lib):
    return bsa_lib


def ok(result):
    assert int(result[0]) == 0, result
    return result[1:]


def kernels(fn):
    """What fn launches, in order: 'tc128', 'rows64x2' (d, row tiles), 'simt64:16:32' (d, rows of a
    prefix and of an own tile), 'merge'."""
    fn()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        fn()
    handle = driver.CUgraph(graph.raw_cuda_graph())
    count = ok(driver.cuGraphGetNodes(handle))[1]
    nodes = ok(driver.cuGraphGetNodes(handle, count))[0]
    names = []
    for node in nodes:
        if (ok(driver.cuGraphNodeGetType(node))[0]
                != driver.CUgraphNodeType.CU_GRAPH_NODE_TYPE_KERNEL):
            continue
        p = ok(driver.cuGraphKernelNodeGetParams(node))[0]
        name = ok(driver.cuFuncGetName(p.func) if int(p.func) else driver.cuKernelGetName(p.kern))
        name = name[0].decode()
        m = re.search(r"prefix_(tc|rows|simt|merge)_kernelI(.*?)EEv", name)
        if m is None:
            continue
        n = re.findall(r"Li(\d+)E", m.group(2) + "E")
        names.append({"tc": "tc" + n[0], "rows": "rows" + "x".join(n),
                      "simt": "simt" + ":".join(n), "merge": "merge"}[m.group(1)])
    return names


def ragged(seed, B, most, own):
    """New and own tokens of B requests, up to `most` new ones."""
    rng = np.random.default_rng(seed)
    nq = [int(x) for x in rng.integers(1, most + 1, B)]
    nq[B // 2] = most
    return nq, [int(rng.integers(q, max(q, own) + 1)) for q in nq]


# dtype, d, heads, kv heads, page, prefix, requests, most new tokens, most own tokens, kernels
PATHS = [
    # few rows a request, the prefix in packed tiles
    (BF16, 64, 4, 4, 32, 20001, 32, 1, 301, ["tc64", "rows64x1", "merge"]),
    (BF16, 64, 8, 2, 16, 20001, 40, 8, 301, ["tc64", "rows64x2", "merge"]),
    (BF16, 64, 8, 1, 64, 40001, 30, 7, 120, ["tc64", "rows64x4", "merge"]),
    (BF16, 128, 8, 2, 64, 33001, 20, 1, 500, ["tc128", "rows128x1", "merge"]),
    (BF16, 128, 8, 2, 128, 8191, 24, 8, 700, ["tc128", "rows128x2", "merge"]),
    (BF16, 128, 8, 2, 16, 8197, 20, 15, 120, ["tc128", "rows128x4", "merge"]),
    # and with the prefix among them
    (BF16, 64, 8, 2, 16, 333, 70, 1, 200, ["rows64x1", "merge"]),
    (BF16, 64, 8, 2, 32, 333, 70, 7, 200, ["rows64x2", "merge"]),
    (BF16, 64, 8, 1, 128, 130, 70, 8, 100, ["rows64x4", "merge"]),
    (BF16, 128, 8, 2, 64, 333, 70, 1, 200, ["rows128x1", "merge"]),
    (BF16, 128, 8, 2, 128, 333, 70, 8, 120, ["rows128x2", "merge"]),
    (BF16, 128, 8, 2, 16, 130, 70, 15, 120, ["rows128x4", "merge"]),
    # one launch
    (BF16, 64, 8, 2, 32, 100, 5, 1, 40, ["rows64x1"]),
    (BF16, 128, 8, 2, 32, 100, 5, 8, 40, ["rows128x2"]),
    (BF16, 64, 8, 1, 16, 100, 5, 8, 40, ["rows64x4"]),
    # requests that fill tiles: prefix and own keys in one pass, in pieces or whole
    (BF16, 64, 8, 2, 16, 700, 3, 300, 400, ["tc64", "merge"]),
    (BF16, 128, 8, 2, 128, 701, 3, 300, 400, ["tc128", "merge"]),
    (BF16, 64, 16, 4, 64, 700, 12, 260, 300, ["tc64"]),
    (BF16, 128, 16, 4, 32, 699, 12, 260, 300, ["tc128"]),
    # and requests that do not: packed tiles for the prefix, the request's for its own keys
    (BF16, 64, 4, 4, 32, 1500, 20, 70, 300, ["tc64", "merge"]),
    (BF16, 128, 8, 8, 16, 1500, 20, 70, 300, ["tc128", "merge"]),
    (F32, 64, 8, 2, 16, 50, 2, 1, 40, ["simt64:16:16"]),
    (F32, 128, 8, 2, 32, 40, 5, 1, 10, ["simt128:32:16"]),
    (F32, 64, 8, 2, 64, 3001, 4, 4, 300, ["simt64:64:16", "merge"]),
    (F32, 128, 8, 2, 16, 1001, 20, 1, 500, ["simt128:64:16", "merge"]),
    (F32, 64, 4, 2, 128, 2001, 4, 1, 300, ["simt64:16:16", "merge"]),
    (F32, 128, 4, 2, 64, 701, 10, 1, 300, ["simt128:32:16", "merge"]),
    (F32, 64, 8, 2, 32, 701, 6, 70, 300, ["simt64:64:64", "merge"]),
    (F32, 128, 8, 1, 16, 701, 6, 70, 300, ["simt128:64:64", "merge"]),
]


@pytest.mark.parametrize("dtype,d,heads,kv_heads,page,prefix,B,most,own,launched", PATHS)
def test_each_kernel(dtype, d, heads, kv_heads, page, prefix, B, most, own, launched):
    nq, lens = ragged(B + most, B, most, own)
    m = Batch(31, dtype, heads, kv_heads, d, page, prefix, nq, lens, decode=most == 1, strided=True)
    assert kernels(m.run) == launched
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix", [0, 700])
@pytest.mark.parametrize("nq", [[1, 5, 0, 8, 3], [40, 1, 129, 64, 2], [1, 1, 0, 1, 1]])
def test_most_new_tokens_need_not_be_named(dtype, prefix, nq):
    """cu_q without max_q: every token of every request is attended."""
    m = Batch(33, dtype, 8, 2, 64, 16, prefix, nq, [max(n, 30) + i for i, n in enumerate(nq)])
    o = torch.full_like(m.q, float("nan"))
    _, lse = bsa.prefix_attn(m.q, m.k, m.v, m.table, m.lens, m.prefix_table, prefix, cu_q=m.cu, o=o)
    m.check(o, lse)


# as PATHS: each way in which a row's result is written
PLACES = [
    (BF16, 64, 8, 2, 32, 100, 5, 1, 40, ["rows64x1"]),
    (BF16, 128, 8, 2, 128, 8191, 24, 8, 700, ["tc128", "rows128x2", "merge"]),
    (BF16, 128, 8, 2, 128, 701, 3, 300, 400, ["tc128", "merge"]),
    (BF16, 64, 16, 4, 64, 700, 12, 260, 300, ["tc64"]),
    (BF16, 128, 16, 4, 32, 699, 12, 260, 300, ["tc128"]),
    (F32, 64, 8, 2, 16, 50, 2, 1, 40, ["simt64:16:16"]),
    (F32, 64, 8, 2, 32, 701, 6, 70, 300, ["simt64:64:64", "merge"]),
]


@pytest.mark.parametrize("dtype,d,heads,kv_heads,page,prefix,B,most,own,launched", PLACES)
@pytest.mark.parametrize("cut", [0, 1, None])
def test_tokens_without_a_slot(dtype, d, heads, kv_heads, page, prefix, B, most, own, launched, cut):
    """A refused request's tokens, single tokens on pages outside the pool and those past the end
    of `slots` are answered with nothing; the others as without `slots`, to the bit."""
    nq, lens = ragged(B + most, B, most, own)
    m = Batch(34, dtype, heads, kv_heads, d, page, prefix, nq, lens, decode=most == 1, pad_tokens=0)
    m.v[int(m.own_ids[1][0]), :, 0] = float("inf")  # of tokens with a slot and without
    o, lse = m.run()
    T = m.q.shape[0]
    top = m.k.shape[0] * page
    slots = np.arange(T) % top
    slots[0] = top - 1
    c = m.cu_list
    slots[c[1] + nq[1] // 2:c[2]] = -1
    slots[T - 1] = top  # behind the pool
    if most > 1:
        slots[1] = 2**31 - 1
    n = {0: 0, 1: T - 1, None: T}[cut]
    none = (slots < 0) | (slots >= top) | (np.arange(T) >= n)
    given = torch.tensor(slots[:n].astype(np.int32), device=DEV)
    got, got_lse = m.run(slots=given)
    assert kernels(lambda: m.run(slots=given)) == launched
    none = torch.as_tensor(none, device=DEV)
    assert none.any() and (n == 0 or not none.all())
    assert (got[none] == 0).all() and (got_lse[none] == -float("inf")).all()
    assert torch.equal(got[~none].view(torch.uint8), o[~none].view(torch.uint8))
    assert torch.equal(got_lse[~none], lse[~none])


class PlacedServer(Server):
    """Hands the slots on, and checks a step whose pages or places may run out."""

    def step(self, q, k, v, new_lens, max_tokens, max_q):
        _, _, cu, slots, _ = bsa.page_tables(self.lens, new_lens, self.table, self.ring, self.free,
                                             self.page, max_tokens, lens_out=self.lens,
                                             free_out=self.free, status=self.status)
        bsa.paged_append(k[:max_tokens], v[:max_tokens], slots, self.k, self.v)
        return bsa.prefix_attn(q, self.k, self.v, self.table, self.lens, self.prefix_table,
                               self.prefix, cu_q=cu, max_q=max_q, slots=slots)

    def moves(self, adds, refused=(), places=None):
        """adds: new tokens of each request (None: done); returns the status bits of the step."""
        before = self.lens.cpu().numpy()
        new = [0 if a is None else int(n) + a for n, a in zip(before, adds)]
        nq = [a or 0 for a in adds]
        T = sum(nq)
        q, k, v = (self.randn(T, h, self.d) for h in (self.heads, self.kv_heads, self.kv_heads))
        self.status.zero_()
        places = T if places is None else places
        o, lse = self.step(q, k, v, torch.tensor(new, dtype=torch.int32, device=DEV), places,
                           max(nq))
        at = 0
        for b, n in enumerate(nq):
            if adds[b] is None:
                self.own[b] = (self.randn(0, self.kv_heads, self.d),) * 2
            put = 0 if b in refused else max(0, min(n, places - at))  # tokens in the cache
            assert (o[at + put:at + n] == 0).all()
            assert (lse[at + put:at + n] == -float("inf")).all()
            if put:
                self.record(b, k[at:at + put], v[at:at + put])
                want, tol = self.want(b, q[at:at + put])
                assert ((o[at:at + put].double() - want).abs() <= tol).all(), b
            at += n
        return int(self.status)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix", [100, 40001])
def test_steps_with_refused_requests(dtype, prefix):
    """Tables, append and attention when pages run out: the refused requests' tokens are answered
    with nothing, the others are served, and the refused ones too once there are pages."""
    s = PlacedServer(dtype=dtype, B=3, prefix=prefix, pool=-(-prefix // 16) + 6)
    assert s.moves([30, 20, 33], refused=[2]) == bsa.PAGES_EXHAUSTED  # 2 + 2 + 3 of 6 pages
    assert s.moves([1, None, 32]) == 0  # takes the last two, frees two
    assert s.lens.tolist() == [31, 0, 32]
    # as many old tokens as new ones, so that every position exists
    assert s.moves([18, 0, 28], refused=[2]) == bsa.PAGES_EXHAUSTED
    assert s.lens.tolist() == [49, 0, 32]
    assert s.moves([None, 0, 1], refused=[2]) == bsa.PAGES_EXHAUSTED
    assert s.moves([0, 9, 28]) == 0
    assert s.lens.tolist() == [0, 9, 60]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_with_too_few_places(dtype):
    """More new tokens than max_tokens: the ones without a slot are answered with nothing."""
    s = PlacedServer(dtype=dtype, B=3)
    assert s.moves([20, 30, 11], places=45) == bsa.PAGES_TOKENS
    assert s.lens.tolist() == [20, 30, 11]


# as PATHS: each way in which a CTA of the tensor-core kernels can give up
WAITS = [
    (BF16, 64, 8, 2, 32, 100, 5, 1, 40, ["rows64x1"]),
    (BF16, 64, 8, 1, 16, 100, 5, 8, 40, ["rows64x4"]),
    (BF16, 128, 8, 2, 128, 333, 70, 8, 120, ["rows128x2", "merge"]),
    (BF16, 128, 8, 2, 64, 33001, 20, 1, 500, ["tc128", "rows128x1", "merge"]),
    (BF16, 64, 8, 2, 16, 20001, 40, 8, 301, ["tc64", "rows64x2", "merge"]),
    (BF16, 128, 8, 2, 128, 701, 3, 300, 400, ["tc128", "merge"]),
    (BF16, 128, 8, 8, 16, 1500, 20, 70, 300, ["tc128", "merge"]),
    (BF16, 64, 16, 4, 64, 700, 12, 260, 300, ["tc64"]),
    (BF16, 128, 16, 4, 32, 699, 12, 260, 300, ["tc128"]),
]


@pytest.fixture
def no_waiting(bsa_lib):
    """The first wait of each role of a CTA runs out."""
    yield lambda: bsa_lib.bsa_selftest_prefix_timeout(1)
    bsa_lib.bsa_selftest_prefix_timeout(0)


@pytest.mark.parametrize("dtype,d,heads,kv_heads,page,prefix,B,most,own,launched", WAITS)
def test_waits_that_run_out(no_waiting, bsa_lib, dtype, d, heads, kv_heads, page, prefix, B, most,
                            own, launched):
    """The kernels end, the status and NaN in every row say so (the workspace holds the results of
    the call before), and the next call is as the one before."""
    nq, lens = ragged(B + most, B, most, own)
    m = Batch(35, dtype, heads, kv_heads, d, page, prefix, nq, lens, decode=most == 1)
    assert kernels(m.run) == launched
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    need = bsa.prefix_attn_workspace_bytes(dtype, len(m.q), B, heads, kv_heads, d, page,
                                           m.table.shape[1], prefix, m.max_q)
    ws = torch.empty(need, device=DEV, dtype=torch.uint8)
    o, lse = m.run(ws=ws, status=status)
    assert int(status) == 0
    no_waiting()
    lost, lost_lse = m.run(ws=ws, status=status)
    bsa_lib.bsa_selftest_prefix_timeout(0)
    assert int(status) != 0 and torch.isnan(lost).all() and torch.isnan(lost_lse).all()
    status.zero_()
    for _ in range(2):
        again, again_lse = m.run(ws=ws, status=status)
        assert int(status) == 0 and torch.equal(again, o) and torch.equal(again_lse, lse)


FAR = [
    (BF16, 130, 3, 1, 40, ["rows128x1"]), (BF16, 130, 70, 1, 200, ["rows128x1", "merge"]),
    (BF16, 20001, 40, 1, 100, ["tc128", "rows128x1", "merge"]),
    (BF16, 300, 8, 200, 260, ["tc128", "merge"]),
    (F32, 130, 3, 1, 40, ["simt128:32:16"]), (F32, 300, 5, 40, 80, ["simt128:64:64", "merge"]),
]


@pytest.fixture(scope="module")
def far_pool(request):
    """Pools of more than 2^31 elements."""
    P = 270_000
    yield [torch.empty(P, 1, 64, 128, device=DEV, dtype=request.param) for _ in range(2)]


@pytest.mark.parametrize("far_pool,prefix,B,most,own,launched", FAR, indirect=["far_pool"])
def test_prefix_and_own_pages_behind_2_to_the_31_elements(far_pool, prefix, B, most, own, launched):
    nq, lens = ragged(B + most, B, most, own)
    m = Batch(32, far_pool[0].dtype, 8, 1, 128, 64, prefix, nq, lens, decode=most == 1)
    pool = m.k.shape[0]
    far = far_pool[0].shape[0] - 1 - np.arange(pool)  # where the batch's pages go
    to = torch.as_tensor(far, device=DEV)
    for big, small in zip(far_pool, (m.k, m.v)):
        big[to] = small
    m.k, m.v = far_pool
    m.prefix_ids, m.own_ids = far[m.prefix_ids], [far[x] for x in m.own_ids]
    m.prefix_table = to[m.prefix_table.long()].int()
    live = m.table < pool
    m.table = torch.where(live, to[m.table.clamp(max=pool - 1).long()].int(), m.table)
    assert kernels(m.run) == launched
    m.check(*m.run())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_serving_steps_behind_a_long_prefix(dtype):
    """Tables advanced in place, then attention in several kernels, step after step."""
    s = Server(dtype=dtype, prefix=40001, pool=2600)
    run_script(s, SCRIPT, s.step)


def test_captured_steps_behind_a_long_prefix():
    """One captured tick of tables, append and three attention kernels, replayed."""
    s = Server(prefix=40001, pool=2600)
    run_script(s, SCRIPT[:1], s.step)
    one = torch.tensor([1, 1, 1, 1, 0, 0], dtype=torch.int32, device=DEV)
    q, k, v = s.randn(4, s.heads, s.d), s.randn(4, s.kv_heads, s.d), s.randn(4, s.kv_heads, s.d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = s.step(q, k, v, s.lens + one, 4, 1)
    for _ in range(20):
        for x in (q, k, v):
            x.copy_(s.randn(*x.shape))
        g.replay()
        for b in range(4):
            s.record(b, k[b:b + 1], v[b:b + 1])
            want, tol = s.want(b, q[b:b + 1])
            assert ((o[b:b + 1].double() - want).abs() <= tol).all()
    assert int(s.status) == 0
