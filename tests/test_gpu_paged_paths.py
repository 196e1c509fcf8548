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
