"""Which kernels a paged batch takes, read from the kernel nodes of a captured call: the cases
that are meant for one form of msa_shared_attend take it, and every instance of its kernels
(query heads per key head, rows of a unit, form) runs against the definition in 64 bits."""
import re

import pytest
import torch
from cuda.bindings import driver

import test_gpu_paged as cases
import top_kv_routing_b200 as msa
from paged_ref import Batch

pytestmark = pytest.mark.gpu


def _do(result):
    assert result[0] == driver.CUresult.CUDA_SUCCESS, result[0]
    return result[1]


def kernels_of(call):
    """Names of the kernels that `call` enqueues on the stream it is given, in order of launch."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        call(stream)
    raw = driver.CUgraph(graph.raw_cuda_graph())
    _, _, count = driver.cuGraphGetNodes(raw)
    err, nodes, count = driver.cuGraphGetNodes(raw, count)
    assert err == driver.CUresult.CUDA_SUCCESS and count == len(nodes)
    names = []
    for node in nodes:
        assert _do(driver.cuGraphNodeGetType(node)) == driver.CUgraphNodeType.CU_GRAPH_NODE_TYPE_KERNEL
        p = _do(driver.cuGraphKernelNodeGetParams(node))
        name = driver.cuFuncGetName(p.func) if int(p.func) else driver.cuKernelGetName(p.kern)
        names.append(_do(name).decode())
    return names


def forms(x):
    """The kernels of one call of a batch: rows<G, 8-row tiles, joins the memory>, memory<G>, blocks<G>."""
    x.call_attend(msa)  # (allocates the workspace)
    found = []
    for name in kernels_of(lambda s: x.call_attend(msa, stream=s)):
        m = re.search(r"rows_kernelILi(\d)ELi(\d)ELb(\d)E", name)
        t = re.search(r"tile_kernelILi(\d)ELb(\d)E", name)
        assert m or t, name
        found.append(("rows", int(m[1]), int(m[2]), m[3] == "1") if m
                     else ("blocks" if t[2] == "1" else "memory", int(t[1])))
    return found


@pytest.mark.parametrize("name", list(cases.CASES))
def test_small_batches_take_the_row_form(name):
    x = Batch(seed=5, **cases.CASES[name])
    assert [f[0] for f in forms(x)] == ["rows"] and not forms(x)[0][3]


@pytest.mark.parametrize("name", list(cases.BLOCKS))
def test_long_blocks_take_the_block_form(name):
    x = Batch(seed=21, **cases._wide(cases.BLOCKS[name]))
    assert forms(x) == [("blocks", x.G)]


@pytest.mark.parametrize("name", list(cases.MANY_ROWS))
def test_many_rows_take_the_memory_form(name):
    x = Batch(seed=21, **cases._wide(cases.MANY_ROWS[name]))
    found = forms(x)
    assert [f[0] for f in found] == ["memory", "rows"] and found[1][3]


@pytest.mark.parametrize("G,new", [(4, 70), (2, 140), (8, 33)])
def test_blocks_of_values_that_are_not_finite(G, new):
    x = Batch([new] * 24, [(37 * b) % 150 for b in range(24)], L=2, H=16, G=G, page=32, groups=[0, 24], mem=[130])
    assert forms(x) == [("blocks", G)]


@pytest.mark.parametrize("G,new", [(4, 20), (1, 100), (8, 33), (2, 64)])
def test_one_row_tile(G, new):
    past = [0, 100, 128 - new, 129, 300, 513, 40, 700, 1, 255]
    x = Batch([new] * 10, past, L=4, H=16, G=G, page=16, groups=[0, 3, 6, 10], mem=[0, 128, 200])
    assert forms(x) == [("blocks", G)]


@pytest.mark.parametrize("B", [511, 513])
def test_blocks_of_many_sequences(B):
    x = Batch([17 + b % 3 for b in range(B)], [(11 * b) % 29 for b in range(B)], H=1, G=8, groups=[0, 5, B - 1],
              mem=[3, 20])
    assert forms(x) == [("blocks", 8)]


# The memory form for every number of query heads per key head and both sizes of the row kernel's
# units: groups of at most one row tile (128 / G tokens), of just more, and of several pairs.
@pytest.mark.parametrize("G,tiles,new,groups,mem", [
    (1, 1, [1] * 258, [0, 128, 257], [300, 150]),
    (1, 1, [1] * 430, [0, 129, 130, 430], [300, 1, 260]),
    (1, 2, [i % 40 for i in range(60)], [0, 30, 59], [400, 150]),
    (2, 1, [1] * 130, [0, 64, 129, 130], [300, 150, 20]),
    (2, 1, [1] * 200, [2, 65, 200], [0, 700]),
    (2, 2, [i % 12 for i in range(60)], [0, 30, 60], [400, 150]),
    (4, 1, [1] * 70, [0, 32, 65, 70], [130, 257, 64]),
    (4, 2, [i % 7 for i in range(50)], [1, 9, 50], [513, 100]),
    (8, 1, [1] * 53 + [0] * 7, [0, 16, 33, 60], [130, 257, 64]),
    (8, 2, [i % 4 for i in range(50)], [1, 9, 50], [513, 100]),
])
def test_memory_form(G, tiles, new, groups, mem):
    x = Batch(new, [(7 * b) % 61 for b in range(len(new))], L=4, H=16, G=G, groups=groups, mem=mem, pad=2, lead=1, seed=51)
    assert forms(x) == [("memory", G), ("rows", G, tiles, True)]
    x.out.fill_(7.0)
    x.call_attend(msa)
    x.check()
    assert x.err.item() == 0
    first = x.out.clone()
    x.call_attend(msa)
    assert torch.equal(first.view(torch.int16), x.out.view(torch.int16))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("tiles,new", [(1, 1), (2, 20)])
def test_row_form(G, tiles, new):
    new = new if tiles == 2 else max(1, 8 // G)
    x = Batch([new, new - 1 or 1, new], [40, 3, 129], L=2, H=2, G=G, groups=[0, 2], mem=[33], seed=52)
    assert forms(x) == [("rows", G, tiles, False)]
    x.out.fill_(7.0)
    x.call_attend(msa)
    x.check()
