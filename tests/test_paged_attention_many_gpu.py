"""dq_paged_attention with so many items that a warp takes each by itself (GPU).

The same formula, inputs and tolerances as in test_paged_attention_gpu.py: a
batch of a hundred and more sequences with 8 key heads leaves every SM several
(sequence, key head) items, whole ones where the page table is short, ranges of
them where it is long.
"""

import math

import pytest
import torch

from test_paged_attention_gpu import BF16, F16, I8, KINDS, call, make, verify

pytestmark = pytest.mark.gpu

HK = 8


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


def ragged(batch, longest, seed):
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(0, longest + 1, (batch,), generator=g)
    n[:6] = torch.tensor([0, 1, longest, 15, 16, -3])
    return n.tolist()


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("longest", [5, 60, 230, 700])
@pytest.mark.parametrize("dim,group", [(64, 4), (64, 16), (128, 1), (128, 12), (256, 2)])
def test_many_items(dq, dtype, cache, longest, dim, group):
    s = make(ragged(130, longest, dim + longest), HK * group, HK, dim, dtype, cache, 16, seed=longest)
    lse = torch.empty(130, HK * group, device="cuda")
    out = call(dq, s, lse=lse)
    verify(s, out, lse)
    assert torch.equal(call(dq, s), out)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("page", [1, 5, 32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (300, 20)])
def test_many_pages_and_windows(dq, dtype, cache, page, window, sinks):
    s = make(ragged(120, 500, page), 16, HK, 128, dtype, cache, page, seed=page)
    verify(s, call(dq, s, window=window, sinks=sinks), window=window, sinks=sinks)


def test_more_heads_than_a_set(dq):
    s = make(ragged(20, 300, 3), 200, 2, 128, BF16, I8, 16, seed=4)  # 100 query heads to a key head
    verify(s, call(dq, s))
    s = make(ragged(400, 40, 3), 96, 4, 64, F16, F16, 16, seed=5)
    verify(s, call(dq, s))


@pytest.mark.parametrize("cache", [I8, BF16])
@pytest.mark.parametrize("longest", [60, 700])
def test_bad_pages_stay_with_their_sequence(dq, cache, longest):
    s = make(ragged(130, longest, 8), 16, HK, 128, BF16, cache, 16, seed=9)
    s["page_table"][2, 0] = -1
    s["page_table"][10, 0] = 2**31 - 1
    s["lengths"][10] = longest
    s["lengths"][20] = 2**31 - 1
    out = call(dq, s)
    bad = torch.zeros(130, dtype=torch.bool, device="cuda")
    bad[[2, 10, 20]] = True
    assert out[bad].isnan().all()
    # the others hold their formula (lengths move the cuts, so not the same bytes as beside other lengths)
    verify({k: (v[~bad] if k in ("q", "page_table", "lengths") else v) for k, v in s.items()}, out[~bad])


@pytest.mark.parametrize("longest", [60, 700])
def test_rows_do_not_depend_on_the_batch(dq, longest):
    s = make(ragged(130, longest, 12), 16, HK, 128, BF16, I8, 16, seed=13)
    whole = call(dq, s)
    part = {k: (v[:7] if k in ("q", "page_table", "lengths") else v) for k, v in s.items()}
    few = call(dq, part)
    verify(part, few)
    verify(part, whole[:7].contiguous())


def test_captured_with_a_long_queue(dq):
    s = make(ragged(130, 700, 14), 16, HK, 128, F16, I8, 16, seed=15)
    want = call(dq, s)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = [call(dq, s) for _ in range(8)]
        for _ in range(3):
            for o in outs:
                o.fill_(math.nan)
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
