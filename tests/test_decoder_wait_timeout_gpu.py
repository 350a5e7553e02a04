"""The bounded waits of the paged attention and linear kernels, made to run out (GPU).

The test build of the library (2 ms limit) leaves one copy out in each kernel:
a tile of key head 0 of sequence 1 in the attention, one K slice of one tile in
each linear kernel. What needed that copy becomes NaN, what did not is exact,
the call ends by itself, and the next call on the same context is exact.
"""

import ctypes

import pytest
import torch

from token_dynamic_quantization_b200 import build as dq_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs(dq_lib, cuda_device):
    """(the product library's helpers, the test build behind the same helpers)."""
    lib = ctypes.CDLL(dq_build.build_wait_test())
    for name in ("dq_w8a8_linear", "dq_paged_attention"):
        getattr(lib, name).argtypes = getattr(dq_lib._lib, name).argtypes
        getattr(lib, name).restype = getattr(dq_lib._lib, name).restype
    return dq_lib, lib


def _both(libs, monkeypatch, f):
    dq, wait = libs
    want = f(dq)

    class Mixed:
        def __getattr__(self, name):
            return getattr(wait if name in ("dq_w8a8_linear", "dq_paged_attention") else real, name)

    real = dq._lib
    monkeypatch.setattr(dq, "_lib", Mixed())
    got = f(dq)
    torch.cuda.synchronize()
    monkeypatch.undo()
    return want, got


# rows, and the outputs that need the missing slice: [rows, columns]
@pytest.mark.parametrize("m,n,rows,cols", [(3, 96, slice(0, 3), slice(16, 32)), (40, 400, slice(0, 40), slice(128, 256)),
                                           (600, 512, slice(256, 512), slice(0, 256)), (600, 511, slice(256, 512), slice(0, 256))])
def test_linear_slice_timeout(libs, monkeypatch, m, n, rows, cols):
    k = 8192
    g = torch.Generator(device="cuda").manual_seed(m)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    b = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    sa, sb = torch.rand(m, generator=g, device="cuda") + 0.5, torch.rand(n, generator=g, device="cuda") + 0.5
    want, got = _both(libs, monkeypatch, lambda dq: dq.w8a8_linear(a, b, sa, sb, activation="silu"))
    bad = got.isnan()
    assert bad.any() and not want.isnan().any()
    needs = torch.zeros_like(bad)
    needs[rows, cols] = True
    assert bad[~needs].sum() == 0 and torch.equal(got[~bad], want[~bad])
    if m > 256:  # tiles may be halved: one half is marked whole
        assert bad[rows, 0:128].all()
    else:
        assert bad[needs].all()
    again = libs[0].w8a8_linear(a, b, sa, sb, activation="silu")
    assert torch.equal(again, want)


@pytest.mark.parametrize("cache", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("lengths", [[300, 2000, 100, 900], [40, 500, 60, 3]])
def test_attention_tile_timeout(libs, monkeypatch, cache, lengths):
    from test_paged_attention_gpu import call, make

    s = make(lengths, 8, 2, 128, torch.bfloat16, cache, 16, seed=3)
    want, got = _both(libs, monkeypatch, lambda dq: call(dq, s))
    bad = got.isnan().all(-1)
    assert got.isnan().any(-1).equal(bad)
    assert bad[1, :4].all()  # the query heads of key head 0 of sequence 1
    # the warp that missed the copy may mark later items of its CTA too, nothing before
    assert not bad[0].any()
    assert torch.equal(got[~bad], want[~bad]) and not want.isnan().any()
    assert torch.equal(call(libs[0], s), want)


@pytest.mark.parametrize("cache", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("longest", [200, 900])
def test_attention_tile_timeout_of_single_warps(libs, monkeypatch, cache, longest):
    from test_paged_attention_gpu import call, make

    s = make([longest - i for i in range(130)], 32, 8, 128, torch.bfloat16, cache, 16, seed=4)
    want, got = _both(libs, monkeypatch, lambda dq: call(dq, s))
    bad = got.isnan().all(-1)
    assert got.isnan().any(-1).equal(bad)
    assert bad[1, :4].all() and not bad[0].any()
    assert torch.equal(got[~bad], want[~bad]) and not want.isnan().any()
    assert torch.equal(call(libs[0], s), want)
