"""The pair kernel of dq_w8a8_linear leaves nothing behind when its CTAs exit (GPU).

Its last tensor-core commits arrive on barriers in both CTAs of a pair, and both wait for them
before they leave: shared memory that a later CTA owns is never written. Products of one K slice
and of a few, whose commits come last of all, run back to back with kernels that fill the same
SMs' shared memory at once (few-token products, 9- to 128-token products and the pair kernel
itself), over and over; every result has to be the same bytes as alone.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


@pytest.mark.parametrize("n", [512, 515])
@pytest.mark.parametrize("k", [16, 128, 640, 896])
def test_back_to_back(dq, k, n):
    g = torch.Generator(device="cuda").manual_seed(k + n)
    codes = lambda r: torch.randint(-127, 128, (r, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)  # noqa: E731
    tokens = (4000, 3, 700, 100, 300)  # the pair kernel, and the two others between its calls
    a, b = codes(max(tokens)), codes(n)
    sa, sb = torch.rand(max(tokens), generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")

    def run(m):
        return dq.w8a8_linear(a[:m], b, sa[:m], sb, activation="relu", out_dtype=torch.bfloat16)

    alone = []
    for m in tokens:
        alone.append(run(m))
        torch.cuda.synchronize()
    want = (a.double() @ b.double().T).float() * (sa[:, None] * sb[None])
    assert torch.equal(alone[0], want[:4000].relu().to(torch.bfloat16))
    for _ in range(10):
        got = [run(m) for _ in range(6) for m in tokens]
        for i, x in enumerate(got):
            assert torch.equal(x, alone[i % len(tokens)])
