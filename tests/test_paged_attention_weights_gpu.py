"""How many bits of a weight dq_paged_attention's products keep (GPU).

The first of every 16 tokens has one score, all others 0: their weight is one number, just
below the middle between two of 16 bits, whose rounding would scale the result as a whole, and
values of one sign hide nothing of it. Bound, relative to the result (all values are positive): half
a step of the output; the weight's bits, 2^-16 beside bf16 caches (a bf16 and a bf16 of the
rest), 2^-20 where f16 is kept in two parts, 2^-11 beside INT8 caches with bf16 outputs; 2^-18 for
exponential, rescalings and sums; the score, a binary32 sum of head_dim equal products and beside
codes of an exact query, (head_dim + 8) 2^-23 of it; and beside codes 2^-13 sum_j p_j v_j for
the 128s that are added to them and taken off again.
"""

import math

import pytest
import torch

from test_paged_attention_gpu import BF16, F16, I8, KINDS, call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("dim,group", [(128, 1), (128, 12), (64, 4), (64, 16), (256, 2)])
@pytest.mark.parametrize("page", [16, 20])
def test_bits_of_a_weight(dq, dim, group, page, dtype, cache):
    n = 400
    s = make([n], group, 1, dim, dtype, cache, page, seed=dim + group)
    s["q"].fill_(0.5)
    j = torch.arange(n, device="cuda")
    at = s["page_table"][0].long()[j // page], 0, j % page
    first = j % 16 == 0
    if cache == I8:
        s["k_cache"][at] = first.to(I8)[:, None].expand(-1, dim)
        s["k_scale"][at] = s["v_scale"][at] = torch.ones(n, device="cuda")
        s["v_cache"][at] = s["v_cache"][at].abs().clamp(min=5)
    else:
        s["k_cache"][at] = first.to(cache)[:, None].expand(-1, dim)
        s["v_cache"][at] = s["v_cache"][at].abs() + 0.125
    v = s["v_cache"][at].double()
    bits = 2.0**-16 if cache == BF16 else (2.0**-11 if cache == I8 and dtype == BF16 else 2.0**-20)
    for whole in (1, 2, 3):
        log2 = whole - math.log2(1 + 0.97 * (2.0**-8 if cache == BF16 else 2.0**-11))
        scale = float(torch.tensor(log2 * math.log(2) / (0.5 * dim), dtype=torch.float32))
        score = torch.where(first, 0.5 * dim * scale, 0.0).double()
        p = torch.softmax(score, 0)
        want = p @ v
        off = want * (bits + 2.0**-18 + 2 * float(score[0]) * (dim + 8) * 2.0**-23)
        if cache == I8:
            off = off + 2.0**-13
        step = torch.finfo(dtype).eps / 2 * torch.exp2(torch.floor(torch.log2(want + off)))
        got = call(dq, s, softmax_scale=scale)[0].double()
        bad = (got - want).abs() > step + off
        assert not bad.any(), (whole, float(((got - want).abs() / want).max()))
