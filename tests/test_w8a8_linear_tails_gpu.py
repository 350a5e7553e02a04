"""dq_w8a8_linear's activations over their tails, against the bounds that dq.h states (GPU).

A product of zero plus a bias is the bias itself, so x is exact. Relative to the value: (x^2 + 8)
2^-22 for GELU, (|u| + 8) 2^-22 for x / (1 + exp(-u)); values below 2^-119 may be zero (never
larger than the value by more than the bound).
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


# the kernels for 8 tokens, 128 tokens, more (32-column rows and turned ones), and any k
@pytest.mark.parametrize("m,n,k", [(1, 8192, 16), (40, 8192, 16), (200, 8192, 16), (200, 8191, 16), (3, 8192, 5)])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_tails(dq, m, n, k, act):
    a, b = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(n, k, dtype=torch.int8, device="cuda")
    ones = torch.ones(max(m, n), device="cuda")
    for low, high in ((-120.0, 20.0), (-14.0, 0.0), (-0.01, 0.01), (1e30, 3e38), (-3e38, -1e3)):
        x = torch.linspace(low, high, n, dtype=torch.float64).float().cuda()
        got = dq.w8a8_linear(a, b, ones[:m], ones[:n], bias=x, activation=act).double()
        d = x.double()
        if act == "gelu":
            # x Phi(x), Phi through its logarithm where it is below binary64's range as well
            want, rel = d * torch.exp(torch.special.log_ndtr(d)), (d * d + 8) * 2.0**-22
        else:
            u = d if act == "silu" else 2 * math.sqrt(2 / math.pi) * (d + 0.044715 * d**3)
            want, rel = d * torch.sigmoid(u), (u.abs() + 8) * 2.0**-22
        want, rel = want.expand_as(got), rel.expand_as(got)
        small = want.abs() < 2.0**-119
        assert not got.isnan().any()
        bad = (got - want).abs() > (rel * want.abs()).clamp(min=2.0**-149)
        assert not (bad & ~small).any(), (low, int((bad & ~small).sum()))
        assert (got[small].abs() <= 2.0**-119 * (1 + 2.0**-10)).all()
