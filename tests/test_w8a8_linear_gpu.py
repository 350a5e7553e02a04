"""dq_w8a8_linear against its formula.

The sum is exact (checked as a binary64 product of integers below 2^53) and
scale, bias, residual and narrowing are single binary32 roundings, so without
an activation the result is compared bit for bit. An activation of the
binary32 value x is compared with the formula in 64 bits at that x:
  SILU and GELU_TANH, x / (1 + exp(-u)): the exponential is 2^-22 off, and its
  argument, rounded a few times, changes it by 4 |u| 2^-24; the quotient and the
  product add 2^-23: at most (|u| + 8) 2^-22 relative.
  GELU: erfc of an argument z = -x / sqrt 2 that is rounded twice changes by 2 z^2
  2^-23 relative, and erfc itself is within 5 units: at most (x^2 + 8) 2^-22.
Then the residual's rounding and half a step of the output's type. Results
that vanish below 1e-30 are compared absolutely.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


def case(m, n, k, out, bias=F32, residual=False, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    b = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    sa = torch.rand(m, generator=g, device="cuda") + 0.5
    sb = (torch.rand(n, generator=g, device="cuda") + 0.5) * spread / (74.0**2 * math.sqrt(k))
    bi = None if bias is None else torch.randn(n, generator=g, device="cuda").to(bias)
    r = torch.randn(m, n, generator=g, device="cuda").to(out) if residual else None
    return a, b, sa, sb, bi, r


def value(a, b, sa, sb, bias):
    """The binary32 value before the activation, bit for bit."""
    acc = (a.double() @ b.double().t()).to(torch.int64)
    x = acc.to(F32) * (sa[:, None] * sb[None, :])
    return x if bias is None else x + bias.float()


def verify(got, args, act="none"):
    a, b, sa, sb, bias, r = args
    x = value(a, b, sa, sb, bias)
    if act in ("none", "relu"):
        want = x if act == "none" else torch.where(x < 0, 0.0, x)
        if r is not None:
            want = want + r.float()
        assert torch.equal(got, want.to(got.dtype))
        return
    d = x.double()
    if act == "gelu":
        want, rel = d * 0.5 * torch.special.erfc(-d / math.sqrt(2)), (d * d + 8) * 2.0**-22
    else:
        u = d if act == "silu" else 2 * math.sqrt(2 / math.pi) * (d + 0.044715 * d**3)
        want, rel = d / (1 + torch.exp(-u)), (u.abs() + 8) * 2.0**-22
    off = rel * want.abs() + 1e-30
    if r is not None:
        want = want + r.double()
        off = off + 2.0**-24 * (want.abs() + off)
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0**-25 if got.dtype == F16 else 0.0
    bad = (got.double() - want).abs() > half * want.abs() + off * (1 + half) + tiny
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))


SHAPES = [(1, 64, 64), (1, 4096, 1024), (2, 130, 528), (7, 1000, 2048), (8, 257, 4096), (9, 128, 128), (16, 4096, 512),
          (17, 33, 1040), (32, 1024, 7168), (33, 200, 256), (48, 777, 1024), (64, 512, 4096), (65, 512, 512),
          (100, 96, 144), (128, 1000, 1024), (129, 256, 2064), (200, 640, 1024), (256, 300, 512), (257, 513, 1040),
          (500, 1, 96), (512, 1024, 1024), (1000, 2051, 1040), (1, 1, 16), (3, 5, 1), (5, 7, 33), (70, 90, 100),
          (1, 2, 131071), (1, 300, 131056), (130, 140, 131056), (2048, 1536, 256), (1500, 4000, 512)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(dq, m, n, k):
    """No bias, no activation: the product's own bits at every shape, and everything at once."""
    args = case(m, n, k, BF16, residual=True, seed=m + n + k)
    got = dq.w8a8_linear(*args[:4], out_dtype=BF16)
    verify(got, (*args[:4], None, None))
    assert torch.equal(got, dq.w8a8_gemm(*args[:4], out_dtype=BF16))
    verify(dq.w8a8_linear(*args[:4], bias=args[4], residual=args[5], activation="silu"), args, "silu")


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("bias", [None, F32, F16, BF16])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_types(dq, out, bias, m):
    for act in ("none", "relu"):
        for residual in (False, True):
            args = case(m, 520, 1024, out, bias, residual, seed=m)
            verify(dq.w8a8_linear(*args[:4], bias=args[4], residual=args[5], activation=act, out_dtype=out), args, act)


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m,k", [(5, 512), (150, 512), (400, 512), (6, 50)])
@pytest.mark.parametrize("spread", [0.01, 3.0, 40.0])
def test_activations(dq, act, out, m, k, spread):
    """Values from near zero to the far tails."""
    args = case(m, 264, k, out, spread=spread, residual=False, seed=m)
    verify(dq.w8a8_linear(*args[:4], bias=args[4], activation=act, out_dtype=out), args, act)


def test_infinite_and_nan_values(dq):
    """Infinite scales and NaN biases follow the formula: relu keeps NaN, silu(+inf) = inf."""
    for m in (4, 140, 400):
        a, b, sa, sb, bias, _ = case(m, 136, 256, F32, seed=1)
        bias[3], bias[5], bias[6] = math.nan, math.inf, -math.inf
        for act in ("none", "relu", "silu"):
            got = dq.w8a8_linear(a, b, sa, sb, bias=bias, activation=act)
            assert got[:, 3].isnan().all() and (got[:, 5] == math.inf).all()
            rest = [j for j in range(136) if j not in (3, 5, 6)]
            assert got[:, rest].isfinite().all()
        assert (dq.w8a8_linear(a, b, sa, sb, bias=bias, activation="relu")[:, 6] == 0).all()


@pytest.mark.parametrize("m,n", [(5, 264), (64, 1000), (300, 264), (300, 261)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_residual_in_place(dq, m, n, out):
    args = case(m, n, 512, out, residual=True, seed=2)
    stream = args[5].clone()
    got = dq.w8a8_linear(*args[:4], bias=args[4], activation="gelu", residual=stream, out=stream)
    assert got is stream
    verify(stream, args, "gelu")


@pytest.mark.parametrize("m", [3, 60, 300])
def test_unaligned_tensors(dq, m):
    """Operands, output and residual off 16-byte boundaries."""
    args = case(m, 256, 512, BF16, BF16, True, seed=3)
    def odd(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    verify(dq.w8a8_linear(odd(args[0]), odd(args[1]), *args[2:4], bias=odd(args[4]), residual=odd(args[5])), args)
    verify(dq.w8a8_linear(*args[:4], bias=args[4], residual=odd(args[5]), out=odd(args[5])), args)


def test_rows_do_not_depend_on_their_number(dq):
    """Which kernel runs depends on the number of tokens; the bits do not."""
    args = case(600, 520, 1024, BF16, residual=True, seed=4)
    want = dq.w8a8_linear(*args[:4], bias=args[4], residual=args[5], activation="gelu")
    for m in (1, 8, 9, 31, 64, 130, 256, 257):
        got = dq.w8a8_linear(args[0][:m], args[1], args[2][:m], args[3], bias=args[4], residual=args[5][:m],
                             activation="gelu")
        assert torch.equal(got, want[:m])


def test_nothing_to_do(dq):
    args = case(4, 8, 64, F32)
    assert dq.w8a8_linear(args[0][:0], args[1], args[2][:0], args[3], bias=args[4]).shape == (0, 8)
    assert dq.w8a8_linear(args[0], args[1][:0], args[2], args[3][:0], bias=args[4][:0]).shape == (4, 0)


@pytest.mark.parametrize("m", [2, 100, 700])
def test_streams_and_graphs(dq, m):
    args = case(m, 1032, 2048, BF16, residual=True, seed=5)
    want = dq.w8a8_linear(*args[:4], bias=args[4], residual=args[5], activation="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = dq.w8a8_linear(*args[:4], bias=args[4], residual=args[5], activation="silu", stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(g):
        for _ in range(3):
            dq.w8a8_linear(*args[:4], bias=args[4], residual=args[5], activation="silu", out=out)
    other = case(m, 1032, 2048, BF16, residual=True, seed=6)
    args[0].copy_(other[0])
    g.replay()
    torch.cuda.synchronize()
    verify(out, args, "silu")
