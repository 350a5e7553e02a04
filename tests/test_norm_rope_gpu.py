"""dq_qk_norm_rope and dq_qk_norm_rope_cache against the formula in 64 bits.

Tolerances, derived from the arithmetic: norm and rotation run in binary32
with about ten roundings on each of the two terms of a rotated channel (the
sum of squares, rsqrt, two products, cos or sin of an angle whose remainder in
units of pi is rounded once, the product and the sum), so the value before the
output's rounding is off by at most 16 * 2^-24 * (|y_a| + |y_b|) = 2^-20 (|y_a| +
|y_b|), y the normed pair. The output adds half a step of its type (and half
the smallest step, for f16 results below its normal range). A code's scale is
the largest such value / 127, and (|y_a| + |y_b|) <= 2 max|row|, so the scale
is within 2^-19 + 2^-24 relative, and a code within 1/2 + 127 * 2^-18 of y /
scale.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


def _inv_freq(rope_dim, device="cuda"):
    if rope_dim == 0:
        return None
    return (10000.0 ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)).float().to(device)


def _case(tokens, hq, hk, dim, dtype, rope_dim, wdtype=F32, seed=0, span=1000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(tokens, hq + 2 * hk, dim, generator=g, device="cuda").to(dtype)
    w = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(wdtype) for _ in range(2)]
    pos = torch.randint(0, span, (tokens,), generator=g, device="cuda").to(torch.int32)
    q, k, v = qkv.split([hq, hk, hk], dim=1)
    return q, k, v, pos, _inv_freq(rope_dim), w


def exact(x, weight, pos, inv_freq, eps, interleaved):
    """(result, |y_a| + |y_b| per channel) in binary64."""
    x = x.double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double()
    out, size = y.clone(), y.abs()
    if inv_freq is not None:
        r = 2 * inv_freq.numel()
        i = torch.arange(r // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        angle = pos.double()[:, None, None] * inv_freq.double()
        ya, yb = y[..., a], y[..., b]
        out[..., a] = ya * angle.cos() - yb * angle.sin()
        out[..., b] = yb * angle.cos() + ya * angle.sin()
        size[..., a] = size[..., b] = ya.abs() + yb.abs()
    return out, size


def check(got, want, size):
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    bad = (got.double() - want).abs() > half * want.abs() + 2.0**-20 * size * (1 + half) + tiny
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


SHAPES = [
    # tokens, q heads, kv heads, dim, rope_dim, interleaved
    (1, 32, 8, 128, 128, False), (5, 4, 1, 64, 64, False), (33, 6, 2, 128, 64, False), (7, 3, 3, 96, 96, True),
    (300, 8, 8, 128, 128, True), (17, 5, 5, 256, 256, False), (9, 2, 1, 80, 40, False), (9, 2, 1, 80, 80, False),
    (4, 3, 1, 20, 10, False), (4, 1, 1, 1, 0, False), (3, 2, 2, 7, 6, True), (11, 2, 1, 256, 0, False),
    (6, 7, 1, 32, 32, False), (2, 2, 1, 16, 16, False), (65, 12, 4, 96, 48, True), (3, 1, 1, 248, 200, False),
    (1200, 16, 2, 64, 64, False),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,hq,hk,dim,rope_dim,interleaved", SHAPES)
def test_norm_rope(dq, tokens, hq, hk, dim, rope_dim, interleaved, dtype):
    q, k, _, pos, freq, (qw, kw) = _case(tokens, hq, hk, dim, dtype, rope_dim)
    q_out, k_out = dq.qk_norm_rope(q, k, pos, freq, qw, kw, epsilon=1e-5, interleaved=interleaved)
    assert q_out.shape == q.shape and q_out.is_contiguous() and k_out.shape == k.shape
    check(q_out, *exact(q, qw, pos, freq, 1e-5, interleaved))
    check(k_out, *exact(k, kw, pos, freq, 1e-5, interleaved))


@pytest.mark.parametrize("wdtype", [F16, BF16, F32, None])
def test_weight_types(dq, wdtype):
    q, k, _, pos, freq, (qw, kw) = _case(6, 4, 2, 128, BF16, 128, wdtype=wdtype or F32)
    if wdtype is None:
        qw = kw = None
    q_out, k_out = dq.qk_norm_rope(q, k, pos, freq, qw, kw)
    check(q_out, *exact(q, qw, pos, freq, 1e-6, False))
    check(k_out, *exact(k, kw, pos, freq, 1e-6, False))


def test_far_and_negative_positions(dq):
    """Positions up to the int32 limits: the angle is reduced in binary64.

    At 2^31 the binary64 product of angle / pi has 2^-53 * 2^31 / pi * 3 roundings
    < 2^-21 of error, times pi: below 2^-19 of a radian; at 2^24 below 2^-26."""
    q, k, _, pos, freq, (qw, kw) = _case(64, 2, 1, 128, BF16, 128)
    pos[:32] = torch.arange(32, device="cuda", dtype=torch.int32) + (1 << 24) - 16
    pos[32], pos[33], pos[34] = 2**31 - 1, -(2**31), -5
    q_out, _ = dq.qk_norm_rope(q, k, pos, freq, qw, kw)
    want, size = exact(q, qw, pos, freq, 1e-6, False)
    near = pos.abs().double() < 2**25
    near[33] = False
    check(q_out[near], want[near], size[near])
    far = ~near
    assert ((q_out[far].double() - want[far]).abs() <= 2.0**-8 * want[far].abs() + (2.0**-19 + 2.0**-20) * size[far]).all()


def test_zero_and_large_rows(dq):
    """A row of zeros stays zero (epsilon keeps it finite); f16 rows at the type's largest value do not overflow."""
    q, k, _, pos, freq, _ = _case(4, 2, 1, 128, F16, 128)
    q = q.clone()
    q[0] = 0
    q[1] = 60000
    q[2] = 6e-8
    q_out, _ = dq.qk_norm_rope(q, k, pos, freq)
    assert (q_out[0] == 0).all()
    check(q_out, *exact(q, None, pos, freq, 1e-6, False))


def test_strides_offsets_and_in_place(dq):
    """Slices of a wider buffer, an odd element offset (scalar path), outputs over the inputs."""
    q, k, _, pos, freq, (qw, kw) = _case(37, 4, 2, 128, BF16, 128)
    want_q, want_k = dq.qk_norm_rope(q.contiguous(), k.contiguous(), pos, freq, qw, kw)
    a = dq.qk_norm_rope(q, k, pos, freq, qw, kw)
    assert torch.equal(a[0], want_q) and torch.equal(a[1], want_k)
    buf = torch.zeros(37 * 6 * 128 + 3, dtype=BF16, device="cuda")[3:].view(37, 6, 128)
    qs, ks = buf[:, :4], buf[:, 4:]
    qs.copy_(q)
    ks.copy_(k)
    b = dq.qk_norm_rope(qs, ks, pos, freq, qw, kw)
    check(b[0], *exact(q, qw, pos, freq, 1e-6, False))
    check(b[1], *exact(k, kw, pos, freq, 1e-6, False))
    dq.qk_norm_rope(qs, ks, pos, freq, qw, kw, out=(qs, ks))
    assert torch.equal(qs, b[0]) and torch.equal(ks, b[1])
    qa, ka = q.clone(), k.clone()
    dq.qk_norm_rope(qa, ka, pos, freq, qw, kw, out=(qa, ka))
    assert torch.equal(qa, want_q) and torch.equal(ka, want_k)


def test_rows_do_not_depend_on_their_neighbours(dq):
    q, k, _, pos, freq, (qw, kw) = _case(400, 32, 8, 128, BF16, 128)
    many = dq.qk_norm_rope(q, k, pos, freq, qw, kw)
    for t in (0, 1, 399):
        one = dq.qk_norm_rope(q[t : t + 1], k[t : t + 1], pos[t : t + 1], freq, qw, kw)
        assert torch.equal(one[0], many[0][t : t + 1]) and torch.equal(one[1], many[1][t : t + 1])


def test_no_tokens(dq):
    q, k, _, pos, freq, _ = _case(0, 4, 2, 64, BF16, 64)
    q_out, k_out = dq.qk_norm_rope(q, k, pos, freq)
    assert q_out.shape == (0, 4, 64) and k_out.shape == (0, 2, 64)


def _cache(pages, hk, page, dim, dtype):
    if dtype == I8:
        mk = lambda: torch.full((pages, hk, page, dim), 77, dtype=I8, device="cuda")  # noqa: E731
        ms = lambda: torch.full((pages, hk, page), -3.0, device="cuda")  # noqa: E731
        return mk(), mk(), ms(), ms()
    mk = lambda: torch.full((pages, hk, page, dim), 77, dtype=dtype, device="cuda")  # noqa: E731
    return mk(), mk(), None, None


@pytest.mark.parametrize("cache", ["same", "int8"])
@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("tokens,hq,hk,dim,rope_dim,interleaved",
                         [SHAPES[0], SHAPES[2], SHAPES[6], SHAPES[8], SHAPES[14], SHAPES[5], (700, 8, 2, 128, 128, False)])
def test_cache_rows(dq, tokens, hq, hk, dim, rope_dim, interleaved, page, cache):
    """Named rows get the key and value (codes: the dynamic quantizer's own for the values), all others stay."""
    q, k, v, pos, freq, (qw, kw) = _case(tokens, hq, hk, dim, BF16, rope_dim, seed=tokens)
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))[:tokens]
    slots = slots.clone()
    if tokens > 4:  # padding and out-of-range slots write nothing
        slots[1], slots[2], slots[3] = -1, pages * page, 2**62
    kc, vc, ks, vs = _cache(pages, hk, page, dim, I8 if cache == "int8" else BF16)
    q_out = dq.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc, vc, ks, vs, qw, kw, epsilon=1e-5,
                                  interleaved=interleaved)
    check(q_out, *exact(q, qw, pos, freq, 1e-5, interleaved))
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live]
    page_of, row_of = at // page, at % page
    touched = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    touched[page_of, row_of] = True
    for c in (kc, vc):
        assert (c.transpose(1, 2)[~touched] == 77).all()
    want, size = exact(k, kw, pos, freq, 1e-5, interleaved)
    if cache == "same":
        check(kc[page_of, :, row_of], want[live], size[live])
        assert torch.equal(vc[page_of, :, row_of], v[live])
        return
    for s in (ks, vs):
        assert (s.transpose(1, 2)[~touched] == -3.0).all()
    vq, vsc, _, _ = dq.dynamic_quant(v.contiguous())
    assert torch.equal(vc[page_of, :, row_of], vq[live]) and torch.equal(vs[page_of, :, row_of], vsc[live])
    scale = want.abs().amax(-1) / 127
    got_scale = ks[page_of, :, row_of].double()
    assert ((got_scale - scale[live]).abs() <= (2.0**-19 + 2.0**-23) * scale[live]).all()
    codes = kc[page_of, :, row_of].double()
    assert ((codes - want[live] / scale[live].clamp_min(1e-300)[..., None]).abs() <= 0.5 + 127 * 2.0**-18).all()


def test_cache_zero_rows(dq):
    """A value row of zeros: scale 0 and codes 0, as the dynamic quantizer writes them."""
    q, k, v, pos, freq, _ = _case(3, 2, 2, 64, F16, 64)
    k, v = k.clone(), v.clone()
    k[1] = 0
    v[2] = 0
    kc, vc, ks, vs = _cache(1, 2, 4, 64, I8)
    dq.qk_norm_rope_cache(q, k, v, pos, freq, torch.arange(3, device="cuda"), kc, vc, ks, vs)
    assert (kc[0, :, 1] == 0).all() and (ks[0, :, 1] == 0).all()
    assert (vc[0, :, 2] == 0).all() and (vs[0, :, 2] == 0).all()


def test_streams_and_graphs(dq):
    """A call on a side stream, and one captured and replayed on new inputs, give the eager call's bytes."""
    q, k, v, pos, freq, (qw, kw) = _case(130, 8, 2, 128, BF16, 128)
    want = dq.qk_norm_rope(q, k, pos, freq, qw, kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = dq.qk_norm_rope(q, k, pos, freq, qw, kw, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    kc, vc, ks, vs = _cache(9, 2, 16, 128, I8)
    slots = torch.arange(130, device="cuda")
    sq, sk, sv = q.contiguous(), k.contiguous(), v.contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dq.qk_norm_rope_cache(sq, sk, sv, pos, freq, slots, kc, vc, ks, vs, qw, kw)
    q2, k2, v2, _, _, _ = _case(130, 8, 2, 128, BF16, 128, seed=9)
    sq.copy_(q2), sk.copy_(k2), sv.copy_(v2)
    g.replay()
    torch.cuda.synchronize()
    kc2, vc2, ks2, vs2 = _cache(9, 2, 16, 128, I8)
    want = dq.qk_norm_rope_cache(q2, k2, v2, pos, freq, slots, kc2, vc2, ks2, vs2, qw, kw)
    for a, b in ((out, want), (kc, kc2), (vc, vc2), (ks, ks2), (vs, vs2)):
        assert torch.equal(a, b)
