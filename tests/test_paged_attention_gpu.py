"""dq_paged_attention against softmax attention in 64 bits.

Tolerances, derived from the arithmetic. A score is a binary32 sum of head_dim
products that are exact (16-bit or code times 16-bit), scaled by a few rounded
factors: off by at most ds = (head_dim + 8) * 2^-23 * |scale| sum_c |q_c K_c| (a
sum's rounding may truncate), which changes its weight by the factor exp(ds).
Beside codes a query is first rounded to integers, a power of two times it, of
which the head's largest lies in [16319, 32639]: each channel is off by at most
half a unit, 0.5 / 16319 max_c |q_c|, and ds grows by |scale| 0.5 / 16319 max_c
|q_c| sum_c |K_c|. Next,
the weight's own exponential, and the running rescalings and sums, are within
2^-18 in all. A weight is rounded to u_p relative before it meets its values:
2^-11 for f16 and INT8 caches, 2^-8 for bf16 (less where it is kept in two
parts), and weights below 2^-32 of the largest may vanish: n * 2^-32. With A =
sum_j p_j |V_j|: |out - exact| <= u_out |exact| + (u_p + 2 exp(ds) - 2 + 2^-18 +
n 2^-32 max|V|/A) A, u_out half a step of the output's type.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, I8 = torch.float16, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


def make(lengths, hq, hk, dim, dtype, cache, page, seed=0, spare=3, q_scale=1.5):
    """Inputs with shuffled pages; rows that no token names hold NaN (or wild codes and NaN scales)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lengths = torch.tensor(lengths, dtype=torch.int32)
    counts = (lengths.clamp_min(0) + page - 1) // page
    total, width = int(counts.sum()) + spare, max(1, int(counts.max())) + 1
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), width), -7, dtype=torch.int32, device="cuda")
    used = (torch.arange(width)[None] < counts[:, None]).cuda()
    table[used] = perm[: int(counts.sum())]
    q = (q_scale * torch.randn(len(lengths), hq, dim, generator=g, device="cuda")).to(dtype)
    named = torch.zeros(total, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths.tolist()):
        j = torch.arange(max(n, 0), device="cuda")
        named[table[b].long()[j // page], j % page] = True
    s = dict(q=q, page_table=table, lengths=lengths.cuda(), k_scale=None, v_scale=None)
    for name in ("k", "v"):
        x = torch.randn(total, hk, page, dim, generator=g, device="cuda")
        if cache == I8:
            scale = x.abs().amax(-1) / 127
            codes = torch.round(x / scale[..., None]).to(I8)
            codes.transpose(1, 2)[~named] = -128
            scale.transpose(1, 2)[~named] = math.nan
            s[name + "_cache"], s[name + "_scale"] = codes, scale
        else:
            x = x.to(cache)
            x.transpose(1, 2)[~named] = math.nan
            s[name + "_cache"] = x
    return s


def call(dq, s, **kw):
    return dq.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["k_scale"],
                              s["v_scale"], **kw)


def verify(s, out, lse=None, window=0, sinks=0, scale=None):
    b, hq, dim = s["q"].shape
    hk, page = s["k_cache"].shape[1:3]
    group, codes = hq // hk, s["k_cache"].dtype == I8
    scale = dim**-0.5 if scale is None else scale
    u_p = 2.0**-8 if s["k_cache"].dtype == BF16 else 2.0**-11
    u_out = torch.finfo(out.dtype).eps / 2
    for i, n in enumerate(s["lengths"].tolist()):
        if n <= 0:
            assert (out[i] == 0).all()
            assert lse is None or (lse[i] == -math.inf).all()
            continue
        j = torch.arange(n, device="cuda")
        if window:
            j = j[(j < sinks) | (j >= n - window)]
        at = s["page_table"][i].long()[j // page]
        k, v = s["k_cache"][at, :, j % page].double(), s["v_cache"][at, :, j % page].double()
        if codes:
            k = k * s["k_scale"][at, :, j % page].double()[..., None]
            v = v * s["v_scale"][at, :, j % page].double()[..., None]
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)  # [n, hq, dim]
        q = s["q"][i].double()
        score = torch.einsum("hd,nhd->hn", q, k) * scale
        ds = ((dim + 8) * 2.0**-23 * abs(scale) * torch.einsum("hd,nhd->hn", q.abs(), k.abs())).amax(-1)
        if codes:
            step = 0.5 / 16319 * q.abs().amax(-1) * abs(scale)
            ds = ds + step * k.abs().sum(-1).amax(0)
        p = torch.softmax(score, -1)
        want = torch.einsum("hn,nhd->hd", p, v)
        a = torch.einsum("hn,nhd->hd", p, v.abs())
        off = (u_p + 2 * torch.expm1(ds) + 2.0**-18)[:, None] * a + len(j) * 2.0**-32 * v.abs().amax(0)
        tiny = 2.0**-25 if out.dtype == F16 else 0.0  # half of f16's smallest step
        bad = (out[i].double() - want).abs() > u_out * want.abs() + off * (1 + u_out) + tiny
        assert not bad.any(), (i, n, int(bad.sum()), float(((out[i].double() - want).abs() / a).max()))
        if lse is not None:
            want = torch.logsumexp(score, -1)
            assert ((lse[i].double() - want).abs() <= ds + 2.0**-18 + 2.0**-23 * want.abs()).all()


KINDS = [(BF16, BF16), (F16, F16), (BF16, I8), (F16, I8)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("hq,hk,dim", [(8, 1, 128), (4, 4, 64), (32, 8, 128), (3, 1, 256), (16, 1, 64), (20, 1, 128),
                                       (6, 2, 80), (2, 1, 7), (48, 2, 64), (12, 12, 256), (64, 1, 128)])
def test_heads_and_types(dq, hq, hk, dim, dtype, cache):
    s = make([1, 77, 0, 300, 33, 16], hq, hk, dim, dtype, cache, 16, seed=dim + hq)
    lse = torch.full((6, hq), 7.0, device="cuda")
    verify(s, call(dq, s, lse=lse), lse)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("page", [1, 3, 16, 20, 64, 128, 1000])
def test_pages(dq, page, dtype, cache):
    """Pages that end inside a tile, and shorter or longer than one."""
    s = make([129, 1, 64, 65, 999, 31], 8, 2, 128, dtype, cache, page, seed=page)
    verify(s, call(dq, s))


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1500])
def test_lengths(dq, length, dtype, cache):
    s = make([length], 8, 2, 128, dtype, cache, 16, seed=length)
    lse = torch.empty(1, 8, device="cuda")
    verify(s, call(dq, s, lse=lse), lse)


@pytest.mark.parametrize("dtype,cache,dim", [(BF16, I8, 128), (F16, F16, 64), (BF16, BF16, 256), (BF16, I8, 40)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (50, 3), (64, 200), (5000, 4), (100, 0), (17, 1000), (0, 9)])
def test_windows(dq, window, sinks, dtype, cache, dim):
    s = make([1, 5, 16, 50, 51, 54, 128, 700, 0, 2000], 8, 2, dim, dtype, cache, 20, seed=window)
    lse = torch.empty(10, 8, device="cuda")
    verify(s, call(dq, s, window=window, sinks=sinks, lse=lse), lse, window, sinks)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("lengths,hq,hk,dim", [
    ([20000], 8, 1, 128), ([9000, 1, 0, 3, 12000], 8, 2, 64), ([70000], 4, 4, 64),
    (list(range(0, 4000, 37)), 4, 1, 128), ([5] * 300, 8, 8, 64), ([4097, 4096, 4095] * 20, 16, 2, 128), ([3000, 2], 16, 2, 256)])
def test_long_and_many(dq, lengths, hq, hk, dim, dtype, cache):
    """Sequences that several CTAs share, short ones beside long ones, more rows than CTAs."""
    s = make(lengths, hq, hk, dim, dtype, cache, 64, seed=len(lengths))
    lse = torch.empty(len(lengths), hq, device="cuda")
    verify(s, call(dq, s, lse=lse), lse)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_peaked_and_extreme_scores(dq, dtype, cache):
    """Rising and falling scores far apart (the running maximum moves often), and a scale of zero or below."""
    s = make([600, 600], 8, 2, 128, dtype, cache, 16, seed=5)
    ramp = torch.linspace(-1, 1, 600, device="cuda")
    for i, r in enumerate((ramp, ramp.flip(0))):
        j = torch.arange(600, device="cuda")
        at = s["page_table"][i].long()[j // 16]
        if cache == I8:
            s["k_scale"][at, :, j % 16] *= r.abs()[:, None] + 1e-3
        else:
            s["k_cache"][at, :, j % 16] *= r[:, None, None].to(cache)
    for scale in (5.0, -5.0, 0.0, 1e-4):
        lse = torch.empty(2, 8, device="cuda")
        verify(s, call(dq, s, softmax_scale=scale, lse=lse), lse, scale=scale)


@pytest.mark.parametrize("size", [1e-6, 1e-3, 1.0, 3e4, 1e20])
def test_value_scales(dq, size):
    """INT8 value scales of any size, and tokens whose scales lie ten binades apart."""
    s = make([700], 8, 2, 128, BF16, I8, 16, seed=7)
    s["v_scale"] *= size
    verify(s, call(dq, s))
    s["v_scale"][::3] *= 2.0**-10
    verify(s, call(dq, s))
    s["v_scale"][1::3] = 0
    verify(s, call(dq, s))


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1e4, 1e30])
def test_query_sizes(dq, size):
    """bf16 queries beyond f16's range beside an INT8 cache."""
    s = make([300, 2], 8, 2, 128, BF16, I8, 16, seed=8)
    s["q"] = (s["q"].float() * size).to(BF16)
    verify(s, call(dq, s, softmax_scale=0.088 / size), scale=0.088 / size)
    s["q"][:, ::2] = 0
    verify(s, call(dq, s, softmax_scale=0.088 / size), scale=0.088 / size)


@pytest.mark.parametrize("dim", [128, 40])
@pytest.mark.parametrize("cache", [BF16, I8])
def test_infinite_and_nan_inputs(dq, cache, dim):
    """NaN in a visible row reaches its own sequence and key head only; what is not visible reaches nobody."""
    s = make([100, 100, 100], 4, 2, dim, BF16, cache, 16, seed=9)
    page, row = int(s["page_table"][1, 2]), 5  # token 37 of sequence 1
    if cache == I8:
        s["k_scale"][page, 1, row] = math.nan
    else:
        s["k_cache"][page, 1, row, 3] = math.nan
    out = call(dq, s)
    assert out[1, 2:].isnan().all()
    assert out[[0, 2]].isfinite().all() and out[1, :2].isfinite().all()
    out = call(dq, s, window=60, sinks=4)  # token 37 is hidden: 100 - 60 = 40
    verify(s, out, window=60, sinks=4)


@pytest.mark.parametrize("dim", [128, 40])
def test_bad_pages_and_lengths_give_nan_rows(dq, dim):
    """Entries outside the cache, and lengths beyond the table, are not followed; their rows are NaN."""
    s = make([100, 90, 80, 70], 4, 2, dim, BF16, I8, 16, seed=10)
    s["page_table"][0, 3] = -1
    s["page_table"][1, 5] = s["k_cache"].shape[0]
    s["lengths"][2] = s["page_table"].shape[1] * 16 + 1
    lse = torch.zeros(4, 4, device="cuda")
    out = call(dq, s, lse=lse)
    assert out[:3].isnan().all() and lse[:3].isnan().all()
    assert out[3].isfinite().all() and lse[3].isfinite().all()
    s["lengths"][2] = 2**31 - 1
    assert call(dq, s)[2].isnan().all()
    s["page_table"][0, 3] = 2**31 - 1
    assert call(dq, s)[0].isnan().all()
    out = call(dq, s, window=20)  # page 3 (tokens 48-63) of sequence 0 is not visible any more
    assert out[0].isfinite().all()


def test_strided_queries_and_scalar_path(dq):
    """q as a slice of a wider row, at an odd element offset, and caches that are not 16-byte aligned."""
    s = make([100, 33, 0], 8, 2, 128, BF16, BF16, 16, seed=11)
    want = call(dq, s)
    wide = torch.zeros(3, 12, 128, dtype=BF16, device="cuda")
    wide[:, 2:10] = s["q"]
    t = dict(s, q=wide[:, 2:10])
    assert torch.equal(call(dq, t), want)
    odd = torch.zeros(3 * 8 * 128 + 1, dtype=BF16, device="cuda")[1:].view(3, 8, 128)
    odd.copy_(s["q"])
    verify(s, call(dq, dict(s, q=odd)))
    for name in ("k_cache", "v_cache"):
        c = s[name]
        o = torch.empty(c.numel() + 1, dtype=c.dtype, device="cuda")[1:].view(c.shape)
        o.copy_(c)
        verify(s, call(dq, dict(s, **{name: o})))


def test_the_same_bytes_every_time(dq):
    s = make([30000, 5, 777, 1234] * 3, 32, 8, 128, BF16, I8, 16, seed=12)
    first = call(dq, s)
    for _ in range(5):
        assert torch.equal(call(dq, s), first)


def test_pages_shared_by_sequences(dq):
    """Two sequences with a common prefix point at the same pages."""
    s = make([96, 96], 8, 2, 128, BF16, I8, 16, seed=13)
    s["page_table"][1, :4] = s["page_table"][0, :4]
    verify(s, call(dq, s))


def test_workspace_streams_and_graphs(dq):
    s = make([9000, 40, 0, 3000], 8, 2, 128, BF16, I8, 16, seed=14)
    want = call(dq, s)
    bytes_ = dq.dq_paged_attention_get_workspace_size(4, 8, 2, 128, dq.DQ_INT8)
    ws = torch.full((max(bytes_, 16),), 255, dtype=torch.uint8, device="cuda")  # no clearing needed
    assert torch.equal(call(dq, s, workspace=ws), want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = call(dq, s, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(g):
        call(dq, s, out=out, workspace=ws)
    for n in ([100, 40, 0, 3000], [1, 1, 0, 1], [8999, 0, 0, 17], [9000, 40, 0, 3000]):  # lengths move between replays
        s["lengths"].copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        verify(s, out)


def test_empty_batch(dq):
    s = make([3], 8, 2, 128, BF16, I8, 16)
    out = dq.paged_attention(s["q"][:0], s["k_cache"], s["v_cache"], s["page_table"][:0], s["lengths"][:0],
                             s["k_scale"], s["v_scale"])
    assert out.shape == (0, 8, 128)
