"""dq_paged_attention beside INT8 caches whose value scales differ by anything (GPU).

Bound, derived from the arithmetic. With p_j the softmax weights, v_j the value scales and
e_j the relative error of weight j: a score is off by at most
  d_j = |scale| ((head_dim + 8) 2^-23 sum_c |q_c K_jc| + 0.5 / 16319 max_c |q_c| sum_c |K_jc|)
(binary32 sums; the query as integers of which the head's largest is at least 16319), its
exponential's argument is rounded twice, 2^-23 |s_j - max s|, and exponential and rescalings are
within 2^-18: e_j = expm1(d_j + 2^-23 |s_j - max s|) + 2^-18. A weight times its value scale is
rounded to f16's 11 bits, 2^-11 at most (a half step would be 2^-12; a subnormal one's
half step is 2^-25, where the largest such product stands at 2^6 at least: 2^-31 of it, for each
token). The codes enter as code + 128 <= 255, and the sum of two tiles (four products at
most) is rounded down by 2^-23 of itself each time before the 128s are taken off: 4 * 2^-23 * 2^8
sum_j p_j v_j. So
  |out - exact| <= sum_j p_j (e_j + 2^-11) |V_j| + sum_j p_j e_j |exact|
                   + 2^-13 sum_j p_j v_j + n 2^-31 128 max_j p_j v_j + half a step of the output.
"""

import math

import pytest
import torch

from test_paged_attention_gpu import BF16, F16, I8, call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


def check(s, out, rows=None):
    b, hq, dim = s["q"].shape
    hk, page = s["k_cache"].shape[1:3]
    scale = dim**-0.5
    for i, n in enumerate(s["lengths"].tolist()):
        if n <= 0 or (rows is not None and i not in rows):
            continue
        j = torch.arange(n, device="cuda")
        at = s["page_table"][i].long()[j // page]
        take = lambda t: t[at, :, j % page].double().repeat_interleave(hq // hk, 1)  # noqa: E731
        k = take(s["k_cache"]) * take(s["k_scale"])[..., None]
        v, vs = take(s["v_cache"]), take(s["v_scale"]).abs().T  # [n, hq, dim], [hq, n]
        v = v * take(s["v_scale"])[..., None]
        q = s["q"][i].double()
        score = torch.einsum("hd,nhd->hn", q, k) * scale
        d = scale * ((dim + 8) * 2.0**-23 * torch.einsum("hd,nhd->hn", q.abs(), k.abs())
                     + 0.5 / 16319 * q.abs().amax(-1)[:, None] * k.abs().sum(-1).T)
        e = torch.expm1(d + 2.0**-23 * (score - score.amax(-1, keepdim=True)).abs()) + 2.0**-18
        p = torch.softmax(score, -1)
        want = torch.einsum("hn,nhd->hd", p, v)
        off = (torch.einsum("hn,nhd->hd", p * (e + 2.0**-11), v.abs()) + (p * e).sum(-1, keepdim=True) * want.abs()
               + (2.0**-13 * (p * vs).sum(-1) + n * 2.0**-24 * (p * vs).amax(-1))[:, None])
        half = torch.finfo(out.dtype).eps / 2
        tiny = torch.finfo(out.dtype).smallest_normal * half
        bad = ~((out[i].double() - want).abs() <= half * want.abs() + off * (1 + half) + tiny)
        assert not bad.any(), (i, n, int(bad.sum()), float(((out[i].double() - want).abs() / want.abs()).max()))


def aim(s, i, token, log2_weight, ratio):
    """Token `token` of sequence i: its value scales times `ratio`, its keys against each head's query, so that its
    weight is about 2^log2_weight of the others'. One query head to a key head."""
    page, dim = s["k_cache"].shape[2], s["q"].shape[2]
    at, row = int(s["page_table"][i, token // page]), token % page
    q = s["q"][i].double()  # [heads, dim]
    codes = torch.round(127 * q / q.abs().amax(-1, keepdim=True))
    s["k_cache"][at, :, row] = codes.to(I8)
    s["k_scale"][at, :, row] = (log2_weight * math.log(2) / ((q * codes).sum(-1) * dim**-0.5)).float()
    s["v_scale"][at, :, row] *= ratio


SHAPES = [  # lengths and channels: one range, ranges that cut a sequence, a warp for each of many (short, long) items
    ([700], 128), ([700], 64), ([700], 256), ([9000, 40], 128), ([60] * 120, 128), ([700] * 120, 128), ([100] * 120, 64)]


@pytest.mark.parametrize("lengths,dim", SHAPES)
@pytest.mark.parametrize("log2_weight,log2_ratio", [(-60, 22), (-60, 28), (-60, 31), (-60, 60), (-200, 90), (-40, 40),
                                                    (-20, 20), (0, 30), (-100, 110), (10, -60)])
@pytest.mark.parametrize("where", [0.0, 0.5, 0.999])
def test_one_large_scale_of_little_weight(dq, lengths, dim, log2_weight, log2_ratio, where):
    """What counts is weight times scale: a huge value scale without weight takes nothing from the others."""
    s = make(lengths, 8, 8, dim, BF16, I8, 16, seed=len(lengths) + dim)
    for i in range(0, len(lengths), 7):
        aim(s, i, int(where * lengths[i]), log2_weight, 2.0**log2_ratio)
    out = call(dq, s)
    check(s, out, rows=[0, 1, len(lengths) // 7 * 7])
    assert torch.equal(call(dq, s), out)


@pytest.mark.parametrize("size", [1e-35, 1e-20, 1e31, 1e33, 1e36, 6e37])
@pytest.mark.parametrize("lengths,dim", [*SHAPES[:6], ([700], 80), ([333, 1, 20], 7)])
def test_scales_over_the_whole_range(dq, lengths, dim, size):
    """Scales from the end of binary32's range to that of bf16 outputs (6e37: values up to 3e38)."""
    s = make(lengths, 8, 2, dim, BF16, I8, 16, seed=33)
    s["v_scale"] *= size
    out = call(dq, s)
    assert out.isfinite().all()
    check(s, out, rows=[0, 1])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim,group", [(128, 4), (128, 16), (64, 16), (256, 3)])
def test_scales_of_every_size_at_once(dq, dtype, dim, group):
    """Scales over sixty binades in any order, peaked scores: every head meets its own largest weight times scale."""
    s = make([2000, 333, 17, 1], 2 * group, 2, dim, dtype, I8, 20, seed=34, q_scale=12.0)
    g = torch.Generator(device="cuda").manual_seed(35)
    s["v_scale"] *= torch.exp2(-60 * torch.rand(s["v_scale"].shape, generator=g, device="cuda"))
    check(s, call(dq, s))


@pytest.mark.parametrize("size", [1e-30, 1e34, 6e37])
@pytest.mark.parametrize("lengths,dim", [([700], 128), ([9000, 40], 128), ([60] * 120, 64), ([300], 256)])
def test_bf16_caches_of_any_size(dq, lengths, dim, size):
    """Values of one sign near the end of bf16's range: their sums before the division would overflow binary32."""
    from test_paged_attention_gpu import verify

    s = make(lengths, 8, 2, dim, BF16, BF16, 16, seed=36)
    s["v_cache"] = (s["v_cache"].float().abs() * size).to(BF16)
    lse = torch.empty(len(lengths), 8, device="cuda")
    out = call(dq, s, lse=lse)
    assert out.isfinite().all()
    verify(s, out, lse)
