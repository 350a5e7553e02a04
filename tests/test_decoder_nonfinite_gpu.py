"""Infinities and NaN in the decoder operators' inputs (GPU).

What the formulas make of them has to come out: nothing that is not finite turns
into an ordinary number on its way, and nothing spreads to rows that do not see it.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, I8 = torch.float16, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


def rope_inputs(tokens, hq, hk, dim, dtype, rope_dim, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = (torch.randn(tokens, h, dim, generator=g, device="cuda").to(dtype) for h in (hq, hk, hk))
    pos = torch.arange(tokens, device="cuda", dtype=torch.int32) + 17
    freq = (10000.0 ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)).float().cuda()
    return q, k, v, pos, freq


# vector kernels (8 and 4 values to a chunk, lane counts of each kind) and the scalar one (20)
@pytest.mark.parametrize("dim,rope_dim", [(128, 128), (64, 64), (96, 48), (256, 256), (40, 40), (20, 10)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_cache_scale_of_a_row_that_is_not_finite(dq, dim, rope_dim, dtype, what):
    """The codes cannot hold it, so the scale does: NaN for that row, all others as without it."""
    q, k, v, pos, freq = rope_inputs(9, 4, 2, dim, dtype, rope_dim)
    pages, page = 3, 4

    def run(k, v):
        c = [torch.zeros(pages, 2, page, dim, dtype=I8, device="cuda") for _ in range(2)]
        s = [torch.zeros(pages, 2, page, device="cuda") for _ in range(2)]
        out = dq.qk_norm_rope_cache(q, k, v, pos, freq, torch.arange(9, device="cuda"), *c, *s)
        return out, c, s

    clean_q, clean_c, clean_s = run(k, v)
    k, v = k.clone(), v.clone()
    k[5, 1, dim - 1], v[6, 0, 3] = what, what  # tokens 5 and 6: rows 1 and 2 of page 1
    got_q, c, s = run(k, v)
    assert torch.equal(got_q, clean_q)
    for i, (row, head) in enumerate(((1, 1), (2, 0))):
        assert s[i][1, head, row].isnan()
        for got, clean in ((c[i], clean_c[i]), (s[i], clean_s[i])):
            got, clean = got.clone(), clean.clone()
            got[1, head, row] = clean[1, head, row] = 0
            assert torch.equal(got, clean)

    # and the attention over that cache: NaN for the key head's queries, nobody else's
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].repeat(2, 1).contiguous()
    for index, head in ((0, 1), (1, 0)):
        caches, scales = list(clean_c), list(clean_s)
        caches[index], scales[index] = c[index], s[index]
        lengths = torch.tensor([9, 5], device="cuda", dtype=torch.int32)  # tokens 0 .. 4 only: finite
        out = dq.paged_attention(got_q[:2].contiguous(), *caches, table, lengths, *scales)
        assert out[0, 2 * head: 2 * head + 2].isnan().all()
        assert out[0, 2 - 2 * head: 4 - 2 * head].isfinite().all() and out[1].isfinite().all()


@pytest.mark.parametrize("dim,rope_dim", [(128, 64), (64, 32), (96, 48), (256, 0), (128, 96), (20, 10)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_channels_past_the_rotation_stay_by_themselves(dq, dim, rope_dim, interleaved, what):
    """An infinite input makes its own channel NaN (inf / inf) and the others 0; an infinite or NaN weight behind
    the rotated channels touches its own channel only."""
    q, k, _, pos, freq = rope_inputs(5, 3, 1, dim, BF16, rope_dim)
    freq = freq if rope_dim else None
    weight = torch.ones(dim, device="cuda")
    clean = dq.qk_norm_rope(q, k, pos, freq, weight, weight, interleaved=interleaved)
    for channel in (rope_dim, dim - 1, (rope_dim + dim) // 2):
        w = weight.clone()
        w[channel] = what
        for got, want in zip(dq.qk_norm_rope(q, k, pos, freq, w, w, interleaved=interleaved), clean):
            assert not got[..., channel].isfinite().any()
            got, want = got.clone(), want.clone()
            got[..., channel] = want[..., channel] = 0
            assert torch.equal(got, want)
        if what != math.inf:
            continue
        x, y = q.clone(), k.clone()
        x[2, 1, channel], y[3, 0, channel] = what, -what
        for (got, want), row in zip(zip(dq.qk_norm_rope(x, y, pos, freq, interleaved=interleaved), clean), ((2, 1), (3, 0))):
            bad = torch.zeros(dim, dtype=torch.bool, device="cuda")
            bad[channel] = True
            assert got[row][bad].isnan().all() and (got[row][~bad] == 0).all()
            got, want = got.clone(), want.clone()
            got[row], want[row] = 0, 0
            assert torch.equal(got, want)


# tensor-core kernel with 64, 128 and 256 channels, with two sets of heads, and the scalar kernel (40)
@pytest.mark.parametrize("dim,group", [(128, 4), (128, 12), (64, 4), (256, 2), (40, 2)])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_scales_that_are_not_finite(dq, dim, group, page, name, what):
    """NaN for the rows that see the token, whatever the signs of scores and codes and however small its weight."""
    from test_paged_attention_gpu import call, make, verify

    s = make([100, 700, 3], 2 * group, 2, dim, BF16, I8, page, seed=21)
    clean = call(dq, s)
    at = int(s["page_table"][1, 37 // page]), 1, 37 % page  # token 37 of sequence 1, key head 1
    # weights from 1 down to nothing, for either sign of the token's scores
    for scale in (dim**-0.5, 40.0, -40.0):
        old = s[name][at].clone()
        want = call(dq, s, softmax_scale=scale)
        s[name][at] = what
        got = call(dq, s, softmax_scale=scale)
        assert got[1, group:].isnan().all()
        assert torch.equal(got[[0, 2]], want[[0, 2]]) and torch.equal(got[1, :group], want[1, :group])
        hidden = call(dq, s, window=600, sinks=4)
        verify(s, hidden, window=600, sinks=4)
        s[name][at] = old
    assert torch.equal(call(dq, s), clean)
