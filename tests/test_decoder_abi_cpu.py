"""Host-side checks of dq_qk_norm_rope(_cache), dq_paged_attention and dq_w8a8_linear, no GPU needed.

Every call is refused (or has nothing to do) before anything is launched, so
the fake pointers are never dereferenced.
"""

import math

import pytest
import torch

FAKE = 0x10000


def call(fn, base, **kw):
    return fn(**{**base, **kw})


def run_cases(fn, base, cases):
    for kw, want in cases:
        assert call(fn, base, **kw) == want, kw


def test_w8a8_linear_refusals(dq_lib):
    d = dq_lib
    base = dict(a=FAKE, b=FAKE, m=256, n=256, k=256, a_scale=FAKE, b_scale=FAKE, bias=FAKE, bias_dtype=d.DQ_F32,
                activation=d.DQ_ACT_GELU, residual=FAKE, out=FAKE, out_dtype=d.DQ_BF16, stream=None)
    run_cases(d.dq_w8a8_linear, base, [
        (dict(m=0, a=None, out=None), d.DQ_OK), (dict(n=0, b=None), d.DQ_OK),
        (dict(m=-1), d.DQ_ERR_BAD_SHAPE), (dict(n=-1), d.DQ_ERR_BAD_SHAPE), (dict(k=0), d.DQ_ERR_BAD_SHAPE),
        (dict(k=1 << 17), d.DQ_ERR_BAD_SHAPE), (dict(m=(1 << 31) + 1), d.DQ_ERR_BAD_SHAPE),
        (dict(out_dtype=d.DQ_INT8), d.DQ_ERR_BAD_DTYPE), (dict(out_dtype=99), d.DQ_ERR_BAD_DTYPE),
        (dict(bias_dtype=d.DQ_INT8), d.DQ_ERR_BAD_DTYPE),
        (dict(activation=5), d.DQ_ERR_BAD_ARGUMENT), (dict(activation=-1), d.DQ_ERR_BAD_ARGUMENT),
        (dict(a=None), d.DQ_ERR_NULL_POINTER), (dict(b=None), d.DQ_ERR_NULL_POINTER),
        (dict(a_scale=None), d.DQ_ERR_NULL_POINTER), (dict(b_scale=None), d.DQ_ERR_NULL_POINTER),
        (dict(out=None), d.DQ_ERR_NULL_POINTER),
        (dict(out=FAKE + 1), d.DQ_ERR_MISALIGNED), (dict(residual=FAKE + 1), d.DQ_ERR_MISALIGNED),
        (dict(bias=FAKE + 2), d.DQ_ERR_MISALIGNED), (dict(a_scale=FAKE + 1), d.DQ_ERR_MISALIGNED),
        (dict(out_dtype=d.DQ_F32, residual=FAKE + 2), d.DQ_ERR_MISALIGNED),
        (dict(bias=None, bias_dtype=99, m=0), d.DQ_OK),
    ])


def rope_base(d):
    return dict(q=FAKE, q_stride=4096, k=FAKE, k_stride=1024, dtype=d.DQ_BF16, tokens=10, q_heads=32, kv_heads=8,
                head_dim=128, q_weight=FAKE, k_weight=FAKE, weight_dtype=d.DQ_F32, epsilon=1e-6, positions=FAKE,
                inv_freq=FAKE, rope_dim=128, interleaved=0, q_out=FAKE, q_out_stride=4096, stream=None)


def rope_cases(d):
    return [
        (dict(tokens=0, q=None, k=None), d.DQ_OK),
        (dict(tokens=-1), d.DQ_ERR_BAD_SHAPE), (dict(tokens=1 << 31), d.DQ_ERR_BAD_SHAPE),
        (dict(q_heads=0), d.DQ_ERR_BAD_SHAPE), (dict(kv_heads=1025), d.DQ_ERR_BAD_SHAPE),
        (dict(head_dim=0), d.DQ_ERR_BAD_SHAPE), (dict(head_dim=257), d.DQ_ERR_BAD_SHAPE),
        (dict(rope_dim=3), d.DQ_ERR_BAD_SHAPE), (dict(rope_dim=130), d.DQ_ERR_BAD_SHAPE),
        (dict(rope_dim=-2), d.DQ_ERR_BAD_SHAPE), (dict(q_stride=4095), d.DQ_ERR_BAD_SHAPE),
        (dict(k_stride=1023), d.DQ_ERR_BAD_SHAPE), (dict(q_out_stride=0), d.DQ_ERR_BAD_SHAPE),
        (dict(dtype=d.DQ_F32), d.DQ_ERR_BAD_DTYPE), (dict(weight_dtype=d.DQ_INT8), d.DQ_ERR_BAD_DTYPE),
        (dict(epsilon=-1e-6), d.DQ_ERR_BAD_ARGUMENT), (dict(epsilon=math.nan), d.DQ_ERR_BAD_ARGUMENT),
        (dict(epsilon=math.inf), d.DQ_ERR_BAD_ARGUMENT), (dict(interleaved=2), d.DQ_ERR_BAD_ARGUMENT),
        (dict(q=None), d.DQ_ERR_NULL_POINTER), (dict(k=None), d.DQ_ERR_NULL_POINTER),
        (dict(q_out=None), d.DQ_ERR_NULL_POINTER), (dict(positions=None), d.DQ_ERR_NULL_POINTER),
        (dict(inv_freq=None), d.DQ_ERR_NULL_POINTER),
        (dict(q=FAKE + 1), d.DQ_ERR_MISALIGNED), (dict(positions=FAKE + 2), d.DQ_ERR_MISALIGNED),
        (dict(q_weight=FAKE + 2), d.DQ_ERR_MISALIGNED), (dict(inv_freq=FAKE + 2), d.DQ_ERR_MISALIGNED),
    ]


def test_qk_norm_rope_refusals(dq_lib):
    d = dq_lib
    base = dict(rope_base(d), k_out=FAKE, k_out_stride=1024)
    run_cases(d.dq_qk_norm_rope, base, rope_cases(d) + [
        (dict(k_out=None), d.DQ_ERR_NULL_POINTER), (dict(k_out=FAKE + 1), d.DQ_ERR_MISALIGNED),
        (dict(k_out_stride=1000), d.DQ_ERR_BAD_SHAPE),
    ])


def test_qk_norm_rope_cache_refusals(dq_lib):
    d = dq_lib
    base = dict(rope_base(d), v=FAKE, v_stride=1024, k_cache=FAKE, v_cache=FAKE, cache_dtype=d.DQ_INT8, k_scale=FAKE,
                v_scale=FAKE, slots=FAKE, num_pages=4, page_size=16)
    run_cases(d.dq_qk_norm_rope_cache, base, rope_cases(d) + [
        (dict(v_stride=1023), d.DQ_ERR_BAD_SHAPE), (dict(num_pages=0), d.DQ_ERR_BAD_SHAPE),
        (dict(page_size=0), d.DQ_ERR_BAD_SHAPE), (dict(num_pages=1 << 31), d.DQ_ERR_BAD_SHAPE),
        (dict(cache_dtype=d.DQ_F16), d.DQ_ERR_BAD_DTYPE), (dict(cache_dtype=d.DQ_INT4X2), d.DQ_ERR_BAD_DTYPE),
        (dict(v=None), d.DQ_ERR_NULL_POINTER), (dict(k_cache=None), d.DQ_ERR_NULL_POINTER),
        (dict(slots=None), d.DQ_ERR_NULL_POINTER), (dict(k_scale=None), d.DQ_ERR_NULL_POINTER),
        (dict(v_scale=FAKE + 2), d.DQ_ERR_MISALIGNED), (dict(slots=FAKE + 4), d.DQ_ERR_MISALIGNED),
        (dict(cache_dtype=d.DQ_BF16, v_cache=FAKE + 1, k_scale=None), d.DQ_ERR_MISALIGNED),
    ])


def test_paged_attention_refusals(dq_lib):
    d = dq_lib
    base = dict(q=FAKE, q_dtype=d.DQ_BF16, q_stride=4096, k_cache=FAKE, v_cache=FAKE, cache_dtype=d.DQ_INT8,
                k_scale=FAKE, v_scale=FAKE, page_table=FAKE, lengths=FAKE, batch=4, q_heads=32, kv_heads=8,
                head_dim=128, num_pages=100, page_size=16, max_pages=10, window=0, sinks=0, softmax_scale=0.1,
                out=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    run_cases(d.dq_paged_attention, base, [
        (dict(batch=0, q=None, out=None), d.DQ_OK),
        (dict(batch=-1), d.DQ_ERR_BAD_SHAPE), (dict(batch=1 << 30), d.DQ_ERR_BAD_SHAPE),
        (dict(q_heads=30), d.DQ_ERR_BAD_SHAPE), (dict(kv_heads=0), d.DQ_ERR_BAD_SHAPE),
        (dict(q_heads=2048), d.DQ_ERR_BAD_SHAPE), (dict(head_dim=512, q_stride=1 << 20), d.DQ_ERR_BAD_SHAPE),
        (dict(q_stride=4095), d.DQ_ERR_BAD_SHAPE), (dict(num_pages=0), d.DQ_ERR_BAD_SHAPE),
        (dict(page_size=0), d.DQ_ERR_BAD_SHAPE), (dict(max_pages=0), d.DQ_ERR_BAD_SHAPE),
        (dict(max_pages=1 << 31), d.DQ_ERR_BAD_SHAPE),
        (dict(q_dtype=d.DQ_F32), d.DQ_ERR_BAD_DTYPE), (dict(cache_dtype=d.DQ_F16), d.DQ_ERR_BAD_DTYPE),
        (dict(window=-1), d.DQ_ERR_BAD_ARGUMENT), (dict(sinks=-1), d.DQ_ERR_BAD_ARGUMENT),
        (dict(softmax_scale=math.nan), d.DQ_ERR_BAD_ARGUMENT), (dict(softmax_scale=math.inf), d.DQ_ERR_BAD_ARGUMENT),
        (dict(q=None), d.DQ_ERR_NULL_POINTER), (dict(k_cache=None), d.DQ_ERR_NULL_POINTER),
        (dict(v_scale=None), d.DQ_ERR_NULL_POINTER), (dict(page_table=None), d.DQ_ERR_NULL_POINTER),
        (dict(lengths=None), d.DQ_ERR_NULL_POINTER), (dict(out=None), d.DQ_ERR_NULL_POINTER),
        (dict(out=FAKE + 1), d.DQ_ERR_MISALIGNED), (dict(lse=FAKE + 2), d.DQ_ERR_MISALIGNED),
        (dict(page_table=FAKE + 2), d.DQ_ERR_MISALIGNED), (dict(k_scale=FAKE + 2), d.DQ_ERR_MISALIGNED),
    ])


def test_paged_attention_workspace_query(dq_lib):
    d = dq_lib
    size = d.dq_paged_attention_get_workspace_size
    # the same for any batch: it depends on the device and the heads
    assert size(1, 32, 8, 128, d.DQ_INT8) == size(5000, 32, 8, 128, d.DQ_INT8)
    for args in ((-1, 32, 8, 128, d.DQ_INT8), (1, 30, 8, 128, d.DQ_INT8), (1, 32, 8, 0, d.DQ_INT8)):
        with pytest.raises(d.DQError) as e:
            size(*args)
        assert e.value.status == d.DQ_ERR_BAD_SHAPE
    with pytest.raises(d.DQError) as e:
        size(1, 32, 8, 128, d.DQ_INT4X2)
    assert e.value.status == d.DQ_ERR_BAD_DTYPE


def test_helpers_check_tensors_on_the_host(dq_lib):
    """Wrong shapes, types, layouts and devices raise before any pointer is passed on."""
    d = dq_lib
    q, k = torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        d.qk_norm_rope(q, k, pos, freq)
    with pytest.raises(TypeError, match="positions"):
        d.qk_norm_rope(q, k, pos.long(), freq)
    with pytest.raises(ValueError, match="positions"):
        d.qk_norm_rope(q, k, pos[:3], freq)
    with pytest.raises(TypeError, match="k must be"):
        d.qk_norm_rope(q, k.half(), pos, freq)
    with pytest.raises(ValueError, match="k must be"):
        d.qk_norm_rope(q, k[:, :, :32], pos, freq)
    with pytest.raises(ValueError, match="q_weight"):
        d.qk_norm_rope(q, k, pos, freq, torch.ones(32))
    with pytest.raises(ValueError, match="densely"):
        d._row_stride("q", q.transpose(1, 2))
    with pytest.raises(ValueError, match="overlap"):
        d._row_stride("q", torch.zeros(1, 8, 64).expand(4, 8, 64))
    with pytest.raises(ValueError, match="densely"):
        d._row_stride("q", torch.zeros(4, 8, 128)[:, :, :64])
    assert d._row_stride("q", torch.zeros(4, 12, 64)[:, 2:10]) == 12 * 64
    assert d._row_stride("q", torch.zeros(1, 12, 64)[:, 2:10]) == 8 * 64
    a, b = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(8, 32, dtype=torch.int8)
    with pytest.raises(ValueError, match="activation"):
        d.w8a8_linear(a, b, torch.ones(4), torch.ones(8), activation="tanh")
    with pytest.raises(ValueError, match="bias"):
        d.w8a8_linear(a, b, torch.ones(4), torch.ones(8), bias=torch.ones(4))
    with pytest.raises(TypeError, match="residual"):
        d.w8a8_linear(a, b, torch.ones(4), torch.ones(8), residual=torch.ones(4, 8), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="K of a"):
        d.w8a8_linear(a, b[:, :16], torch.ones(4), torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        d.w8a8_linear(a, b, torch.ones(4), torch.ones(8))
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    codes, scales = cache.to(torch.int8), torch.ones(3, 2, 16)
    table, lengths = torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        d.paged_attention(q, cache, cache, table, lengths)
    for kw, error, match in [
        (dict(k_cache=cache.half()), TypeError, "k_cache"), (dict(v_cache=cache[:2]), ValueError, "v_cache"),
        (dict(k_cache=codes, v_cache=codes), ValueError, "needs k_scale"),
        (dict(k_cache=codes, v_cache=codes, k_scale=scales, v_scale=scales[:, :, :8]), ValueError, "v_scale"),
        (dict(k_cache=codes, v_cache=codes, k_scale=scales, v_scale=scales.half()), TypeError, "v_scale"),
        (dict(page_table=table.long()), TypeError, "page_table"), (dict(page_table=table[:3]), ValueError, "page_table"),
        (dict(lengths=lengths[:3]), ValueError, "lengths"), (dict(lse=torch.ones(4, 2)), ValueError, "lse"),
        (dict(out=torch.ones(4, 8, 64)), TypeError, "out"), (dict(q=q[:, :, :32]), ValueError, "k_cache"),
        (dict(k_cache=cache.transpose(0, 2)), ValueError, "k_cache"),
    ]:
        with pytest.raises(error, match=match):
            d.paged_attention(**{**dict(q=q, k_cache=cache, v_cache=cache, page_table=table, lengths=lengths), **kw})
    slots = torch.arange(4)
    base = dict(q=q, k=k, v=k, positions=pos, inv_freq=freq, slots=slots, k_cache=cache, v_cache=cache)
    for kw, error, match in [
        (dict(v=k[:3]), ValueError, "v must"), (dict(slots=slots.int()), TypeError, "slots"),
        (dict(slots=slots[:2]), ValueError, "slots"), (dict(k_cache=cache[:, :1]), ValueError, "k_cache"),
        (dict(out=q.half()), TypeError, "out"), (dict(inv_freq=freq.double()), TypeError, "inv_freq"), ({}, ValueError, "CUDA"),
    ]:
        with pytest.raises(error, match=match):
            d.qk_norm_rope_cache(**{**base, **kw})
