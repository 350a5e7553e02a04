"""Calls that the decoder operators' documentation allows at its edges (GPU).

First calls inside a capture, calls of several threads at once, tensors past
2^31 elements (the same rows somewhere else give the same bytes), windows at the
end of their type, value scales of either sign.
"""

import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


FIRST = """
import torch
from token_dynamic_quantization_b200 import dq
g = torch.Generator(device="cuda").manual_seed(1)
q = torch.randn(3, 8, 128, generator=g, device="cuda").bfloat16()
k = torch.randn(3, 2, 128, generator=g, device="cuda").bfloat16()
pos = torch.arange(3, device="cuda", dtype=torch.int32)
freq = torch.rand(64, generator=g, device="cuda")
slots = torch.tensor([0, 17, 40], device="cuda")
cache = [torch.zeros(6, 2, 16, 128, dtype=torch.int8, device="cuda") for _ in range(2)]
scale = [torch.zeros(6, 2, 16, device="cuda") for _ in range(2)]
table = torch.arange(6, device="cuda", dtype=torch.int32).reshape(3, 2)
table = torch.cat([table] * 40, 1).contiguous()
lengths = torch.tensor([1, 1100, 9], device="cuda", dtype=torch.int32)
w = torch.randint(-127, 128, (1024, 1024), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
x = {m: torch.randint(-127, 128, (m, 1024), generator=g, device="cuda", dtype=torch.int32).to(torch.int8) for m in (3, 40, 300)}
s = {m: torch.rand(m, generator=g, device="cuda") for m in (3, 40, 300, 1024)}
torch.cuda.synchronize()

def run():
    qr = dq.qk_norm_rope_cache(q, k, k, pos, freq, slots, *cache, *scale)
    out = [qr, *dq.qk_norm_rope(q, k, pos, freq), dq.paged_attention(qr, *cache, table, lengths, *scale)]
    return out + [dq.w8a8_linear(x[m], w, s[m], s[1024], activation="gelu") for m in x]

stream = torch.cuda.Stream()
with torch.cuda.stream(stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = run()
    graph.replay()
torch.cuda.synchronize()
for a, b in zip(captured, run()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_calls_inside_a_capture(dq):
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_threads(dq):
    from test_paged_attention_gpu import call, make

    s = make([700, 3, 90, 2000], 8, 2, 128, torch.bfloat16, torch.int8, 16, seed=9)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(-127, 128, (512, 1024), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    a = torch.randint(-127, 128, (200, 1024), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    sa, sb = torch.rand(200, generator=g, device="cuda"), torch.rand(512, generator=g, device="cuda")
    freq, pos = torch.rand(64, generator=g, device="cuda"), torch.arange(4, device="cuda", dtype=torch.int32)

    def once(stream):
        q, _ = dq.qk_norm_rope(s["q"], s["q"], pos, freq, stream=stream)
        return [q, call(dq, s, stream=stream)] + [dq.w8a8_linear(a[:m], w, sa[:m], sb, stream=stream) for m in (5, 60, 200)]

    want = once(None)
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in range(4)]

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    got = once(None)
                    streams[i].synchronize()
                    wrong.extend(i for x, y in zip(got, want) if not torch.equal(x, y))
        except Exception as e:
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("dim,page,dtype", [(128, 16, torch.int8), (128, 5, torch.int8), (80, 16, torch.int8),
                                            (128, 16, torch.bfloat16)])
def test_caches_past_32_bits(dq, dim, page, dtype):
    hk, codes = 4, dtype == torch.int8
    pages = (2**31 // (hk * page * dim) + 100) * (2 if codes else 1)  # past 2^32 bytes either way
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.stack([torch.randperm(90, generator=g, device="cuda")[:12] for _ in range(2)]).int()
    lengths = torch.tensor([12 * page - 3, 2 * page + 1], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 8, dim, generator=g, device="cuda").bfloat16()
    tokens = 90 * page
    k = torch.randn(tokens, hk, dim, generator=g, device="cuda").bfloat16()
    v = torch.randn(tokens, hk, dim, generator=g, device="cuda").bfloat16()
    qs = torch.zeros(tokens, 1, dim, device="cuda", dtype=torch.bfloat16)
    pos, freq = torch.arange(tokens, device="cuda", dtype=torch.int32), torch.rand(dim // 4, generator=g, device="cuda")
    out = []
    for count in (90, pages):
        cache = [torch.zeros(count, hk, page, dim, dtype=dtype, device="cuda") for _ in range(2)]
        scale = [torch.zeros(count, hk, page, device="cuda") if codes else None for _ in range(2)]
        first = count - 90
        dq.qk_norm_rope_cache(qs, k, v, pos, freq, first * page + torch.arange(tokens, device="cuda"), *cache, *scale)
        att = dq.paged_attention(q, *cache, table + first, lengths, *scale)
        out.append([att] + [t[first:].clone() for t in cache + scale if t is not None])
        assert not cache[0][:first][-200:].any()
        del cache, scale
    for a, b in zip(*out):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,k", [(70000, 32768, 16), (66000, 32769, 16), (140000, 40, 16384), (3, 140000, 16384),
                                   (100, 140000, 16384)])
def test_linear_past_32_bits(dq, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(4)
    codes = lambda r: torch.randint(-127, 128, (r, k), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    a, b = codes(m), codes(n)
    sa, sb = torch.rand(m, generator=g, device="cuda") * 2.0**-8, torch.rand(n, generator=g, device="cuda")
    out = dq.w8a8_linear(a, b, sa, sb, activation="relu", out_dtype=torch.float16)
    # the last rows of either operand on their own, other kernels among them
    rows, cols = min(m, 100), min(n, 300)
    part = dq.w8a8_linear(a[m - rows:], b[n - cols:], sa[m - rows:], sb[n - cols:], activation="relu", out_dtype=torch.float16)
    assert torch.equal(out[m - rows:, n - cols:], part)
    want = (a[m - 2:].double() @ b[:50].double().T * (sa[m - 2:].double()[:, None] * sb[:50].double())).relu()
    # three roundings of binary32 and one of binary16, half of whose smallest step is 2^-25
    off = (out[m - 2:, :50].double() - want).abs()
    assert (off <= want * (2.0**-11 + 4 * 2.0**-24) + 2.0**-25).all()
    del out, a, b
    torch.cuda.empty_cache()


def test_norm_rope_past_32_bits(dq):
    tokens, heads = 2**31 // (64 * 128) + 300, 64
    q = torch.zeros(tokens, heads, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    q[-40:] = torch.randn(40, heads, 128, generator=g, device="cuda").bfloat16()
    k = q[:, :1].clone()
    pos, freq = torch.arange(tokens, device="cuda", dtype=torch.int32), torch.rand(64, generator=g, device="cuda")
    want = dq.qk_norm_rope(q[-40:].contiguous(), k[-40:].contiguous(), pos[-40:].contiguous(), freq)
    k_out = torch.empty(tokens, 1, 128, dtype=torch.bfloat16, device="cuda")
    got = dq.qk_norm_rope(q, k, pos, freq, out=(q, k_out))  # in place
    assert torch.equal(got[0][-40:], want[0]) and torch.equal(got[1][-40:], want[1])
    assert not got[0][:-40].any()
    del q, got, k, k_out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("window,sinks", [(2**62, 2**62), (2**63 - 1, 2**63 - 1), (100, 2**63 - 1), (2**63 - 1, 0)])
@pytest.mark.parametrize("dim", [128, 80])
def test_windows_at_the_end_of_their_type(dq, window, sinks, dim):
    from test_paged_attention_gpu import call, make, verify

    s = make([700, 3, 90, 130], 8, 2, dim, torch.float16, torch.float16, 16, seed=11)
    verify(s, call(dq, s, window=window, sinks=sinks))  # every token is visible, as without a window


@pytest.mark.parametrize("dim", [128, 80])
def test_scales_of_either_sign(dq, dim):
    from test_paged_attention_gpu import call, make, verify

    s = make([700, 3, 90, 130], 8, 2, dim, torch.bfloat16, torch.int8, 16, seed=12)
    for name, big in (("k_scale", 1.0), ("v_scale", 2.0**20)):
        flip = torch.rand(s[name].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(13)) < 0.5
        s[name] = torch.where(flip, -big * s[name], s[name])
    verify(s, call(dq, s))
