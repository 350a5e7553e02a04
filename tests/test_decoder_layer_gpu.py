"""The decoder's operators in a run, as a serving step uses them (GPU).

A new token per sequence: dynamic_quant -> w8a8_linear (queries, keys and values,
with a bias) -> qk_norm_rope_cache (INT8 pages) -> paged_attention -> dynamic_quant
-> w8a8_linear (output projection onto the residual, in place). Every step's result
is compared with its formula in 64 bits on that step's own inputs, so the bounds
are those of one operator each; then the run is repeated, and captured and
replayed, for the same bytes. The cache is filled by prompt calls first.

Bounds. Linear: the int32 sum is exact, its conversion and each later operation
round once to binary32 (2^-24 of a value at most (|product| + |bias|), five of
them), then half a step of bf16. Norm and rotation: a binary32 sum of 128
squares, a reciprocal root, two products and a rotation of two products, the
angle within 2^-32 of a turn and its sine within 2^-22: 2^-19 of the pair's
length, then the output's rounding; codes: half a step beside that. Attention:
the bound of its own test, 2^-11 of the weights and scores within (128 + 8) *
2^-23 * scale * sum |q K|, beside INT8 caches a query within 2^-15 of its head's
largest channel.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HK, DIM, HIDDEN, PAGE, BASE = 8, 2, 128, 640, 16, 10000.0


@pytest.fixture(scope="module")
def dq(dq_lib, cuda_device):
    return dq_lib


class Layer:
    def __init__(self, lengths, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
        self.n = (HQ + 2 * HK) * DIM
        self.w_qkv, self.s_qkv = codes(self.n, HIDDEN), (rnd(self.n).abs() + 0.5) * 2.0**-11
        self.bias = (0.1 * rnd(self.n)).to(torch.bfloat16)
        self.w_out, self.s_out = codes(HIDDEN, HQ * DIM), (rnd(HIDDEN).abs() + 0.5) * 2.0**-11
        self.q_weight, self.k_weight = 1 + 0.1 * rnd(DIM), 1 + 0.1 * rnd(DIM)
        self.inv_freq = (BASE ** (-torch.arange(0, DIM, 2, device="cuda", dtype=torch.float64) / DIM)).float()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")  # the new token included; 0: padding
        b, longest = len(lengths), max(lengths)
        pages = (longest + PAGE - 1) // PAGE
        perm = torch.randperm(b * pages + 2, generator=g, device="cuda").to(torch.int32)
        self.table = perm[: b * pages].reshape(b, pages).contiguous()
        self.spare = perm[b * pages:]
        shape = (b * pages + 2, HK, PAGE, DIM)
        self.cache = [torch.full(shape, 77, dtype=torch.int8, device="cuda") for _ in range(2)]
        self.scale = [torch.full(shape[:3], 5.0, device="cuda") for _ in range(2)]
        self.x = rnd(b, HIDDEN).to(torch.bfloat16)
        self.prompt = [rnd(max(n - 1, 0), self.n).to(torch.bfloat16) for n in lengths]
        # where the new token goes; a padded sequence's goes nowhere
        last = (self.lengths - 1).clamp_min(0).long()
        slot = self.table.gather(1, (last // PAGE)[:, None])[:, 0].long() * PAGE + last % PAGE
        self.slots = torch.where(self.lengths > 0, slot, -1)
        self.positions = (self.lengths - 1).clamp_min(0)

    def split(self, qkv):
        q, k, v = qkv.split([HQ * DIM, HK * DIM, HK * DIM], dim=1)
        return q.unflatten(1, (HQ, DIM)), k.unflatten(1, (HK, DIM)), v.unflatten(1, (HK, DIM))

    def fill(self, dq):
        for b, qkv in enumerate(self.prompt):
            t = qkv.shape[0]
            if t == 0:
                continue
            j = torch.arange(t, device="cuda")
            slots = self.table[b].long()[j // PAGE] * PAGE + j % PAGE
            dq.qk_norm_rope_cache(*self.split(qkv), j.int(), self.inv_freq, slots, *self.cache, *self.scale,
                                  q_weight=self.q_weight, k_weight=self.k_weight)

    def step(self, dq, x):
        """Every intermediate result; x itself becomes the layer's output."""
        s = {}
        s["codes"], s["scale"], *_ = dq.dynamic_quant(x)
        s["qkv"] = dq.w8a8_linear(s["codes"], self.w_qkv, s["scale"], self.s_qkv, bias=self.bias, out_dtype=torch.bfloat16)
        s["q"] = dq.qk_norm_rope_cache(*self.split(s["qkv"]), self.positions, self.inv_freq, self.slots, *self.cache,
                                       *self.scale, q_weight=self.q_weight, k_weight=self.k_weight)
        s["att"] = dq.paged_attention(s["q"], *self.cache, self.table, self.lengths, *self.scale)
        s["codes2"], s["scale2"], *_ = dq.dynamic_quant(s["att"].flatten(1))
        s["out"] = dq.w8a8_linear(s["codes2"], self.w_out, s["scale2"], self.s_out, residual=x, out=x,
                                  out_dtype=torch.bfloat16)
        return s


def quantized_ok(x, codes, scale):
    want = x.double().abs().amax(-1) / 127
    assert ((scale.double() - want).abs() <= want * 2.0**-22).all()
    # half a step, and the binary32 division's rounding of a quotient up to 127
    assert ((codes.double() * scale.double()[:, None] - x.double()).abs() <= scale.double()[:, None] * (0.5 + 2.0**-15)).all()


def linear_ok(got, codes, scale, w, w_scale, bias=None, residual=None):
    prod = codes.double() @ w.double().T * (scale.double()[:, None] * w_scale.double()[None])
    size = prod.abs()
    want = prod
    for extra in (bias, residual):
        if extra is not None:
            want, size = want + extra.double(), size + extra.double().abs()
    assert ((got.double() - want).abs() <= want.abs() * 2.0**-8 + size * 5 * 2.0**-24 * (1 + 2.0**-8)).all()


def rotated(x, weight, positions, inv_freq):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
    angle = positions.double()[:, None] * inv_freq.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = y[..., : DIM // 2], y[..., DIM // 2:]
    length = torch.cat([(a.square() + b.square()).sqrt()] * 2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1), length


@pytest.mark.parametrize("lengths", [[1], [37, 1, 0, 200], [5] * 21 + [0, 700], [33] * 140])
def test_decode_step(dq, lengths):
    layer = Layer(lengths, seed=len(lengths))
    layer.fill(dq)
    before = [t.clone() for t in layer.cache + layer.scale]
    x = layer.x.clone()
    s = layer.step(dq, x)
    n = layer.lengths.tolist()

    quantized_ok(layer.x, s["codes"], s["scale"])
    linear_ok(s["qkv"], s["codes"], s["scale"], layer.w_qkv, layer.s_qkv, bias=layer.bias)
    q, k, v = layer.split(s["qkv"])
    want, length = rotated(q, layer.q_weight, layer.positions, layer.inv_freq)
    assert ((s["q"].double() - want).abs() <= want.abs() * 2.0**-8 + length * 2.0**-18).all()

    # the cache: the new rows, and nothing else
    live = layer.slots >= 0
    page, row = layer.slots[live] // PAGE, layer.slots[live] % PAGE
    for i, (x64, size) in enumerate((rotated(k, layer.k_weight, layer.positions, layer.inv_freq), (v.double(), v.double().abs()))):
        codes, scale = layer.cache[i][page, :, row].double(), layer.scale[i][page, :, row].double()
        top = x64[live].abs().amax(-1)
        assert ((scale - top / 127).abs() <= top / 127 * 2.0**-17).all()
        assert ((codes * scale[..., None] - x64[live]).abs() <= scale[..., None] * (0.5 + 2.0**-9)).all()
        layer_cache, old = layer.cache[i].clone(), before[i]
        layer_cache[page, :, row] = old[page, :, row]
        assert torch.equal(layer_cache, old)
        scales = layer.scale[i].clone()
        scales[page, :, row] = before[2 + i][page, :, row]
        assert torch.equal(scales, before[2 + i])

    for b, t in enumerate(n):
        if t == 0:
            assert (s["att"][b] == 0).all()
            continue
        j = torch.arange(t, device="cuda")
        pages = layer.table[b].long()[j // PAGE]
        K, V = (layer.cache[i][pages, :, j % PAGE].double() * layer.scale[i][pages, :, j % PAGE].double()[..., None]
                for i in range(2))  # [t, HK, DIM]
        qb = s["q"][b].double().view(HK, HQ // HK, DIM)
        score = torch.einsum("kgd,tkd->kgt", qb, K) * DIM**-0.5
        size = torch.einsum("kgd,tkd->kgt", qb.abs(), K.abs()) * DIM**-0.5
        # a query beside codes is within 2^-15 of its head's largest channel
        size = size * (DIM + 8) * 2.0**-23 + torch.einsum("kg,tk->kgt", qb.abs().amax(-1), K.abs().sum(-1)) * DIM**-0.5 * 2.0**-15
        p = score.softmax(-1)
        want = torch.einsum("kgt,tkd->kgd", p, V)
        weight = torch.einsum("kgt,tkd->kgd", p, V.abs())
        tol = want.abs() * 2.0**-8 + weight * (2.0**-11 + 2 * (size.amax(-1, keepdim=True).exp() - 1) + 2.0**-17) + 1e-12
        assert ((s["att"][b].double().view_as(want) - want).abs() <= tol).all()

    quantized_ok(s["att"].flatten(1), s["codes2"], s["scale2"])
    linear_ok(s["out"], s["codes2"], s["scale2"], layer.w_out, layer.s_out, residual=layer.x)
    assert s["out"].data_ptr() == x.data_ptr()

    # again (the step writes the same rows of the cache), then captured and replayed
    again = layer.x.clone()
    r = layer.step(dq, again)
    for name in s:
        assert torch.equal(r[name], s[name]), name
    for t, old in zip(layer.cache + layer.scale, before):
        t.copy_(old)
    held = layer.x.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = layer.step(dq, held)
        for _ in range(2):
            held.copy_(layer.x)
            graph.replay()
    torch.cuda.synchronize()
    for name in s:
        assert torch.equal(captured[name], s[name]), name
