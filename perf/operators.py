"""The attention half of a decoder layer around the quantizers, one operator a case.

  norm_rope   RMS norms of every query and key head with the position rotation in the
              same pass, the keys (and values) written out or into a paged cache that
              holds 16-bit values or int8 codes with a scale for each token and head
  attention   one new token of each sequence over that cache, any lengths, with an
              optional sliding window beside a few first tokens that stay visible
  linear      the W8A8 product with bias, activation and residual in its epilogue

`own` chooses between the plain forms below and the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "int8": 1}


def listed():
    return [
        # ---- norms, rotation and cache writes
        # one sequence generating: a single token enters a 16-bit cache, where the call's latency counts
        dict(name="rope_decode_1", op="norm_rope", tokens=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             cache="bf16", page=16, rope_dim=128, interleaved=False, weight="bf16", pad=0),
        # a prompt whose queries and keys go to the attention as they are: no cache
        dict(name="rope_prompt_8192", op="norm_rope", tokens=8192, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             cache="none", page=16, rope_dim=128, interleaved=False, weight="bf16", pad=0),
        # a long prompt filling an int8 cache
        dict(name="rope_int8_16384", op="norm_rope", tokens=16384, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             cache="int8", page=64, rope_dim=128, interleaved=False, weight="f32", pad=0),
        # a padded, ragged batch: half of each head rotated, adjacent pairs, few heads, odd token count
        dict(name="rope_partial_1003", op="norm_rope", tokens=1003, q_heads=12, kv_heads=4, dim=96, dtype="f16",
             cache="int8", page=24, rope_dim=48, interleaved=True, weight="f16", pad=3),
        # ---- attention of one new token over the paged cache
        # a chat's first tokens: the shortest cache, latency
        dict(name="attn_1x127_int8", op="attention", batch=1, max_len=127, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", cache="int8", page=16, window=0, sinks=0, pad=0),
        # one long document: the cache's length is the only parallel axis
        dict(name="attn_1x131072_bf16", op="attention", batch=1, max_len=131072, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", cache="bf16", page=64, window=0, sinks=0, pad=0),
        # a serving batch with lengths from short to 8192 and padded rows, int8 cache
        dict(name="attn_64x8192_int8", op="attention", batch=64, max_len=8192, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", cache="int8", page=16, window=0, sinks=0, pad=4),
        # the window with its first tokens, sixteen query heads to a key head, pages that are no multiple of a tile
        dict(name="attn_window_48x6000", op="attention", batch=48, max_len=6000, q_heads=64, kv_heads=4, dim=64,
             dtype="f16", cache="f16", page=20, window=2048, sinks=4, pad=0),
        # ---- the product
        # one token through a projection: the weights are all there is to read
        dict(name="linear_1x4096x4096", op="linear", m=1, n=4096, k=4096, out="bf16", bias="bf16",
             act="silu", residual=False),
        # a decode batch through a wide projection with the residual stream added
        dict(name="linear_48x7168x8192", op="linear", m=48, n=7168, k=8192, out="bf16", bias="f32",
             act="none", residual=True),
        # a prompt through a projection, everything in the epilogue
        dict(name="linear_4096x4096x4096", op="linear", m=4096, n=4096, k=4096, out="bf16", bias="bf16",
             act="gelu", residual=True),
        # ragged in every direction, 32-bit output
        dict(name="linear_1000x2051x1040", op="linear", m=1000, n=2051, k=1040, out="f32", bias="f32",
             act="gelu_tanh", residual=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_rope", "attention", "linear"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "norm_rope":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8])
        dim = rng.choice([64, 80, 96, 128, 256])
        tokens = _log(rng, 1, min(16384, 16384 * 48 * 128 // ((group + 2) * kv_heads * dim)))
        return dict(op=op, tokens=tokens, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, dtype=dtype,
                    cache=rng.choice(["none", dtype, "int8"]), page=rng.choice([1, 16, 24, 64, 128]),
                    rope_dim=dim // rng.choice([1, 1, 2]), interleaved=rng.random() < 0.3,
                    weight=rng.choice([dtype, "f32"]), pad=rng.randint(0, min(3, tokens - 1)))
    if op == "attention":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 7, 8, 16])
        dim, cache = rng.choice([64, 128, 128, 256]), rng.choice([dtype, "int8", "int8"])
        batch = _log(rng, 1, 128)
        most = min(131072, 64 * 8192 * 8 * 128 // (batch * kv_heads * dim * BYTES[cache]))
        length = _log(rng, 1, most)
        window = _log(rng, 64, 8192) if rng.random() < 0.3 else 0
        return dict(op=op, batch=batch, max_len=length, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    dtype=dtype, cache=cache, page=rng.choice([1, 16, 20, 64, 128]), window=window,
                    sinks=rng.randint(0, 8) if window else 0, pad=rng.randint(0, min(3, batch - 1)))
    m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), 16 * _log(rng, 4, 512)
    m = max(1, min(m, 4096 ** 3 // (n * k)))
    out = rng.choice(["bf16", "f16", "f32"])
    return dict(op=op, m=m, n=n, k=k, out=out, bias=rng.choice(["none", "f32", "bf16"]),
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), residual=rng.random() < 0.5)


# ---------------------------------------------------------------- sizes that follow from a case


def _lengths(c):
    """Cached tokens of each sequence: evenly spread up to the longest, then rows of padding."""
    rows = c["batch"] - c["pad"]
    return [max(1, round(c["max_len"] * (i + 1) / rows)) for i in range(rows)] + [0] * c["pad"]


def _visible(c):
    return [n if c["window"] == 0 or n <= c["window"] else c["window"] + min(c["sinks"], n - c["window"])
            for n in _lengths(c)]


def work(case):
    c = case
    if c["op"] == "norm_rope":
        heads, kv, d, e = c["q_heads"], c["kv_heads"], c["dim"], BYTES[c["dtype"]]
        live = c["tokens"] - c["pad"]
        if c["cache"] == "none":
            moved = c["tokens"] * (heads + kv) * d * e * 2
        else:
            row = d * BYTES[c["cache"]] + (4 if c["cache"] == "int8" else 0)
            moved = c["tokens"] * heads * d * e * 2 + live * 2 * kv * (d * e + row) + c["tokens"] * 8
        return {"bytes": moved + c["tokens"] * 4, "flops": c["tokens"] * (heads + kv) * d * 7}
    if c["op"] == "attention":
        seen, d = sum(_visible(c)), c["dim"]
        row = 2 * d * BYTES[c["cache"]] + (8 if c["cache"] == "int8" else 0)
        pages = sum(-(-n // c["page"]) for n in _visible(c))
        moved = seen * c["kv_heads"] * row + 2 * c["batch"] * c["q_heads"] * d * BYTES[c["dtype"]] + 4 * pages
        return {"bytes": moved + 4 * c["batch"], "flops": 4 * seen * c["q_heads"] * d}
    m, n, k = c["m"], c["n"], c["k"]
    moved = (m + n) * k + 4 * (m + n) + m * n * BYTES[c["out"]] * (2 if c["residual"] else 1)
    return {"bytes": moved + (0 if c["bias"] == "none" else n * BYTES[c["bias"]]), "flops": 2 * m * n * k}


# ---------------------------------------------------------------- inputs


def _pool(c, shape, g, device):
    """A cache's rows as quantizing N(0, 1) keys or values leaves them: (rows, scales or None)."""
    x = torch.randn(shape, generator=g, device=device, dtype=torch.float16)
    if c["cache"] != "int8":
        return x.to(DTYPES[c["cache"]]), None
    scale = x.abs().amax(-1, keepdim=True).float() / 127
    return torch.round(x / scale).to(torch.int8), scale.squeeze(-1).contiguous()


def prepare(case, seed):
    c, device = case, torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(int(seed))
    s = dict(case=dict(case))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)

    if c["op"] == "norm_rope":
        t, hq, hk, d, dt = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]]
        # q, k and v are slices of one projection's output
        s["qkv"] = normal(t, (hq + 2 * hk) * d, dtype=dt)
        s["q_weight"] = (1 + normal(d, scale=0.1)).to(DTYPES[c["weight"]])
        s["k_weight"] = (1 + normal(d, scale=0.1)).to(DTYPES[c["weight"]])
        start = int(torch.randint(0, 100000, (1,), generator=g, device=device))
        s["positions"] = (start + torch.arange(t, device=device)).to(torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rope_dim"], 2, dtype=torch.float64) / c["rope_dim"])).float().to(device)
        if c["cache"] != "none":
            pages = -(-t // c["page"]) + 1
            slots = torch.randperm(pages, generator=g, device=device)[:, None] * c["page"] + torch.arange(c["page"], device=device)
            s["slots"] = slots.reshape(-1)[:t].clone()
            if c["pad"]:
                s["slots"][-c["pad"]:] = -1
            kind = torch.int8 if c["cache"] == "int8" else DTYPES[c["cache"]]
            for name in ("k", "v"):
                s[name + "_cache"] = torch.zeros(pages, hk, c["page"], d, dtype=kind, device=device)
                s[name + "_scale"] = torch.zeros(pages, hk, c["page"], device=device) if kind == torch.int8 else None
        return s
    if c["op"] == "attention":
        b, hq, hk, d, page = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        lengths = torch.tensor(_lengths(c))[torch.randperm(b, generator=torch.Generator().manual_seed(int(seed)))]
        counts = (lengths + page - 1) // page
        total, width = int(counts.sum()), max(1, int(counts.max()))
        used = (torch.arange(width)[None] < counts[:, None]).to(device)
        table = torch.zeros(b, width, dtype=torch.int32, device=device)
        table[used] = torch.randperm(total, generator=g, device=device).to(torch.int32)
        s["page_table"], s["lengths"] = table, lengths.to(torch.int32).to(device)
        s["q"] = normal(b, hq, d, dtype=DTYPES[c["dtype"]], scale=1.5)
        s["k_cache"], s["k_scale"] = _pool(c, (total, hk, page, d), g, device)
        s["v_cache"], s["v_scale"] = _pool(c, (total, hk, page, d), g, device)
        return s
    m, n, k = c["m"], c["n"], c["k"]

    def codes(rows):
        return torch.round(normal(rows, k, scale=32.0).clamp(-127, 127)).to(torch.int8)

    s["a"], s["b"] = codes(m), codes(n)
    s["a_scale"] = torch.rand(m, generator=g, device=device) * 0.02 + 0.01
    s["b_scale"] = (torch.rand(n, generator=g, device=device) * 0.5 + 0.75) / (32 * math.sqrt(k) * 0.64)
    s["bias"] = None if c["bias"] == "none" else normal(n, dtype=DTYPES[c["bias"]], scale=0.5)
    s["residual"] = normal(m, n, dtype=DTYPES[c["out"]]) if c["residual"] else None
    return s


# ---------------------------------------------------------------- one pass


def _plain_norm_rope(s):
    c = s["case"]
    t, hq, hk, d, r = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["rope_dim"]
    q, k, v = s["qkv"].float().split([hq * d, hk * d, hk * d], dim=-1)
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def norm(x, heads, weight):
        x = x.reshape(t, heads, d)
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()

    def rotate(x):
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., : r // 2], x[..., r // 2 : r]
            y[..., : r // 2], y[..., r // 2 : r] = a * cos - b * sin, b * cos + a * sin
        return y

    dt = DTYPES[c["dtype"]]
    out = {"q": rotate(norm(q, hq, s["q_weight"])).to(dt)}
    k = rotate(norm(k, hk, s["k_weight"]))
    if c["cache"] == "none":
        return dict(out, k=k.to(dt))
    live = s["slots"] >= 0
    at = s["slots"][live]
    page, row = at // c["page"], at % c["page"]
    for name, x in (("k", k), ("v", v.reshape(t, hk, d))):
        x = x[live]
        if c["cache"] != "int8":
            s[name + "_cache"][page, :, row] = x.to(dt)
            out[name + "_cache"] = s[name + "_cache"]
            continue
        scale = x.abs().amax(-1) / 127
        codes = torch.round(x / scale.clamp_min(1e-38)[..., None])
        s[name + "_cache"][page, :, row] = codes.to(torch.int8)
        s[name + "_scale"][page, :, row] = scale
        out[name + "_scale"] = s[name + "_scale"]
        out[name + "_cache"] = (s[name + "_cache"].float() * s[name + "_scale"][..., None]).to(dt)
    return out


def _plain_attention(s):
    c = s["case"]
    b, hq, hk, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    n = s["lengths"].long()[:, None]
    j = torch.arange(s["page_table"].shape[1] * c["page"], device=n.device)
    page, row = s["page_table"].long()[:, j // c["page"]], j % c["page"]

    def rows(name):  # [b, hk, tokens, d]
        x = s[name + "_cache"][page, :, row].float()
        return (x if s[name + "_scale"] is None else x * s[name + "_scale"][page, :, row][..., None]).transpose(1, 2)

    seen = j < n
    if c["window"]:
        seen = seen & ((j < c["sinks"]) | (j >= n - c["window"]))
    seen = seen[:, None, None]
    q = s["q"].float().reshape(b, hk, hq // hk, d)
    score = (q @ rows("k").transpose(2, 3)) * d**-0.5
    top = score.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ rows("v")) / total, 0.0)
    return out.reshape(b, hq, d).to(DTYPES[c["dtype"]])


def _activate(x, name):
    if name == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x**3)))
    return x / (1 + torch.exp(-x)) if name == "silu" else x


def _plain_linear(s):
    c = s["case"]
    x = (s["a"].float() @ s["b"].float().t()) * (s["a_scale"][:, None] * s["b_scale"])
    if s["bias"] is not None:
        x = x + s["bias"].float()
    x = _activate(x, c["act"])
    if s["residual"] is not None:
        x = x + s["residual"].float()
    return x.to(DTYPES[c["out"]])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "attention": _plain_attention, "linear": _plain_linear}[c["op"]](s)
    from token_dynamic_quantization_b200 import dq

    if c["op"] == "linear":
        return dq.w8a8_linear(s["a"], s["b"], s["a_scale"], s["b_scale"], bias=s["bias"], activation=c["act"],
                              residual=s["residual"], out_dtype=DTYPES[c["out"]])
    if c["op"] == "attention":
        return dq.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["k_scale"],
                                  s["v_scale"], window=c["window"], sinks=c["sinks"])
    t, hq, hk, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].view(t, hq + 2 * hk, d).split([hq, hk, hk], dim=1)
    if c["cache"] == "none":
        q, k = dq.qk_norm_rope(q, k, s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], epsilon=1e-6,
                               interleaved=c["interleaved"])
        return {"q": q, "k": k}
    q = dq.qk_norm_rope_cache(q, k, v, s["positions"], s["inv_freq"], s["slots"], s["k_cache"], s["v_cache"],
                              s["k_scale"], s["v_scale"], s["q_weight"], s["k_weight"], epsilon=1e-6,
                              interleaved=c["interleaved"])
    if c["cache"] != "int8":
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}

    def values(codes, scale):  # the codes as the values that they stand for
        return dq.dequant_per_token(codes.view(-1, d), scale.view(-1), out_dtype=DTYPES[c["dtype"]]).view(codes.shape)

    return {"q": q, "k_cache": values(s["k_cache"], s["k_scale"]), "k_scale": s["k_scale"],
            "v_cache": values(s["v_cache"], s["v_scale"]), "v_scale": s["v_scale"]}


# ---------------------------------------------------------------- the definitions, in 64 bits


def _exact_norm_rope(c, s):
    t, hq, hk, d, r = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["rope_dim"]
    x = s["qkv"].double().view(t, hq + 2 * hk, d)
    pair = torch.arange(r // 2, device=x.device)
    first, second = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + r // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), s["positions"].double()[:, None, None] * s["inv_freq"].double())

    def head(rows, weight):
        y = rows / (rows.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * weight.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": head(x[:, :hq], s["q_weight"])}
    k, v = head(x[:, hq : hq + hk], s["k_weight"]), x[:, hq + hk :]
    if c["cache"] == "none":
        return dict(out, k=k)
    keep = (s["slots"] >= 0).nonzero().squeeze(1)
    for name, rows in (("k", k), ("v", v)):
        pool = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device=x.device).transpose(1, 2).reshape(-1, hk, d)
        if c["cache"] == "int8":
            scale = rows.abs().amax(-1, keepdim=True) / 127
            rows = torch.round(rows / scale.clamp_min(1e-300)) * scale
            steps = torch.zeros(pool.shape[:2], dtype=torch.float64, device=x.device)
            steps[s["slots"][keep]] = scale[keep].squeeze(-1)
            out[name + "_scale"] = steps.view(-1, c["page"], hk).transpose(1, 2)
        pool[s["slots"][keep]] = rows[keep]
        out[name + "_cache"] = pool.view(-1, c["page"], hk, d).transpose(1, 2)
    return out


def _exact_attention(c, s):
    b, hq, hk, d, page = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        tokens = list(range(n))
        if c["window"] and n > c["window"]:
            tokens = list(range(min(c["sinks"], n - c["window"]))) + list(range(n - c["window"], n))
        j = torch.tensor(tokens, device=out.device)
        at = s["page_table"][i].long()[j // page]
        for h in range(hk):
            k, v = s["k_cache"][at, h, j % page].double(), s["v_cache"][at, h, j % page].double()
            if c["cache"] == "int8":
                k = k * s["k_scale"][at, h, j % page].double()[:, None]
                v = v * s["v_scale"][at, h, j % page].double()[:, None]
            q = s["q"][i, h * (hq // hk) : (h + 1) * (hq // hk)].double()
            out[i, h * (hq // hk) : (h + 1) * (hq // hk)] = torch.softmax(q @ k.t() / math.sqrt(d), -1) @ v
    return out


def _exact_linear(c, s):
    x = torch.mm(s["a"].double(), s["b"].double().t())
    x = x * s["a_scale"].double()[:, None] * s["b_scale"].double()[None, :]
    x = x if s["bias"] is None else x + s["bias"].double()
    x = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[c["act"]](x)
    return x if s["residual"] is None else x + s["residual"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "attention": _exact_attention, "linear": _exact_linear}[case["op"]](case, s)
