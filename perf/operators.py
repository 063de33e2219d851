"""The attention side of a decode layer, case by case: rotary positions, the quantised paged key-value
cache, and attention of one new token per sequence over it.

Sizes are those of the 27B-class layer that the benchmark runs (QKV 5120 -> 7168, O 5120 -> 5120: 40 query
heads and 8 key-value heads of 128) and generic ones around it.
"""
import math

import torch

own = False

BF16, E4M3, NVFP4 = "bf16", "e4m3", "nvfp4"


# ---- cases ---------------------------------------------------------------------------------------

def _rope(name, tokens, heads, head_dim, rot, layout, scaling, start, x, y):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "head_dim": head_dim, "rot": rot,
            "layout": layout, "scaling": scaling, "start": start, "x": x, "y": y}


def _cache(name, fmt, tokens, kv_heads, head_dim, page, rotary):
    return {"name": name, "op": "cache", "fmt": fmt, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim,
            "page": page, "rotary": rotary}


def _attn(name, fmt, batch, longest, ragged, q_heads, kv_heads, head_dim, page, window):
    return {"name": name, "op": "attn", "fmt": fmt, "batch": batch, "longest": longest, "ragged": ragged,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "window": window}


def listed():
    return [
        # One user's decode step: q and k heads of one QKV row, in bf16.  Latency only.
        _rope("rope_one_token", 1, 48, 128, 128, "half", "none", 1000, "bf16", "bf16"),
        # A decode batch of odd width at scattered far positions, half of the head rotated in adjacent
        # pairs; fp32 rows, as the one-user product writes them.
        _rope("rope_users_interleaved", 33, 48, 128, 64, "interleaved", "linear", 700000, "f32", "bf16"),
        # A prompt chunk of a context stretched past its trained length.
        _rope("rope_prompt_yarn", 4096, 48, 128, 128, "half", "yarn", 250000, "bf16", "bf16"),
        # The 32-user decode step writing one token each, in the weights' own 4-bit format.
        _cache("cache_users_nvfp4", NVFP4, 32, 8, 128, 64, False),
        # A prompt chunk written in bf16, keys rotated on the way.
        _cache("cache_prompt_bf16_rotary", BF16, 2048, 8, 128, 16, True),
        # A long prompt of odd length, wide heads, in 8 bits.
        _cache("cache_prompt_e4m3", E4M3, 8191, 4, 256, 128, False),
        # The first tokens of one user's answer: latency only.
        _attn("attn_one_user_short", NVFP4, 1, 100, False, 40, 8, 128, 64, 0),
        # One user with a long context: few rows, all the work along the cache.  The most bytes.
        _attn("attn_one_user_long", BF16, 1, 131072, False, 40, 8, 128, 256, 0),
        # The 32-user decode batch of the benchmark over ragged contexts, 4-bit cache.
        _attn("attn_users_nvfp4", NVFP4, 32, 16384, True, 40, 8, 128, 64, 0),
        # Small heads in 8 bits, small pages.
        _attn("attn_users_e4m3", E4M3, 8, 32768, True, 16, 2, 64, 16, 0),
        # Many users with short contexts.
        _attn("attn_many_short", NVFP4, 256, 512, True, 40, 8, 128, 64, 0),
        # Wide heads under a sliding window.
        _attn("attn_window", BF16, 16, 8192, True, 16, 4, 256, 48, 1024),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attn", "attn"])
    if op == "rope":
        head_dim = rng.choice([64, 80, 128, 192, 256])
        heads = rng.randint(1, 48)
        rot = 16 * rng.randint(1, head_dim // 16)
        tokens = _log(rng, 1, max(1, 4096 * 48 * 128 // (heads * head_dim)) if heads * head_dim > 6144 else 4096)
        return _rope(None, tokens, heads, head_dim, rot, rng.choice(["half", "interleaved"]),
                     rng.choice(["none", "linear", "yarn"]), _log(rng, 1, 1000000), rng.choice(["bf16", "f32"]),
                     rng.choice(["bf16", "f32"]))
    fmt = rng.choice([BF16, E4M3, NVFP4])
    kv_heads, page = rng.randint(1, 8), 16 * rng.randint(1, 16)
    if op == "cache":
        head_dim = rng.choice([64, 80, 96, 128, 192, 256])
        return _cache(None, fmt, _log(rng, 1, 8191), min(kv_heads, 1024 // head_dim), head_dim, page,
                      fmt == BF16 and rng.random() < 0.5)
    head_dim = rng.choice([64, 80, 96, 128, 192, 256])
    batch = _log(rng, 1, 256)
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    # At most the largest listed case's cache, whatever the lengths drawn.
    most = 32 * 16384 * 8 * 128 // (4 * batch * kv_heads * head_dim) // (1 if group <= 5 else 4)
    longest = _log(rng, 1, max(1, min(131072, most)))
    window = rng.choice([0, 0, 0, _log(rng, 1, longest)])
    return _attn(None, fmt, batch, longest, rng.random() < 0.7, group * kv_heads, kv_heads, head_dim, page, window)


# ---- inputs --------------------------------------------------------------------------------------

def _floats(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _channels(gen, n):
    """Uneven channel sizes, as keys have them."""
    return torch.exp(0.5 * _floats(gen, n))


ROPE_BASE, YARN_FACTOR, YARN_TRAINED, LINEAR_FACTOR = 1.0e6, 8.0, 32768, 4.0


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        # The rotated heads lie in wider rows: the value heads follow them in a QKV row.
        t, h, d = case["tokens"], case["heads"], case["head_dim"]
        row = (h + 8) * d
        x = _floats(gen, t, row).to(torch.bfloat16 if case["x"] == "bf16" else torch.float32)
        if t > 256:     # a prompt chunk
            pos = case["start"] + torch.arange(t, device="cuda")
        else:           # a decode batch: every user somewhere else
            pos = torch.randint(0, case["start"] + 1, (t,), generator=gen, device="cuda")
        return {"x": x[:, :h * d].view(t, h, d), "pos": pos.to(torch.int32)}
    ps, hk, d = case["page"], case["kv_heads"], case["head_dim"]
    if case["op"] == "cache":
        t = case["tokens"]
        kv = _floats(gen, t, 2 * hk, d)
        kv[:, :hk] *= _channels(gen, d)
        kv = kv.to(torch.bfloat16)
        pages = (t + ps - 1) // ps + 3
        if t > 256:     # a prompt: pages in any order, each filled in turn; it starts inside its first page
            first = int(seed) % ps
            order = torch.randperm(pages, generator=gen, device="cuda")
            at = first + torch.arange(t, device="cuda")
            slots, pos = order[at // ps] * ps + at % ps, at
        else:           # a decode batch: one token each, in pages of their own
            pages = t + 1
            order = torch.randperm(pages, generator=gen, device="cuda")[:t]
            slots = order * ps + torch.randint(0, ps, (t,), generator=gen, device="cuda")
            pos = torch.randint(0, 100000, (t,), generator=gen, device="cuda")
        return {"k": kv[:, :hk], "v": kv[:, hk:], "slots": slots, "pos": pos.to(torch.int32), "pages": pages}
    b, hq, longest = case["batch"], case["q_heads"], case["longest"]
    width = (longest + ps - 1) // ps
    if case["ragged"]:
        lens = torch.randint(1, longest + 1, (b,), generator=gen, device="cuda")
        if b > 4:
            lens[b // 2] = 0            # a free place in the batch
        lens[b - 1] = longest
    else:
        lens = torch.full((b,), longest, device="cuda")
    pages = b * width + 1
    table = torch.randperm(pages, generator=gen, device="cuda")[:b * width].view(b, width)
    q = (1.5 * _floats(gen, b, hq, d)).to(torch.bfloat16)
    k = torch.empty(pages * ps, hk, d, dtype=torch.bfloat16, device="cuda")
    k.normal_(generator=gen)
    k *= _channels(gen, d).to(torch.bfloat16)
    v = torch.empty_like(k).normal_(generator=gen)
    return {"q": q, "k": k, "v": v, "table": table.to(torch.int32), "lens": lens.to(torch.int32), "pages": pages}


def _turns(case):
    """(fp64 angle per position of each pair, factor on the rotated values) of a case's rotary positions."""
    rot, scaling = case.get("rot", case["head_dim"]), case.get("scaling", "none")
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = ROPE_BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / LINEAR_FACTOR, 1.0
    if scaling == "yarn":
        # Pairs that turn more than 32 times over the trained length stay, those under one turn are
        # slowed by the factor, and a ramp over the pair index joins them.
        def pair(turns):
            return rot * math.log(YARN_TRAINED / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / YARN_FACTOR * ramp, 0.1 * math.log(YARN_FACTOR) + 1.0
    return f, 1.0


# ---- plain forms ---------------------------------------------------------------------------------

def _rotate(x, pos, turns, factor, layout):
    """x [tokens][heads][head_dim] in fp32, rotated in fp32 with angles taken in 64 bits."""
    rot = 2 * turns.numel()
    angle = pos.to(torch.float64)[:, None] * turns
    c = (torch.cos(angle) * factor).float()[:, None, :]
    s = (torch.sin(angle) * factor).float()[:, None, :]
    y = x.float().clone()
    if layout == "half":
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    else:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return y


def _encode(x, fmt):
    """x [...][head_dim] as the format's codes and scales."""
    if fmt == BF16:
        return (x.to(torch.bfloat16),)
    x = x.float()
    if fmt == E4M3:
        amax = x.abs().amax(-1, keepdim=True)
        f, e = torch.frexp(amax)                    # amax = f 2^e, f in [0.5, 1)
        e = (e - 9 + (f > 0.875).int()).clamp(min=-110)
        e = torch.where(amax > 0, e, torch.full_like(e, -110))
        return torch.ldexp(x, -e).to(torch.float8_e4m3fn), e.to(torch.int8)
    b = x.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    a = b.abs() / torch.where(s > 0, s, torch.ones_like(s))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(s > 0, code + 8 * torch.signbit(b).to(torch.uint8), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.squeeze(-1)


def _decode(parts, fmt):
    """The fp32 values that codes and scales stand for."""
    if fmt == BF16:
        return parts[0].float()
    if fmt == E4M3:
        return torch.ldexp(parts[0].float(), parts[1].int())
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=parts[0].device)
    code = torch.stack((parts[0] & 15, parts[0] >> 4), -1).flatten(-2)
    return (values[code.int()].unflatten(-1, (-1, 16)) * parts[1].float()[..., None]).flatten(-2)


def _take(cache, index):
    return tuple(part.view(torch.uint8)[index].view(part.dtype) if part.dtype == torch.float8_e4m3fn else part[index]
                 for part in cache)


def _put(cache, index, parts):
    return [old.view(torch.uint8).index_put_((index,), new.view(torch.uint8)) if old.dtype == torch.float8_e4m3fn
            else old.index_put_((index,), new) for old, new in zip(cache, parts)]


def _attend(q, k, v, valid, scale):
    """q [b][hk][g][d], k and v [b][hk][l][d], valid [b][l]; fp32.  Rows with nothing valid give 0 and -inf."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = s.masked_fill(~valid[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + torch.log(total)).squeeze(-1)


# ---- what is measured ----------------------------------------------------------------------------

def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    d = case["head_dim"]
    if case["op"] == "rope" or case.get("rotary"):
        st["turns"], st["factor"] = _turns(case)
    if own:
        # A serving program keeps its frequency table, its cache in the library's layout, and the
        # marshalled arguments of its calls.
        from bit_quantized_decode_amd import binding as B
        fmt = {BF16: B.NVFP4_KV_BF16, E4M3: B.NVFP4_KV_E4M3, NVFP4: B.NVFP4_KV_NVFP4}
        dtypes = {"bf16": torch.bfloat16, "f32": torch.float32}
        table = None
        if "turns" in st:
            scaling = {"none": None, "linear": ("linear", LINEAR_FACTOR), "yarn": ("yarn", YARN_FACTOR, YARN_TRAINED)}
            table = B.rope_table(case.get("rot", d), base=ROPE_BASE, layout=case.get("layout", "half"),
                                 scaling=scaling[case.get("scaling", "none")], device="cuda")
        if case["op"] == "rope":
            st["call"] = B.rope_prepared(st["x"], st["pos"], table, dtype=dtypes[case["y"]])
            return st
        cache = B.KvCache(st["pages"], case["page"], case["kv_heads"], d, fmt[case["fmt"]], device="cuda")
        if case["op"] == "cache":
            st["write"] = B.kv_append_prepared(cache, st["k"], st["v"], st["slots"],
                                               positions=None if table is None else st["pos"], table=table)
            st["read"] = B.kv_read_prepared(cache, st["slots"], dtype=torch.bfloat16)
            return st
        B.kv_append(cache, st.pop("k"), st.pop("v"), torch.arange(st["pages"] * case["page"], device="cuda"))
        st["call"] = B.attn_decode_prepared(st["q"], cache, st["table"], st["lens"], scale=d ** -0.5,
                                            window=case["window"], lse=True)
        return st
    if case["op"] == "cache":
        n = st["pages"] * case["page"]
        empty = torch.zeros(1, case["kv_heads"], d, device="cuda")
        st["cache"] = [[part.expand(n, *part.shape[1:]).clone() if part.dtype != torch.float8_e4m3fn
                        else part.view(torch.uint8).expand(n, *part.shape[1:]).clone().view(part.dtype)
                        for part in _encode(empty, case["fmt"])] for _ in range(2)]
    elif case["op"] == "attn":
        st["cache"] = [_encode(st.pop(name), case["fmt"]) for name in ("k", "v")]
    return st


def run(st):
    case = st["case"]
    if own:
        if case["op"] == "cache":
            st["write"]()
            return st["read"]()
        return st["call"]()
    if case["op"] == "rope":
        y = _rotate(st["x"], st["pos"], st["turns"], st["factor"], case["layout"])
        return y.to(torch.bfloat16) if case["y"] == "bf16" else y
    fmt = case["fmt"]
    if case["op"] == "cache":
        k = _rotate(st["k"], st["pos"], st["turns"], st["factor"], "half") if case["rotary"] else st["k"]
        _put(st["cache"][0], st["slots"], _encode(k, fmt))
        _put(st["cache"][1], st["slots"], _encode(st["v"], fmt))
        return (_decode(_take(st["cache"][0], st["slots"]), fmt).to(torch.bfloat16),
                _decode(_take(st["cache"][1], st["slots"]), fmt).to(torch.bfloat16))
    b, hq, hk, d, ps = (case[n] for n in ("batch", "q_heads", "kv_heads", "head_dim", "page"))
    at = torch.arange(case["longest"], device="cuda")
    lens = st["lens"][:, None]
    valid = (at < lens) & ((at >= lens - case["window"]) if case["window"] else (at >= 0))
    rows = st["table"].long()[:, at // ps] * ps + at % ps
    k, v = (_decode(_take(part, rows), fmt).transpose(1, 2).contiguous() for part in st["cache"])
    q = st["q"].float().view(b, hk, hq // hk, d)
    o, lse = _attend(q, k, v, valid, d ** -0.5)
    return o.view(b, hq, d).to(torch.bfloat16), lse.view(b, hq)


def _row_bytes(fmt, head_dim):
    """Bytes of one token's k or v of one head."""
    return {BF16: 2 * head_dim, E4M3: head_dim + 1, NVFP4: head_dim // 2 + head_dim // 16}[fmt]


def _tokens(case):
    """Cached tokens that a case attends over: the mean of its lengths, whatever the seed."""
    b, longest, w = case["batch"], case["longest"], case["window"]
    seen = (lambda n: min(n, w)) if w else (lambda n: n)
    if not case["ragged"]:
        return b * seen(longest)
    inner = sum(seen(n) for n in range(1, longest + 1)) / longest
    return seen(longest) + inner * (b - 1 - (b > 4))


def work(case):
    d = case["head_dim"]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        size = {"bf16": 2, "f32": 4}
        return {"bytes": n * d * (size[case["x"]] + size[case["y"]]) + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    hk = case["kv_heads"]
    if case["op"] == "cache":
        rows = 2 * case["tokens"] * hk
        # Written: values in, cache out.  Read back: cache in, values out.
        return {"bytes": rows * (4 * d + 2 * _row_bytes(case["fmt"], d)) + 8 * case["tokens"], "flops": 4 * rows * d}
    tokens = _tokens(case)
    return {"bytes": 2 * tokens * hk * _row_bytes(case["fmt"], d) + case["batch"] * case["q_heads"] * (4 * d + 4),
            "flops": 4 * tokens * case["q_heads"] * d}


# ---- the definition, in 64 bits ------------------------------------------------------------------

def _nearest(x, grid):
    """The grid value nearest to each x >= 0, ties to the even index; past the last, the last."""
    up = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
    below, above = x - grid[up - 1], grid[up] - x
    even = torch.where(up % 2 == 0, up, up - 1)
    return grid[torch.where(below < above, up - 1, torch.where(above < below, up, even))]


def _e4m3_grid():
    low = [m * 2.0 ** -9 for m in range(8)]
    return torch.tensor(low + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device="cuda")


def _stored(x, fmt):
    """The fp64 values a cache of this format holds for x."""
    if fmt == BF16:
        return x.to(torch.bfloat16).double()
    x = x.double()
    if fmt == E4M3:
        amax = x.abs().amax(-1, keepdim=True).clamp(min=1e-300)
        size = torch.exp2(torch.ceil(torch.log2(amax / 448.0)).clamp(min=-110.0))
        size = torch.where(amax > 448.0 * size, 2 * size, size)     # should the logarithm have been off
        size = torch.where((amax <= 224.0 * size) & (size > 2.0 ** -110), size / 2, size)
        return torch.copysign(_nearest((x / size).abs(), _e4m3_grid()) * size, x)
    b = x.unflatten(-1, (-1, 16))
    scale = _nearest(b.abs().amax(-1, keepdim=True) / 6.0, _e4m3_grid())
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    y = _nearest(b.abs() / scale.clamp(min=2.0 ** -9), grid) * scale
    return torch.copysign(y, b).flatten(-2)


def _turned(x, pos, case):
    """x in fp64, its pairs turned as complex numbers."""
    turns, factor = _turns(case)
    rot = 2 * turns.numel()
    w = torch.polar(torch.full((), factor, dtype=torch.float64, device="cuda").expand(pos.numel(), rot // 2).contiguous(),
                    pos.double()[:, None] * turns)[:, None, :]
    y = x.double().clone()
    first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case.get("layout", "half") == "half"
                     else (slice(0, rot, 2), slice(1, rot, 2)))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "rope":
        return _turned(st["x"], st["pos"], case)
    fmt = case["fmt"]
    if case["op"] == "cache":
        if case["rotary"]:      # the values before their one rounding
            return _turned(st["k"], st["pos"], case), _stored(st["v"], fmt)
        return _stored(st["k"], fmt), _stored(st["v"], fmt)
    b, hq, hk, d, ps = (case[n] for n in ("batch", "q_heads", "kv_heads", "head_dim", "page"))
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    for i in range(b):
        first = max(0, lens[i] - case["window"]) if case["window"] else 0
        if lens[i] <= first:
            continue
        at = torch.arange(first, lens[i], device="cuda")
        rows = st["table"][i].long()[at // ps] * ps + at % ps
        k, v = _stored(st["k"][rows], fmt), _stored(st["v"][rows], fmt)
        for h in range(hk):
            own_heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            s = st["q"][i, own_heads].double() @ k[:, h].t() / math.sqrt(d)
            lse[i, own_heads] = torch.logsumexp(s, -1)
            out[i, own_heads] = torch.softmax(s, -1) @ v[:, h]
    return out, lse
