"""Reading less of a long key-value cache, case by case: attention of a batch over a prefix that all its
sequences share, attention over the pages that a cheap score selects (page bounds, selection, attention), and
eviction of pages by the attention weight that they have had.

Sizes are those of the 27B-class layer that the benchmark runs (40 query heads and 8 key-value heads of 128)
and generic ones around it.
"""
import math

import torch

own = False

BF16, E4M3, NVFP4 = "bf16", "e4m3", "nvfp4"


# ---- cases ---------------------------------------------------------------------------------------

def _shared(name, fmt, batch, prefix, longest, q_heads, kv_heads, head_dim, page):
    return {"name": name, "op": "shared", "fmt": fmt, "batch": batch, "prefix": prefix, "longest": longest,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page}


def _bounds(name, fmt, pages, kv_heads, head_dim, page):
    return {"name": name, "op": "bounds", "fmt": fmt, "pages": pages, "kv_heads": kv_heads, "head_dim": head_dim,
            "page": page}


def _sparse(name, fmt, batch, longest, ragged, budget, q_heads, kv_heads, head_dim, page):
    return {"name": name, "op": "sparse", "fmt": fmt, "batch": batch, "longest": longest, "ragged": ragged,
            "budget": budget, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page}


def _weigh(name, fmt, batch, longest, ragged, q_heads, kv_heads, head_dim, page, window, decay):
    return {"name": name, "op": "weigh", "fmt": fmt, "batch": batch, "longest": longest, "ragged": ragged,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "window": window,
            "decay": decay}


def _evict(name, batch, longest, budget, sink, recent, kv_heads, page):
    return {"name": name, "op": "evict", "batch": batch, "longest": longest, "budget": budget, "sink": sink,
            "recent": recent, "kv_heads": kv_heads, "page": page}


def listed():
    return [
        # A few users just after a common instruction: latency counts.
        _shared("shared_few_short", NVFP4, 4, 1000, 40, 40, 8, 128, 64),
        # The 32-user decode batch of the benchmark under one long document, 4-bit cache.
        _shared("shared_users_nvfp4", NVFP4, 32, 32768, 512, 40, 8, 128, 64),
        # Many samples of one prompt: the prefix is a large matrix product.  The most operations.
        _shared("shared_many_bf16", BF16, 200, 8192, 128, 40, 8, 128, 16),
        # Wide heads in 8 bits, an odd number of users and of prefix tokens.
        _shared("shared_wide_e4m3", E4M3, 7, 50001, 300, 16, 4, 256, 48),
        # One user's newest full pages, and a whole prompt's.
        _bounds("bounds_users", NVFP4, 32, 8, 128, 64),
        _bounds("bounds_prompt", BF16, 2048, 8, 128, 64),
        # One user with a long context attending to a thirty-second of it.
        _sparse("sparse_one_user", BF16, 1, 131072, False, 64, 40, 8, 128, 64),
        # The 32-user decode batch over ragged contexts, an eighth of the longest.
        _sparse("sparse_users_nvfp4", NVFP4, 32, 16384, True, 64, 40, 8, 128, 32),
        # The whole cache read, with the weights of its pages besides: one long user, ragged users.
        _weigh("weigh_one_user", E4M3, 1, 65536, False, 40, 8, 128, 64, 0, 1.0),
        _weigh("weigh_users_nvfp4", NVFP4, 32, 8192, True, 40, 8, 128, 64, 0, 0.9),
        # Half of the pages of every user given back; one user with a very long table.
        _evict("evict_users", 32, 16384, 128, 1, 4, 8, 64),
        _evict("evict_one_user", 1, 131072, 1000, 4, 16, 8, 16),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "bounds", "sparse", "sparse", "weigh", "weigh", "evict"])
    fmt = rng.choice([BF16, E4M3, NVFP4])
    kv_heads, page = rng.randint(1, 8), 16 * rng.randint(1, 8)
    head_dim = rng.choice([64, 80, 96, 128, 192, 256])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    if op == "evict":
        longest = _log(rng, 1, 131072 * page // 64)
        pages = -(-longest // page)
        batch = _log(rng, 1, max(1, min(256, 65536 // (pages * kv_heads))))
        return _evict(None, batch, longest, _log(rng, 1, pages), rng.randint(0, 4), rng.randint(1, 8), kv_heads, page)
    if op == "bounds":
        most = 2048 * 8 * 64 * 128 // (kv_heads * page * head_dim)
        return _bounds(None, fmt, _log(rng, 1, most), kv_heads, head_dim, page)
    if op == "shared":
        batch = _log(rng, 1, 200)
        longest = _log(rng, 1, 1000)
        # At most the largest listed case's operations and scores, and its cache's values.
        most = min(200 * 8192 * 40 * 128 // (batch * group * kv_heads * max(head_dim, 128)),
                   32768 * 8 * 128 // (kv_heads * head_dim)) - longest
        return _shared(None, fmt, batch, _log(rng, 1, max(1, most)), longest, group * kv_heads, kv_heads, head_dim, page)
    batch = _log(rng, 1, 64)
    most = 131072 * 8 * 128 // (batch * kv_heads * head_dim) // (1 if group <= 5 else 4)
    longest = _log(rng, 1, max(1, min(131072, most)))
    ragged = rng.random() < 0.7
    if op == "sparse":
        budget = _log(rng, 1, max(1, 4096 // page))
        return _sparse(None, fmt, batch, longest, ragged, budget, group * kv_heads, kv_heads, head_dim, page)
    window = rng.choice([0, 0, 0, _log(rng, 1, longest)])
    return _weigh(None, fmt, batch, longest, ragged, group * kv_heads, kv_heads, head_dim, page, window,
                  rng.choice([1.0, 0.9, 0.5]))


# ---- inputs --------------------------------------------------------------------------------------

def _floats(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _channels(gen, n):
    """Uneven channel sizes, as keys have them."""
    return torch.exp(0.5 * _floats(gen, n))


def _lengths(gen, case):
    b, longest = case["batch"], case["longest"]
    if case.get("ragged", True):
        lens = torch.randint(1, longest + 1, (b,), generator=gen, device="cuda")
        if b > 4:
            lens[b // 2] = 0            # a free place in the batch, or a sequence without a token of its own
        lens[b - 1] = longest
        return lens.to(torch.int32)
    return torch.full((b,), longest, dtype=torch.int32, device="cuda")


def _keys(gen, slots, hk, d, page=None):
    """Keys and values in bf16.  `page`: keys lie around a direction of their page's own, as those of neighbouring
    tokens do (what makes a page's bounds tell pages apart)."""
    k = torch.empty(slots, hk, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    if page:
        k.view(-1, page, hk, d).add_(_floats(gen, slots // page, 1, hk, d).to(torch.bfloat16))
    k *= _channels(gen, d).to(torch.bfloat16)
    return k, torch.empty_like(k).normal_(generator=gen)


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ps, hk = case["page"], case["kv_heads"]
    if case["op"] == "bounds":
        d, n = case["head_dim"], case["pages"]
        k, v = _keys(gen, n * ps, hk, d)
        return {"k": k, "v": v, "pool": n, "which": torch.randperm(n, generator=gen, device="cuda").to(torch.int32)}
    b, width = case["batch"], -(-case["longest"] // ps)
    lens = _lengths(gen, case)
    if case["op"] == "shared":
        first = -(-case["prefix"] // ps)
        pool = first + b * width + 1
        order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        st = {"lens": lens, "pool": pool, "prefix_pages": order[:first].clone(),
              "prefix_len": torch.full((1,), case["prefix"], dtype=torch.int32, device="cuda"),
              "table": order[first:first + b * width].view(b, width).clone()}
    else:
        pool = b * width + 1
        table = torch.randperm(pool, generator=gen, device="cuda")[:b * width].view(b, width).to(torch.int32)
        st = {"lens": lens, "pool": pool, "table": table}
    if case["op"] in ("weigh", "evict"):
        # Attention weight gathers on few pages: the first and a heavy-tailed rest.
        w = torch.exp(2.0 * _floats(gen, b, hk, width))
        w[..., 0] += 100.0
        st["weights"] = w
    if case["op"] == "evict":
        # Pages of the middle that are gone already.
        gone = torch.rand(b, width, generator=gen, device="cuda") < 0.05
        st["table"] = torch.where(gone, torch.full_like(st["table"], -1), st["table"])
        return st
    hq, d = case["q_heads"], case["head_dim"]
    st["q"] = (1.5 * _floats(gen, b, hq, d)).to(torch.bfloat16)
    st["k"], st["v"] = _keys(gen, pool * ps, hk, d, ps if case["op"] == "sparse" else None)
    return st


# ---- plain forms ---------------------------------------------------------------------------------

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
        return torch.ldexp(x, -e).to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.int8)
    b = x.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    a = b.abs() / torch.where(s > 0, s, torch.ones_like(s))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(s > 0, code + 8 * torch.signbit(b).to(torch.uint8), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.squeeze(-1).view(torch.uint8)


def _decode(parts, fmt):
    """The fp32 values that codes and scales stand for."""
    if fmt == BF16:
        return parts[0].float()
    if fmt == E4M3:
        return torch.ldexp(parts[0].view(torch.float8_e4m3fn).float(), parts[1].int())
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=parts[0].device)
    code = torch.stack((parts[0] & 15, parts[0] >> 4), -1).flatten(-2)
    return (values[code.int()].unflatten(-1, (-1, 16)) * parts[1].view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _read(parts, index, fmt):
    return _decode(tuple(p[index] for p in parts), fmt)


def _sizes(case):
    return tuple(case[n] for n in ("batch", "q_heads", "kv_heads", "head_dim", "page"))


def _weights(s):
    """Scores [...][n], -inf where there is nothing -> (terms, their sum, lse); a row with nothing: zeros and -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, torch.ones_like(total)), (m + torch.log(total)).squeeze(-1)


def _run_shared(st, case):
    b, hq, hk, d, ps = _sizes(case)
    g, prefix, longest = hq // hk, case["prefix"], case["longest"]
    scale, fmt = d ** -0.5, case["fmt"]
    at = torch.arange(prefix, device="cuda")
    rows = st["prefix_pages"].long()[at // ps] * ps + at % ps
    kp, vp = (_read(part, rows, fmt).transpose(0, 1).contiguous() for part in st["cache"])    # [hk][prefix][d]
    at = torch.arange(longest, device="cuda")
    rows = st["table"].long()[:, at // ps] * ps + at % ps
    ko, vo = (_read(part, rows, fmt).transpose(1, 2).contiguous() for part in st["cache"])    # [b][hk][longest][d]
    q = st["q"].float().view(b, hk, g, d)
    sp = torch.matmul(q.transpose(0, 1).reshape(hk, b * g, d), kp.transpose(1, 2))
    sp = sp.view(hk, b, g, prefix).transpose(0, 1) * scale
    so = torch.matmul(q, ko.transpose(2, 3)) * scale
    so = so.masked_fill((at >= st["lens"][:, None])[:, None, None, :], -math.inf)
    p, total, lse = _weights(torch.cat((sp, so), -1))
    o = torch.matmul(p[..., :prefix].transpose(0, 1).reshape(hk, b * g, prefix), vp)
    o = o.view(hk, b, g, d).transpose(0, 1) + torch.matmul(p[..., prefix:], vo)
    return (o / total).reshape(b, hq, d).to(torch.bfloat16), lse.view(b, hq)


def _run_bounds(st, case):
    ps, hk, d = case["page"], case["kv_heads"], case["head_dim"]
    which = st["which"].long()
    rows = which[:, None] * ps + torch.arange(ps, device="cuda")
    k = _read(st["cache"][0], rows, case["fmt"])                                    # [n][ps][hk][d]
    st["bounds"][which] = torch.stack((k.amin(1), k.amax(1)), 2).to(torch.bfloat16)
    return st["bounds"]


def _select(st, case):
    """(chosen pages [b][hk][budget] in ascending order of place, -1 behind them; their tokens [b])."""
    b, hq, hk, d, ps = _sizes(case)
    g, budget = hq // hk, case["budget"]
    table, lens = st["table"].long(), st["lens"].long()
    width = table.shape[1]
    q = st["q"].double().view(b, hk, g, d)
    q = torch.cat((q.clamp(max=0.0), q.clamp(min=0.0)), -1)
    bounds = st["bounds"].view(-1, hk, 2 * d)
    score = torch.empty(b, hk, width, dtype=torch.float64, device="cuda")
    for i in range(b):
        lohi = bounds[table[i]].double().transpose(0, 1).contiguous()               # [hk][width][2 d]
        score[i] = torch.matmul(q[i], lohi.transpose(1, 2)).amax(1)
    blocks = (lens + ps - 1) // ps
    place = torch.arange(width, device="cuda")
    score = score.masked_fill((place >= blocks[:, None])[:, None], -math.inf)
    score = score.masked_fill((place == blocks[:, None] - 1)[:, None], math.inf)    # the newest one
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    if width < budget:
        order = torch.nn.functional.pad(order, (0, budget - width), value=width)
    count = blocks.clamp(max=budget)
    behind = (torch.arange(budget, device="cuda") >= count[:, None])[:, None]
    chosen = order[..., :budget].masked_fill(behind, width).sort(-1).values
    pages = torch.nn.functional.pad(table, (0, 1), value=-1)[:, None].expand(b, hk, width + 1).gather(2, chosen)
    tokens = torch.where(count > 0, (count - 1) * ps + (lens - 1) % ps + 1, count)
    return pages.to(torch.int32), tokens.to(torch.int32)


def _run_sparse(st, case):
    b, hq, hk, d, ps = _sizes(case)
    pages, tokens = _select(st, case)
    at = torch.arange(case["budget"] * ps, device="cuda")
    rows = pages.long().clamp(min=0)[..., at // ps] * ps + at % ps                  # [b][hk][budget * ps]
    head = torch.arange(hk, device="cuda")[:, None]
    k, v = (_read(part, (rows, head), case["fmt"]) for part in st["cache"])
    s = torch.matmul(st["q"].float().view(b, hk, hq // hk, d), k.transpose(2, 3)) * d ** -0.5
    s = s.masked_fill((at >= tokens[:, None])[:, None, None], -math.inf)
    p, total, lse = _weights(s)
    o = torch.matmul(p, v) / total
    return o.reshape(b, hq, d).to(torch.bfloat16), lse.view(b, hq), pages, tokens


def _run_weigh(st, case):
    b, hq, hk, d, ps = _sizes(case)
    width = st["table"].shape[1]
    at = torch.arange(width * ps, device="cuda")
    lens = st["lens"][:, None]
    valid = (at < lens) & ((at >= lens - case["window"]) if case["window"] else (at >= 0))
    rows = st["table"].long()[:, at // ps] * ps + at % ps
    k, v = (_read(part, rows, case["fmt"]).transpose(1, 2).contiguous() for part in st["cache"])
    s = torch.matmul(st["q"].float().view(b, hk, hq // hk, d), k.transpose(2, 3)) * d ** -0.5
    p, total, lse = _weights(s.masked_fill(~valid[:, None, None], -math.inf))
    o = torch.matmul(p, v) / total
    mass = (p / total).sum(2).view(b, hk, width, ps).sum(-1)
    return o.reshape(b, hq, d).to(torch.bfloat16), lse.view(b, hq), case["decay"] * st["weights"] + mass


def _run_evict(st, case):
    """(kept pages [b][budget] in order, their tokens [b], dropped pages [b][width] in order, kept weights [b][hk][budget])."""
    b, hk, ps, budget = case["batch"], case["kv_heads"], case["page"], case["budget"]
    table, lens, weights = st["table"].long(), st["lens"].long(), st["weights"]
    width = table.shape[1]
    blocks = ((lens + ps - 1) // ps)[:, None]
    place = torch.arange(width, device="cuda")
    there = (table >= 0) & (place < blocks) | (place == blocks - 1)
    # The newest ones first, then the oldest, then by weight.
    rank = weights.double().sum(1)
    rank = torch.where(place < case["sink"], math.inf, rank)
    keys = [torch.where(there, rank, -math.inf), torch.where(there & (place >= blocks - case["recent"]), place + 1, 0)]
    order = torch.sort(keys[0], dim=-1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(keys[1].gather(1, order), dim=-1, descending=True, stable=True).indices)
    if width < budget:
        order = torch.nn.functional.pad(order, (0, budget - width), value=width)
    count = there.sum(1).clamp(max=budget)
    chosen = order[:, :budget].masked_fill(torch.arange(budget, device="cuda") >= count[:, None], width).sort(-1).values
    pages = torch.nn.functional.pad(table, (0, 1), value=-1).gather(1, chosen)
    moved = torch.nn.functional.pad(weights, (0, 1)).gather(2, chosen[:, None].expand(b, hk, budget))
    tokens = torch.where(count > 0, (count - 1) * ps + (lens - 1) % ps + 1, count)
    dropped = there & (table >= 0)
    dropped = torch.nn.functional.pad(dropped, (0, 1)).scatter(1, chosen, False)[:, :width]
    first = torch.sort(torch.where(dropped, place, width), -1).values
    freed = torch.nn.functional.pad(table, (0, 1), value=-1).gather(1, first)
    return pages.to(torch.int32), tokens.to(torch.int32), freed.to(torch.int32), moved


# ---- what is measured ----------------------------------------------------------------------------

def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        # A serving program keeps its cache in the library's layout and the marshalled arguments of its calls.
        from bit_quantized_decode_amd import binding as B
        scale = None if case["op"] == "evict" else case["head_dim"] ** -0.5
        fmt = {BF16: B.NVFP4_KV_BF16, E4M3: B.NVFP4_KV_E4M3, NVFP4: B.NVFP4_KV_NVFP4}[case.get("fmt", BF16)]
        if case["op"] == "evict":
            st["call"] = B.kv_evict_prepared(st["weights"], st["table"], st["lens"], case["page"], case["budget"],
                                             sink=case["sink"], recent=case["recent"])
            return st
        cache = B.KvCache(st["pool"], case["page"], case["kv_heads"], case["head_dim"], fmt, device="cuda")
        B.kv_append(cache, st.pop("k"), st.pop("v"), torch.arange(st["pool"] * case["page"], device="cuda"))
        if case["op"] == "shared":
            st["call"] = B.attn_shared_prepared(st["q"], cache, st["prefix_pages"], st["prefix_len"], st["table"], st["lens"],
                                                scale=scale, lse=True)
        elif case["op"] == "bounds":
            st["call"] = B.kv_bounds_prepared(cache, st["which"])
        elif case["op"] == "sparse":
            bounds = B.kv_bounds(cache, torch.arange(st["pool"], dtype=torch.int32, device="cuda"))
            st["select"] = B.kv_select_prepared(st["q"], cache, bounds, st["table"], st["lens"], case["budget"])
            pages, tokens = st["select"].outputs
            st["call"] = B.attn_decode_prepared(st["q"], cache, pages, tokens, scale=scale, lse=True)
        else:
            st["call"] = B.attn_weigh_prepared(st["q"], cache, st["table"], st["lens"], st["weights"], decay=case["decay"],
                                               weights_out=torch.empty_like(st["weights"]), scale=scale,
                                               window=case["window"], lse=True)
        return st
    if case["op"] != "evict":
        st["cache"] = [_encode(st.pop(name), case["fmt"]) for name in ("k", "v")]
    if case["op"] in ("bounds", "sparse"):
        hk, d, ps = case["kv_heads"], case["head_dim"], case["page"]
        st["bounds"] = torch.zeros(st["pool"], hk, 2, d, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "sparse":
            for i in range(0, st["pool"], 256):
                part = tuple(p[i * ps:(i + 256) * ps] for p in st["cache"][0])
                k = _decode(part, case["fmt"]).view(-1, ps, hk, d)
                st["bounds"][i:i + 256] = torch.stack((k.amin(1), k.amax(1)), 2).to(torch.bfloat16)
    return st


_PLAIN = {"shared": _run_shared, "bounds": _run_bounds, "sparse": _run_sparse, "weigh": _run_weigh, "evict": _run_evict}


def run(st):
    case = st["case"]
    if not own:
        return _PLAIN[case["op"]](st, case)
    if case["op"] == "sparse":
        pages, tokens = st["select"]()
        return *st["call"](), pages, tokens
    return st["call"]()


def _row_bytes(fmt, head_dim):
    """Bytes of one token's k or v of one head."""
    return {BF16: 2 * head_dim, E4M3: head_dim + 1, NVFP4: head_dim // 2 + head_dim // 16}[fmt]


def _mean(case, of):
    """The sum over the batch of of(length): the mean over a case's random lengths, whatever the seed."""
    b, longest = case["batch"], case["longest"]
    if not case.get("ragged", True):
        return b * of(longest)
    inner = sum(of(n) for n in range(1, longest + 1)) / longest
    return of(longest) + inner * (b - 1 - (b > 4))


def work(case):
    op, hk, ps = case["op"], case["kv_heads"], case["page"]
    if op == "evict":
        pages = _mean(case, lambda n: -(-n // ps))
        width, budget, b = -(-case["longest"] // ps), case["budget"], case["batch"]
        # Weights, table and lengths in; kept pages and weights, dropped pages, lengths out.
        return {"bytes": round(pages * (4 * hk + 4) + b * (8 + 4 * width + budget * (4 + 4 * hk))), "flops": round(pages * hk)}
    d = case["head_dim"]
    row = _row_bytes(case["fmt"], d)
    if op == "bounds":
        tokens = case["pages"] * ps * hk
        return {"bytes": tokens * row + case["pages"] * (hk * 4 * d + 4), "flops": 2 * tokens * d}
    b, hq = case["batch"], case["q_heads"]
    rows = b * hq * (4 * d + 4)                     # q in, o and lse out
    if op == "shared":
        tokens = _mean(case, lambda n: n)
        return {"bytes": round(2 * (case["prefix"] + tokens) * hk * row + rows + 4 * b),
                "flops": round(4 * (b * case["prefix"] + tokens) * hq * d)}
    if op == "sparse":
        # Bounds are looked at only where there is a choice.
        scored = _mean(case, lambda n: 0 if -(-n // ps) <= case["budget"] else -(-n // ps) - 1)
        tokens = _mean(case, lambda n: n if -(-n // ps) <= case["budget"] else (case["budget"] - 1) * ps + (n - 1) % ps + 1)
        return {"bytes": round(scored * hk * 4 * d + 2 * tokens * hk * row + rows + 4 * b * hk * case["budget"]),
                "flops": round(2 * scored * hq * d + 4 * tokens * hq * d)}
    w = case["window"]
    tokens = _mean(case, lambda n: min(n, w) if w else n)
    width = -(-case["longest"] // ps)
    return {"bytes": round(2 * tokens * hk * row + rows + 8 * b * hk * width), "flops": round(4 * tokens * hq * d)}


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


def _slots(pages, tokens, ps):
    at = torch.arange(tokens, device="cuda")
    return pages.long()[at // ps] * ps + at % ps


def exact(case, seed):
    st = _inputs(case, seed)
    op, hk, ps = case["op"], case["kv_heads"], case["page"]
    if op == "evict":
        return _exact_evict(st, case)
    d, fmt = case["head_dim"], case["fmt"]
    if op == "bounds":
        out = torch.empty(st["pool"], hk, 2, d, dtype=torch.float64, device="cuda")
        for i in range(0, st["pool"], 64):
            k = _stored(st["k"][i * ps:(i + 64) * ps], fmt).view(-1, ps, hk, d).sort(1).values
            out[i:i + 64] = torch.stack((k[:, 0], k[:, -1]), 2)
        return out
    b, hq = case["batch"], case["q_heads"]
    g = hq // hk
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    if op == "shared":
        rows = _slots(st["prefix_pages"], case["prefix"], ps)
        for h in range(hk):
            kp, vp = (_stored(st[n][rows, h], fmt) for n in ("k", "v"))
            for i in range(b):
                mine = _slots(st["table"][i], lens[i], ps)
                k, v = (torch.cat((p, _stored(st[n][mine, h], fmt))) for p, n in ((kp, "k"), (vp, "v")))
                s = st["q"][i, h * g:(h + 1) * g].double() @ k.t() / math.sqrt(d)
                lse[i, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
                out[i, h * g:(h + 1) * g] = torch.softmax(s, -1) @ v
        return out, lse
    if op == "sparse":
        pages = torch.full((b, hk, case["budget"]), -1, dtype=torch.int32, device="cuda")
        tokens = torch.zeros(b, dtype=torch.int32, device="cuda")
        for i in range(b):
            blocks = -(-lens[i] // ps)
            if not blocks:
                continue
            count = min(blocks, case["budget"])
            tokens[i] = (count - 1) * ps + lens[i] - (blocks - 1) * ps
            held = st["k"].view(-1, ps, hk, d)[st["table"][i, :blocks].long()]
            for h in range(hk):
                k = _stored(held[:, :, h], fmt)                             # [blocks][ps][d]
                low, high = k.amin(1), k.amax(1)
                q = st["q"][i, h * g:(h + 1) * g].double()
                best = torch.full((blocks,), -math.inf, dtype=torch.float64, device="cuda")
                for r in range(g):
                    best = torch.maximum(best, torch.maximum(q[r] * low, q[r] * high).sum(-1))
                order = torch.sort(best[:-1], descending=True, stable=True).indices[:count - 1]
                chosen = torch.cat((order.sort().values, torch.tensor([blocks - 1], device="cuda")))
                pages[i, h, :count] = st["table"][i][chosen]
                mine = _slots(pages[i, h], int((count - 1) * ps + lens[i] - (blocks - 1) * ps), ps)
                k, v = (_stored(st[n][mine, h], fmt) for n in ("k", "v"))
                s = q @ k.t() / math.sqrt(d)
                lse[i, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
                out[i, h * g:(h + 1) * g] = torch.softmax(s, -1) @ v
        return out, lse, pages, tokens
    weights = case["decay"] * st["weights"].double()
    for i in range(b):
        first = max(0, lens[i] - case["window"]) if case["window"] else 0
        if lens[i] <= first:
            continue
        mine = _slots(st["table"][i], lens[i], ps)[first:]
        page = torch.arange(first, lens[i], device="cuda") // ps
        for h in range(hk):
            k, v = (_stored(st[n][mine, h], fmt) for n in ("k", "v"))
            s = st["q"][i, h * g:(h + 1) * g].double() @ k.t() / math.sqrt(d)
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            out[i, h * g:(h + 1) * g] = p @ v
            weights[i, h].index_add_(0, page, p.sum(0))
    return out, lse, weights


def _exact_evict(st, case):
    b, hk, ps, budget = case["batch"], case["kv_heads"], case["page"], case["budget"]
    table, weights = st["table"].cpu(), st["weights"].double().cpu()
    width = table.shape[1]
    pages = torch.full((b, budget), -1, dtype=torch.int32)
    freed = torch.full((b, width), -1, dtype=torch.int32)
    tokens = torch.zeros(b, dtype=torch.int32)
    moved = torch.zeros(b, hk, budget, dtype=torch.float64)
    for i, n in enumerate(st["lens"].tolist()):
        blocks = -(-n // ps)
        there = [j for j in range(blocks) if table[i, j] >= 0 or j == blocks - 1]
        heavy = weights[i].sum(0).tolist()
        last = [j for j in reversed(there) if j >= blocks - case["recent"]]
        rest = [j for j in there if j < blocks - case["recent"]]
        first = [j for j in rest if j < case["sink"]]
        rest = sorted((j for j in rest if j >= case["sink"]), key=lambda j: (-heavy[j], j))
        keep = sorted((last + first + rest)[:budget])
        drop = [j for j in there if j not in set(keep) and table[i, j] >= 0]
        for at, j in enumerate(keep):
            pages[i, at] = table[i, j]
            moved[i, :, at] = weights[i, :, j]
        for at, j in enumerate(drop):
            freed[i, at] = table[i, j]
        if keep:
            tokens[i] = (len(keep) - 1) * ps + n - (blocks - 1) * ps
    return pages.cuda(), tokens.cuda(), freed.cuda(), moved.cuda()
