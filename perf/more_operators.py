"""The calls of a server of many requests and what measures them: packed prompts and an 8-bit paged cache.

Three families, each with its plain form (elementary torch operations in 32 bits, or 64 where 32 lose what
matters) and its value in 64 bits:

* ``append``  new keys and values of every sequence into a paged cache of e4m3 bytes with one scale, a power of
              two, for each page and head, the keys rotated (NeoX) on the way;
* ``paged``   attention of the few new tokens of a serving step over that cache: one token, a run of tokens, or a
              tree of drafted ones;
* ``packed``  causal attention over whole prompts of different lengths that follow each other in one buffer, with
              grouped heads.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BASE = 10000.0
TOP = 448.0       # largest e4m3 value
FLOOR = -32       # smallest exponent of a scale


def listed():
    return [
        # one new token of 8 sequences: the call between the projection and the attention, where latency is all
        {"name": "append_token", "op": "append", "type": "bf16", "batch": 8, "kv_heads": 4, "tokens": 1, "total": 0, "cap": 5000,
         "dim": 64, "rope": 64, "page": 16, "factors": False},
        # the prompts of 6 requests, 16384 tokens, into new pages, k and v views of the packed projection
        {"name": "append_prompts", "op": "append", "type": "bf16", "batch": 6, "kv_heads": 8, "tokens": 0, "total": 16384, "cap": 0,
         "dim": 128, "rope": 128, "page": 64, "factors": False},
        # the next parts of long prompts, into pages begun before, odd sizes, part of the head rotated, divisors
        {"name": "append_parts", "op": "append", "type": "f16", "batch": 3, "kv_heads": 2, "tokens": 0, "total": 2309, "cap": 3001,
         "dim": 80, "rope": 48, "page": 48, "factors": True},
        # one token for each of 4 sequences over short caches: latency
        {"name": "paged_short", "op": "paged", "type": "f16", "batch": 4, "heads": 16, "kv_heads": 4, "tokens": 1, "cap": 700,
         "dim": 64, "page": 16, "window": 0, "sinks": 0, "tree": False},
        # one token for each of 32 sequences over caches of up to 16385 keys
        {"name": "paged_token", "op": "paged", "type": "bf16", "batch": 32, "heads": 32, "kv_heads": 8, "tokens": 1, "cap": 16385,
         "dim": 128, "page": 64, "window": 0, "sinks": 0, "tree": False},
        # one long sequence: few rows, a long axis
        {"name": "paged_long", "op": "paged", "type": "bf16", "batch": 1, "heads": 8, "kv_heads": 1, "tokens": 1, "cap": 200003,
         "dim": 128, "page": 128, "window": 0, "sinks": 0, "tree": False},
        # a tree of 31 drafted tokens for 4 sequences, window layer
        {"name": "paged_tree", "op": "paged", "type": "f16", "batch": 4, "heads": 16, "kv_heads": 4, "tokens": 31, "cap": 5000,
         "dim": 64, "page": 32, "window": 4096, "sinks": 4, "tree": True},
        # three new tokens of 12 sequences under a window with first keys, odd sizes
        {"name": "paged_window", "op": "paged", "type": "bf16", "batch": 12, "heads": 6, "kv_heads": 2, "tokens": 3, "cap": 9001,
         "dim": 80, "page": 48, "window": 2000, "sinks": 70, "tree": False},
        # five short prompts, the library's smallest head
        {"name": "packed_short", "op": "packed", "type": "f16", "batch": 5, "heads": 2, "kv_heads": 2, "total": 200, "dim": 32,
         "window": 0, "sinks": 0, "skew": False},
        # a batch of prompts of 400 to 1900 tokens
        {"name": "packed_prompts", "op": "packed", "type": "bf16", "batch": 8, "heads": 16, "kv_heads": 4, "total": 8192, "dim": 128,
         "window": 0, "sinks": 0, "skew": False},
        # one long prompt among short ones
        {"name": "packed_long", "op": "packed", "type": "bf16", "batch": 4, "heads": 32, "kv_heads": 8, "total": 8192, "dim": 128,
         "window": 0, "sinks": 0, "skew": True},
        # a window layer with first keys, odd sizes
        {"name": "packed_window", "op": "packed", "type": "f16", "batch": 7, "heads": 12, "kv_heads": 4, "total": 6001, "dim": 72,
         "window": 500, "sinks": 1, "skew": False},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    heads = rng.choice([(2, 2), (8, 1), (6, 2), (16, 4), (16, 16), (12, 4), (5, 1), (32, 8)])
    kind = rng.choice(["append", "paged", "paged", "packed"])
    dtype = rng.choice(["bf16", "f16"])
    if kind == "packed":
        batch = _log(rng, 1, 40)
        case = {"op": "packed", "type": dtype, "batch": batch, "heads": heads[0], "kv_heads": heads[1],
                "total": _log(rng, max(17, batch), 8192), "dim": 8 * rng.randint(4, 16),
                "window": rng.choice([0, 0, _log(rng, 16, 2048)]), "sinks": rng.choice([0, 1, 4, 130]), "skew": rng.random() < 0.4}
        dear = work(listed()[10])["flops"]
        while work(case)["flops"] > dear:  # no dearer than the listed long prompt
            case["total"] = case["total"] * 7 // 8
        return case
    dim, page = 16 * rng.randint(2, 8), rng.choice([16, 32, 48, 64, 128, 256])
    batch = _log(rng, 1, 32)
    if kind == "append":
        if rng.random() < 0.5:  # new tokens, as many for each sequence
            tokens = rng.choice([1, 1, 2, rng.randint(3, 64)])
            return {"op": "append", "type": dtype, "batch": batch, "kv_heads": heads[1], "tokens": tokens, "total": 0,
                    "cap": _log(rng, 64, 9000), "dim": dim, "rope": rng.choice([dim, dim, dim // 2]), "page": page,
                    "factors": rng.random() < 0.3}
        most = min(16384, 16384 * 8 * 128 // (heads[1] * dim))
        return {"op": "append", "type": dtype, "batch": batch, "kv_heads": heads[1], "tokens": 0, "total": _log(rng, 2 * batch + 16, most),
                "cap": rng.choice([0, 0, _log(rng, 16, 4000)]), "dim": dim, "rope": rng.choice([dim, dim, dim // 2]), "page": page,
                "factors": rng.random() < 0.3}
    tokens = rng.choice([1, 1, 2, rng.randint(3, 64)])
    return {"op": "paged", "type": dtype, "batch": batch, "heads": heads[0], "kv_heads": heads[1], "tokens": tokens,
            "cap": _log(rng, 200, min(200000, max(201, 16384 * 32 * 8 // (batch * max(8, heads[1] * (1 + tokens // 8)))))),
            "dim": dim, "page": page, "window": rng.choice([0, 0, _log(rng, 64, 4096)]), "sinks": rng.choice([0, 4, 70]),
            "tree": tokens > 2 and rng.random() < 0.7}


def _parts(total, batch, skew):
    """`total` tokens as `batch` lengths of at least one: from short to long, or the first taking most."""
    weight = [1.0 + 4.0 * b / max(1, batch - 1) for b in range(batch)]
    if skew:
        weight[0] = 3.0 * sum(weight)
    free = total - batch
    lens = [1 + int(free * w / sum(weight)) for w in weight]
    lens[-1] += total - sum(lens)
    return lens


def _lengths(case):
    """(lengths of the sequences with their new tokens, how many of them are new)."""
    B = case["batch"]
    if case["op"] == "packed":
        lens = _parts(case["total"], B, case["skew"])
        return lens, lens
    if case["op"] == "append" and case["total"]:
        new = _parts(case["total"], B, False)
        before = [(case["cap"] * (b + 1)) // B for b in range(B)]
        return [x + y for x, y in zip(before, new)], new
    n, T = case["cap"], case["tokens"]
    return [max(min(n, T), n - (n * 2 * b) // (3 * B) - 3 * b) for b in range(B)], [min(n, T)] * B


def _tree(tokens, seed):
    """Ancestor bits (itself among them) of each node of a random tree, in a signed 64-bit word each."""
    g = torch.Generator().manual_seed(seed)
    bits = [1]
    for t in range(1, tokens):
        bits.append(bits[int(torch.randint(0, t, (1,), generator=g))] | (1 << t))
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, K, D = DTYPES[case["type"]], case["batch"], case["kv_heads"], case["dim"]
    lens, new = _lengths(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    s = {"case": case, "scale": D ** -0.5}
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    if case["op"] == "packed":  # views of the projection's output [total, H + 2 K, D]
        H = case["heads"]
        qkv = normal(1, case["total"], H + 2 * K, D).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + K].transpose(1, 2), qkv[:, :, H + K:].transpose(1, 2)
        s["cu"] = ints(starts)
        return s
    # the cache: pages in any order, three of them nobody's, values as they are after many appends
    page = case["page"]
    most = max(-(-n // page) for n in lens)
    n_pages = B * most + 3
    order = torch.randperm(n_pages, generator=g, device="cuda")[:B * most]
    s["table"] = order.to(torch.int32).view(B, most)
    s["len"] = ints(lens)
    for name in "kv":
        x = normal(n_pages, K, page, D).mul_(torch.exp2(normal(n_pages, K, 1, 1)))
        scale = _power(x.abs().amax((2, 3)))
        s[name + "_pages"], s[name + "_scale"] = x.div_(scale[:, :, None, None]).to(torch.float8_e4m3fn), scale
    if case["op"] == "append":
        s["cu"] = None
        if case["total"]:
            qkv = normal(1, case["total"], 2 * K, D).to(dt)
            s["cu"] = ints(starts)
        else:
            qkv = normal(B, case["tokens"], 2 * K, D).to(dt)
        s["k"], s["v"] = qkv[:, :, :K].transpose(1, 2), qkv[:, :, K:].transpose(1, 2)
        s["factors"] = 1 + 7 * torch.rand(case["rope"] // 2, generator=g, device="cuda") if case["factors"] else None
        return s
    s["q"] = normal(B, case["tokens"], case["heads"], D).to(dt).transpose(1, 2)
    s["tree"] = None
    if case["tree"]:
        s["tree"] = torch.tensor([_tree(case["tokens"], seed * 100 + b) for b in range(B)], dtype=torch.int64, device="cuda")
    return s


def run(state):
    c = state["case"]
    if own:
        return _library(state, c)
    return {"append": _plain_append, "paged": _plain_paged, "packed": _plain_packed}[c["op"]](state, c)


def _library(s, c):
    import vision_encoder_flash_gb300 as vef

    window = c.get("window") or None
    if c["op"] == "packed":
        return vef.forward_packed(s["q"], s["k"], s["v"], s["cu"], window=window, n_sinks=c["sinks"], scale=s["scale"])
    cache = (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["len"])
    if c["op"] == "append":
        vef.append_paged(s["k"], s["v"], *cache, cu_seqlens=s["cu"], rope_dims=c["rope"], base=BASE, factors=s["factors"])
        return cache[:4]
    return vef.forward_paged(s["q"], *cache, tree_mask=s["tree"], window=window, n_sinks=c["sinks"], scale=s["scale"])


# ---------------------------------------------------------------- the plain forms

def _power(amax):
    """The smallest power of two whose e4m3 values reach `amax`."""
    m, e = torch.frexp(amax / TOP)  # amax / 448 = m 2^e, 1/2 <= m < 1
    e = torch.where(m > 0.5, e, e - 1).clamp_min(FLOOR)
    return torch.exp2(torch.where(amax > 0, e, torch.full_like(e, FLOOR)).double()).float()


def _places(s, c):
    """Of each new token, in the order of the buffer: its sequence and its row of the sequence."""
    B = c["batch"]
    if s["cu"] is None:
        T = c["tokens"]
        b = torch.arange(B, device="cuda").repeat_interleave(T)
        i, n = torch.arange(T, device="cuda").repeat(B), T
    else:
        cu, t = s["cu"].long(), torch.arange(c["total"], device="cuda")
        b = torch.bucketize(t, cu[1:], right=True)
        i, n = t - cu[b], (cu[1:] - cu[:-1])[b]
    return b, s["len"].long()[b] - n + i, i


def _plain_append(s, c):
    page, half = c["page"], c["rope"] // 2
    b, row, i = _places(s, c)
    P, r = s["table"].long()[b, row // page], row % page
    inv = BASE ** (torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 / c["rope"]))
    if s["factors"] is not None:
        inv = inv / s["factors"].double()
    theta = row.double()[:, None, None] * inv
    cos, sin = torch.cos(theta).float(), torch.sin(theta).float()
    first = torch.zeros(s["k_scale"].shape[0], device="cuda")  # pages whose row 0 is written start anew
    first = first.index_put((P,), (r == 0).float(), accumulate=True)
    older = row[i == 0] if s["cu"] is not None else row.view(c["batch"], -1)[:, 0]
    old_page, old_rows = s["table"].long().gather(1, (older // page)[:, None])[:, 0], older % page
    for name in "kv":
        x = s[name].transpose(1, 2).flatten(0, 1).float()  # [tokens, K, D]
        if name == "k":
            a, z = x[..., :half], x[..., half:2 * half]
            x = torch.cat([a * cos - z * sin, a * sin + z * cos, x[..., 2 * half:]], -1)
        pages, scale = s[name + "_pages"].view(torch.uint8), s[name + "_scale"]
        top = torch.zeros_like(scale).index_reduce_(0, P, x.abs().amax(-1), "amax")
        was = torch.where(first[:, None] > 0, torch.zeros_like(scale), scale)
        now = torch.where(top > 0, torch.maximum(was, _power(top)), scale)
        # the rows before the new ones, in the one page of each sequence that has such
        held = pages[old_page].view(torch.float8_e4m3fn).float() * (scale / now)[old_page][:, :, None, None]
        before = torch.arange(page, device="cuda")[None, :] < old_rows[:, None]
        held = torch.where(before[:, None, :, None], held.to(torch.float8_e4m3fn).view(torch.uint8), pages[old_page])
        pages[old_page] = held
        pages[P, :, r] = (x / now[P][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(now)
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _paged_visible(s, c):
    """[B, 1, 1, tokens, rows of the cache]: which of them each new token sees."""
    T, dev, cap = c["tokens"], "cuda", s["table"].shape[1] * c["page"]
    t = torch.arange(T, device=dev)
    first = s["len"].long()[:, None] - T  # cache row of the first new token
    anc = (t[None, :, None] >= t[None, None, :]).expand(c["batch"], T, T) if s["tree"] is None else \
        ((s["tree"][:, :, None] >> t[None, None, :]) & 1).bool()
    pos = first + anc.sum(-1) - 1  # a new token's position: behind its ancestors
    j = torch.arange(cap, device=dev)[None, :]
    u = j - first  # which new token a cache row holds
    new = (u >= 0) & (u < T)
    keypos = torch.where(new, pos.gather(1, u.clamp(0, T - 1)), j)[:, None, :]
    path = anc.gather(2, u.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
    seen = ((u < 0)[:, None, :] | (new[:, None, :] & path)) & ((keypos > pos[..., None] - (c["window"] or (cap + T))) | (keypos < c["sinks"]))
    return seen[:, None, None]


def _plain_paged(s, c):
    B, H, K, D = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    table = s["table"].long()

    def rows(name):  # [B, K, 1, rows, D] in 32 bits
        x = s[name + "_pages"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        return x.mul_(s[name + "_scale"][table][..., None, None]).transpose(1, 2).flatten(2, 3)[:, :, None]

    q = s["q"].float().unflatten(1, (K, H // K))
    x = (torch.matmul(q, rows("k").transpose(-1, -2)) * s["scale"]).masked_fill_(~_paged_visible(s, c), -math.inf)
    return torch.matmul(_weights(x), rows("v")).flatten(1, 2).to(DTYPES[c["type"]])


def _weights(x):
    """Softmax over the last dimension, zeros where it is -infinity throughout; in place."""
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    return x.div_(x.sum(-1, keepdim=True).clamp_min(1e-30))


def _plain_packed(s, c):
    """Every sequence padded to the longest."""
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    most = max(_lengths(c)[0])
    cu, i = s["cu"].long(), torch.arange(most, device="cuda")
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i[None]).clamp_max(c["total"] - 1)  # [B, most]

    def rows(x):
        return x[0].float()[:, at].transpose(0, 1)  # [B, heads, most, D]

    q, k, v = rows(s["q"]).unflatten(1, (K, H // K)), rows(s["k"])[:, :, None], rows(s["v"])[:, :, None]
    p, j = i[:, None], i[None, :]
    seen = (j <= p) & ((j > p - (c["window"] or most)) | (j < c["sinks"]))
    x = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).masked_fill_(~seen, -math.inf)
    out = torch.matmul(_weights(x), v).flatten(1, 2).to(DTYPES[c["type"]])  # [B, H, most, D]
    t = torch.arange(c["total"], device="cuda")
    b = torch.bucketize(t, cu[1:], right=True)
    return out[b, :, t - cu[b]].transpose(0, 1)[None]


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "paged": _exact_paged, "packed": _exact_packed}[case["op"]](s, case)


def _exact_append(s, c):
    """What the bytes stand for in units of their scale, before the rounding to 8 bits; the scales."""
    page, half, (lens, new) = c["page"], c["rope"] // 2, _lengths(c)
    freq = torch.exp(torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 * math.log(BASE) / c["rope"]))
    if s["factors"] is not None:
        freq = freq / s["factors"].double()
    pools = {n: s[n + "_pages"].double() for n in "kv"}
    scales = {n: s[n + "_scale"].double() for n in "kv"}
    table, at = s["table"].tolist(), 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for name in "kv":
            x = (s[name][0, :, at:at + m] if c["total"] else s[name][b]).double()  # [K, m, D]
            if name == "k":
                pos = torch.arange(n - m, n, device="cuda", dtype=torch.float64)
                z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous())
                z = z * torch.polar(torch.ones((), device="cuda", dtype=torch.float64), pos[:, None] * freq)
                x = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
            done = 0
            while done < m:
                row = n - m + done
                lo, take, where = row % page, min(page - row % page, m - done), table[b][row // page]
                part = x[:, done:done + take]
                e = torch.ceil(torch.log2(part.abs().amax((1, 2)) / TOP) - 1e-12).clamp_min(FLOOR)
                old, scale = scales[name][where], 2.0 ** e
                if lo:
                    scale = torch.maximum(scale, old)
                    pools[name][where, :, :lo] *= (old / scale)[:, None, None]
                scales[name][where] = scale
                pools[name][where, :, lo:lo + take] = part / scale[:, None, None]
                done += take
        at += m
    return pools["k"], pools["v"], scales["k"], scales["v"]


def _exact_paged(s, c):
    """One head of one sequence at a time."""
    H, K, T, D, page = c["heads"], c["kv_heads"], c["tokens"], c["dim"], c["page"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    for b, L in enumerate(_lengths(c)[0]):
        words = [(1 << (t + 1)) - 1 for t in range(T)] if s["tree"] is None else [int(x) & (2 ** 64 - 1) for x in s["tree"][b]]
        depth = [bin(x).count("1") - 1 for x in words]
        at = torch.tensor([L - T + d for d in depth], device="cuda")
        key_at = torch.cat([torch.arange(L - T, device="cuda"), at])
        path = torch.tensor([[(x >> u) & 1 for u in range(T)] for x in words], device="cuda").bool()
        seen = torch.cat([torch.ones(T, L - T, device="cuda", dtype=torch.bool), path], 1)
        if c["window"]:
            seen = seen & ((at[:, None] - key_at[None, :] < c["window"]) | (key_at[None, :] < c["sinks"]))
        ids = s["table"][b, :-(-L // page)].long()
        for e in range(K):
            k, v = ((s[n + "_pages"][:, e].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                     * s[n + "_scale"][ids, e].double()[:, None, None]).flatten(0, 1)[:L] for n in "kv")
            for h in range(e * (H // K), (e + 1) * (H // K)):
                w = torch.softmax((s["q"][b, h].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf), -1)
                out[b, h] = w @ v
    return out


def _exact_packed(s, c):
    H, K = c["heads"], c["kv_heads"]
    out, at = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64), 0
    for n in _lengths(c)[0]:
        i = torch.arange(n, device="cuda")
        hidden = i[:, None] < i[None, :]
        if c["window"]:
            hidden = hidden | ((i[:, None] - i[None, :] >= c["window"]) & (i[None, :] >= c["sinks"]))
        for h in range(H):
            q, k, v = (s[x][0, y, at:at + n].double() for x, y in (("q", h), ("k", h // (H // K)), ("v", h // (H // K))))
            out[0, h, at:at + n] = torch.softmax((q @ k.T * s["scale"]).masked_fill(hidden, -math.inf), -1) @ v
        at += n
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, K, D = case["batch"], case["kv_heads"], case["dim"]
    lens, new = _lengths(case)
    if case["op"] == "append":  # k and v in 16 bits in, 8 bits and the scales out
        n, pages = sum(new), sum(-(-x // case["page"]) - (x - y) // case["page"] for x, y in zip(lens, new))
        return {"bytes": n * K * D * 6 + pages * (K * 8 + 4), "flops": n * K * (8 * D + 3 * case["rope"])}
    H, W, sinks = case["heads"], case["window"], case["sinks"]
    if case["op"] == "packed":
        return {"bytes": sum(lens) * (H + K) * 4 * D, "flops": sum(_pairs(n, W or n, sinks) for n in lens) * H * D * 4}
    T = case["tokens"]
    keys = sum(n if not W else min(n, W + T + sinks) for n in lens)
    return {"bytes": keys * K * 2 * D + 4 * B * H * T * D, "flops": keys * T * H * D * 4}


def _pairs(n, window, sinks):
    """Visible (query, key) pairs of n queries over their own n keys."""
    w, full = min(window, n), min(window, n) * (min(window, n) + 1) // 2
    inside = full + (n - w) * w
    extra = max(0, n - w)  # query w + x sees min(sinks, x + 1) keys before its window
    a = min(extra, sinks)
    return inside + a * (a + 1) // 2 + (extra - a) * sinks
