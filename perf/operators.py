"""The decoder-side attention operators and the calls that measure them.

Three families, each with its plain form (elementary torch operations in 32 bits, or 64 where 32 lose what
matters), its library call and its value in 64 bits:

* ``qk``      RMS norm of every q and k row (one head of one token) and the NeoX rotation, in one pass, and
              its gradients;
* ``window``  causal attention in which a query sees the last ``window`` keys and the first ``n_sinks`` ones,
              with grouped heads, per-sequence lengths, and its gradients;
* ``cached``  the same attention for the few new tokens of a serving step over a cache of keys and values:
              one token, a run of tokens, or a tree of drafted ones.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
BASE = 10000.0


def listed():
    return [
        # one new token of 8 sequences: the call between the projection and the cache, where latency is all
        {"name": "qk_token", "op": "qk", "grad": False, "type": "bf16", "batch": 8, "heads": 16, "kv_heads": 4, "n": 1,
         "dim": 64, "rope": 64, "packed": False, "weights": True, "far": 100000},
        # the library's odd image shape (16 heads, 4100 rows of 72) in its own type, no weights
        {"name": "qk_rows72", "op": "qk", "grad": False, "type": "f32", "batch": 1, "heads": 16, "kv_heads": 16, "n": 4100,
         "dim": 72, "rope": 72, "packed": False, "weights": False, "far": 0},
        # a large prompt batch, q and k read in place from the packed projection [batch, n, heads, dim]
        {"name": "qk_prompt", "op": "qk", "grad": False, "type": "bf16", "batch": 4, "heads": 32, "kv_heads": 8, "n": 4096,
         "dim": 128, "rope": 128, "packed": True, "weights": True, "far": 0},
        # a training step's way back through the same pass
        {"name": "qk_grad", "op": "qk", "grad": True, "type": "bf16", "batch": 4, "heads": 16, "kv_heads": 4, "n": 4096,
         "dim": 128, "rope": 128, "packed": True, "weights": True, "far": 0},
        # the same with odd sizes and a rotation of part of the head
        {"name": "qk_grad_part", "op": "qk", "grad": True, "type": "f16", "batch": 2, "heads": 6, "kv_heads": 2, "n": 1025,
         "dim": 80, "rope": 48, "packed": False, "weights": True, "far": 5000},
        # the library's smallest shape, a short prompt
        {"name": "window_short", "op": "window", "grad": False, "type": "f16", "batch": 1, "heads": 2, "kv_heads": 2, "n": 64,
         "dim": 32, "window": 32, "sinks": 2, "ragged": False},
        # a long prompt under a window, grouped heads
        {"name": "window_prompt", "op": "window", "grad": False, "type": "bf16", "batch": 1, "heads": 16, "kv_heads": 4, "n": 8192,
         "dim": 128, "window": 1024, "sinks": 4, "ragged": False},
        # prompts of different lengths padded to one, odd sizes
        {"name": "window_padded", "op": "window", "grad": False, "type": "f16", "batch": 3, "heads": 12, "kv_heads": 4, "n": 2309,
         "dim": 72, "window": 500, "sinks": 1, "ragged": True},
        # a training step of a window layer: forward and gradients
        {"name": "window_train", "op": "window", "grad": True, "type": "bf16", "batch": 2, "heads": 16, "kv_heads": 4, "n": 4096,
         "dim": 64, "window": 1024, "sinks": 4, "ragged": False},
        # a training step of a full causal layer, odd sizes, one key head for all
        {"name": "window_train_full", "op": "window", "grad": True, "type": "f16", "batch": 2, "heads": 5, "kv_heads": 1, "n": 1111,
         "dim": 96, "window": 0, "sinks": 0, "ragged": True},
        # one token for each of 32 sequences over caches of up to 16385 keys
        {"name": "cached_token", "op": "cached", "type": "bf16", "batch": 32, "heads": 32, "kv_heads": 8, "tokens": 1, "cap": 16385,
         "dim": 128, "window": 0, "sinks": 0, "tree": False},
        # a tree of 31 drafted tokens for 4 sequences, window layer
        {"name": "cached_tree", "op": "cached", "type": "f16", "batch": 4, "heads": 16, "kv_heads": 4, "tokens": 31, "cap": 5000,
         "dim": 64, "window": 4096, "sinks": 4, "tree": True},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    heads = rng.choice([(2, 2), (8, 1), (6, 2), (16, 4), (16, 16), (12, 4), (5, 1), (32, 8)])
    dim = 8 * rng.randint(4, 16)
    kind = rng.choice(["qk", "qk_grad", "window", "window_grad", "cached"])
    if kind.startswith("qk"):
        batch = _log(rng, 1, 8)
        most = min(8192, (4 * 40 * 4096 * 128 * 2 // (3 if kind == "qk_grad" else 2)) // (batch * sum(heads) * dim * 2))
        return {"op": "qk", "grad": kind == "qk_grad", "type": rng.choice(["bf16", "f16", "f32"]), "batch": batch,
                "heads": heads[0], "kv_heads": heads[1], "n": _log(rng, 1, most), "dim": dim,
                "rope": rng.choice([dim, dim, dim // 2]), "packed": rng.random() < 0.5, "weights": rng.random() < 0.75,
                "far": rng.choice([0, 0, 7777, 500000])}
    if kind.startswith("window"):
        batch = rng.randint(1, 3)
        most = int(math.sqrt(2 * 16 * 4096 * 4096 / (batch * heads[0])))
        case = {"op": "window", "grad": kind == "window_grad", "type": rng.choice(["bf16", "f16"]), "batch": batch,
                "heads": heads[0], "kv_heads": heads[1], "n": _log(rng, 17, min(8192, most)), "dim": dim,
                "window": rng.choice([0, _log(rng, 16, 2048), _log(rng, 16, 2048)]), "sinks": rng.choice([0, 1, 4, 130]),
                "ragged": rng.random() < 0.5}
        while work(case)["flops"] > 1e11:  # no dearer than the listed training step
            case["n"] = case["n"] * 7 // 8
        return case
    batch = _log(rng, 1, 32)
    tokens = rng.choice([1, 1, 2, rng.randint(3, 64)])
    return {"op": "cached", "type": rng.choice(["bf16", "f16"]), "batch": batch, "heads": heads[0], "kv_heads": heads[1],
            "tokens": tokens, "cap": _log(rng, 200, max(201, 16384 * 32 * 8 // (batch * max(8, heads[1] * (1 + tokens // 8))))),
            "dim": dim, "window": rng.choice([0, 0, _log(rng, 64, 4096)]), "sinks": rng.choice([0, 4, 70]),
            "tree": tokens > 2 and rng.random() < 0.7}


def _lengths(case):
    """The sequences' lengths: the first is the whole buffer, the others shorter."""
    n, batch = case.get("n") or case["cap"], case["batch"]
    if case["op"] == "window" and not case["ragged"]:
        return [n] * batch
    return [max(min(n, case.get("tokens", 1)), n - (n * 2 * b) // (3 * batch) - 3 * b) for b in range(batch)]


def _tree(tokens, seed):
    """Ancestor bits (itself among them) of each node of a random tree, in a signed 64-bit word each."""
    g = torch.Generator().manual_seed(seed)
    bits = [1]
    for t in range(1, tokens):
        bits.append(bits[int(torch.randint(0, t, (1,), generator=g))] | (1 << t))
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["type"]]
    B, H, K, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def rows(heads, n):
        return normal(B, heads, n, D)

    s = {"case": case}
    if case["op"] == "qk":
        n = case["n"]
        if case["packed"]:  # the projection's output [B, n, H + 2 K, D]; q and k are views of it
            qkv = normal(B, n, H + 2 * K, D)
            s["q"], s["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + K].transpose(1, 2)
        else:
            s["q"], s["k"] = rows(H, n), rows(K, n)
        s["wq"] = s["wk"] = s["pos"] = None
        if case["weights"]:
            s["wq"] = 1 + 0.25 * torch.randn(D, generator=g, device="cuda")
            s["wk"] = 1 + 0.25 * torch.randn(D, generator=g, device="cuda")
        if case["far"]:  # each sequence at its own place
            first = torch.randint(0, case["far"], (B, 1), generator=g, device="cuda")
            s["pos"] = (first + torch.arange(n, device="cuda")).to(torch.int32)
        if case["grad"]:
            s["dq"], s["dk"] = rows(H, n), rows(K, n)
        return s
    s["scale"] = D ** -0.5
    s["len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["op"] == "window":
        n = case["n"]
        s["q"], s["k"], s["v"] = rows(H, n), rows(K, n), rows(K, n)
        s["kv_len"] = s["q_start"] = None
        if case["ragged"]:
            s["kv_len"], s["q_start"] = s["len"], torch.zeros(B, dtype=torch.int32, device="cuda")
        if case["grad"]:
            s["dout"] = rows(H, n)
        return s
    s["q"], s["k"], s["v"] = rows(H, case["tokens"]), rows(K, case["cap"]), rows(K, case["cap"])
    s["tree"] = None
    if case["tree"]:
        s["tree"] = torch.tensor([_tree(case["tokens"], seed * 100 + b) for b in range(B)], dtype=torch.int64, device="cuda")
    return s


def run(state):
    c = state["case"]
    if own:
        return _library(state, c)
    if c["op"] == "qk":
        return _plain_qk_grad(state, c) if c["grad"] else _plain_qk(state, c)
    if c["op"] == "cached":
        return _plain_attention(state, c, _cached_visible(state, c))[0]
    return _plain_train(state, c) if c["grad"] else _plain_attention(state, c, _window_visible(state, c))[0]


def _library(s, c):
    import vision_encoder_flash_gb300 as vef

    if c["op"] == "qk":
        how = dict(rope_dims=c["rope"], positions=s["pos"], base=BASE, eps=EPS)
        if c["grad"]:
            got = vef.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], **how)
            return got if c["weights"] else got[:2]
        return vef.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], **how)
    window = c["window"] or None
    if c["op"] == "cached":
        return vef.forward_cached(s["q"], s["k"], s["v"], s["len"], tree_mask=s["tree"], window=window, n_sinks=c["sinks"],
                                  scale=s["scale"])
    how = dict(window=window, n_sinks=c["sinks"], scale=s["scale"], kv_len=s["kv_len"], q_start=s["q_start"])
    if not c["grad"]:
        return vef.forward_window(s["q"], s["k"], s["v"], **how)
    out, lse = vef.forward_window(s["q"], s["k"], s["v"], return_lse=True, **how)
    return (out,) + tuple(vef.backward_window(s["dout"], s["q"], s["k"], s["v"], out, lse, **how))


# ---------------------------------------------------------------- the plain forms

def _angles(s, c):
    """cos and sin [B or 1, 1, n, rope / 2] of the rows' positions, the angles in 64 bits."""
    half, n = c["rope"] // 2, c["n"]
    inv = BASE ** (torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 / c["rope"]))
    pos = torch.arange(n, device="cuda")[None] if s["pos"] is None else s["pos"]
    theta = (pos.double()[..., None] * inv)[:, None]
    return torch.cos(theta).float(), torch.sin(theta).float()


def _turn(x, cos, sin, half):
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)


def _plain_qk(s, c):
    cos, sin = _angles(s, c)

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _turn(y if w is None else y * w, cos, sin, c["rope"] // 2).to(DTYPES[c["type"]])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_qk_grad(s, c):
    cos, sin = _angles(s, c)

    def one(x, w, d):
        x, g = x.float(), _turn(d.float(), cos, -sin, c["rope"] // 2)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        gw = g if w is None else g * w
        dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
        return dx.to(DTYPES[c["type"]]), (g * n).sum((0, 1, 2), dtype=torch.float64).float()

    (dq, dwq), (dk, dwk) = one(s["q"], s["wq"], s["dq"]), one(s["k"], s["wk"], s["dk"])
    return (dq, dk, dwq, dwk) if c["weights"] else (dq, dk)


def _window_visible(s, c):
    """[B, 1, 1, n, n]: which keys each query row sees."""
    i = torch.arange(c["n"], device="cuda")
    p, j = i[:, None], i[None, :]
    seen = (j <= p) & ((j > p - (c["window"] or c["n"])) | (j < c["sinks"]))
    return (seen[None] & (p[None] < s["len"].long()[:, None, None]))[:, None, None]


def _cached_visible(s, c):
    """[B, 1, 1, tokens, cap]: which cache rows each new token sees."""
    T, dev = c["tokens"], "cuda"
    t = torch.arange(T, device=dev)
    first = s["len"].long()[:, None] - T  # cache row of the first new token
    anc = (t[None, :, None] >= t[None, None, :]).expand(c["batch"], T, T) if s["tree"] is None else \
        ((s["tree"][:, :, None] >> t[None, None, :]) & 1).bool()
    pos = first + anc.sum(-1) - 1  # a new token's position: behind its ancestors
    j = torch.arange(c["cap"], device=dev)[None, :]
    u = j - first  # which new token a cache row holds
    new = (u >= 0) & (u < T)
    keypos = torch.where(new, pos.gather(1, u.clamp(0, T - 1)), j)[:, None, :]
    path = anc.gather(2, u.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
    p = pos[..., None]
    seen = ((u < 0)[:, None, :] | (new[:, None, :] & path)) & ((keypos > p - (c["window"] or (c["cap"] + T))) | (keypos < c["sinks"]))
    return seen[:, None, None]


def _plain_attention(s, c, seen):
    """The output, and the weights of every (query, key) with the operands in 32 bits."""
    B, H, K = c["batch"], c["heads"], c["kv_heads"]
    q = s["q"].float().unflatten(1, (K, H // K))
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    x = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    w = x.div_(x.sum(-1, keepdim=True).clamp_min(1e-30))
    return torch.matmul(w, v).flatten(1, 2).to(DTYPES[c["type"]]), (q, k, v, w)


def _plain_train(s, c):
    out, (q, k, v, w) = _plain_attention(s, c, _window_visible(s, c))
    dt, shape = DTYPES[c["type"]], q.shape
    do = s["dout"].float().view(shape)
    dv = torch.matmul(w.transpose(-1, -2), do).sum(2)
    dw = torch.matmul(do, v.transpose(-1, -2))
    ds = (dw - (dw * w).sum(-1, keepdim=True)) * w * s["scale"]
    dq, dk = torch.matmul(ds, k).flatten(1, 2), torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return out, dq.to(dt), dk.to(dt), dv.to(dt)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(s, case)
    return _exact_attention(s, case)


def _exact_qk(s, c):
    B, n, half = c["batch"], c["n"], c["rope"] // 2
    pos = s["pos"].double() if s["pos"] is not None else torch.arange(n, device="cuda", dtype=torch.float64).expand(B, n)
    freq = torch.exp(torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 * math.log(BASE) / c["rope"]))
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), pos[:, :, None] * freq)  # [B, n, half]
    outs, sums = [], []
    for name, weight in (("q", "wq"), ("k", "wk")):
        x, w = s[name].double(), s[weight]
        w = torch.ones(c["dim"], device="cuda", dtype=torch.float64) if w is None else w.double()
        rms = ((x ** 2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
        g = s["d" + name].double() if c["grad"] else (x / rms) * w
        z = torch.complex(g[..., :half].contiguous(), g[..., half:2 * half].contiguous())
        z = z * (turn.conj() if c["grad"] else turn)[:, None]
        g = torch.cat([z.real, z.imag, g[..., 2 * half:]], -1)
        if not c["grad"]:
            outs.append(g)
            continue
        sums.append((g * x / rms).sum((0, 1, 2)))
        h = g * w
        outs.append(h / rms - x * (h * x).sum(-1, keepdim=True) / (c["dim"] * rms ** 3))
    return tuple(outs + sums) if c["weights"] else tuple(outs)


def _exact_attention(s, c):
    """One head of one sequence at a time, over the rows that it sees."""
    H, K, grad = c["heads"], c["kv_heads"], c.get("grad", False)
    lens = [int(x) for x in s["len"]]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(out), *(torch.zeros(s["k"].shape, device="cuda", dtype=torch.float64) for _ in range(2))
    for b in range(c["batch"]):
        L = lens[b]
        if c["op"] == "window":
            at = key_at = torch.arange(L, device="cuda")
            allowed = at[:, None] >= key_at[None, :]
        else:
            T = c["tokens"]
            words = [(1 << (t + 1)) - 1 for t in range(T)] if s["tree"] is None else [int(x) & (2 ** 64 - 1) for x in s["tree"][b]]
            depth = [bin(x).count("1") - 1 for x in words]
            at = torch.tensor([L - T + d for d in depth], device="cuda")
            key_at = torch.cat([torch.arange(L - T, device="cuda"), at])
            path = torch.tensor([[(x >> u) & 1 for u in range(T)] for x in words], device="cuda").bool()
            allowed = torch.cat([torch.ones(T, L - T, device="cuda", dtype=torch.bool), path], 1)
        if c["window"]:
            allowed = allowed & ((at[:, None] - key_at[None, :] < c["window"]) | (key_at[None, :] < c["sinks"]))
        rows = at.numel()
        hidden = ~allowed
        for h in range(H):
            e = h // (H // K)
            q, k, v = s["q"][b, h, :rows].double(), s["k"][b, e, :L].double(), s["v"][b, e, :L].double()
            p = torch.softmax((q @ k.T * s["scale"]).masked_fill(hidden, -math.inf), -1)
            out[b, h, :rows] = p @ v
            if grad:
                do = s["dout"][b, h, :rows].double()
                ds = p * (do @ v.T - (do * out[b, h, :rows]).sum(-1, keepdim=True))
                dv[b, e, :L] += p.T @ do
                dq[b, h, :rows] = ds @ k * s["scale"]
                dk[b, e, :L] += ds.T @ q * s["scale"]
    return (out, dq, dk, dv) if grad else out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, H, K, D, size = case["batch"], case["heads"], case["kv_heads"], case["dim"], BYTES[case["type"]]
    if case["op"] == "qk":
        rows = B * case["n"] * (H + K)
        return {"bytes": rows * D * size * (3 if case["grad"] else 2) + (16 * D if case["weights"] else 0)
                + (4 * B * case["n"] if case["far"] else 0), "flops": rows * D * (14 if case["grad"] else 7)}
    W, sinks = case["window"], case["sinks"]
    lens = _lengths(case)
    if case["op"] == "window":
        pairs = sum(_pairs(n, W or n, sinks) for n in lens)
        tokens, passes = sum(lens), (2 if case["grad"] else 1)
        heads = (H * (4 if case["grad"] else 2) + K * 2 * passes) * D * size
        return {"bytes": tokens * heads, "flops": pairs * H * D * (14 if case["grad"] else 4)}
    T = case["tokens"]
    keys = sum(n if not W else min(n, W + T + sinks) for n in lens)
    return {"bytes": keys * K * 2 * D * size + 2 * B * H * T * D * size, "flops": keys * T * H * D * 4}


def _pairs(n, window, sinks):
    """Visible (query, key) pairs of n queries over their own n keys."""
    w, full = min(window, n), min(window, n) * (min(window, n) + 1) // 2
    inside = full + (n - w) * w
    extra = max(0, n - w)  # query w + x sees min(sinks, x + 1) keys before its window
    a = min(extra, sinks)
    return inside + a * (a + 1) // 2 + (extra - a) * sinks
