"""The decoder calls together, as a layer uses them: a training step from the
packed projection to its gradient, and serving from the prompt over single
tokens to a tree of drafted ones."""
import numpy as np
import pytest

import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, f64, normal

pytestmark = pytest.mark.gpu

B, H, K, D = 2, 6, 2, 64
WINDOW, SINKS, BASE, EPS = 70, 3, 10000.0, 1e-6


@pytest.fixture(scope="module")
def td():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a CUDA device")
    from vision_encoder_flash_gb300 import build
    build.build()
    vef.load_library()
    return torch, torch.device("cuda", 0)


def reference(torch, qkv, wq, wk, lens):
    """The layer in f64: norm, rotation, windowed attention of each sequence's
    own rows (those behind its length give zeros)."""
    n = qkv.shape[1]
    q, k, v = (t.transpose(1, 2) for t in qkv.split((H, K, K), dim=2))
    pos = torch.arange(n, device=qkv.device, dtype=torch.float64)
    theta = pos[:, None] * BASE ** (torch.arange(D // 2, device=qkv.device, dtype=torch.float64) * (-2.0 / D))

    def turned(x, w):
        y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat([a * theta.cos() - b * theta.sin(), a * theta.sin() + b * theta.cos()], -1)

    q, k = turned(q, wq), turned(k, wk)
    k, v = (t.repeat_interleave(H // K, 1) for t in (k, v))
    i, j = torch.arange(n, device=qkv.device)[:, None], torch.arange(n, device=qkv.device)[None]
    seen = (j <= i) & ((j > i - WINDOW) | (j < SINKS))
    x = (q @ k.transpose(2, 3) * D ** -0.5).masked_fill(~seen, float("-inf"))
    own = (torch.arange(n, device=qkv.device)[None] < lens[:, None]).double()[:, None, :, None]
    return torch.softmax(x, -1) @ v * own


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_training_step(td, name):
    torch, dev = td
    n, lens = 333, torch.tensor([333, 250], dtype=torch.int32, device=dev)
    start = torch.zeros(B, dtype=torch.int32, device=dev)
    qkv = normal(torch, (B, n, H + 2 * K, D), name, 1, dev)
    wq, wk = (1 + 0.2 * normal(torch, (D,), "f32", 2 + i, dev) for i in range(2))
    dout = normal(torch, (B, H, n, D), name, 4, dev)
    how = dict(window=WINDOW, n_sinks=SINKS, scale=D ** -0.5, kv_len=lens, q_start=start)

    def step():
        q, k, v = (t.transpose(1, 2) for t in qkv.split((H, K, K), dim=2))
        qr, kr = vef.qk_norm_rope(q, k, wq, wk, base=BASE, eps=EPS)
        out, lse = vef.forward_window(qr, kr, v, return_lse=True, **how)
        grad = torch.empty_like(qkv)  # the packed gradient, written in place
        gq, gk, gv = (t.transpose(1, 2) for t in grad.split((H, K, K), dim=2))
        vef.backward_window(dout, qr, kr, v, out, lse, dq=gq, dk=gk, dv=gv, **how)
        _, _, gwq, gwk = vef.qk_norm_rope_backward(gq, gk, q, k, wq, wk, base=BASE, eps=EPS, dq=gq, dk=gk)
        return out, grad, gwq, gwk

    got = step()
    x = [t.double().requires_grad_() for t in (qkv, wq, wk)]
    want = reference(torch, *x, lens)
    want.backward(dout.double())
    # forward four roundings (q and k, weights, result), backward five more
    # (weights, their gradients, dq / dk, the norm's result), each of at most u
    # in its own norm, and a softmax of scores of size one amplifies by less than 2
    u = HALF_STEP[name]
    for a, b, what in zip(got, (want.detach(), x[0].grad, x[1].grad, x[2].grad), ("out", "dqkv", "dwq", "dwk")):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel <= (8 if what == "out" else 18) * u, f"{what}: {rel:.2e}"
    assert vef.device_status() == 0
    # the step captured and replayed on other values
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    qkv.copy_(normal(torch, qkv.shape, name, 11, dev))
    g.replay()
    torch.cuda.synchronize(dev)
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))


def test_serving(td):
    """Prompt, single tokens and a tree against the whole sequence at once."""
    torch, dev = td
    n, prompt, steps = 220, 190, 6
    qkv = normal(torch, (B, n, H + 2 * K, D), "bf16", 21, dev)
    wq, wk = (1 + 0.2 * normal(torch, (D,), "f32", 22 + i, dev) for i in range(2))
    q, k, v = (t.transpose(1, 2) for t in qkv.split((H, K, K), dim=2))
    how = dict(window=WINDOW, n_sinks=SINKS, scale=D ** -0.5)
    qr, kr = vef.qk_norm_rope(q, k, wq, wk, base=BASE, eps=EPS)
    whole = vef.forward_window(qr, kr, v, **how)
    # both paths round weights and results by u: each is within (2 u + 2^-13)
    # max |v| of the formula
    near = 2 * (2 * HALF_STEP["bf16"] + 2.0 ** -13) * float(v.abs().max())
    cache_k, cache_v = (torch.full((B, K, 256, D), float("nan"), dtype=qkv.dtype, device=dev) for _ in range(2))

    def append(first, rows):
        part = slice(first, first + rows)
        qn, _ = vef.qk_norm_rope(q[:, :, part], k[:, :, part], wq, wk, pos0=first, base=BASE, eps=EPS,
                                 k_out=cache_k[:, :, part])
        cache_v[:, :, part] = v[:, :, part]
        return qn, torch.full((B,), first + rows, dtype=torch.int32, device=dev)

    qn, lens = append(0, prompt)
    out = vef.forward_window(qn, cache_k, cache_v, kv_len=lens, q_start=torch.zeros_like(lens), **how)
    assert np.abs(f64(out) - f64(whole[:, :, :prompt])).max() <= near
    for s in range(steps):
        qn, lens = append(prompt + s, 1)
        out = vef.forward_cached(qn, cache_k, cache_v, lens, **how)
        assert np.abs(f64(out) - f64(whole[:, :, prompt + s:prompt + s + 1])).max() <= near
    # a tree: tokens 0, 2, 3, 5 are the next of the sequence, 1 and 4 other drafts
    at, path, words = prompt + steps, [0, 2, 3, 5], [1, 0b11, 0b101, 0b1101, 0b10101, 0b101101]
    depth = torch.tensor([bin(w).count("1") - 1 for w in words], dtype=torch.int32, device=dev)
    take = torch.tensor([at + int(d) if i in path else 7 * i for i, d in enumerate(depth)], device=dev)
    qn, kn = vef.qk_norm_rope(q[:, :, take].contiguous(), k[:, :, take].contiguous(), wq, wk, base=BASE, eps=EPS,
                              positions=(at + depth)[None].expand(B, 6).contiguous())
    cache_k[:, :, at:at + 6], cache_v[:, :, at:at + 6] = kn, v[:, :, take]
    lens = torch.full((B,), at + 6, dtype=torch.int32, device=dev)
    mask = torch.tensor([words] * B, dtype=torch.int64, device=dev)
    out = vef.forward_cached(qn, cache_k, cache_v, lens, tree_mask=mask, **how)
    assert np.abs(f64(out[:, :, path]) - f64(whole[:, :, at:at + 4])).max() <= near
    assert vef.device_status() == 0
