"""The serving calls as a layer of a server uses them: norm of q and k, prompts of
different lengths into the cache and through attention, then steps of new
tokens and of a drafted tree, against the f64 oracle over the values that the
cache holds; captured, on threads, across devices' streams."""
import threading

import numpy as np
import pytest

from oracle import decoder as od
from oracle import serving as osv
import vision_encoder_flash_gb300 as vef
from decoder_util import HALF_STEP, TINY, assert_within, f64, normal
from serving_util import ints, pool, values

pytestmark = pytest.mark.gpu

B, H, K, D, PAGE, MOST = 3, 8, 2, 64, 16, 40


@pytest.fixture(scope="module")
def td():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a CUDA device")
    from vision_encoder_flash_gb300 import build
    build.build()
    vef.load_library()
    return torch, torch.device("cuda", 0)


class Layer:
    """The caches of one layer, and the projections of seeded steps."""

    def __init__(self, td, name, window=None, sinks=0):
        self.torch, self.dev = td
        torch, dev = td
        self.name, self.how = name, dict(window=window, n_sinks=sinks, scale=D ** -0.5)
        self.k, self.v, _ = pool(torch, B * MOST + 1, K, PAGE, D, "tokens", dev)
        self.ks, self.vs = (torch.zeros(B * MOST + 1, K, device=dev) for _ in range(2))
        order = torch.randperm(B * MOST, generator=torch.Generator().manual_seed(3)) + 1
        self.table = order.to(torch.int32).view(B, MOST).to(dev)
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.wq, self.wk = (torch.linspace(0.5, 1.5, D, device=dev) for _ in range(2))

    def cache(self):
        return self.k, self.v, self.ks, self.vs, self.table, self.lens

    def projection(self, rows, seed, batch=1):
        x = normal(self.torch, (batch, rows, H + 2 * K, D), self.name, seed, self.dev).transpose(1, 2)
        return x[:, :H], x[:, H:H + K], x[:, H + K:]

    def prompts(self, lens, seed):
        q, k, v = self.projection(sum(lens), seed)
        starts = np.concatenate([[0], np.cumsum(lens)])
        cu = ints(self.torch, starts.tolist(), self.dev)
        pos = ints(self.torch, [[i for n in lens for i in range(n)]], self.dev)
        qr, kr = vef.qk_norm_rope(q, k, self.wq, self.wk, positions=pos)
        self.lens += ints(self.torch, lens, self.dev)
        vef.append_paged(kr, v, *self.cache(), cu_seqlens=cu)
        return vef.forward_packed(qr, kr, v, cu, **self.how), (qr, kr, v, starts)

    def step(self, tokens, seed, words=None):
        """New tokens of each sequence: norm alone, then the rotation on the way into the cache."""
        torch, dev = self.torch, self.dev
        q, k, v = self.projection(tokens, seed, batch=B)
        _, kn = vef.qk_norm_rope(q[:, :0], k, None, self.wk, rope_dims=0)
        self.lens += tokens
        depth = torch.arange(tokens) if words is None else torch.tensor([bin(w).count("1") - 1 for w in words])
        pos = (self.lens[:, None] - tokens + depth.to(dev)[None]).to(torch.int32).contiguous()
        vef.append_paged(kn, v, *self.cache(), rope_dims=D, positions=pos)
        qr, _ = vef.qk_norm_rope(q, k[:, :0], self.wq, None, positions=pos)
        mask = None if words is None else torch.tensor([words] * B, dtype=torch.int64, device=dev)
        return vef.forward_paged(qr, *self.cache(), tree_mask=mask, **self.how), qr

    def check_step(self, out, qr, words=None):
        """Against the oracle over what the cache holds."""
        k, v, ks, vs = values(self.k), values(self.v), f64(self.ks), f64(self.vs)
        lens, table = self.lens.tolist(), self.table.tolist()
        T = qr.shape[2]
        for b in range(B):
            n = lens[b]
            kk, vv, sv = (osv.gathered(x, s, table[b], n)[0][None] for x, s in ((k, ks), (v, vs), (np.ones_like(v), vs)))
            seen = od.cached_visible(T, n, self.how["window"], self.how["n_sinks"], n, words)[None]
            want, bound = osv.paged_attention(f64(qr)[b:b + 1], kk, vv, sv[..., 0], seen, float(np.float32(D ** -0.5)),
                                              HALF_STEP[self.name])
            assert_within(f64(out)[b:b + 1], want, bound, f"sequence {b}", tiny=2 * TINY[self.name])


@pytest.mark.parametrize("name,window,sinks", [("bf16", None, 0), ("f16", 100, 3)])
def test_prompts_then_steps(td, name, window, sinks):
    torch, dev = td
    layer = Layer(td, name, window, sinks)
    lens = [150, 1, 333]
    out, (qr, kr, v, starts) = layer.prompts(lens, 10)
    for b, n in enumerate(lens):
        part = [f64(x)[:, :, starts[b]:starts[b] + n] for x in (qr, kr, v)]
        seen = od.window_visible(n, n, window, sinks, n, 0)[None]
        want, _, _, bound, _, _ = od.attention(*part, seen, float(np.float32(D ** -0.5)), HALF_STEP[name])
        assert_within(out[:, :, starts[b]:starts[b] + n], want, bound, f"prompt {b}", tiny=2 * TINY[name])
        # the cache holds the prompt's keys and values: within half a step of e4m3, or of its
        # smallest, in units of the page's scale
        for pages, scales, x in ((layer.k, layer.ks, part[1]), (layer.v, layer.vs, part[2])):
            held, _ = osv.gathered(values(pages), f64(scales), layer.table.tolist()[b], n)
            unit, _ = osv.gathered(np.ones(tuple(pages.shape)), f64(scales), layer.table.tolist()[b], n)
            assert np.all(np.abs(held - x[0]) <= 2.0 ** -4 * np.abs(x[0]) * (1 + 2.0 ** -20) + 2.0 ** -10 * unit)
    for i in range(20):  # over a page's end
        layer.check_step(*layer.step(1, 20 + i))
    layer.check_step(*layer.step(5, 50))
    words = [0b1, 0b11, 0b101, 0b1011, 0b10101]
    before = layer.lens.clone()
    layer.check_step(*layer.step(5, 60, words), words)
    layer.lens.copy_(before + 2)  # two of the drafted tokens are kept: the others' rows are written again
    layer.check_step(*layer.step(3, 70))
    assert vef.device_status() == 0


def test_a_step_in_two_graphs(td):
    """Two layers' steps captured, replayed on two streams at once for forty tokens."""
    torch, dev = td
    layers = [Layer(td, "bf16"), Layer(td, "bf16")]
    eager = [Layer(td, "bf16"), Layer(td, "bf16")]
    for i, l in enumerate(layers + eager):
        l.prompts([200, 30, 77], 90 + i % 2)
    inputs = [[normal(torch, (B, h, 1, D), "bf16", 95 + h + 10 * i, dev) for h in (H, K, K)] for i in range(2)]

    def step(l, x):
        l.lens.add_(1)
        vef.append_paged(x[1], x[2], *l.cache(), rope_dims=D)
        return vef.forward_paged(x[0], *l.cache(), **l.how)

    graphs = []
    for l, x in zip(layers, inputs):
        start = l.lens.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(l, x)
        l.lens.copy_(start)
        graphs.append((g, out))
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for t in range(40):
        for i, x in enumerate(inputs):
            for j, y in enumerate(x):
                y.copy_(normal(torch, y.shape, "bf16", 200 + 10 * t + j + 5 * i, dev))
        for s, (g, _) in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream(dev))
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize(dev)
        for (_, out), l, x in zip(graphs, eager, inputs):
            assert torch.equal(out, step(l, x))
    assert vef.device_status() == 0


def test_threads(td):
    """Four host threads, each with a layer and a stream of its own."""
    torch, dev = td

    def serve(layer):
        outs = [layer.prompts([120, 40, 9], 300)[0]]
        for t in range(12):
            outs.append(layer.step(1 + t % 3, 310 + t)[0])
        return outs

    want = serve(Layer(td, "f16", 64, 2))
    torch.cuda.synchronize(dev)
    errors = []

    def worker():
        try:
            torch.cuda.set_device(dev)
            stream = torch.cuda.Stream(dev)
            with torch.cuda.stream(stream):
                got = serve(Layer(td, "f16", 64, 2))
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    errors.append("different results")
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=worker) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and vef.device_status() == 0


CAPTURE = """
import sys
import torch
import vision_encoder_flash_gb300 as vef
dev = torch.device("cuda:0")
torch.manual_seed(1)
q = torch.randn(1, 4, 300, 64, device=dev).bfloat16()
k, v = (torch.randn(1, 2, 300, 64, device=dev).bfloat16() for _ in range(2))
pk, pv = (torch.randint(0, 120, (8, 2, 64, 64), dtype=torch.uint8, device=dev) for _ in range(2))
ks, vs = (torch.full((8, 2), 0.125, device=dev) for _ in range(2))
table = torch.arange(8, dtype=torch.int32, device=dev).view(1, 8)
lens = torch.full((1,), 300, dtype=torch.int32, device=dev)
cu = torch.tensor([0, 170, 300], dtype=torch.int32, device=dev)

def append():
    vef.append_paged(k, v, pk, pv, ks, vs, table, lens, rope_dims=64)
    return pk, pv, ks, vs

def paged():
    return (vef.forward_paged(q[:, :, :5], pk, pv, ks, vs, table, lens, scale=0.125),)

def packed():
    return vef.forward_packed(q, k, v, cu, scale=0.125, return_lse=True)

call = dict(append=append, paged=paged, packed=packed)[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert all(torch.equal(a, b) for a, b in zip(got, call()))
assert vef.device_status() == 0
print("captured")
"""


@pytest.mark.parametrize("call", ["append", "paged", "packed"])
def test_first_call_in_a_capture(call):
    """What a call sets up once must not disturb a capture that is a process's first call."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", CAPTURE, call], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
