"""Shared by the GPU tests of the serving calls: caches, packed rows."""
import numpy as np

from decoder_util import dtype, f64, normal  # noqa: F401


def ints(torch, x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def pool(torch, n_pages, heads, page, dim, layout, dev, fill=0x7f):
    """(k_pages, v_pages, everything they are views of): "heads" [n, H, page, D], "tokens" [n,
    page, H, D] seen so, "both" k and v in one buffer with 16 bytes of padding a row; all
    bytes NaN (or `fill`)."""
    f8 = torch.float8_e4m3fn
    if layout == "heads":
        big = torch.full((2, n_pages, heads, page, dim), fill, dtype=torch.uint8, device=dev)
        k, v = big[0], big[1]
    elif layout == "tokens":
        big = torch.full((2, n_pages, page, heads, dim), fill, dtype=torch.uint8, device=dev)
        k, v = big[0].transpose(1, 2), big[1].transpose(1, 2)
    else:
        big = torch.full((n_pages, page, 2, heads, dim + 16), fill, dtype=torch.uint8, device=dev)
        k, v = big[:, :, 0, :, :dim].transpose(1, 2), big[:, :, 1, :, :dim].transpose(1, 2)
    return k.view(f8), v.view(f8), big


def values(pages):
    """f64 values of a pool."""
    return pages.float().double().cpu().numpy()


def filled(torch, shape, lens, page, seed, dev, layout="heads", spread=2.0, spare=2, v_spread=None):
    """A cache [.., K, page, D] of sequences of these lengths, quantised here: k_pages, v_pages, k_scale,
    v_scale, table, kv_len.  Pages in random order, of scales 2^(+-spread); what no row
    holds is NaN."""
    K, D = shape
    rng = np.random.default_rng(seed)
    most = max(1, max(-(-max(n, 1) // page) for n in lens))
    n_pages = most * len(lens) + spare
    table = rng.permutation(n_pages)[:most * len(lens)].reshape(len(lens), most)
    k, v, _ = pool(torch, n_pages, K, page, D, layout, dev)
    scales = []
    for x, s in ((k, spread), (v, spread if v_spread is None else v_spread)):
        scale = 2.0 ** np.rint(rng.normal(size=(n_pages, K)) * s - 6)
        data = np.clip(rng.normal(size=(n_pages, K, page, D)) * 100, -440, 440)
        for b, n in enumerate(lens):
            for i in range(most):
                data[table[b, i], :, max(0, min(page, n - i * page)):] = np.nan
        x.view(torch.uint8).copy_(torch.from_numpy(data).float().to(torch.float8_e4m3fn).view(torch.uint8).to(dev))
        scales.append(torch.from_numpy(scale).float().to(dev))
    return k, v, *scales, ints(torch, table.tolist(), dev), ints(torch, lens, dev)
