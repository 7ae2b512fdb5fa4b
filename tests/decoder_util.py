"""Shared by the GPU tests of the decoder calls: inputs, layouts, bounds."""
import numpy as np

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # of one rounding, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half a step below the smallest normals


def dtype(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(torch, shape, name, seed, dev, scale=1.0):
    """Seeded normal values of the type, on the device."""
    x = np.random.default_rng(seed).normal(size=shape) * scale
    return torch.from_numpy(x).to(dev).to(dtype(torch, name))


def laid_out(torch, x, layout):
    """The same values in another layout: "plain", "packed" ([B, N, H, D]
    seen as [B, H, N, D]), or "padded" (a part of a larger buffer whose other
    elements are NaN)."""
    B, H, N, D = x.shape
    if layout == "plain":
        return x.contiguous()
    if layout == "packed":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    big = torch.full((B + 1, H, N + 5, D + 24), float("nan"), dtype=x.dtype, device=x.device)
    big[:B, :, 3:3 + N, 8:8 + D] = x
    return big[:B, :, 3:3 + N, 8:8 + D]


def assert_within(got, want, bound, what, u=0.0, tiny=0.0):
    """|got - want| <= bound + u |want| + tiny, element by element."""
    got = f64(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == want.shape, what
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    over = np.abs(got - want) - (bound + u * np.abs(want) + tiny)
    i = np.unravel_index(int(np.argmax(over)), over.shape) if over.size else None
    assert over.size == 0 or over[i] <= 0, (
        f"{what}: at {tuple(int(x) for x in i)} got {got[i]!r}, want {want[i]!r}, "
        f"{int((over > 0).sum())} of {over.size} outside")
