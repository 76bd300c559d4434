"""Helpers of the tests of a block's operators: 64-bit references and error bounds.

A bound counts roundings: the store to a type is off by at most half a step,
``finfo(t).eps / 2`` of the value (for values below the smallest normal one, of that),
and a sum of terms in 32 bits by at most (its additions) * 2^-24 of the terms'
absolute sum."""
import torch

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


def store_error(ref, dtype):
    f = torch.finfo(dtype)
    return ref.abs().clamp(min=f.smallest_normal) * (f.eps / 2)


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound elementwise (float64 tensors on one device)."""
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        k = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {k}: got "
            f"{float(got.reshape(-1)[k])} want {float(ref.reshape(-1)[k])} within "
            f"{float(bound.expand_as(ref).reshape(-1)[k])}")


def strided(t, pad, device="cuda", offset=0):
    """A copy of matrix t whose rows are ``pad`` elements apart from being contiguous,
    starting ``offset`` elements into its storage, and that storage (filled with NaN)."""
    r, c = t.shape
    store = torch.full((r * (c + pad) + offset + 8,), float("nan"), dtype=t.dtype, device=device)
    view = store.as_strided((r, c), (c + pad, 1), offset)
    view.copy_(t)
    return view, store


def act64(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "sigmoid":
        return torch.sigmoid(z)
    return z


def slope64(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) * (2 * torch.pi) ** -0.5
    if name == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    if name == "sigmoid":
        return torch.sigmoid(z) * torch.sigmoid(-z)
    return torch.ones_like(z)
