"""Helpers of the operator tests: types, strided tensors and the error bound
of one rounding.  No operator arithmetic lives here."""
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# unit roundoff: half the distance between neighbours at 1
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # smallest step


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def strided(g, n, d, dtype, pad=0, shift=0, std=1.0, mean=0.0):
    """[n, d] rows of a buffer whose rows are pad elements longer, starting shift elements in."""
    buf = randn(g, n * (d + pad) + shift, dtype=dtype, std=std, mean=mean)
    return buf[shift:].reshape(n, d + pad)[:, :d]


def empty_strided(n, d, dtype, pad=0, shift=0, fill=None):
    buf = torch.empty(n * (d + pad) + shift, dtype=dtype, device="cuda")
    if fill is not None:
        buf.fill_(fill)
    return buf[shift:].reshape(n, d + pad)[:, :d]


def close(got, want, dt, extra, what=""):
    """|got - want| <= u |want| + extra (elementwise; one rounding to dt plus the fp32 arithmetic's error)."""
    got, want = got.double(), want.double()
    lim = U[dt] * want.abs() + extra + TINY[dt]
    bad = ~((got - want).abs() <= lim)
    if bool(bad.any()):
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got.reshape(-1)[i].item()} for {want.reshape(-1)[i].item()}")
