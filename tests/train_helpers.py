"""Shared by the tests of the training-step operators: inputs drawn on the GPU
and comparisons with references in 64 bits.

Tolerances are derived, not tuned.  EPS is the largest relative error of one
fp32 rounding and HALF that of one rounding to bf16.  A sum of n terms in fp32,
in any order, is off by at most n * EPS * (sum of the terms' magnitudes).  The
noise of operands that are rounded to bf16 before a product is the sum of
independent errors, each at most HALF of its term, hence of standard deviation
HALF / sqrt(3) * sqrt(sum of squared terms); six standard deviations bound the
millions of values of a test."""
import torch

EPS = 2.0 ** -24
HALF = 2.0 ** -8    # 8 significant bits: half a unit in the last place of 1.0
NOISE = 6 * HALF / 3 ** 0.5


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def within(got, ref, tol):
    """|got - ref| <= tol everywhere, and got finite."""
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        t = tol[i] if torch.is_tensor(tol) else tol
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} values off; first at {at}: "
                             f"got {got[i].item()}, want {ref[i].item()} +- {float(t)}")


def rounded(ref, dtype):
    """The error of rounding ref to dtype (with room for the value rounded being slightly off)."""
    return ref.abs() * (1.01 * HALF if dtype == torch.bfloat16 else 2 * EPS)


def workspace(n):
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in every type
