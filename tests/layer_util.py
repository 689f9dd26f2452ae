"""Plain forms in 64 bits of the 4-bit base products and rotary positions, for the tests
of the frozen part of a layer, with the bounds their tests hold the kernels to.

A value computed in 32 bits is off by at most u = 2^-24 of its size at each step; one
rounding to bf16 is off by at most 2^-8 of the value (half of torch.finfo's eps)."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def groups_of(d_in, group):
    return -(-d_in // (group or d_in))


def random_weight(gen, d_out, d_in, group, with_zero, std=0.02):
    """q, scale, zero (CPU): scales as 16-bit floats hold them."""
    g = groups_of(d_in, group)
    q = torch.randint(256, (d_out, d_in // 2), generator=gen, dtype=torch.uint8)
    scale = (torch.rand(d_out, g, generator=gen) * std / 4 + std / 16).half().float()
    zero = torch.randint(16, (d_out, g), generator=gen, dtype=torch.uint8) if with_zero else None
    return q, scale, zero


def integer_weight(gen, d_out, d_in, group, with_zero):
    """As random_weight with scales that are powers of two: integer inputs then give sums
    that 32 bits hold exactly."""
    q, scale, zero = random_weight(gen, d_out, d_in, group, with_zero)
    scale = 2.0 ** -torch.randint(3, tuple(scale.shape), generator=gen).float()
    return q, scale, zero


def levels(w, d_in, group):
    """(q - zero, scale, zero) of every weight, in 64 bits [d_out][d_in]."""
    q, scale, zero = w
    v = torch.empty(q.shape[0], d_in, dtype=torch.float64)
    v[:, 0::2] = (q & 15).double()
    v[:, 1::2] = (q >> 4).double()
    of = torch.arange(d_in) // (group or d_in)
    z = torch.full_like(v, 8.0) if zero is None else zero.double()[:, of]
    return v - z, scale.double()[:, of], z


def base_sum(x, w, d_in, group):
    """sum_k x W and the bound of its error in the kernel's order of 32-bit sums.

    The kernel forms sum x (16 + q) and (16 + z) sum x over each group and subtracts them.
    Every product and partial sum is at most m = sum |x| ((16 + q) + (16 + z)) s, and a
    term passes at most: 3 products (fp32 x in three pieces) of a block of 128, each
    accumulated with an error of u (2u if the matrix core cuts off instead of rounding),
    the two operations of the group's factor, one addition per group, and 8 of the join."""
    d, s, z = levels(w, d_in, group)
    x = x.double()
    y = x @ (d * s).t()
    m = x.abs() @ ((d + 2 * z + 32) * s.abs()).t()
    pieces = 3 if x.dtype != torch.bfloat16 else 1
    steps = 2 * (128 * pieces + 4 + 4 * groups_of(d_in, 128) + 8)
    return y, steps * U32 * m


def act64(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    if kind == "gelu":
        return 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def check_within(got, want, bound, what):
    got = got.detach().cpu().double()
    err = (got - want).abs()
    worst = (err / bound.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert bool((err <= bound).all()), f"{what}: worst error / bound {worst:.3f}, error {err.max():.3e}"
    return worst


def guarded(rows, cols, dtype, offset=0, fill=7.0):
    """A contiguous device tensor [rows][cols] inside a larger one of `fill`, `offset`
    elements past a 16-byte boundary; returns (tensor, check that the rest is untouched)."""
    n = rows * cols
    whole = torch.full((n + 1024,), fill, dtype=dtype, device="cuda")
    lo = 256 + offset

    def intact():
        rest = torch.cat((whole[:lo], whole[lo + n:]))
        assert bool((rest == fill).all()), "wrote outside of its rows"
    return whole[lo:lo + n].view(rows, cols), intact
