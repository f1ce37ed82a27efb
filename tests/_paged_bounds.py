"""Bounds of paged_attn_m1 by how a call holds its weights, derived from the kernel's arithmetic.

Relative to the weight of the largest score (1), a weight p enters the product with the values as

  bf16 cache                two bf16 parts: each rounding leaves at most 2^-8 of what it rounds,
                            2^-16 p together; bf16's exponents reach as far as fp32's.
  fp16 cache                two fp16 parts of 2^7 p or more: 2^-11 twice, 2^-22 p, and never less
                            than half of fp16's smallest step, 2^-25, which is 2^-32 of the largest.
  q8 cache, fp16 queries    p times a value scale as two fp16 parts: 2^-22 of it, or half a step.
  q8 cache, bf16 queries    the same as one fp16 part: 2^-11 of it, or half a step.

A q8 group's products are kept times 2^(22 - e), e the exponent of the largest of the group's scales
so far (scale >= 2^(e - 16)): half a step is 2^-25 * 2^(e - 22) <= 2^-31 of that scale, times |int8|.

The output's own rounding is half a unit in the last place: at most 2^-8 of it in bf16 (8 significant
bits), 2^-11 in fp16, or half of fp16's smallest step.
"""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def of_weight(dtype, q8):
    """Relative error of a weight above the smallest steps."""
    if q8:
        return 2.0 ** -22 if dtype is torch.float16 else 2.0 ** -11
    return 2.0 ** -22 if dtype is torch.float16 else 2.0 ** -16


def tolerance(out, p, v, dtype, ds, depth, v_scales=None):
    """Bound of |output - out| for out = p @ v: p [n] normalised weights, v [n, D] (double).

    ds: error of a score; depth: terms of the longest chain of fp32 additions; v_scales [n, D / 32]
    of a q8 cache.  A relative error of every weight and of their sum by 2 ds moves the output by
    4 ds sum p|v|; a chain of additions by depth * 2^-23 of it.
    """
    q8 = v_scales is not None
    tol = U[dtype] * out.abs() + (4 * ds + of_weight(dtype, q8) + depth * 2.0 ** -23) * (p[:, None] * v.abs()).sum(0)
    if q8:
        most = v_scales.abs().amax(0).repeat_interleave(32)  # of each column's group
        tol = tol + 2.0 ** -31 * p.max() * most * (v.abs() / v_scales.abs().repeat_interleave(32, 1).clamp(min=1e-300)).sum(0)
    elif dtype is torch.float16:
        tol = tol + 2.0 ** -32 * p.max() * v.abs().sum(0)
    return tol + (2.0 ** -25 if dtype is torch.float16 else 0.0)
