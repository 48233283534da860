"""A cache whose top-k result shows how many bits of the weights enter the product with V.

In one group of 16 tokens of every unit, one key is zero (score 0, the maximum, weight 1, value 0)
and three are -e_0, with values of one: query head g, whose first element is b_g, weighs them by
p = 2^(-b_g log2(e) / sqrt(d)).  All other keys are -8000 e_0 and weigh exactly 0.  The result is

    out = 3 p / (1 + 3 p)   in every column,

whatever lies in the other elements of q.  p is picked so that its first two bf16 pieces leave more
than 2^-17.7 of it: a product that loses them is off by that much, and

  - the score is one exact product; its scaling and the scale's own rounding move the exponent by
    at most 2 * 2^-24 * |exponent|, |exponent| < 2, so p by ln 2 * 2^-22, and the exponential by
    2^-22 more: together under 1.7 * 2^-22 of p, and under that much of out (p stands in both sums)
  - three equal products and their sums inside the matrix instruction, which truncates at 2^-23 of
    the largest: three additions of pieces, at most 3 * 2^-23
  - the sum of four weights: 3 * 2^-24; joining the warps' results by factors of exactly 1 and 0
    adds nothing; the division 2^-22

so a result that keeps every bit is off by less than (1.7 / 4 + 3 / 8 + 3 / 16 + 1 / 4) 2^-20 =
1.24 * 2^-20 relative.
"""
import math

import torch

BOUND = 1.24 * 2.0 ** -20
LEFT = 2.0 ** -17.7


def bf16(x):
    return x.to(torch.bfloat16).double()


def pieces(p):
    """What one, two and three bf16 pieces of p (float64) add up to."""
    hi = bf16(p)
    lo = bf16(p - hi)
    return hi, hi + lo, hi + lo + bf16(p - hi - lo)


def weight(b, d):
    return torch.exp2(-b * (1.4426950408889634 / math.sqrt(d)))


def heads(d):
    """bf16 values b (float64) whose weights, also when p is off by 2^-21, leave more than LEFT
    behind their second piece; exponents stay below 2."""
    b = torch.arange(64, 2048).double() / 128
    b = b[(b == bf16(b)) & (b * 1.4427 / math.sqrt(d) < 2)]
    keep = torch.ones(len(b), dtype=torch.bool)
    for off in (-1, 0, 1):
        p = weight(b, d) * (1 + off * 2.0 ** -21)
        keep &= ((p - pieces(p)[1]).abs() / p) > LEFT
    return b[keep]


def result(p):
    return 3 * p / (1 + 3 * p)
