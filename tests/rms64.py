"""How far a decode's output may be from float64 as a whole: a relative root mean
square, which a single block of a long context left out or counted twice exceeds
many times over (test_rms64.py), where a bound per element that adds up every
rounding's worst case does not notice it."""
import math

import torch


def limit(dtype, ref=None, group=64):
    """Twice the expected error of outputs of many tokens with independent values.

    A rounding to p bits is off by up to half a step h = 2^-p of a value with
    mantissa m in [1, 2): relative error uniform in +-h / m, root mean square
    h / sqrt(3) sqrt(E 1/m^2) = 0.425 h for log-uniform m (E 1/m^2 = 3 / (8 ln 2)).
      * the output: h = eps / 2 of its type;
      * the weights a_t = p_t s_t: h = 2^-11, independent from token to token, each
        times (c - 7.5) s of its row.  That is V less the middle of its row's range,
        whose square is 1.2 V^2 on average for normal rows of 64 (the middle of the
        range of 64 normal values has variance 0.2): a relative 0.425 h sqrt(1.2)
        of the output, whose own square is the sum of w^2 V^2.
    Everything else is float32.  Twice that leaves room for how few tokens carry an
    output and how few outputs are averaged.

    With ref [H, D], for every group: outputs below the type's normal range (2^-14
    in fp16, which means of values of 2^-12 over 320 tokens are) lie on a grid of
    its smallest step, u = 2^-24, so their rounding is off by up to u / 2 however
    small they are, u / sqrt(12) root mean square."""
    half = torch.finfo(dtype).eps / 2
    squares = half ** 2 + 1.2 * 2.0 ** -22
    if ref is None:
        return 2 * 0.425 * math.sqrt(squares)
    step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    size2 = ref.double().unflatten(-1, (-1, group)).pow(2).mean((0, 2))
    return 2 * (0.425 ** 2 * squares + step ** 2 / 12 / size2).sqrt()


def relative(out, ref, group=64):
    """Relative root mean square error of out [H, D] for every group of the row."""
    o, r = (x.double().cpu().unflatten(-1, (-1, group)) for x in (out, ref))
    return ((o - r).pow(2).mean((0, 2)) / r.pow(2).mean((0, 2))).sqrt()
