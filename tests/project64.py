"""Norms, E4M3 quantisers and the block-scaled product in 64 bits, on the CPU, and how
far the kernels may be from them."""
import torch

GROUP = 128


def groups(x, n=GROUP):
    return -(-x // n)


def spread(scales, rows, cols, block_rows):
    """Scales per element."""
    s = scales.double().repeat_interleave(GROUP, 1)[:, :cols]
    return s.repeat_interleave(block_rows, 0)[:rows]


def values(codes, scales, block_rows=1):
    """What codes [R, D] (uint8 or float8) stand for."""
    c = codes.view(torch.float8_e4m3fn).double()
    return c * spread(scales, *c.shape, block_rows)


def quantise(x, block_rows=1):
    """Codes (uint8) and scales of x [R, D] by the definition, in float32."""
    R, D = x.shape
    nr, nd = groups(R, block_rows), groups(D)
    g = torch.zeros(nr * block_rows, nd * GROUP)
    g[:R, :D] = x.float()
    g = g.view(nr, block_rows, nd, GROUP)
    a = torch.where(g.isnan(), 0.0, g.abs()).amax((1, 3), keepdim=True)
    b = a.clamp(min=2.0 ** -100)
    scale = torch.where(a > 0, b / 448, 1.0)
    # (448 / b would be 448 times b's reciprocal: two roundings)
    codes = (g * torch.full_like(b, 448).div(b)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(nr * block_rows, nd * GROUP)[:R, :D].contiguous(), scale.view(nr, nd)


def total(x, residual):
    """x + residual as it is kept: a float32 sum rounded to the type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(h, weight, eps):
    """The norm of h [..., D] in 64 bits."""
    d = h.double()
    return d / (d.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


# The norm in float32: a thread adds at most 32 squares, 5 exchanges and at most 32
# partial sums follow, all of one sign: the sum is off by at most 69 roundings of
# 2^-24, its root by half of that; the division, eps, the root and the two products
# add 5 more.
NORM = 40 * 2.0 ** -24


def norm_bound(y, dtype):
    """The norm rounded once to 16 bits; fp16 has steps of 2^-24 below 2^-14."""
    half = torch.finfo(dtype).eps / 2
    return y.abs() * (half + NORM * (1 + half)) + (2.0 ** -25 if dtype == torch.float16 else 0)


def codes_bound(y, scales, off=NORM):
    """|value - y|: half a step of E4M3 (2^-4 of the value, 2^-10 scales below 2^-6
    scales), of a y that is `off` by itself and by its scale."""
    s = spread(scales, *y.shape, 1)
    return y.abs() * (2.0 ** -4 + 3 * off + 2.0 ** -22) + s * 2.0 ** -10


def matmul(a, sa, b, sb):
    """out, and the sum of its terms' magnitudes."""
    x, y = values(a, sa), values(b, sb, GROUP)
    return x @ y.t(), x.abs() @ y.abs().t()


def matmul_bound(size, k, out, dtype):
    """A group is summed by four instructions of 32 products each, aligned to the largest
    and cut below 2^-23 of it: 4 x 33 steps of 2^-23 of the sum of magnitudes at most.
    Each group's scales and addition round by 2^-24 in float32; out rounds once."""
    off = size * (4 * 33 * 2.0 ** -23 + (groups(k) + 2) * 2.0 ** -24)
    half = 0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    return off * (1 + half) + out.abs() * half + (2.0 ** -25 if dtype == torch.float16 else 0)
