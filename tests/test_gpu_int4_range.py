"""4-bit decode over values of any size: rows and groups of very different scales,
rows without a scale beside them, and queries up to the stated limits."""
import math

import pytest
import torch

import plain64
import rms64
from test_gpu_int4 import DTYPES, Case, gen, randn

pytestmark = pytest.mark.gpu
F16, BF16 = DTYPES


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    import pagedattention_decode_kvp_gb300 as kvp
    _build.build()
    kvp.load_library()


def widened(c, max_blocks):
    """The same case with wider tables (the automatic split)."""
    more = torch.full((c.tables.shape[0], max_blocks - c.tables.shape[1]), -1, dtype=torch.int32)
    c.tables = torch.cat([c.tables, more], 1)
    return c


def check_all(c, dtype, rms=False):
    """One pass, given partitions, balanced pieces."""
    ref, tol = plain64.decode4(c.q, c.kc, c.vc, c.ks, c.vs, c.tables, c.lens, c.scale)
    for way, pb in (("one pass", 0), ("one block a partition", 1), ("partitions", 3),
                    ("balanced", -1)):
        if pb < 0:
            widened(c, 70)
        out = c.run(max(pb, 0))
        assert torch.isfinite(out).all(), way
        err = (out.cpu().double() - ref).abs()
        worst = float((err / tol.clamp(min=1e-300)).max())
        assert (err <= tol).all(), f"{way}: worst error is {worst:.3g} of the bound"
        for b in range(len(ref)) if rms else ():
            e = rms64.relative(out[b], ref[b])
            assert (e < rms64.limit(dtype, ref[b])).all(), (way, b, e)


def test_zero_rows_beside_one_large_row():
    """Equal scores, 16 rows of zeros and one of +-1e30: a 17th of it."""
    k, v = torch.zeros(17, 1, 64), torch.zeros(17, 1, 64)
    v[16] = torch.linspace(-1e30, 1e30, 64)
    c = Case([17], 2, 1, 64, BF16, k=[k], v=[v])
    check_all(c, BF16)


@pytest.mark.parametrize("dtype,size", [(F16, 13), (F16, -12)] +
                         [(BF16, s) for s in (40, -40, 80, -80, 110, -110, 125)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [5, 16, 150])
def test_rows_without_a_scale_beside_rows_of_any_size(dtype, size, D, at):
    """Rows of one value (0, ordinary, or as large as the others) before and after
    rows of size 2^size, in a block (at 5), across warps and across runs; scores
    equal and not."""
    n = 200
    rows = (torch.randn(n, 1, D, generator=gen(1)).clamp(-2.9, 2.9) * 2.0 ** size).to(dtype)
    flat = torch.randn(n, 1, 1, generator=gen(2)).expand(-1, -1, D)
    early = (torch.arange(n) < at)[:, None, None]
    v, k = [], []
    for const in (torch.zeros_like(flat), flat, flat.clamp(-2.9, 2.9) * 2.0 ** size):
        for first in (True, False):
            v.append(torch.where(early == first, const.to(dtype), rows))
            k.append(torch.zeros(n, 1, D) if first else randn((n, 1, D), dtype, 7))
    c = Case([n] * 6, 3, 1, D, dtype, seed=5, k=k, v=v)
    check_all(c, dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [0, 100, 126])
def test_large_rows_without_a_scale_under_rising_scores(D, size):
    """Scores that climb by over 100 powers of two, values that only the zeros
    carry."""
    n = 300
    direction = torch.sign(torch.randn(D, generator=gen(1)))
    k = [(direction * torch.arange(n)[:, None, None] * f).to(BF16) for f in (0.5 / D, 2.0 / D)]
    v = [(torch.randn(n, 1, 1, generator=gen(2)).clamp(-1.9, 1.9) * 2.0 ** size)
         .expand(-1, -1, D).to(BF16)] * 2
    q = (direction * math.sqrt(D)).expand(2, 2, D).to(BF16).contiguous()
    check_all(Case([n] * 2, 2, 1, D, BF16, k=k, v=v, q=q), BF16)


GROUPS = [(F16, 9, -9), (F16, 12, -12), (F16, -10, 12)] + \
    [(BF16, a, b) for a, b in ((0, -18), (-20, 0), (12, -12), (-15, 15), (30, -30), (-50, 50),
                               (110, -100))]


@pytest.mark.parametrize("dtype,a,b", GROUPS)
def test_two_groups_of_different_scale(dtype, a, b):
    """head_dim 128: each group of 64 is as exact as if the other were not there,
    at one ratio throughout or one that changes from token to token."""
    n = 320
    v = []
    for grade in (lambda t: 1.0, lambda t: t / n, lambda t: 1 - t / n, lambda t: float(t % 2)):
        f = torch.tensor([grade(t) for t in range(n)])[:, None, None, None]
        x = torch.randn(n, 2, 2, 64, generator=gen(3)).clamp(-2.9, 2.9)
        v.append((x * torch.exp2(f * torch.tensor([float(a), float(b)])[:, None]))
                 .flatten(2).to(dtype))
    c = Case([n] * 4, 8, 2, 128, dtype, seed=9, v=v)
    check_all(c, dtype)
    steady = Case([n], 8, 2, 128, dtype, seed=9, v=v[:1])
    check_all(steady, dtype, rms=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [118.99, 115.0, 111.5, 80.0, -115.0, -124.0])
def test_queries_at_the_stated_limits(D, size):
    """bf16 queries of almost 2^119 (times the scale of 2^-3 and 2^-3.5 below 2^116)
    and down to 2^-126, with keys that keep the scores ordinary."""
    n = 90
    q = torch.rand(1, 6, D, generator=gen(4)) * 2.0 ** size
    q[0, 3, 5] = 2.0 ** size
    k = [(torch.randn(n, 2, D, generator=gen(5)).clamp(-2.9, 2.9) * 2.0 ** -size).to(BF16)]
    c = Case([n], 6, 2, D, BF16, seed=14, k=k, q=q.to(BF16))
    check_all(c, BF16)


@pytest.mark.parametrize("dtype,size", [(F16, 12), (BF16, 30), (BF16, -90), (BF16, 110)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [100, 5000, 8700])
def test_sizes_that_change_in_the_middle_of_a_long_run(dtype, size, D, at):
    """From one token on, in a run of two slices of its block table, or for one block
    alone; whole, in pieces of all contexts and in partitions."""
    n = 9011
    x = torch.randn(n, 1, D, generator=gen(1)).clamp(-2.9, 2.9)
    t = torch.arange(n)[:, None, None]
    big = torch.tensor(2.0 ** size)
    v = [(x * torch.where(t >= at, big, torch.tensor(1.0))).to(dtype),
         (x * torch.where((t >= at) & (t < at + 16), big, torch.tensor(1.0))).to(dtype)]
    c = Case([n, n], 2, 1, D, dtype, seed=3, v=v)
    ref, tol = plain64.decode4(c.q, c.kc, c.vc, c.ks, c.vs, c.tables, c.lens, c.scale)
    for pb in (0, 1024, 100):
        out = c.run(pb)
        err = (out.cpu().double() - ref).abs()
        assert (err <= tol).all(), (pb, float((err / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("dtype,size", [(F16, 12), (BF16, 60), (BF16, -100)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_short_runs_of_any_size(dtype, size, D):
    """A warp for each of many runs: ordinary, without a scale, large, and both."""
    B = 700
    lens, v = [1 + (7 * b * b) % 45 for b in range(B)], []
    for b, n in enumerate(lens):
        x = torch.randn(n, 1, D, generator=gen(b)).clamp(-2.9, 2.9)
        if b % 4 == 1:
            x = x[..., :1].expand(-1, -1, D)
        if b % 4 >= 2:
            x = x * torch.where((torch.arange(n) >= n // 2)[:, None, None] | (b % 4 == 2),
                                2.0 ** size, 1.0)
        v.append(x.to(dtype))
    c = Case(lens, 1, 1, D, dtype, seed=8, v=v)
    c.check(c.run())
