"""Norms of rows whose squares leave float32's range, and of every size beside each other."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import project64 as ref
from test_gpu_int4 import bits, randn

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def rows(D, seed):
    """Rows of N(0, 1), each at a size of its own: the ends of bf16, where sums of squares
    overflow (2^64 / sqrt(D)) or vanish, and one element far above or below its row."""
    sizes = [0, 57, 60, 1, 62, 63, 100, 125, -39, -41, -60, -75, 0, -100, -126, 40, -20]
    x = randn((len(sizes) + 4, D), torch.float64, seed).clamp(-3.9, 3.9)
    x[:len(sizes)] *= 2.0 ** torch.tensor(sizes, dtype=torch.float64)[:, None]
    x[-4, D // 2] = 2.0 ** 127
    x[-3] *= 2.0 ** -90
    x[-3, D - 1] = 2.0 ** -50
    x[-2] = 2.0 ** 127
    x[-1, :-1] = 0
    x[-1, -1] = 2.0 ** -133
    return x.to(BF16)


def bound(want):
    """norm_bound, and half a step of bf16 below its normal range.  (The powers of two that
    such rows are scaled by are exact.)"""
    return ref.norm_bound(want, BF16) + 2.0 ** -134


# every kernel of the norm: D up to 64, 128, 256, 512, 1024, ... 32768
DIMS = [8, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200,
        16384, 16392, 32768]


@pytest.mark.parametrize("eps", [1e-5, 0.0, 1e-29, 2.0 ** -140])
@pytest.mark.parametrize("D", DIMS)
def test_rows_of_every_size(D, eps):
    x, w = rows(D, D), (1 + 0.3 * randn((D,), F32, 3)).to(BF16)
    out = torch.empty_like(x, device="cuda")
    kvp.kvp_rms_norm(out, x.cuda(), w.cuda(), eps)
    want = ref.norm(x, w, torch.tensor(eps, dtype=F32).double())
    assert want.isfinite().all()
    assert ((out.cpu().double() - want).abs() <= bound(want)).all()


@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("H,D", [(1, 64), (5, 64), (7, 128), (3, 200), (2, 512), (3, 1000)])
def test_heads_of_every_size(H, D, eps):
    """Rows of different sizes in one warp, in place and inside a projection."""
    x = rows(D, 5)
    T = len(x) // H
    qkv = torch.ones((T, H + 2, D), dtype=BF16)
    qkv[:, 1:1 + H] = x[:T * H].view(T, H, D)
    w = (1 + 0.3 * randn((D,), F32, 3)).to(BF16)
    want = ref.norm(qkv[:, 1:1 + H], w, torch.tensor(eps, dtype=F32).double())
    dev = qkv.cuda()
    kvp.kvp_rms_norm(dev[:, 1:1 + H], dev[:, 1:1 + H], w.cuda(), eps)
    assert ((dev[:, 1:1 + H].cpu().double() - want).abs() <= bound(want)).all()
    assert (dev[:, 0] == 1).all() and (dev[:, -1] == 1).all()


@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("D", [64, 128, 144, 272, 528, 1040, 2064, 4112, 8208, 32768])
def test_codes_and_sums_of_every_size(D, eps):
    x, w = rows(D, D), (1 + 0.3 * randn((D,), F32, 3)).to(BF16)
    r = x.roll(1, 1) * 0.25
    h = ref.total(x, r)
    want = ref.norm(h, w, torch.tensor(eps, dtype=F32).double())
    codes = torch.empty((len(x), D), dtype=U8, device="cuda")
    scales, total = torch.empty((len(x), ref.groups(D)), device="cuda"), torch.empty_like(x, device="cuda")
    kvp.kvp_rms_norm_fp8(codes, scales, x.cuda(), w.cuda(), eps, residual=r.cuda(), residual_out=total)
    assert torch.equal(bits(total), bits(h))
    c, s = codes.cpu(), scales.cpu()
    assert ((ref.values(c, s) - want).abs() <= ref.codes_bound(want, s)).all()


@pytest.mark.parametrize("D", [64, 128, 512, 1024, 8192])
def test_zeros_infinities_and_nan(D):
    """A row of zeros is zeros (NaN without eps); an infinity leaves zeros and one NaN; neither
    touches the rows beside it."""
    x, w = rows(D, 1), torch.ones(D, dtype=BF16)
    clean = torch.empty_like(x, device="cuda")
    kvp.kvp_rms_norm(clean, x.cuda(), w.cuda(), 1e-5)
    x[0], x[3, 1], x[15, 2] = 0, float("inf"), float("nan")
    out = torch.empty_like(clean)
    kvp.kvp_rms_norm(out, x.cuda(), w.cuda(), 1e-5)
    assert (out[0] == 0).all() and out[15].isnan().all()
    assert out[3, 1].isnan() and (out[3, 2:] == 0).all() and out[3, 0] == 0
    rest = [i for i in range(len(x)) if i not in (0, 3, 15)]
    assert torch.equal(bits(out[rest]), bits(clean[rest]))
    kvp.kvp_rms_norm(out, x.cuda(), w.cuda(), 0.0)
    assert out[0].isnan().all() and not out[rest].isnan().any()


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
@pytest.mark.parametrize("T,D", [(64, 8192), (300, 128), (5, 4096)])
def test_the_same_norm_gives_the_same_bits(T, D, dtype):
    """Whatever the outputs held before, and between other calls."""
    x, r, w = (randn(s, dtype, i).cuda() for i, s in enumerate([(T, D), (T, D), (D,)]))
    other = randn((T, D), dtype, 9).cuda()

    def all_of(x, fill):
        out, total, mine = (torch.full_like(x, fill) for _ in range(3))
        codes, scales = (torch.full((T, n), fill, dtype=d, device="cuda")
                         for n, d in ((D, U8), (ref.groups(D), F32)))
        again = [torch.full_like(t, fill) for t in (codes, scales)]
        kvp.kvp_rms_norm(out, x, w, 1e-5, residual=r, residual_out=total)
        kvp.kvp_rms_norm_fp8(codes, scales, x, w, 1e-5, residual=r, residual_out=mine)
        kvp.kvp_quantise_fp8(*again, x)
        return [bits(t) for t in (out, total, mine, codes, scales, *again)]

    first = all_of(x, 0)
    for i in range(1, 20):
        all_of(other, i)
        for a, b in zip(first, all_of(x, i)):
            assert torch.equal(a, b)
