"""Norms and quantisers of so many rows that what they read and write passes 32 bits."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import project64 as ref
from test_gpu_int4 import bits, randn

pytestmark = pytest.mark.gpu

F16, F32, U8 = torch.float16, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def tall(R, D, seed):
    """[R, D], zeros but for some rows, the last ones among them; those rows."""
    at = torch.tensor([0, 1, 2 ** 20 + 3, R // 2, R // 2 + 1, R - 129, R - 2, R - 1])
    x = torch.zeros((R, D), dtype=F16, device="cuda")
    few = randn((len(at), D), F16, seed)
    x[at.cuda()] = few.cuda()
    return x, few, at


@pytest.mark.parametrize("R,D", [(2 ** 24 + 3, 128), (2 ** 29 + 77, 16)])
def test_codes_and_scales(R, D):
    """Codes past 2^31 bytes; with 16 columns the scales too."""
    x, few, at = tall(R, D, 1)
    w = (1 + 0.3 * randn((D,), F32, 2)).to(F16)
    codes = torch.full((R, D), 9, dtype=U8, device="cuda")
    scales = torch.full((R, ref.groups(D)), 9.0, device="cuda")
    kvp.kvp_rms_norm_fp8(codes, scales, x, w.cuda(), 1e-5)
    c, s = codes[at.cuda()].cpu(), scales[at.cuda()].cpu()
    want = ref.norm(few, w, 1e-5)
    assert ((ref.values(c, s) - want).abs() <= ref.codes_bound(want, s)).all()
    codes[at.cuda()], scales[at.cuda()] = 0, 1
    assert not codes.any() and (scales == 1).all()

    codes.fill_(9), scales.fill_(9)
    kvp.kvp_quantise_fp8(codes, scales, x)
    want, ws = ref.quantise(few)
    assert torch.equal(codes[at.cuda()].cpu(), want) and torch.equal(scales[at.cuda()].cpu(), ws)
    codes[at.cuda()], scales[at.cuda()] = 0, 1
    assert not codes.any() and (scales == 1).all()

    codes.fill_(9)
    scales = torch.full((ref.groups(R), ref.groups(D)), 9.0, device="cuda")
    kvp.kvp_quantise_fp8(codes, scales, x, block_rows=128)
    for i in {int(i) // 128 for i in at}:
        rows = slice(128 * i, min(R, 128 * i + 128))
        want, ws = ref.quantise(x[rows].cpu(), 128)
        assert torch.equal(codes[rows].cpu(), want) and torch.equal(scales[i:i + 1].cpu(), ws)
        codes[rows], scales[i] = 0, 1
    assert not codes.any() and (scales == 1).all()


def test_the_most_rows_of_a_norm():
    """2^31 - 1 rows, in place."""
    R, D = 2 ** 31 - 1, 8
    x, few, at = tall(R, D, 3)
    w = (1 + 0.3 * randn((D,), F32, 2)).to(F16)
    kvp.kvp_rms_norm(x, x, w.cuda(), 1e-5)
    want = ref.norm(few, w, 1e-5)
    assert ((x[at.cuda()].cpu().double() - want).abs() <= ref.norm_bound(want, F16)).all()
    x[at.cuda()] = 0
    assert not x.view(torch.int64).any()


def test_a_residual_of_many_rows():
    R, D = 2 ** 27 + 5, 32
    x, few, at = tall(R, D, 4)
    w = (1 + 0.3 * randn((D,), F32, 2)).to(F16)
    out = torch.full_like(x, 9)
    kvp.kvp_rms_norm(out, x, w.cuda(), 1e-5, residual=x, residual_out=x)
    h = ref.total(few, few)
    want = ref.norm(h, w, 1e-5)
    assert torch.equal(bits(x[at.cuda()]), bits(h))
    assert ((out[at.cuda()].cpu().double() - want).abs() <= ref.norm_bound(want, F16)).all()
    x[at.cuda()], out[at.cuda()] = 0, 0
    assert not x.view(torch.int64).any() and not out.view(torch.int64).any()
