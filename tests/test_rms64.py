"""The criterion of rms64.py: outputs rounded as a kernel rounds them pass, outputs
without one block, without one token, or with a block twice do not."""
import pytest
import torch

import rms64


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [1000, 9000, 20011])
def test_a_lost_block_shows(dtype, n):
    D, H = 64, 8
    v = torch.randn(n, D, generator=gen(1), dtype=torch.float64)
    p = torch.randn(H, n, generator=gen(2), dtype=torch.float64).exp()
    ref = (p @ v) / p.sum(1, keepdim=True)
    top = rms64.limit(dtype)
    # a kernel's roundings
    low, high = v.amin(1, keepdim=True), v.amax(1, keepdim=True)
    s, mid = (high - low) / 15, (high + low) / 2
    a = (p[:, :, None] * s).float().half().double()[..., 0]
    out = (a @ ((v - mid) / s) + p @ mid) / p.sum(1, keepdim=True)
    assert (rms64.relative(out.to(dtype), ref) < top).all()
    tokens = torch.randint(0, n, (50,), generator=gen(3)).tolist() + [0, n - 1]
    for t in tokens:
        lost, block = torch.ones(n, dtype=torch.float64), torch.ones(n, dtype=torch.float64)
        lost[t] = 0
        block[t // 16 * 16:t // 16 * 16 + 16] = 0
        for keep, sure in ((block, True), (2 - block, True), (lost, dtype == torch.float16)):
            w = p * keep
            err = rms64.relative(((w @ v) / w.sum(1, keepdim=True)).to(dtype), ref)
            assert not sure or (err > top).all(), (t, float(err))
