"""The serving step of the README, run as it stands there."""
import os
import re

import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import plain64
from test_gpu_int4 import randn

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def serving_step():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    step, = (b for b in blocks if "kvp_release_tables" in b)
    return step


@pytest.mark.parametrize("finished,new", [([0, 1, 0, 0], [1, 0, 1, 1]), ([1, 0, 0, 0], [0, 2, 0, 3]),
                                          ([0, 0, 0, 1], [1, 1, 1, 4])])
def test_each_request_attends_with_its_own_query(finished, new):
    """Also beside requests that finish, or get no or several new tokens."""
    B, Hq, Hkv, D, MB, NB, T = 4, 4, 2, 64, 6, 30, 16
    z = dict(dtype=torch.int32, device="cuda")
    f = dict(dtype=torch.float16, device="cuda")
    before = [20, 5, 33, 47]
    tables = torch.full((B, MB), -1, **z)
    at = 0
    for b, n in enumerate(before):
        k = -(-n // 16)
        tables[b, :k] = torch.arange(at, at + k, **z)
        at += k
    v = dict(kvp=kvp, torch=torch, B=B, Hq=Hq, Hkv=Hkv, D=D, tables=tables,
             lens=torch.tensor(before, **z), finished=torch.tensor(finished, **z),
             new_lens=torch.tensor(new, **z), free_blocks=torch.arange(NB, **z).flip(0).contiguous(),
             free_count=torch.tensor([NB - at], **z), slots=torch.zeros(T, **z),
             query_start=torch.zeros(B + 1, **z), positions=torch.zeros(T, **z),
             qkv=randn((T, Hq + 2 * Hkv, D), torch.float16, 2).cuda(),
             q_out=torch.full((T, Hq, D), float("nan"), **f),
             out=torch.full((B, Hq, D), float("nan"), **f),
             k_codes=torch.zeros((NB, Hkv, 16, D // 2), dtype=torch.uint8, device="cuda"),
             v_codes=torch.zeros((NB, Hkv, 16, D // 2), dtype=torch.uint8, device="cuda"),
             k_pairs=torch.zeros((NB, Hkv, 16, D // 64, 2), **f),
             v_pairs=torch.zeros((NB, Hkv, 16, D // 64, 2), **f),
             cos_sin=plain64.angles(128, D).cuda())
    pools = [v[n] for n in ("k_codes", "v_codes", "k_pairs", "v_pairs")]
    x = randn((2, NB * 16, Hkv, D), torch.float16, 1).cuda()
    kvp.kvp_append_int4(x[0], x[1], *pools, torch.arange(NB * 16, **z))
    exec(serving_step(), v)
    after = [(0 if e else n) + k for e, n, k in zip(finished, before, new)]
    assert v["lens"].tolist() == after
    ends = torch.tensor(new).cumsum(0)
    q = v["q_out"].cpu()[(ends - 1).clamp(min=0)]
    live = [b for b in range(B) if new[b] > 0]
    for b in live:  # the last new token of request b, rotated by its position
        want = plain64.rotate(v["qkv"].cpu()[int(ends[b]) - 1, None, :Hq], v["cos_sin"].cpu(),
                              [torch.tensor([after[b] - 1])], (D // 2,), False)
        assert torch.equal(q[b], want[0])
    ref, tol = plain64.decode4(q, *(t.cpu() for t in pools), v["tables"].cpu(), v["lens"].cpu(),
                               D ** -0.5)
    for b in live:
        assert ((v["out"][b].cpu().double() - ref[b]).abs() <= tol[b]).all(), b
