"""4-bit decode of long contexts: the error of the outputs as a whole (rms64), which a
block or token lost or read twice where a context is cut exceeds."""
import pytest
import torch

import plain64
import rms64
from test_gpu_int4 import DTYPES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    import pagedattention_decode_kvp_gb300 as kvp
    _build.build()
    kvp.load_library()


LONG = [([20011], 8, 1, 128, (0, 1024)), ([9011, 3000, 1500, 6345], 8, 1, 64, (0, 100)),
        ([2500, 1017, 2499], 8, 8, 64, (0,)), ([1100, 1099, 1088], 32, 16, 128, (0, 7)),
        ([1040, 128, 129, 1999], 2, 1, 128, (0, 16)), ([8300, 9000], 8 * 229, 1, 128, (0,)),
        ([1999, 700, 1437, 348, 792], 16, 1, 128, (0,))]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,Hq,kv,D,parts", LONG)
def test_error_of_long_contexts_as_a_whole(dtype, lens, Hq, kv, D, parts):
    """Where contexts are cut, by themselves or together, into pieces, segments and
    partitions: a block lost or read twice at a cut exceeds the limit."""
    c = Case(lens, Hq, kv, D, dtype, seed=33, max_blocks=max(70, -(-max(lens) // 16)))
    step = max(1, Hq // 16)  # (query heads looked at)
    heads = list(range(0, Hq, step)) if kv == 1 else list(range(Hq))
    ref = torch.stack([reference(c, b, heads) for b in range(len(lens))])
    for pb in parts:
        out = c.run(pb)[:, heads]
        for b in range(len(lens)):
            e = rms64.relative(out[b], ref[b])
            assert (e < rms64.limit(dtype, ref[b])).all(), (pb, b, e)


def reference(c, b, heads):
    """float64 attention of request b's given query heads."""
    n, Hq, kv = int(c.lens[b]), c.q.shape[1], c.kc.shape[1]
    ids = c.tables[b, :-(-n // 16)].long()

    def values(codes, pairs):  # [kv, n, D]
        x = plain64.values4(codes[ids], pairs[ids])
        return x.transpose(0, 1).flatten(1, 2)[:, :n]

    k, v = values(c.kc, c.ks), values(c.vc, c.vs)
    of = torch.tensor([h // (Hq // kv) for h in heads])
    s = torch.einsum("hd,hnd->hn", c.q[b, heads].double(), k[of]) if kv > 1 else \
        c.q[b, heads].double() @ k[0].T
    w = torch.softmax(s * c.scale, 1)
    return torch.einsum("hn,hnd->hd", w, v[of]) if kv > 1 else w @ v[0]
