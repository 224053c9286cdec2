"""Rotary positions fused with the append, on the GPU: bit for bit against the
float32 definition, and against float64 within that definition's roundings."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import plain64
from test_gpu_int4 import DTYPES, bits, distinct_slots, empty_pools, gen, randn

pytestmark = pytest.mark.gpu

P = 700  # positions in the tests' table


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


class Step:
    """q, k, v as slices of one projection's output, with `gap` unused elements
    behind each token."""

    def __init__(self, T, Hq, kv, D, R, sections, dtype, seed=1, gap=0, padding=True):
        width = (Hq + 2 * kv) * D + gap
        self.qkv = randn((T, width), dtype, seed)
        rows = self.qkv[:, :(Hq + 2 * kv) * D].unflatten(1, (-1, D))
        self.q, self.k, self.v = rows[:, :Hq], rows[:, Hq:Hq + kv], rows[:, Hq + kv:]
        self.NB = -(-T // 16) + 2
        self.slots = distinct_slots(T, self.NB, seed + 1, padding)
        A = len(sections)
        self.pos = torch.randint(0, P, (A, T), generator=gen(seed + 2)).to(torch.int32)
        self.pos[:, 0] = torch.tensor([0, P - 1, 0, P - 1][:A])
        self.cs = plain64.angles(P, R)
        self.sections = sections
        g = self.qkv.cuda()
        rows = g[:, :(Hq + 2 * kv) * D].unflatten(1, (-1, D))
        self.gpu = rows[:, :Hq], rows[:, Hq:Hq + kv], rows[:, Hq + kv:]

    def want(self, interleaved, x):
        return plain64.rotate(x, self.cs, self.pos, self.sections, interleaved)


SHAPES = [  # T, Hq, kv, D, R, sections, gap
    (1, 1, 1, 64, 64, (32,), 0),
    (5, 8, 2, 64, 32, (16,), 8),
    (64, 64, 8, 128, 128, (16, 24, 24), 0),
    (33, 6, 3, 128, 64, (7, 0, 25), 16),
    (40, 5, 5, 128, 16, (1, 2, 3, 2), 0),
    (17, 12, 1, 64, 48, (8, 16), 0),
    (9, 0, 4, 128, 112, (56,), 0),
    (1500, 8, 2, 128, 128, (10, 18, 18, 18), 0),
    (2100, 16, 4, 64, 64, (8, 12, 12), 24),
    # several tokens to a warp, and units that no power of two divides
    (9001, 1, 1, 128, 128, (16, 24, 24), 0),
    (7001, 1, 1, 64, 48, (8, 16), 8),
    (5003, 7, 1, 128, 64, (7, 0, 25), 16),
    (4001, 8, 2, 64, 32, (16,), 8),
    (2502, 5, 5, 128, 112, (56,), 0),
    (12007, 0, 1, 64, 64, (32,), 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope_append_bit_exact(dtype, interleaved, shape):
    T, Hq, kv, D, R, sections, gap = shape
    s = Step(T, Hq, kv, D, R, sections, dtype, seed=T, gap=gap)
    kc = torch.full((s.NB, kv, 16, D), 3.0, dtype=dtype)
    gk, gv = kc.cuda(), kc.cuda()
    q_out = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda") if Hq else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvp.kvp_rope_append(q_out, s.gpu[0] if Hq else None, s.gpu[1], s.gpu[2], gk, gv, s.cs.cuda(),
                        s.pos.cuda(), s.slots.cuda(), sections=sections, interleaved=interleaved,
                        status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    assert torch.equal(bits(gk), bits(plain64.scatter(kc, s.want(interleaved, s.k), s.slots)))
    assert torch.equal(bits(gv), bits(plain64.scatter(kc, s.v, s.slots)))
    if Hq:
        want = s.want(interleaved, s.q)
        want[s.slots < 0] = 5.0  # padding rows are left as they are
        assert torch.equal(bits(q_out), bits(want))
        # against 64 bits: two products, a sum and the 16-bit rounding
        ref = plain64.rotate(s.q, s.cs, s.pos, sections, interleaved, torch.float64)
        live = s.slots >= 0
        big = plain64.rotate(s.q.abs(), s.cs.abs() * torch.tensor([1.0]), s.pos, sections,
                             interleaved, torch.float64).abs()
        size = s.q.double().abs().amax(-1, keepdim=True) * 2 + big
        half = torch.finfo(dtype).eps / 2
        tol = half * ref.abs() * (1 + half) + 2.0 ** -22 * size + torch.finfo(dtype).tiny * half
        assert ((q_out.cpu().double() - ref).abs() <= tol)[live].all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope_append_int4_is_rope_then_quantise(dtype, interleaved, shape):
    T, Hq, kv, D, R, sections, gap = shape
    s = Step(T, Hq, kv, D, R, sections, dtype, seed=T + 7, gap=gap)
    kc, vc, ks, vs = empty_pools(s.NB, kv, D, dtype)
    g = [t.cuda() for t in (kc, vc, ks, vs)]
    q_out = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda") if Hq else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvp.kvp_rope_append_int4(q_out, s.gpu[0] if Hq else None, s.gpu[1], s.gpu[2], *g, s.cs.cuda(),
                             s.pos.cuda(), s.slots.cuda(), sections=sections,
                             interleaved=interleaved, status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    for x, codes, pairs, gc, gp in ((s.want(interleaved, s.k), kc, ks, g[0], g[2]),
                                    (s.v, vc, vs, g[1], g[3])):
        c, p = plain64.quantise4(x)
        assert torch.equal(gc.cpu(), plain64.scatter(codes, plain64.pack4(c), s.slots))
        want = plain64.scatter(pairs, p, s.slots)
        assert ((bits(gp) == bits(want)) | (gp.cpu() == want)).all()
    if Hq:
        want = s.want(interleaved, s.q)
        want[s.slots < 0] = 5.0
        assert torch.equal(bits(q_out), bits(want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope_append_in_place(dtype):
    """q_out may be q, here a slice of the projection's output."""
    s = Step(50, 8, 2, 128, 128, (16, 24, 24), dtype, seed=3)
    kc = torch.zeros((s.NB, 2, 16, 128), dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    kvp.kvp_rope_append(s.gpu[0], s.gpu[0], s.gpu[1], s.gpu[2], kc, vc, s.cs.cuda(), s.pos.cuda(),
                        s.slots.cuda(), sections=s.sections)
    want = s.want(False, s.q)
    want[s.slots < 0] = s.q[s.slots < 0]
    assert torch.equal(bits(s.gpu[0]), bits(want))
    assert torch.equal(bits(s.gpu[1]), bits(s.k)) and torch.equal(bits(s.gpu[2]), bits(s.v))


@pytest.mark.parametrize("T", [6, 3000])
@pytest.mark.parametrize("int4", [False, True])
def test_rope_append_bad_position_or_slot(T, int4):
    dtype, D, kv, Hq = torch.float16, 64, 2, 4
    s = Step(T, Hq, kv, D, D, (10, 22), dtype, seed=4, padding=False)
    bad = [1, 3, 4]
    s.pos[1, bad[0]] = P
    s.pos[0, bad[1]] = -1
    s.slots[bad[2]] = s.NB * 16
    q_out = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (s.cs.cuda(), s.pos.cuda(), s.slots.cuda())
    if int4:
        kc, vc, ks, vs = empty_pools(s.NB, kv, D, dtype)
        g = [t.cuda() for t in (kc, vc, ks, vs)]
        kvp.kvp_rope_append_int4(q_out, *s.gpu, *g, *args, sections=(10, 22), status=status)
    else:
        kc = torch.full((s.NB, kv, 16, D), 3.0, dtype=dtype)
        g = [kc.cuda(), kc.cuda()]
        kvp.kvp_rope_append(q_out, *s.gpu, *g, *args, sections=(10, 22), status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    s.pos.clamp_(0, P - 1)
    want_q, k = s.want(False, s.q), s.want(False, s.k)
    want_q[bad] = 0
    assert torch.equal(bits(q_out), bits(want_q))
    slots = s.slots.clone()
    slots[bad] = -1
    rows = plain64.pack4(plain64.quantise4(k)[0]) if int4 else k
    assert torch.equal(bits(g[0]), bits(plain64.scatter(kc, rows, slots)))


def test_rope_append_no_tokens_is_a_no_op():
    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.ones((2, 1, 16, 64), dtype=torch.float16, device="cuda")
    x = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    kvp.kvp_rope_append(x, x, x, x, kc, kc, plain64.angles(4, 64).cuda(),
                        torch.empty(0, **i32), torch.empty(0, **i32))
    assert (kc == 1).all()
