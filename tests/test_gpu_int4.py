"""4-bit pools on the GPU: the quantising append, the read-back and the block
copy bit for bit against their float32 definition, the decode against float64
within a bound derived from its roundings (plain64.decode4)."""
import math

import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import plain64

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(dtype)


def empty_pools(NB, kv, D, dtype):
    """Pools of a byte pattern that nothing writes by chance, and NaN pairs."""
    codes = torch.full((NB, kv, 16, D // 2), 0xA5, dtype=torch.uint8)
    pairs = torch.full((NB, kv, 16, D // 64, 2), float("nan"), dtype=dtype)
    return codes, codes.clone(), pairs, pairs.clone()


def bits(t):
    return t.cpu().contiguous().view(torch.int16) if t.dtype in DTYPES else t.cpu()


def distinct_slots(T, NB, seed, padding=True):
    s = torch.randperm(NB * 16, generator=gen(seed))[:T].to(torch.int32)
    if padding and T > 3:
        s[torch.rand(T, generator=gen(seed + 1)) < 0.2] = -1
    return s


def special_rows(T, kv, D, dtype, seed):
    """Rows where a quantiser can go wrong: zeros, constants, the type's largest
    and smallest magnitudes, values half way between codes, one outlier."""
    x = randn((T, kv, D), dtype, seed)
    big = torch.finfo(dtype).max
    rows = [torch.zeros(D), torch.full((D,), 3.25), torch.full((D,), -0.0),
            torch.randn(D, generator=gen(seed)) * 1e-7, torch.arange(D) * 2.0 ** -24,
            (torch.arange(D) % 31) * 0.5, (torch.arange(D) % 31) * 0.5 - 7.0,
            torch.where(torch.arange(D) == 17, 500.0, 0.01), torch.arange(D) - D / 2.0]
    if dtype == torch.float16:
        rows += [torch.where(torch.arange(D) % 2 == 0, big, -big)]
    else:  # the range has to stay finite in float32
        rows += [torch.where(torch.arange(D) % 2 == 0, 1.5e38, -1.5e38),
                 torch.randn(D, generator=gen(seed)) * 1e-38,
                 torch.randn(D, generator=gen(seed + 2)) * 1e-39]
    for i, r in enumerate(rows):
        if i < T:
            x[i, 0] = r.to(dtype)
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,kv", [(1, 1), (5, 3), (37, 2), (300, 8), (1111, 5), (11003, 1),
                                  (7001, 2), (4003, 3)])
def test_append_and_read_int4_bit_exact(dtype, D, T, kv):
    NB = -(-T // 16) + 3
    key, value = special_rows(T, kv, D, dtype, 11), special_rows(T, kv, D, dtype, 12).flip(0)
    slots = distinct_slots(T, NB, 5)
    kc, vc, ks, vs = empty_pools(NB, kv, D, dtype)
    g = [t.cuda() for t in (kc, vc, ks, vs)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvp.kvp_append_int4(key.cuda(), value.cuda(), *g, slots.cuda(), status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    for x, codes, pairs, got_c, got_p in ((key, kc, ks, g[0], g[2]), (value, vc, vs, g[1], g[3])):
        c, p = plain64.quantise4(x)
        # every other slot keeps its bytes; a zero of either sign is the same zero
        want_c = plain64.scatter(codes, plain64.pack4(c), slots)
        want_p = plain64.scatter(pairs, p, slots)
        assert torch.equal(got_c.cpu(), want_c)
        got_p = got_p.cpu()
        same = (bits(got_p) == bits(want_p)) | (got_p == want_p)
        assert same.all()
    # reading back: one float32 and one 16-bit rounding; padding rows are kept
    ko = torch.full((T, kv, D), 7.0, dtype=dtype, device="cuda")
    vo = ko.clone()
    kvp.kvp_read_int4(ko, vo, *g, slots.cuda(), status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    for x, got in ((key, ko), (value, vo)):
        c, p = plain64.quantise4(x)
        want = plain64.values4(plain64.pack4(c), p, torch.float32).to(dtype)
        want[slots < 0] = 7.0
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_int4_error_is_half_a_step(dtype):
    """A value is at most half a code step from its source, plus what rounding
    the scale (half a step of the type, 15 codes) and the value itself add."""
    x = randn((64, 4, 128), dtype, 3) + randn((1, 1, 128), dtype, 4)
    c, p = plain64.quantise4(x)
    got = plain64.values4(plain64.pack4(c), p)
    half = torch.finfo(dtype).eps / 2
    s = p[..., :1].double().expand(-1, -1, -1, 64).flatten(-2)
    assert ((got - x.double()).abs() <= s * (0.5 + 15 * half) * (1 + 2.0 ** -20)).all()


def test_read_int4_same_slot_twice_and_bad_slot():
    D, kv, NB = 128, 2, 4
    x = randn((3, kv, D), torch.float16, 8)
    g = [t.cuda() for t in empty_pools(NB, kv, D, torch.float16)]
    kvp.kvp_append_int4(x.cuda(), x.cuda(), *g, torch.tensor([5, 63, 0], dtype=torch.int32).cuda())
    slots = torch.tensor([63, 63, 64, -1, 5], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ko = torch.full((5, kv, D), 9.0, dtype=torch.float16, device="cuda")
    vo = ko.clone()
    kvp.kvp_read_int4(ko, vo, *g, slots, status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    assert torch.equal(ko[0], ko[1]) and (ko[2] == 0).all() and (ko[3] == 9).all()
    c, p = plain64.quantise4(x)
    want = plain64.values4(plain64.pack4(c), p, torch.float32).half()
    assert torch.equal(ko[0].cpu(), want[1]) and torch.equal(vo[4].cpu(), want[0])


def test_append_int4_bad_slot_sets_status_and_skips():
    D, kv, NB = 64, 2, 2
    kc, vc, ks, vs = empty_pools(NB, kv, D, torch.bfloat16)
    g = [t.cuda() for t in (kc, vc, ks, vs)]
    x = randn((2, kv, D), torch.bfloat16, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvp.kvp_append_int4(x.cuda(), x.cuda(), *g, torch.tensor([32, 3], dtype=torch.int32).cuda(),
                        status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    c, _ = plain64.quantise4(x)
    want = plain64.scatter(kc, plain64.pack4(c), torch.tensor([-1, 3]))
    assert torch.equal(g[0].cpu(), want)


@pytest.mark.parametrize("D,kv", [(64, 1), (128, 3)])
def test_copy_blocks_int4_bit_exact(D, kv):
    NB = 20
    codes = [torch.randint(0, 256, (NB, kv, 16, D // 2), generator=gen(i), dtype=torch.uint8)
             for i in (1, 2)]
    pairs = [randn((NB, kv, 16, D // 64, 2), torch.float16, i) for i in (3, 4)]
    cp = torch.tensor([[3, 10], [3, 11], [7, 0], [5, 5], [19, 12]], dtype=torch.int32)
    g = [t.cuda() for t in codes + pairs]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvp.kvp_copy_blocks_int4(*g, cp.cuda(), status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    for was, now in zip(codes + pairs, g):
        want = was.clone()
        for a, b in cp.tolist():
            want[b] = was[a]
        assert torch.equal(now.cpu(), want)
    kvp.kvp_copy_blocks_int4(*g, torch.tensor([[1, 20], [2, 4]], dtype=torch.int32).cuda(),
                             status=status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    assert torch.equal(g[0][4].cpu(), codes[0][2])


# ------------------------------------------------------------------ decode
class Case:
    """Pools filled for the given lengths; every slot past a context, and every
    block of nobody, holds NaN pairs and random codes."""

    def __init__(self, lens, Hq, kv, D, dtype, seed=1, k=None, v=None, q=None, max_blocks=None,
                 spare=9):
        self.lens = torch.tensor(lens, dtype=torch.int32)
        blocks = [-(-n // 16) for n in lens]
        NB = sum(blocks) + spare
        MB = max_blocks or max(1, max(blocks))
        perm = torch.randperm(NB, generator=gen(seed)).tolist()
        self.tables = torch.full((len(lens), MB), -1, dtype=torch.int32)
        self.kc = torch.randint(0, 256, (NB, kv, 16, D // 2), generator=gen(seed + 1),
                                dtype=torch.uint8)
        self.vc = self.kc.flip(0).clone()
        self.ks = torch.full((NB, kv, 16, D // 64, 2), float("nan"), dtype=dtype)
        self.vs = self.ks.clone()
        at = 0
        for b, n in enumerate(lens):
            ids = perm[at:at + blocks[b]]
            at += blocks[b]
            self.tables[b, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
            if n == 0:
                continue
            kx = k[b] if k is not None else \
                randn((n, kv, D), dtype, seed + 10 + b) + randn((1, kv, D), dtype, seed + 5)
            vx = v[b] if v is not None else randn((n, kv, D), dtype, seed + 1000 + b)
            pos = torch.arange(n)
            blk, off = torch.tensor(ids)[pos // 16], pos % 16
            for x, codes, pairs in ((kx, self.kc, self.ks), (vx, self.vc, self.vs)):
                c, p = plain64.quantise4(x.to(dtype))
                codes[blk, :, off] = plain64.pack4(c)
                pairs[blk, :, off] = p
        self.q = q if q is not None else randn((len(lens), Hq, D), dtype, seed + 3)
        self.scale = 1.0 / math.sqrt(D)
        self.pools = [t.cuda() for t in (self.kc, self.vc, self.ks, self.vs)]

    def workspace(self, pb=0):
        n = kvp.kvp_decode_workspace_bytes(self.q.shape[0], self.q.shape[1],
                                           kvp.cache_desc_int4(self.kc), self.tables.shape[1], pb,
                                           kv_int4=True)
        return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None

    def run(self, pb=0, status=None, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda")
        kvp.kvp_attention_decode_int4(out, self.q.cuda(), *self.pools, self.tables.cuda(),
                                      self.lens.cuda(), self.scale, workspace=self.workspace(pb),
                                      partition_blocks=pb, status=status, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        ref, tol = plain64.decode4(self.q, self.kc, self.vc, self.ks, self.vs, self.tables,
                                   self.lens, self.scale)
        err = (out.cpu().double() - ref).abs()
        assert torch.isfinite(out).all()
        worst = (err / tol.clamp(min=1e-300)).max()
        assert (err <= tol).all(), f"worst error is {float(worst):.3g} of the bound"


HEADS = [(1, 1), (2, 1), (6, 2), (8, 1), (5, 5), (12, 1), (16, 2), (17, 1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,kv", HEADS)
@pytest.mark.parametrize("pb,max_blocks", [(0, 40), (3, 40), (8, 40), (0, 70)])
def test_decode_int4_shapes(dtype, D, Hq, kv, pb, max_blocks):
    """One pass (tables of up to 64 blocks), given partitions, balanced pieces."""
    c = Case([1, 15, 16, 17, 100, 257, 530, 0, 48], Hq, kv, D, dtype, seed=Hq + D,
             max_blocks=max_blocks)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(pb, status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    c.check(out)
    assert torch.count_nonzero(out[7]) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_int4_one_token_is_its_value(dtype):
    c = Case([1, 1], 4, 2, 128, dtype, seed=6)
    out = c.run()
    for b in range(2):
        v = plain64.values4(c.vc[c.tables[b, 0].long(), :, 0], c.vs[c.tables[b, 0].long(), :, 0])
        want = v.repeat_interleave(2, 0)
        # one weight of 1: its fp16 product with the scale, the centre in float32
        s = c.vs[c.tables[b, 0].long(), :, 0, :, 0].double().repeat_interleave(64, -1)
        tol = 2.0 ** -11 * 7.5 * s.repeat_interleave(2, 0) + \
            torch.finfo(dtype).eps / 2 * want.abs() * 1.001 + 2.0 ** -20
        assert ((out[b].cpu().double() - want).abs() <= tol).all()


def graded(n, kv, D, dtype, exps, seed):
    """Rows whose sizes are powers of two: exps(t) for token t."""
    x = torch.randn(n, kv, D, generator=gen(seed))
    e = torch.tensor([float(exps(t)) for t in range(n)])
    return (x * torch.exp2(e)[:, None, None]).to(dtype)


V_SIZES = {
    "one token dwarfs the rest": lambda t: 12 if t == 40 else -6,
    "first block tiny": lambda t: -20 if t < 16 else 0,
    "growing": lambda t: min(14, t // 12 - 10),
    "shrinking": lambda t: 12 - min(30, t // 8),
    "alternating": lambda t: 10 if t % 2 else -10,
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", sorted(V_SIZES))
def test_decode_int4_value_scales_of_any_size(dtype, sizes):
    lens = [300, 61]
    v = [graded(n, 2, 128, dtype, V_SIZES[sizes], 50 + n) for n in lens]
    c = Case(lens, 8, 2, 128, dtype, seed=21, v=v)
    c.check(c.run())
    c.check(c.run(4))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_decode_int4_constant_rows(dtype, D):
    """Rows of one value have scale 0 and carry everything in the zero: alone,
    and before or after rows that have a scale."""
    n = 200
    flat = torch.randn(n, 2, 1, generator=gen(3)).expand(-1, -1, D).to(dtype)
    some = randn((n, 2, D), dtype, 4, 1e-3)
    first = torch.where((torch.arange(n) < 48)[:, None, None], flat, some)
    last = torch.where((torch.arange(n) >= 150)[:, None, None], flat, some)
    zero = torch.zeros(n, 2, D, dtype=dtype)
    c = Case([n] * 4, 8, 2, D, dtype, seed=5, v=[flat, first, last, zero],
             k=[flat, some, zero, first])
    out = c.run()
    c.check(out)
    c.check(c.run(2))
    assert torch.count_nonzero(out[3]) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_int4_scores_that_rise_and_fall(dtype):
    """Scores that climb by more than the weights' headroom from block to block
    (the reference has to follow), jump once, or fall away."""
    n, D = 400, 128
    direction = torch.sign(torch.randn(D, generator=gen(1)))
    k = []
    for f in (lambda t: t / 4.0, lambda t: 60.0 if t == 333 else -20.0, lambda t: -t / 4.0):
        size = torch.tensor([f(t) for t in range(n)])
        k.append((direction * size[:, None, None] / 8 + 0.02 *
                  torch.randn(n, 1, D, generator=gen(2))).to(dtype))
    q = (direction * torch.tensor([1.0, -1.0, 0.25, 4.0])[:, None]).expand(3, 4, D)
    c = Case([n] * 3, 4, 1, D, dtype, seed=9, k=k, q=q.to(dtype).contiguous())
    c.check(c.run())
    c.check(c.run(5))


@pytest.mark.parametrize("dtype,factor", [(torch.float16, 60000.0), (torch.float16, 6e-8),
                                          (torch.bfloat16, 1e20), (torch.bfloat16, 1e-30)])
def test_decode_int4_queries_of_any_size(dtype, factor):
    """The query operand is scaled by a power of two; K is scaled the other way
    here so that the scores stay ordinary."""
    n, D = 90, 64
    q = torch.rand(1, 6, D, generator=gen(4)) * factor
    k = [(torch.randn(n, 2, D, generator=gen(5)) / factor)
         .clamp(-6e4, 6e4).to(dtype)]
    c = Case([n], 6, 2, D, dtype, seed=14, k=k, q=q.to(dtype))
    c.check(c.run())


def test_decode_int4_bad_id_in_one_piece_of_a_long_context():
    c = Case([4000, 4000], 8, 2, 128, torch.float16, seed=18)
    good = c.run()
    c.tables[0, 200] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(0, status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    assert torch.count_nonzero(out[0]) == 0 and torch.equal(out[1], good[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_int4_long_context(dtype):
    c = Case([20011], 8, 1, 128, dtype, seed=31)
    c.check(c.run())
    c.check(c.run(1024))  # one CTA walks 16384 tokens


def test_decode_int4_split_phases_and_repeats_give_the_same_bits():
    c = Case([900, 33, 2000], 16, 2, 128, torch.float16, seed=4)
    whole = c.run(16)
    assert torch.equal(whole, c.run(16))
    out, ws = torch.zeros_like(whole), c.workspace(16)
    args = (out, c.q.cuda(), *c.pools, c.tables.cuda(), c.lens.cuda(), c.scale)
    for phase in (kvp.KVP_PHASE_PARTIAL, kvp.KVP_PHASE_REDUCE | kvp.KVP_DECODE_MERGE_RUNS):
        kvp.kvp_attention_decode_int4(*args, workspace=ws, partition_blocks=16, phases=phase)
    torch.cuda.synchronize()
    assert torch.equal(out, whole)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,kv,B", [(128, 16, 1, 9), (64, 8, 8, 40), (128, 32, 32, 3),
                                       (64, 921, 307, 2)])
def test_decode_int4_balanced_pieces(dtype, D, Hq, kv, B):
    """Ragged contexts whose pieces cut some of them once, some often and some
    not at all, with empty ones between; more kv heads than pieces."""
    lens = [(700 * (i % 3) + 37 * i * i) % 1500 for i in range(B)]
    lens[0], lens[-1] = 1999, 1
    if B > 4:
        lens[2] = lens[3] = 0
        lens[4] = 16
    c = Case(lens, Hq, kv, D, dtype, seed=B, max_blocks=126)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(0, status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    c.check(out)
    assert torch.equal(out, c.run(0))


@pytest.mark.parametrize("lens", [[1040], [8 * 16], [8 * 16 + 1, 7], [129, 0, 2000, 0],
                                  [16] * 200, [1] * 500, [40] * 130 + [3000] + [40] * 7])
def test_decode_int4_balanced_edges(lens):
    """Pieces that end with a context, one-block contexts, more requests than
    threads of a CTA, one long context among short ones."""
    c = Case(lens, 2, 1, 128, torch.float16, seed=len(lens), max_blocks=190)
    c.check(c.run())


def test_decode_int4_workspace_is_all_that_is_written():
    """The balanced decode writes its workspace only; what lies behind stays."""
    c = Case([3000, 10, 500], 16, 2, 128, torch.bfloat16, seed=3)
    n = c.workspace().numel()
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((5,) + c.q.shape[1:], 9.0, dtype=c.q.dtype, device="cuda")
    kvp.kvp_attention_decode_int4(out[1:4], c.q.cuda(), *c.pools, c.tables.cuda(), c.lens.cuda(),
                                  c.scale, workspace=ws[:n])
    c.check(out[1:4])
    assert (ws[n:] == 0x5A).all() and (out[0] == 9).all() and (out[4] == 9).all()


@pytest.mark.parametrize("pb,max_blocks", [(0, 7), (2, 7), (0, 90)])
def test_decode_int4_bad_table_or_length_zeroes_the_rows(pb, max_blocks):
    c = Case([100, 40, 70], 8, 2, 64, torch.float16, seed=8, max_blocks=max_blocks)
    good = c.run(pb)
    for b, entry, value, length in ((0, 6, 10 ** 6, 100), (1, 0, -3, 40),
                                    (2, 0, 0, 16 * max_blocks + 1), (0, 0, 0, -1)):
        was = c.tables[b, entry].clone(), c.lens[b].clone()
        c.lens[b] = length
        if length == int(was[1]):
            c.tables[b, entry] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = c.run(pb, status)
        assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
        assert torch.count_nonzero(out[b]) == 0
        others = [i for i in range(3) if i != b]
        assert torch.equal(out[others], good[others])
        c.tables[b, entry], c.lens[b] = was


def test_decode_int4_blocks_past_4_gib():
    """Codes of the pool's last blocks lie past 2^32 bytes."""
    D, kv, NB, dtype = 128, 128, 36000, torch.float16
    assert NB * kv * 16 * D // 2 > 2 ** 32
    small = Case([200], kv, kv, D, dtype, seed=17, spare=0)
    nb = small.kc.shape[0]
    kc = torch.empty((NB, kv, 16, D // 2), dtype=torch.uint8, device="cuda")
    ks = torch.empty((NB, kv, 16, D // 64, 2), dtype=dtype, device="cuda")
    vc, vs = torch.empty_like(kc), torch.empty_like(ks)
    slots = (torch.arange(200) + (NB - 13) * 16).to(torch.int32).cuda()
    pos = torch.arange(200)
    blk = small.tables[0].long()[pos // 16]
    for big, src in zip((kc, vc, ks, vs), small.pools):
        big[-13:] = 0
        big[slots.long() // 16, :, slots.long() % 16] = src[blk.cuda(), :, (pos % 16).cuda()]
    assert nb == 13
    out = torch.empty(small.q.shape, dtype=dtype, device="cuda")
    tables = (torch.arange(13, dtype=torch.int32) + NB - 13)[None].cuda()
    kvp.kvp_attention_decode_int4(out, small.q.cuda(), kc, vc, ks, vs, tables, small.lens.cuda(),
                                  small.scale, workspace=small.workspace())
    assert torch.equal(out, small.run())
    # the append and the read-back reach them as well
    x = randn((200, kv, D), dtype, 3).cuda()
    kvp.kvp_append_int4(x, x, kc, vc, ks, vs, slots)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    kvp.kvp_read_int4(ko, vo, kc, vc, ks, vs, slots)
    c, p = plain64.quantise4(x.cpu())
    assert torch.equal(ko.cpu(), plain64.values4(plain64.pack4(c), p, torch.float32).to(dtype))
    assert torch.equal(ko, vo)


def test_decode_int4_in_two_captured_graphs():
    """Two captured decodes, each with its own workspace, replayed together on two
    streams, give what eager calls give."""
    cases = [Case([3000, 50], 8, 1, 128, torch.bfloat16, seed=s) for s in (41, 42)]
    want = [c.run(16) for c in cases]
    graphs = []
    for c in cases:
        out, q, t, n, ws = (torch.zeros_like(want[0]), c.q.cuda(), c.tables.cuda(), c.lens.cuda(),
                            c.workspace(16))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvp.kvp_attention_decode_int4(out, q, *c.pools, t, n, c.scale, workspace=ws,
                                          partition_blocks=16)
        graphs.append((g, out, (q, t, n, ws)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (g, out, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    for (_, out, _), w in zip(graphs, want):
        assert torch.equal(out, w)


def test_decode_int4_balanced_in_two_captured_graphs():
    """The same for the automatic split, whose pieces leave notes for the merge."""
    cases = [Case([3000, 50, 0, 1777], 8, 1, 128, torch.float16, seed=s, max_blocks=200)
             for s in (43, 44)]
    want = [c.run() for c in cases]
    graphs = []
    for c in cases:
        out, q, t, n, ws = (torch.zeros_like(want[0]), c.q.cuda(), c.tables.cuda(), c.lens.cuda(),
                            c.workspace())
        assert ws is not None
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvp.kvp_attention_decode_int4(out, q, *c.pools, t, n, c.scale, workspace=ws)
        graphs.append((g, out, (q, t, n, ws)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (g, out, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    for (_, out, _), w in zip(graphs, want):
        assert torch.equal(out, w)


@pytest.mark.parametrize("given", [False, True])
def test_int4_entry_points_use_the_stream(given):
    """On a side stream behind a long wait, current or passed as `stream`: inputs
    that arrive on that stream are seen."""
    T, kv, D, NB = 300, 2, 128, 30
    x = randn((T, kv, D), torch.float16, 1).cuda()
    slots = torch.randperm(NB * 16, generator=gen(2))[:T].to(torch.int32).cuda()
    pairs = torch.tensor([[0, NB], [3, NB + 1]], dtype=torch.int32, device="cuda")
    tables = torch.arange(NB, dtype=torch.int32, device="cuda")[None]
    lens = torch.full((1,), NB * 16, dtype=torch.int32, device="cuda")
    q = randn((1, 4, D), torch.float16, 3).cuda()

    def run(late, side):
        kc, vc, ks, vs = (t.cuda() for t in empty_pools(NB + 2, kv, D, torch.float16))
        for t in (kc, vc, ks, vs):
            t.zero_()
        key, ko, vo = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
        out = torch.zeros_like(q)
        kw = dict(stream=side) if given and late else {}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            if late:
                torch.cuda._sleep(20_000_000)
            key.copy_(x)
            if kw:
                with torch.cuda.stream(torch.cuda.default_stream()):
                    calls(key, kc, vc, ks, vs, ko, vo, out, kw)
            else:
                calls(key, kc, vc, ks, vs, ko, vo, out, kw)
        torch.cuda.synchronize()
        return kc, vc, ks, vs, ko, vo, out

    def calls(key, kc, vc, ks, vs, ko, vo, out, kw):
        kvp.kvp_append_int4(key, key, kc, vc, ks, vs, slots, **kw)
        kvp.kvp_copy_blocks_int4(kc, vc, ks, vs, pairs, **kw)
        kvp.kvp_read_int4(ko, vo, kc, vc, ks, vs, slots, **kw)
        kvp.kvp_attention_decode_int4(out, q, kc, vc, ks, vs, tables, lens, 0.1, **kw)

    want = run(False, torch.cuda.default_stream())
    assert want[-1].abs().max() > 0
    for a, b in zip(run(True, torch.cuda.Stream()), want):
        assert torch.equal(bits(a) if a.is_floating_point() else a,
                           bits(b) if b.is_floating_point() else b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_int4_infinities_stay_in_their_rows(dtype):
    T, kv, D, NB = 70, 3, 128, 6
    x, y = randn((T, kv, D), dtype, 5), randn((T, kv, D), dtype, 6)
    for i, v in enumerate((float("inf"), -float("inf"), float("nan"))):
        x[7 * i, i, 3 + 40 * i] = v
        y[7 * i + 1, i, 90 - 40 * i] = v
    kc, vc, ks, vs = (t.cuda() for t in empty_pools(NB, kv, D, dtype))
    slots = torch.arange(T, dtype=torch.int32)
    kvp.kvp_append_int4(x.cuda(), y.cuda(), kc, vc, ks, vs, slots.cuda())
    for rows, codes, pairs in ((x, kc, ks), (y, vc, vs)):
        c, s = plain64.quantise4(rows.nan_to_num(0, 0, 0))
        fine = rows.isfinite().all(-1)
        codes, pairs = codes.cpu(), pairs.cpu()
        assert torch.equal(codes[slots.long() // 16, :, slots.long() % 16][fine],
                           plain64.pack4(c)[fine])
        assert torch.equal(bits(pairs[slots.long() // 16, :, slots.long() % 16])[fine],
                           bits(s)[fine])


def test_decode_int4_balanced_runs_longer_than_the_staged_table():
    """So many query heads that one piece is left: its runs span several slices of
    their block tables."""
    c = Case([8300, 0, 9000], 8 * 229, 1, 128, torch.float16, seed=51, max_blocks=600)
    c.check(c.run())
    c.tables[2, 540] = 10 ** 6  # in the second slice
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(0, status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    assert torch.count_nonzero(out[2]) == 0 and torch.count_nonzero(out[0]) > 0


@pytest.mark.parametrize("Hq,kv,lens", [(8, 1, [9011, 3000, 1, 0, 6345]), (8, 8, [2500, 17, 2499]),
                                        (32, 16, [1100, 1099, 1088, 1])])
def test_decode_int4_contexts_cut_by_themselves(Hq, kv, lens):
    """Few blocks for the GPU: every context is cut alone, into runs of one size."""
    c = Case(lens, Hq, kv, 64, torch.bfloat16, seed=61, max_blocks=600)
    out = c.run()
    c.check(out)
    for i in range(len(lens)):  # a failed context leaves the others' bits
        if lens[i] < 1000:
            continue
        keep = c.tables[i, lens[i] // 16 - 1].clone()
        c.tables[i, lens[i] // 16 - 1] = -5
        bad = c.run()
        c.tables[i, lens[i] // 16 - 1] = keep
        assert torch.count_nonzero(bad[i]) == 0
        others = [j for j in range(len(lens)) if j != i]
        assert torch.equal(bad[others], out[others])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,kv,B,most,pb", [(64, 32, 20, 500, 0), (8, 1, 650, 40, 0),
                                             (33, 11, 60, 200, 5), (40, 1, 130, 17, 1)])
def test_decode_int4_many_short_runs(dtype, D, Hq, kv, B, most, pb):
    """More runs than CTAs of four warps fit the GPU: a warp for each."""
    lens = [1 + (i * i * 7 + 3 * i) % most for i in range(B)]
    lens[1], lens[B // 2], lens[-1] = 0, most, 16
    c = Case(lens, Hq, kv, D, dtype, seed=71)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(pb, status)
    assert kvp.kvp_read_status(status) == kvp.KVP_OK
    c.check(out)
    assert torch.count_nonzero(out[1]) == 0
    assert torch.equal(out, c.run(pb))
    c.tables[B // 2, 0] = c.kc.shape[0]
    c.lens[5] = 16 * c.tables.shape[1] + 1
    bad = c.run(pb, status)
    assert kvp.kvp_read_status(status) == kvp.KVP_ERR_BAD_BLOCK
    assert torch.count_nonzero(bad[B // 2]) == 0 and torch.count_nonzero(bad[5]) == 0
    rest = [i for i in range(B) if i not in (5, B // 2)]
    assert torch.equal(bad[rest], out[rest])
