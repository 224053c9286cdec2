"""The block-scaled product in every kind of cut that its plan makes: each shape is listed with
the tile and the split that it is there for, and the plan is asked whether it still takes them."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import project64 as ref
from test_gpu_int4 import bits

pytestmark = pytest.mark.gpu

F8, U8, F32 = torch.float8_e4m3fn, torch.uint8, torch.float32
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


# (tokens, splits): rows of a per tile (256: pairs) and CTAs that share a tile's k.
# Every cut that is made, with remainders of rows, columns and k.
CUTS = [((16, 1), 1, 130, 16), ((16, 2), 1, 7530, 1584), ((16, 3), 1, 69, 1744),
        ((16, 4), 1, 73, 2000), ((16, 5), 1, 65, 3808), ((16, 6), 1, 65, 5280),
        ((16, 7), 1, 74, 6160), ((16, 8), 1, 66, 8160), ((32, 1), 1769, 289, 16),
        ((32, 2), 1711, 138, 1936), ((32, 3), 1231, 134, 1424), ((32, 4), 1599, 66, 2336),
        ((32, 5), 779, 129, 3136), ((32, 6), 599, 131, 5136), ((32, 7), 595, 129, 6160),
        ((32, 8), 466, 129, 9120), ((64, 1), 38, 20322, 16), ((64, 2), 33, 13619, 5040),
        ((64, 3), 1588, 134, 2640), ((64, 4), 35, 4849, 5040), ((64, 5), 1674, 131, 5024),
        ((128, 1), 67, 13318, 16), ((128, 2), 66, 7687, 3008), ((128, 3), 2458, 134, 3120),
        ((128, 4), 1948, 129, 6928), ((128, 5), 1692, 131, 9264), ((128, 6), 1257, 131, 15888),
        ((256, 1), 75, 20746, 16)]
# Groups of one CTA beyond the spans of scales that are staged (16 groups each, two of them; by
# pairs 8, four of them): 17, 31, 33, 49, 64 and 65 of them.
SPANS = [((16, 1), 1, 11777, 2096), ((16, 1), 1, 16781, 3936), ((16, 1), 1, 13173, 4160),
         ((16, 1), 1, 12550, 6240), ((16, 1), 1, 17453, 8176), ((16, 1), 1, 17074, 8272),
         ((16, 8), 1, 65, 16752), ((16, 3), 1, 4826, 11744), ((16, 2), 1, 7297, 8320),
         ((16, 2), 1, 7255, 12304), ((16, 2), 1, 7914, 16384), ((16, 2), 1, 7765, 16528),
         ((32, 1), 2473, 129, 2080), ((32, 1), 17, 19811, 3872), ((32, 1), 20, 21149, 4176),
         ((32, 1), 17, 20595, 6224), ((32, 1), 17, 21991, 8128), ((32, 1), 17, 22897, 8320),
         ((32, 3), 17, 7654, 6272), ((32, 3), 17, 6123, 11904), ((32, 3), 17, 6173, 12368),
         ((32, 2), 17, 9938, 12320), ((32, 2), 20, 8155, 16288), ((32, 2), 17, 10742, 16416),
         ((64, 1), 35, 20039, 2176), ((64, 1), 36, 19523, 3888), ((64, 1), 35, 19686, 4160),
         ((64, 1), 35, 20533, 6176), ((64, 1), 33, 19805, 8192), ((64, 1), 34, 19743, 8320),
         ((64, 3), 1540, 131, 6288), ((64, 4), 34, 4773, 15664), ((64, 4), 1193, 129, 16752),
         ((64, 2), 34, 13118, 12304), ((64, 2), 33, 13562, 16272), ((64, 2), 34, 13046, 16608),
         ((128, 1), 129, 8038, 2064), ((128, 1), 132, 7850, 3856), ((128, 1), 66, 13341, 4192),
         ((128, 1), 67, 13314, 6224), ((128, 1), 69, 13834, 8192), ((128, 1), 66, 13441, 8320),
         ((128, 3), 2459, 130, 6176), ((128, 2), 68, 6449, 7936), ((128, 2), 65, 6577, 8352),
         ((128, 2), 67, 6455, 12336), ((128, 2), 75, 6501, 16304), ((128, 2), 66, 6490, 16624),
         ((256, 1), 137, 10499, 2144), ((256, 1), 132, 10575, 3872), ((256, 1), 138, 10389, 4160),
         ((256, 1), 140, 11673, 6256), ((256, 1), 137, 10090, 8144), ((256, 1), 132, 10818, 8208)]
# Sizes that a layer has.
LAYERS = [((16, 2), 1, 10240, 8192), ((32, 4), 64, 4096, 4096), ((64, 1), 33, 32000, 4096),
          ((64, 3), 64, 10240, 8192), ((128, 1), 128, 10240, 8192), ((128, 2), 256, 4096, 4096),
          ((256, 1), 517, 4096, 4096), ((256, 1), 1100, 10240, 2048)]
# One shape of each tile, in one CTA and in a cluster, for what does not need them all.
EACH = [((16, 1), 3, 11777, 2096), ((16, 3), 16, 4100, 2064), ((32, 1), 20, 21149, 4176),
        ((32, 3), 17, 7654, 6272), ((64, 1), 50, 19686, 1040), ((64, 4), 61, 4849, 5040),
        ((128, 1), 128, 13341, 1168), ((128, 2), 100, 7687, 3008), ((256, 1), 270, 10575, 1296)]


def name(s):
    return f"{s[0][0]}x{s[0][1]}-{s[1]}x{s[2]}x{s[3]}"


def sizes(shape):
    """The shape's sizes, once its plan is seen to be the one that it is listed for."""
    cut, M, N, K = shape
    assert kvp.kvp_matmul_fp8_plan(M, N, K) == cut
    return M, N, K


def operands(M, N, K, seed, integers=False):
    """As in test_gpu_project, made on the GPU.  `integers`: whole codes to 8, scales of 1/2, 1
    and 2 that change from group to group; every sum is exact in float32 (below 2^22, in steps
    of 1/4)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    G, GN = ref.groups(K), ref.groups(N)
    if integers:
        a, b = (torch.randint(-8, 9, (n, K), **kw).to(torch.float16).to(F8) for n in (M, N))
        sa, sb = (2.0 ** torch.randint(-1, 2, (n, G), **kw) for n in (M, GN))
    else:
        a, b = (torch.randn((n, K), dtype=torch.float16, **kw).mul_(60).to(F8) for n in (M, N))
        sa, sb = (torch.exp(torch.randn((n, G), **kw)) / 448 for n in (M, GN))
    return a.view(U8), sa.float(), b.view(U8), sb.float()


def outputs(M, N, dtype):
    """Places for a result: whole rows, rows 16-byte aligned inside others, and odd ones; and
    what lies beside them."""
    aligned, odd = -(-N // 16) * 16 + 32, (N | 1) + 8
    for shape, first in (((M + 1, N), 0), ((M + 1, aligned), 16), ((M + 1, odd), 3)):
        whole = torch.full(shape, 9.0, dtype=dtype, device="cuda")
        yield whole, whole[:M, first:first + N]


def untouched(whole, out):
    """(whole may be written through `out` alone)"""
    out.fill_(9)
    return bool((whole == 9).all())


@pytest.mark.parametrize("shape", CUTS + SPANS + LAYERS + EACH, ids=name)
def test_whole_numbers(shape):
    """Exact, and rounded once in 16 bits: every element has its place and its scales."""
    M, N, K = sizes(shape)
    args = operands(M, N, K, M + N + K, integers=True)
    want, _ = ref.matmul(*args)
    assert want.abs().max() < 60000
    for dtype in (F32, BF16, F16):
        for whole, out in outputs(M, N, dtype):
            kvp.kvp_matmul_fp8(out, *args)
            assert torch.equal(bits(out), bits(want.to(dtype))), (dtype, out.stride())
            assert untouched(whole, out)


@pytest.mark.parametrize("shape", CUTS + SPANS[::5] + LAYERS + EACH, ids=name)
def test_against_64_bits(shape):
    M, N, K = sizes(shape)
    args = operands(M, N, K, M + N + K)
    want, size = ref.matmul(*args)
    for dtype in (F32, BF16, F16):
        out = torch.empty((M, N), dtype=dtype, device="cuda")
        kvp.kvp_matmul_fp8(out, *args)
        assert ((out.double() - want).abs() <= ref.matmul_bound(size, K, want, dtype)).all()


@pytest.mark.parametrize("shape", EACH, ids=name)
def test_strided_operands(shape):
    M, N, K = sizes(shape)
    a, sa, b, sb = operands(M, N, K, 1)
    want, out = (torch.empty((M, N), dtype=F32, device="cuda") for _ in range(2))
    kvp.kvp_matmul_fp8(want, a, sa, b, sb)
    wide_a, wide_b = (torch.full((n, w), 0x7f, dtype=U8, device="cuda")
                      for n, w in ((M, K + 48), (N, 2 * K)))
    wide_a[:, 16:16 + K], wide_b[:, K:] = a, b
    kvp.kvp_matmul_fp8(out, wide_a[:, 16:16 + K].view(F8), sa, wide_b[:, K:], sb)
    assert torch.equal(bits(out), bits(want))


@pytest.mark.parametrize("shape", EACH, ids=name)
def test_nan_stays_in_its_row_and_column(shape):
    """Codes that are NaN, and scales that are none or infinite."""
    M, N, K = sizes(shape)
    a, sa, b, sb = operands(M, N, K, 11)
    clean, out = (torch.empty((M, N), dtype=F32, device="cuda") for _ in range(2))
    kvp.kvp_matmul_fp8(clean, a, sa, b, sb)
    a[M // 2, K - 3], b[131, 7], b[N - 1, K - 1] = 0x7f, 0xff, 0x7f
    sa[M - 1, -1], sb[3, 0] = float("nan"), float("inf")
    kvp.kvp_matmul_fp8(out, a, sa, b, sb)
    rows, cols = [M // 2, M - 1], [131, N - 1]
    assert out[rows].isnan().all() and out[:, cols].isnan().all()
    assert not out[:, 3 * 128:4 * 128].isfinite().any()
    rest = torch.ones((M, N), dtype=torch.bool, device="cuda")
    rest[rows], rest[:, cols], rest[:, 3 * 128:4 * 128] = False, False, False
    assert torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("shape", EACH, ids=name)
def test_scales_far_apart(shape):
    """Groups far above and below the others, and scales near the ends of what is allowed."""
    M, N, K = sizes(shape)
    a, sa, b, sb = operands(M, N, K, 3)
    sa[:, 2] *= 2.0 ** 60
    sb[:, 5] *= 2.0 ** -40
    sa[:, 7], sb[:, 7] = 2.0 ** -100, 2.0 ** 100
    sa[M // 2] *= 2.0 ** -50
    want, size = ref.matmul(a, sa, b, sb)
    out = torch.empty((M, N), dtype=F32, device="cuda")
    kvp.kvp_matmul_fp8(out, a, sa, b, sb)
    assert ((out.double() - want).abs() <= ref.matmul_bound(size, K, want, F32)).all()


@pytest.mark.parametrize("shape", [((32, 1), 20, 21149, 4176), ((64, 4), 61, 4849, 5040),
                                   ((128, 2), 100, 7687, 3008), ((256, 1), 270, 10575, 1296)], ids=name)
def test_offsets_past_32_bits(shape):
    """Results and codes whose last rows lie past 2^31 elements, and bytes."""
    M, N, K = sizes(shape)
    a, sa, b, sb = operands(M, N, K, 5)
    want = torch.empty((M, N), dtype=BF16, device="cuda")
    kvp.kvp_matmul_fp8(want, a, sa, b, sb)
    for n, x in ((M, a), (N, b)):
        step = (2 ** 31 // (n - 1) // 16 + 2) * 16
        far = torch.empty((n - 1) * step + K, dtype=U8, device="cuda").as_strided((n, K), (step, 1))
        far.copy_(x)
        out = torch.empty_like(want)
        kvp.kvp_matmul_fp8(out, far if x is a else a, sa, far if x is b else b, sb)
        assert torch.equal(bits(out), bits(want))
        del far
    for odd in (0, 1):      # (16-byte stores, and others)
        step = (2 ** 31 // (M - 1) // 8 + 2) * 8 + odd
        far = torch.empty((M - 1) * step + N, dtype=BF16, device="cuda").as_strided((M, N), (step, 1))
        kvp.kvp_matmul_fp8(far, a, sa, b, sb)
        assert torch.equal(bits(far), bits(want))
        del far


def test_more_rows_than_2_to_30():
    """Rows behind which twice their number does not fit 32 bits; results past 2^31."""
    M, N, K = 2 ** 30 + 300, 3, 16
    a = torch.zeros((M, K), dtype=U8, device="cuda")
    rows = torch.tensor([0, 1, 255, 256, 2 ** 29 + 7, 2 ** 30 - 1, 2 ** 30, M - 45, M - 1], device="cuda")
    few, _, b, sb = operands(len(rows), N, K, 2, integers=True)
    a[rows] = few
    sa = torch.full((M, 1), 2.0, device="cuda")
    out = torch.full((M, N), 9.0, dtype=BF16, device="cuda")
    kvp.kvp_matmul_fp8(out, a, sa, b, sb)
    want, _ = ref.matmul(few, sa[:len(rows)], b, sb)
    assert torch.equal(bits(out[rows]), bits(want.to(BF16)))
    out[rows] = 0
    assert not out.any()


def test_captured_cuts_on_two_streams():
    """Every tile, whole and shared, in two graphs that share their inputs and are replayed side
    by side: the same bits as alone."""
    calls = [operands(*sizes(s), seed=i) for i, s in enumerate(EACH)]
    want = [torch.empty(s[1:3], dtype=BF16, device="cuda") for s in EACH]
    for o, c in zip(want, calls):
        kvp.kvp_matmul_fp8(o, *c)
    torch.cuda.synchronize()
    sides = []
    for side in range(2):
        outs = [torch.zeros_like(o) for o in want]
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for i in range(2 * len(EACH)):
                j = (i * (side + 1) + side) % len(EACH)
                kvp.kvp_matmul_fp8(outs[j], *calls[j])
        sides.append((stream, graph, outs))
    for _ in range(5):
        for stream, graph, _ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, outs in sides:
        for o, v in zip(outs, want):
            assert torch.equal(bits(o), bits(v))


def test_a_status_word_keeps_its_first_error():
    """A product that goes well writes nothing; after a wait that gave up (the products' own is
    one of the self-test's, all of which have to) the word says so, whatever runs behind it."""
    clean, timeout = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    kvp.kvp_selftest_wait_timeout(timeout, 5_000_000)
    for i, s in enumerate(EACH):
        args = operands(*sizes(s), seed=i)
        out = torch.empty(s[1:3], dtype=BF16, device="cuda")
        kvp.kvp_matmul_fp8(out, *args, status=clean)
        kvp.kvp_matmul_fp8(out, *args, status=timeout)
    assert kvp.kvp_read_status(clean) == kvp.KVP_OK
    assert kvp.kvp_read_status(timeout) == kvp.KVP_ERR_TIMEOUT
