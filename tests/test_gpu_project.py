"""Norms, E4M3 quantisers and the block-scaled product on the GPU."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import project64 as ref
from test_gpu_int4 import DTYPES, bits, randn

pytestmark = pytest.mark.gpu

F8, U8, F32 = torch.float8_e4m3fn, torch.uint8, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def gpu(*shape, dtype, fill=0):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


def weight(D, dtype, seed):
    return (1 + 0.3 * randn((D,), torch.float32, seed)).to(dtype)


# ------------------------------------------------------------------ norms
DIMS = [8, 24, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 5000, 8192,
        8200, 16384, 16392, 32768]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", DIMS)
def test_norm(D, dtype):
    T = 5 if D > 4096 else 37
    x, r, w = randn((T, D), dtype, 1), 3 * randn((T, D), dtype, 2), weight(D, dtype, 3)
    x[3] = 0
    r[3] = 0
    if T > 5:
        x[4] *= 1000.0 if dtype == torch.float16 else 1e15
    for res in (None, r):
        h = ref.total(x, res)
        want = ref.norm(h, w, 1e-5)
        out, total = gpu(T + 1, D, dtype=dtype, fill=7), gpu(T + 1, D, dtype=dtype, fill=7)
        kw = {} if res is None else dict(residual=res.cuda(), residual_out=total[:T])
        kvp.kvp_rms_norm(out[:T], x.cuda(), w.cuda(), 1e-5, **kw)
        assert ((out[:T].cpu().double() - want).abs() <= ref.norm_bound(want, dtype)).all()
        assert (out[T] == 7).all() and (total[T] == 7).all()
        assert res is None or torch.equal(bits(total[:T].cpu()), bits(h))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,D", [(1, 1, 64), (3, 5, 64), (33, 7, 128), (130, 64, 128), (9, 3, 192),
                                   (2, 12, 2048), (1, 8, 64), (17, 2, 72)])
def test_norm_of_heads(T, H, D, dtype):
    """Heads that are a slice of a projection's output, normed in place and elsewhere."""
    qkv, w = randn((T, H + 3, D), dtype, 4).cuda(), weight(D, dtype, 5).cuda()
    before = qkv.clone()
    x = qkv[:, 2:2 + H]
    want = ref.norm(x.cpu(), w.cpu(), 1e-6)
    out = gpu(T, H, D, dtype=dtype)
    kvp.kvp_rms_norm(out, x, w, 1e-6)
    assert ((out.cpu().double() - want).abs() <= ref.norm_bound(want, dtype)).all()
    kvp.kvp_rms_norm(x, x, w, 1e-6)
    assert torch.equal(bits(x), bits(out))
    for rest in (slice(0, 2), slice(2 + H, None)):
        assert torch.equal(bits(qkv[:, rest]), bits(before[:, rest]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_in_place_and_strided(dtype):
    T, D = 19, 1040
    x, r, w = (randn((T, D), dtype, i).cuda() for i in (1, 2, 3))
    out, total = gpu(T, D, dtype=dtype), gpu(T, D, dtype=dtype)
    kvp.kvp_rms_norm(out, x, w[0], 1e-5, residual=r, residual_out=total)
    wide = gpu(T, 3 * D + 8, dtype=dtype, fill=3)
    a, b = wide[:, 8:8 + D], wide[:, 16 + D:16 + 2 * D]
    a.copy_(x), b.copy_(r)
    before = wide.clone()
    kvp.kvp_rms_norm(a, a, w[0], 1e-5, residual=b, residual_out=b)
    assert torch.equal(bits(a), bits(out)) and torch.equal(bits(b), bits(total))
    a.copy_(x), b.copy_(r)
    assert torch.equal(bits(wide), bits(before))     # (nothing beside them)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_numbers_that_are_none(dtype):
    """A row with an infinity or a NaN spoils itself alone; eps carries a row of zeros."""
    x, w = randn((6, 256), dtype, 1).cuda(), weight(256, dtype, 2).cuda()
    clean = gpu(6, 256, dtype=dtype)
    kvp.kvp_rms_norm(clean, x, w, 1e-5)
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    out = gpu(6, 256, dtype=dtype)
    kvp.kvp_rms_norm(out, x, w, 1e-5)
    assert out[1].isnan().all() and out[3, 200].isnan()
    for i in (0, 2, 4, 5):
        assert torch.equal(bits(out[i]), bits(clean[i]))
    codes, scales = gpu(6, 256, dtype=U8), gpu(6, 2, dtype=F32)
    kvp.kvp_rms_norm_fp8(codes, scales, x, w, 1e-5)
    good, gs = gpu(6, 256, dtype=U8), gpu(6, 2, dtype=F32)
    x[1, 7], x[3, 200] = 0, 0
    kvp.kvp_rms_norm_fp8(good, gs, x, w, 1e-5)
    assert codes[1].view(F8).float().isnan().all()
    for i in (0, 2, 4, 5):
        assert torch.equal(codes[i], good[i]) and torch.equal(scales[i], gs[i])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [16, 48, 64, 128, 144, 256, 272, 512, 1024, 1040, 2064, 4096, 7168, 8192,
                               12304, 32768])
def test_norm_in_codes(D, dtype):
    T = 5 if D > 4096 else 21
    x, r, w = randn((T, D), dtype, 1), 3 * randn((T, D), dtype, 2), weight(D, dtype, 3)
    x[2], r[2] = 0, 0
    x[:, : D // 2] *= 50
    for res in (None, r):
        h = ref.total(x, res)
        want = ref.norm(h, w, 1e-5)
        codes, scales = gpu(T + 1, D, dtype=U8, fill=9), gpu(T + 1, ref.groups(D), dtype=F32, fill=9)
        total = gpu(T, D, dtype=dtype)
        kw = {} if res is None else dict(residual=res.cuda(), residual_out=total)
        kvp.kvp_rms_norm_fp8(codes[:T], scales[:T], x.cuda(), w.cuda(), 1e-5, **kw)
        assert (codes[T] == 9).all() and (scales[T] == 9).all()
        assert res is None or torch.equal(bits(total.cpu()), bits(h))
        c, s = codes[:T].cpu(), scales[:T].cpu()
        assert ((ref.values(c, s) - want).abs() <= ref.codes_bound(want, s)).all()
        # the scale is the largest magnitude's
        pad = torch.zeros(T, ref.groups(D) * 128, dtype=torch.float64)
        pad[:, :D] = want.abs()
        most = pad.view(T, -1, 128).amax(-1) / 448
        most[most == 0] = 1
        assert ((s.double() - most).abs() <= most * (2 * ref.NORM)).all()


# ------------------------------------------------------------------ quantisers
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("R,D", [(1, 16), (1, 128), (7, 144), (65, 1040), (128, 256), (129, 272),
                                 (300, 4096), (1000, 64)])
def test_quantise(R, D, block, dtype):
    """Bit-exact with the definition; strided rows; rows behind are left alone."""
    x = randn((R, D), dtype, 1) * torch.logspace(-3, 3, D).to(dtype)
    x[R // 2, : min(D, 130)] = 0
    want, ws = ref.quantise(x, block)
    wide = gpu(R, D + 24, dtype=dtype, fill=9)
    wide[:, 8:8 + D] = x.cuda()
    codes = gpu(R + 1, D + 32, dtype=U8, fill=9)
    scales = gpu(ws.shape[0] + 1, ws.shape[1], dtype=F32, fill=9)
    kvp.kvp_quantise_fp8(codes[:R, 16:16 + D], scales[:-1], wide[:, 8:8 + D], block_rows=block)
    assert torch.equal(codes[:R, 16:16 + D].cpu(), want)
    assert torch.equal(scales[:-1].cpu(), ws)
    assert (codes[R] == 9).all() and (codes[:, :16] == 9).all() and (codes[:, 16 + D:] == 9).all()
    assert (scales[-1] == 9).all()


@pytest.mark.parametrize("block", [1, 128])
def test_quantise_sizes_and_ties(block):
    """Every 16-bit magnitude, the smallest and largest among them, ties of the codes'
    steps, NaN and infinities."""
    for dtype in DTYPES:
        every = torch.arange(2 ** 15, dtype=torch.int32).to(torch.int16).view(dtype)
        x = every[every.isfinite()]
        x = x[: len(x) // 128 * 128].view(-1, 128).clone()
        x[:, ::3] *= -1
        want, ws = ref.quantise(x, block)
        codes, scales = gpu(*x.shape, dtype=U8), gpu(*ws.shape, dtype=F32)
        kvp.kvp_quantise_fp8(codes, scales, x.cuda(), block_rows=block)
        assert torch.equal(codes.cpu(), want) and torch.equal(scales.cpu(), ws)
    # ties: multiples of half a step of a group whose largest is 448 * 2^k
    x = torch.arange(-448, 448, 7, dtype=torch.float32).to(torch.bfloat16).view(1, 128)
    x = torch.cat([x, x.flip(1)], 0) / 16
    x[:, 0] = 28.0
    want, ws = ref.quantise(x, block)
    codes, scales = gpu(2, 128, dtype=U8), gpu(*ws.shape, dtype=F32)
    kvp.kvp_quantise_fp8(codes, scales, x.cuda(), block_rows=block)
    assert torch.equal(codes.cpu(), want) and torch.equal(scales.cpu(), ws)
    x = randn((256, 256), torch.float16, 5)
    x[3, 5], x[200, 130] = float("nan"), float("-inf")
    codes, scales = gpu(256, 256, dtype=U8), gpu(256 // block, 2, dtype=F32)
    kvp.kvp_quantise_fp8(codes, scales, x.cuda(), block_rows=block)
    v = ref.values(codes.cpu(), scales.cpu(), block)
    assert v[3, 5].isnan() and v[200, 130].isnan() and scales[200 // block, 1].isinf()
    clean = x.clone()
    clean[3, 5] = clean[200, 130] = 0
    want, ws = ref.quantise(clean, block)
    same = torch.ones_like(x, dtype=torch.bool)
    same[3, 5] = False
    first = 200 // block * block
    same[first:first + block, 128:] = False
    assert torch.equal(codes.cpu()[same], want[same])


# ------------------------------------------------------------------ product
def operands(M, N, K, seed, integers=False):
    """Codes and scales; `integers`: whole codes to 8 and scales of 1/2, 1 and 2, every
    sum of which is exact in float32."""
    g = torch.Generator().manual_seed(seed)
    G, GN = ref.groups(K), ref.groups(N)
    if integers:
        a, b = (torch.randint(-8, 9, (n, K), generator=g).float().to(F8) for n in (M, N))
        sa, sb = (2.0 ** torch.randint(-1, 2, (n, G), generator=g) for n in (M, GN))
    else:
        a, b = ((60 * torch.randn((n, K), generator=g)).clamp(-448, 448).to(F8) for n in (M, N))
        sa, sb = (torch.exp(torch.randn((n, G), generator=g)) / 448 for n in (M, GN))
    return a.view(U8), sa.float(), b.view(U8), sb.float()


SHAPES = [(1, 768, 512), (1, 1, 16), (2, 100, 48), (7, 129, 128), (16, 128, 144), (17, 256, 272),
          (32, 1000, 1024), (33, 64, 4096), (48, 4096, 512), (63, 130, 1040), (64, 10240, 1024),
          (65, 257, 2048), (100, 333, 656), (127, 128, 128), (128, 512, 4096), (129, 1281, 384),
          (200, 77, 8192), (256, 256, 256), (257, 640, 1152), (517, 2048, 1024), (1000, 1, 512),
          (1024, 1024, 16), (2049, 1100, 640), (260, 9800, 400), (2500, 2000, 272),
          (5000, 1030, 144), (2305, 2304, 4224), (513, 13000, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_whole_numbers(M, N, K):
    """Exact in float32, and rounded once in 16 bits: every element has its place."""
    a, sa, b, sb = operands(M, N, K, M + N, integers=True)
    want, _ = ref.matmul(a, sa, b, sb)
    args = [x.cuda() for x in (a, sa, b, sb)]
    for dtype in (F32, torch.bfloat16, torch.float16):
        if dtype == torch.float16 and want.abs().max() > 60000:
            continue
        out = gpu(M + 1, N + 8, dtype=dtype, fill=9)
        kvp.kvp_matmul_fp8(out[:M, 3:3 + N], *args)
        assert torch.equal(bits(out[:M, 3:3 + N].cpu()), bits(want.to(dtype)))
        assert (out[M] == 9).all() and (out[:, :3] == 9).all() and (out[:, 3 + N:] == 9).all()


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[0] * s[1] * s[2] < 10 ** 9])
def test_product(M, N, K, dtype):
    a, sa, b, sb = operands(M, N, K, 7 * M + N)
    want, size = ref.matmul(a, sa, b, sb)
    out = gpu(M, N, dtype=dtype)
    kvp.kvp_matmul_fp8(out, *(x.cuda() for x in (a, sa, b, sb)))
    assert ((out.cpu().double() - want).abs() <= ref.matmul_bound(size, K, want, dtype)).all()


@pytest.mark.parametrize("M", [3, 40, 130, 700])
def test_product_of_strided_operands(M):
    N, K = 200, 400
    a, sa, b, sb = operands(M, N, K, M)
    want = gpu(M, N, dtype=F32)
    kvp.kvp_matmul_fp8(want, a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    wide_a, wide_b = gpu(M, K + 48, dtype=U8, fill=0x7f), gpu(N, 2 * K, dtype=U8, fill=0x7f)
    wide_a[:, 16:16 + K], wide_b[:, K:] = a.cuda(), b.cuda()
    wide = gpu(M, 3 * N + 1, dtype=F32, fill=9)
    kvp.kvp_matmul_fp8(wide[:, N:2 * N], wide_a[:, 16:16 + K].view(F8), sa.cuda(), wide_b[:, K:],
                       sb.cuda())
    assert torch.equal(bits(wide[:, N:2 * N]), bits(want))
    assert (wide[:, :N] == 9).all() and (wide[:, 2 * N:] == 9).all()


@pytest.mark.parametrize("M", [1, 5, 64, 130, 600])
def test_nan_codes_stay_in_their_row_and_column(M):
    N, K = 300, 512
    a, sa, b, sb = operands(M, N, K, 11)
    clean, out = gpu(M, N, dtype=F32), gpu(M, N, dtype=F32)
    kvp.kvp_matmul_fp8(clean, *(x.cuda() for x in (a, sa, b, sb)))
    a[M // 2, 300], b[131, 7] = 0x7f, 0xff
    kvp.kvp_matmul_fp8(out, *(x.cuda() for x in (a, sa, b, sb)))
    assert out[M // 2].isnan().all() and out[:, 131].isnan().all()
    rest = torch.ones(M, N, dtype=torch.bool)
    rest[M // 2], rest[:, 131] = False, False
    assert torch.equal(out.cpu()[rest], clean.cpu()[rest])


@pytest.mark.parametrize("M", [1, 64, 300])
def test_scales_of_very_different_size(M):
    """A group far below the others, and scales near the ends of what is allowed."""
    N, K = 256, 1024
    a, sa, b, sb = operands(M, N, K, 3)
    sa[:, 2] *= 2.0 ** 60
    sb[:, 5] *= 2.0 ** -40
    sa[:, 7], sb[:, 7] = 2.0 ** -100, 2.0 ** 100
    want, size = ref.matmul(a, sa, b, sb)
    out = gpu(M, N, dtype=F32)
    kvp.kvp_matmul_fp8(out, *(x.cuda() for x in (a, sa, b, sb)))
    assert ((out.cpu().double() - want).abs() <= ref.matmul_bound(size, K, want, F32)).all()


def test_empty_calls():
    z = gpu(0, 256, dtype=torch.float16)
    w = gpu(256, dtype=torch.float16)
    codes, scales = gpu(0, 256, dtype=U8), gpu(0, 2, dtype=F32)
    kvp.kvp_rms_norm(z, z, w, 1e-5)
    kvp.kvp_rms_norm_fp8(codes, scales, z, w, 1e-5)
    for block in (1, 128):
        kvp.kvp_quantise_fp8(codes, scales, z, block_rows=block)
    kvp.kvp_matmul_fp8(gpu(0, 128, dtype=F32), codes, scales, gpu(128, 256, dtype=U8),
                       gpu(1, 2, dtype=F32))
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements, and bytes, apart."""
    T, D, N, step = 3, 256, 136, 2 ** 31 + 64
    a, sa, b, sb = operands(T, N, D, 5)
    want = gpu(T, N, dtype=torch.bfloat16)
    kvp.kvp_matmul_fp8(want, a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    far = torch.empty(2 * step + D, dtype=torch.bfloat16, device="cuda")
    wide = far.as_strided((T, D), (step, 1))
    bytes_ = far.view(U8).as_strided((T, D), (step, 1))
    bytes_.copy_(a.cuda())
    out = gpu(T, N, dtype=torch.bfloat16)
    kvp.kvp_matmul_fp8(out, bytes_, sa.cuda(), b.cuda(), sb.cuda())
    assert torch.equal(bits(out), bits(want))
    kvp.kvp_matmul_fp8(wide[:, :N], a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    assert torch.equal(bits(wide[:, :N]), bits(want))
    x, w = randn((T, D), torch.bfloat16, 6).cuda(), weight(D, torch.bfloat16, 7).cuda()
    y = torch.empty_like(x)
    kvp.kvp_rms_norm(y, x, w, 1e-5)
    wide.copy_(x)
    kvp.kvp_rms_norm(wide, wide, w, 1e-5)
    assert torch.equal(bits(wide), bits(y))
    codes, scales = gpu(T, D, dtype=U8), gpu(T, 2, dtype=F32)
    kvp.kvp_quantise_fp8(codes, scales, y)
    kvp.kvp_quantise_fp8(bytes_, scales, y)
    assert torch.equal(bytes_.cpu(), codes.cpu())
    many = 2 ** 24 + 3                                  # rows x scales past 2^31 bytes
    x = torch.zeros((many, 128), dtype=torch.float16, device="cuda")
    x[-1, 5] = 7
    out = torch.empty_like(x)
    kvp.kvp_rms_norm(out, x, gpu(128, dtype=torch.float16, fill=1), 1e-6)
    assert out[-1, 5] > 11 and not out[:-1].any()


# ------------------------------------------------------------------ together
def layer(T, hidden, Hq, Hkv, D, dtype, seed):
    """What a layer's attention keeps: norms, quantised weights, pools."""
    f = dict(dtype=dtype, device="cuda")
    n_qkv = (Hq + 2 * Hkv) * D
    L = {"w1": weight(hidden, dtype, seed).cuda(), "w2": weight(hidden, dtype, seed + 1).cuda(),
         "wq": weight(D, dtype, seed + 2).cuda(), "wk": weight(D, dtype, seed + 3).cuda()}
    for name, n, k in (("qkv", n_qkv, hidden), ("o", hidden, Hq * D)):
        w = (randn((n, k), torch.float32, seed + n) * k ** -0.5).to(dtype).cuda()
        L[name], L[name + "_s"] = gpu(n, k, dtype=U8), gpu(ref.groups(n), ref.groups(k), dtype=F32)
        kvp.kvp_quantise_fp8(L[name], L[name + "_s"], w, block_rows=128)
    NB = -(-T // 16) + 2
    L["kc"], L["vc"] = torch.zeros((NB, Hkv, 16, D), **f), torch.zeros((NB, Hkv, 16, D), **f)
    L["ws"] = gpu(1 << 22, dtype=U8)
    return L


def attention_block(L, x, residual, cos_sin, positions, slots, tables, lens, Hq, Hkv, D, status=None):
    """norm -> projection -> head norms -> rotary append -> decode -> projection -> norm."""
    T, hidden = x.shape
    dt = x.dtype
    codes, scales = gpu(T, hidden, dtype=U8), gpu(T, ref.groups(hidden), dtype=F32)
    h = torch.empty_like(x)
    kvp.kvp_rms_norm_fp8(codes, scales, x, L["w1"], 1e-5, residual=residual, residual_out=h)
    qkv = torch.empty((T, Hq + 2 * Hkv, D), dtype=dt, device="cuda")
    kvp.kvp_matmul_fp8(qkv.view(T, -1), codes, scales, L["qkv"], L["qkv_s"], status=status)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kvp.kvp_rms_norm(q, q, L["wq"], 1e-6)
    kvp.kvp_rms_norm(k, k, L["wk"], 1e-6)
    q_out = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    kvp.kvp_rope_append(q_out, q, k, v, L["kc"], L["vc"], cos_sin, positions, slots, status=status)
    att = torch.empty_like(q_out)
    kvp.kvp_attention_decode(att, q_out, L["kc"], L["vc"], tables, lens, D ** -0.5,
                             workspace=L["ws"], status=status)
    c2, s2 = gpu(T, Hq * D, dtype=U8), gpu(T, ref.groups(Hq * D), dtype=F32)
    kvp.kvp_quantise_fp8(c2, s2, att.view(T, -1))
    o = torch.empty_like(x)
    kvp.kvp_matmul_fp8(o, c2, s2, L["o"], L["o_s"], status=status)
    y, h2 = torch.empty_like(x), torch.empty_like(x)
    kvp.kvp_rms_norm(y, o, L["w2"], 1e-5, residual=h, residual_out=h2)
    return {"codes": codes, "scales": scales, "h": h, "qkv": qkv, "q_out": q_out, "att": att, "c2": c2,
            "s2": s2, "o": o, "y": y, "h2": h2}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,hidden,Hq,Hkv,D", [(4, 512, 8, 2, 64), (33, 1040, 8, 8, 128),
                                               (150, 2048, 16, 4, 128)])
def test_a_layers_attention(T, hidden, Hq, Hkv, D, dtype):
    """Every step from the tensors that the step before left, one token per request."""
    import plain64
    L = layer(T, hidden, Hq, Hkv, D, dtype, 20)
    x, r = randn((T, hidden), dtype, 1), 2 * randn((T, hidden), dtype, 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    cs = plain64.angles(64, D).cuda()
    NB = L["kc"].shape[0]
    slots = (torch.arange(T) * 16 % (NB * 16) + torch.arange(T) * 16 // (NB * 16)).to(torch.int32)
    positions = torch.zeros(T, **i32)
    tables = (slots // 16).view(T, 1).cuda()
    lens = (slots % 16 + 1).cuda()
    got = attention_block(L, x.cuda(), r.cuda(), cs, positions, slots.cuda(), tables, lens, Hq, Hkv, D)
    g = {k: v.cpu() for k, v in got.items()}
    h = ref.total(x, r)
    assert torch.equal(bits(g["h"]), bits(h))
    want = ref.norm(h, L["w1"].cpu(), 1e-5)
    assert ((ref.values(g["codes"], g["scales"]) - want).abs()
            <= ref.codes_bound(want, g["scales"])).all()
    want, size = ref.matmul(g["codes"], g["scales"], L["qkv"].cpu(), L["qkv_s"].cpu())
    v = g["qkv"].view(T, -1)[:, (Hq + Hkv) * D:]     # (q and k are normed in place)
    bound = ref.matmul_bound(size, hidden, want, dtype)
    assert ((v.double() - want[:, -v.shape[1]:]).abs() <= bound[:, -v.shape[1]:]).all()
    for first, n, w in ((0, Hq, "wq"), (Hq, Hkv, "wk")):
        raw = want.view(T, -1, D)[:, first:first + n].to(dtype)   # one rounding either way
        y = ref.norm(raw, L[w].cpu(), 1e-6)
        rel = 2 * torch.finfo(dtype).eps
        close = (g["qkv"][:, first:first + n].double() - y).abs()
        assert (close <= rel * (y.abs() + y.abs().amax(-1, keepdim=True))).all()
    want, ws = ref.quantise(g["att"].view(T, -1))
    assert torch.equal(g["c2"], want) and torch.equal(g["s2"], ws)
    want, size = ref.matmul(g["c2"], g["s2"], L["o"].cpu(), L["o_s"].cpu())
    assert ((g["o"].double() - want).abs() <= ref.matmul_bound(size, Hq * D, want, dtype)).all()
    h2 = ref.total(g["o"], h)
    assert torch.equal(bits(g["h2"]), bits(h2))
    want = ref.norm(h2, L["w2"].cpu(), 1e-5)
    assert ((g["y"].double() - want).abs() <= ref.norm_bound(want, dtype)).all()


@pytest.mark.parametrize("T", [3, 80])
def test_captured_and_on_side_streams(T):
    """The block captured twice, replayed side by side on two streams, with inputs that
    change between replays; the same bits as an eager run."""
    import plain64
    hidden, Hq, Hkv, D, dtype = 512, 8, 2, 64, torch.bfloat16
    cs = plain64.angles(64, D).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    pos, slots = torch.zeros(T, **i32), torch.arange(T, **i32)
    tables, lens = (slots // 16).view(T, 1).contiguous(), slots % 16 + 1
    sides = []
    for i in range(2):
        L = layer(T, hidden, Hq, Hkv, D, dtype, 40 + i)
        x, r = randn((T, hidden), dtype, i).cuda(), randn((T, hidden), dtype, 9 + i).cuda()
        args = (L, x, r, cs, pos, slots, tables, lens, Hq, Hkv, D)
        attention_block(*args)
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = attention_block(*args)
        sides.append((args, stream, graph, out))
    for seed in (100, 200):
        for i, (args, *_) in enumerate(sides):
            args[1].copy_(randn((T, hidden), dtype, seed + i))
        torch.cuda.synchronize()
        for _, stream, graph, _ in sides:
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for args, _, _, out in sides:
            want = attention_block(*args)
            for name in want:
                assert torch.equal(bits(out[name]), bits(want[name])), name


@pytest.mark.parametrize("M,N,K", [(1, 768, 4096), (64, 2048, 4096), (130, 1000, 2048),
                                   (1500, 1536, 1024)])
def test_the_same_call_gives_the_same_bits(M, N, K):
    args = [x.cuda() for x in operands(M, N, K, 1)]
    outs = [gpu(M, N, dtype=F32) for _ in range(4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        kvp.kvp_matmul_fp8(o, *args, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(bits(o), bits(outs[0]))


def test_captured_products_beside_other_work():
    """Products cut over clusters, by pairs and in one piece, captured into two graphs that
    share their inputs, replayed on two streams beside an FP8 decode and a norm: the same
    bits as alone."""
    shapes = [(64, 2048, 4096), (1, 512, 2048), (128, 4096, 1024), (2600, 2048, 1024), (33, 8200, 256)]
    calls = [[t.cuda() for t in operands(*s, seed=s[0])] for s in shapes]
    want = [gpu(M, N, dtype=torch.bfloat16) for M, N, _ in shapes]
    for o, c in zip(want, calls):
        kvp.kvp_matmul_fp8(o, *c)
    B, Hkv, D, MB = 16, 2, 128, 64
    codes = torch.randint(0, 120, (2, B * MB, Hkv, 16, D), dtype=U8).cuda()
    pool_scales = torch.rand((2, B * MB, Hkv, 16)).cuda()
    tables = torch.arange(B * MB, dtype=torch.int32, device="cuda").view(B, MB)
    lens = torch.full((B,), 16 * MB, dtype=torch.int32, device="cuda")
    q = randn((B, 8, D), torch.bfloat16, 1).cuda()
    x, w = randn((500, 1024), torch.bfloat16, 2).cuda(), weight(1024, torch.bfloat16, 3).cuda()

    def decode(out, ws):
        kvp.kvp_attention_decode_fp8(out, q, *codes, *pool_scales, tables, lens, 0.05, workspace=ws,
                                     partition_blocks=16)

    nbytes = kvp.kvp_decode_workspace_bytes(B, 8, kvp.cache_desc(codes[0]), MB, 16, kv_fp8=True)
    ws = [gpu(nbytes, dtype=U8) for _ in range(2)]
    att, norm = torch.empty_like(q), torch.empty_like(x)
    decode(att, ws[0])
    kvp.kvp_rms_norm(norm, x, w, 1e-5)
    torch.cuda.synchronize()
    sides = []
    for side in range(2):
        outs = [gpu(M, N, dtype=torch.bfloat16) for M, N, _ in shapes]
        rest = torch.empty_like(q), torch.empty_like(x)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for i in range(10):
                j = (i * (side + 1) + side) % len(shapes)
                kvp.kvp_matmul_fp8(outs[j], *calls[j])
                decode(rest[0], ws[side])
                kvp.kvp_rms_norm(rest[1], x, w, 1e-5)
        sides.append((stream, graph, outs, rest))
    for _ in range(5):
        for stream, graph, *_ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, outs, rest in sides:
        for o, v in zip(outs, want):
            assert torch.equal(bits(o), bits(v))
        assert torch.equal(bits(rest[0]), bits(att)) and torch.equal(bits(rest[1]), bits(norm))


def test_tensors_of_another_place_are_refused():
    a, sa, b, sb = operands(2, 128, 128, 1)
    out = gpu(2, 128, dtype=F32)
    for i in range(4):
        args = [x.cuda() for x in (a, sa, b, sb)]
        args[i] = args[i].cpu()
        with pytest.raises(ValueError):
            kvp.kvp_matmul_fp8(out, *args)
    x = gpu(2, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        kvp.kvp_rms_norm(x, x, x[0].cpu(), 1e-5)
    with pytest.raises(ValueError):
        kvp.kvp_quantise_fp8(gpu(2, 128, dtype=U8), torch.zeros(2, 1), x)


def test_the_readmes_projections():
    """The README's lines, as they stand there."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md"), encoding="utf-8") as f:
        lines, = (b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "matmul_fp8" in b)
    T, hidden, Hq, Hkv, D, dt = 5, 512, 4, 2, 64, torch.bfloat16
    L = layer(T, hidden, Hq, Hkv, D, dt, 60)
    x, r = randn((T, hidden), dt, 1).cuda(), randn((T, hidden), dt, 2).cuda()
    out = randn((T, Hq, D), dt, 3).cuda()
    v = dict(kvp=kvp, T=T, Hq=Hq, Hkv=Hkv, x=x.clone(), residual=r.clone(), norm_weight=L["w1"],
             codes=gpu(T, hidden, dtype=U8), scales=gpu(T, 4, dtype=F32), qkv_codes=L["qkv"],
             qkv_scales=L["qkv_s"], qkv=gpu(T, Hq + 2 * Hkv, D, dtype=dt), q_weight=L["wq"],
             k_weight=L["wk"], out=out, out_codes=gpu(T, Hq * D, dtype=U8),
             out_scales=gpu(T, 2, dtype=F32), o_codes=L["o"], o_scales=L["o_s"])
    exec(lines, v)
    assert torch.equal(bits(v["residual"]), bits(ref.total(x.cpu(), r.cpu())))
    codes, scales = ref.quantise(out.cpu().view(T, -1))
    assert torch.equal(v["out_codes"].cpu(), codes) and torch.equal(v["out_scales"].cpu(), scales)
    want, size = ref.matmul(codes, scales, L["o"].cpu(), L["o_s"].cpu())
    assert ((v["x"].cpu().double() - want).abs()
            <= ref.matmul_bound(size, Hq * D, want, dt)).all()
    want, size = ref.matmul(v["codes"].cpu(), v["scales"].cpu(), L["qkv"].cpu(), L["qkv_s"].cpu())
    got = v["qkv"].cpu().view(T, -1).double()[:, (Hq + Hkv) * D:]
    assert ((got - want[:, -got.shape[1]:]).abs()
            <= ref.matmul_bound(size, hidden, want, dt)[:, -got.shape[1]:]).all()


# ------------------------------------------------------------------ the compiled way
def arguments(dtype):
    """Arguments of every entry point, in the order of the compiled functions."""
    T, D, N = 5, 272, 130
    x, r = randn((T, D), dtype, 1).cuda(), randn((T, D), dtype, 2).cuda()
    out, total, w = gpu(T, D, dtype=dtype), gpu(T, D, dtype=dtype), weight(D, dtype, 3).cuda()
    codes, scales = gpu(T, D, dtype=U8), gpu(T, 3, dtype=F32)
    a, sa, b, sb = (t.cuda() for t in operands(T, N, D, 4))
    status = gpu(1, dtype=torch.int32)
    return {"rms_norm": [out, x, w, 1e-5, r, total],
            "rms_norm_fp8": [codes, scales, x, w, 1e-5, r, total],
            "quantise_fp8": [codes, scales, x, 1],
            "matmul_fp8": [gpu(T, N, dtype=dtype), a, sa, b, sb, status]}


def by_python(name, args):
    """The same call by the public function on an explicit stream, which takes the way
    through Python."""
    kw = dict(stream=torch.cuda.current_stream())
    if name.startswith("rms"):
        kw.update(residual=args[-2], residual_out=args[-1])
        args = args[:-2]
    elif name == "quantise_fp8":
        kw.update(block_rows=args[-1])
        args = args[:-1]
    else:
        kw.update(status=args[-1])
        args = args[:-1]
    getattr(kvp, "kvp_" + name)(*args, **kw)


NAMES = ["rms_norm", "rms_norm_fp8", "quantise_fp8", "matmul_fp8"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", NAMES)
def test_both_ways_give_the_same(name, dtype):
    a, b = arguments(dtype)[name], arguments(dtype)[name]
    assert getattr(kvp._calls(), name)(*a) == kvp.KVP_OK
    by_python(name, b)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        if isinstance(x, torch.Tensor):
            assert torch.equal(bits(x), bits(y))
    # without what may be left out, and of other types
    if name.startswith("rms"):
        assert getattr(kvp._calls(), name)(*a[:-2], None, None) == kvp.KVP_OK
    if name == "rms_norm":
        heads = gpu(3, 7, 64, dtype=dtype)[:, 2:5]
        assert kvp._calls().rms_norm(heads, heads, gpu(64, dtype=dtype), 0.5, None,
                                     None) == kvp.KVP_OK
    if name == "matmul_fp8":
        for out in (a[0], gpu(5, 130, dtype=F32), gpu(5, 140, dtype=dtype)[:, 3:133]):
            assert kvp._calls().matmul_fp8(out, a[1].view(F8), a[2], a[3].view(F8), a[4],
                                           None) == kvp.KVP_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_what_is_not_in_order_is_left_alone(name):
    """Every tensor in turn of another type, on the CPU, one row short, with strided rows
    or something else altogether: not called, and nothing written."""
    call = getattr(kvp._calls(), name)
    good = arguments(torch.float16)[name]
    before = [x.clone() if isinstance(x, torch.Tensor) else x for x in good]
    for i, x in enumerate(good):
        if not isinstance(x, torch.Tensor):
            continue
        wide = torch.zeros((*x.shape[:-1], 2 * x.shape[-1]), dtype=x.dtype, device="cuda")
        bad = [x.double(), x.cpu(), "x", 3, wide[..., ::2], x[None]]
        if not (name == "matmul_fp8" and i == 5):
            bad += [x[:-1], None]
        if x.dim() > 1:
            bad.append(x.t().contiguous().t())
        for y in bad:
            if isinstance(y, torch.Tensor) and y.is_cuda and y.shape == x.shape and \
                    y.dtype == x.dtype and y.is_contiguous():
                continue
            if name == "matmul_fp8" and i == 5 and getattr(y, "dtype", None) == x.dtype and y.is_cuda:
                continue                     # (a status word of any shape)
            assert call(*good[:i], y, *good[i + 1:]) is None, (i, getattr(y, "shape", y))
    for i, x in enumerate(good):
        if isinstance(x, (int, float)):
            for y in ("1", None, 2.5 if isinstance(x, int) else 1, 2 ** 40, 64):
                assert call(*good[:i], y, *good[i + 1:]) is None
    torch.cuda.synchronize()
    for x, y in zip(good, before):
        if isinstance(x, torch.Tensor):
            assert torch.equal(bits(x), bits(y))
