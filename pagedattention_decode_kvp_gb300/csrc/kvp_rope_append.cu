// kvp_rope_append.cu -- the write side of a layer's attention, fused:
//   * rope_append: rotate q and k by positions on one to four axes (time,
//     height, width, ...), write q out and scatter K (rotated) and V to their
//     slots of a 16-bit cache; rope_append_int4 quantises them on the way;
//   * append_int4: quantise K/V rows to 4-bit codes with one (scale, zero) pair
//     per 64 elements and scatter them;
//   * read_int4: the rows of given slots as the 16-bit values they stand for.
//
// Rotation of a row x with R = rotary_dim, pair i of R/2 on axis a(i):
//   y_i = x_i cos - x_j sin,  y_j = x_j cos + x_i sin,
// (i, j) = (i, i + R/2) or (2i, 2i + 1); cos and sin are float32 table entries
// of position positions[a(i), t].  Every product and sum is rounded to float32
// by itself (no fused multiply-add) and y once to the 16-bit type, so that the
// result does not depend on how a compiler contracts the expression.
//
// Quantisation of a group of 64 elements (float32, IEEE division):
//   z = min x,  s = RN16((max x - min x) / 15),
//   c = s > 0 ? min(15, rint((x - z) / s)) : 0,   value = s * c + z.
// z is an element, so it is exact in the 16-bit type; s carries half a step of
// that type, which moves the largest value by at most 15 * 2^-9 = 0.03 steps of
// the code (bf16), against the code's own half step.
//
// Bound by HBM for prompts and by latency for a step.  D / 16 lanes share a
// row; a lane holds two 16-byte chunks, chosen so that both elements of every
// split-half pair are its own, and uses its 8 (cos, sin) pairs for every head
// of the token it works on.  Measured, prompts of 33098 tokens, 32 kv heads of
// 128 (shares of the measured copy bandwidth): rotation with a 16-bit append 237
// us (0.98 to 1.02), 4-bit append 137 us (0.72), read-back 110 us (0.90);
// rotation with a 4-bit append, 8191 tokens of 64 + 8 heads, 56 us (0.79).  The
// 4-bit appends are held by the quantiser, 395 instructions for four K and four V
// rows, and by the wait for rows, of which none is on its way meanwhile: 44% of the
// warps are resident, the issue slots 66% full, and global memory is the first
// stall.  More CTAs per SM (with the 8 at 140 us: 139 with 9, 142 with 10, spilling)
// or the next rows' loads in registers (138 at 6 CTAs, 150 at 8, spilling) do not
// change that, nor does one check over all of a lane's elements (157: exact ties are
// common).  A step of 64 tokens takes 2.8 to 3.1 us.
#include <algorithm>

#include "kvp_device.cuh"
#include "kvp_serve.h"

namespace kvp {
namespace {

constexpr int kRowThreads = 128;

// Two 16-byte chunks of a row, as packed 16-bit pairs.
struct RowPair {
  uint4 a, b;
};

__device__ __forceinline__ RowPair load_pair(const uint16_t* row, int ca, int cb) {
  RowPair r;
  r.a = *reinterpret_cast<const uint4*>(row + ca * 8);
  r.b = *reinterpret_cast<const uint4*>(row + cb * 8);
  return r;
}

__device__ __forceinline__ void store_pair(uint16_t* row, int ca, int cb, const RowPair& r) {
  *reinterpret_cast<uint4*>(row + ca * 8) = r.a;
  *reinterpret_cast<uint4*>(row + cb * 8) = r.b;
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = dev::unpack2<kBf16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool kBf16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(dev::pack2<kBf16>(x[0], x[1]), dev::pack2<kBf16>(x[2], x[3]),
                    dev::pack2<kBf16>(x[4], x[5]), dev::pack2<kBf16>(x[6], x[7]));
}

__device__ __forceinline__ void rotate_pair(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  const float b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = a;
  y = b;
}

// Which chunks of a row lane c holds, and which of them are rotated.  Split
// halves: the rotated lanes hold chunks c and c + R/16, whose elements pair up;
// the other lanes share the unrotated rest.  Adjacent pairs lie within chunks.
struct LaneChunks {
  int a, b;
  bool rot_a, rot_b;
};

template <int D, bool kRope>
__device__ __forceinline__ LaneChunks lane_chunks(const RowParams& p, int c) {
  constexpr int L = D / 16;
  LaneChunks k;
  if (!kRope || p.interleaved) {
    k.a = c;
    k.b = c + L;
    k.rot_a = kRope && k.a * 8 < p.rotary_dim;
    k.rot_b = kRope && k.b * 8 < p.rotary_dim;
  } else {
    const int half = p.rotary_dim / 16;  // chunks of one half
    const bool rot = c < half;
    k.a = rot ? c : 2 * half + (c - half);
    k.b = rot ? c + half : 2 * half + (L - half) + (c - half);
    k.rot_a = k.rot_b = rot;
  }
  return k;
}

template <bool kBf16>
__device__ __forceinline__ void rotate(RowPair& r, const LaneChunks& k, bool interleaved,
                                       const float (&cs)[8], const float (&sn)[8]) {
  if (!k.rot_a && !k.rot_b) return;
  float x[8], y[8];
  unpack8<kBf16>(r.a, x);
  unpack8<kBf16>(r.b, y);
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k.rot_a) rotate_pair(x[2 * j], x[2 * j + 1], cs[j], sn[j]);
      if (k.rot_b) rotate_pair(y[2 * j], y[2 * j + 1], cs[4 + j], sn[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) rotate_pair(x[j], y[j], cs[j], sn[j]);
  }
  r.a = pack8<kBf16>(x);
  r.b = pack8<kBf16>(y);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (kBf16) {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r =
        __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (kBf16) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r =
        __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Codes of 8 elements (element e in bits 4e .. 4e + 3).  With d = x - z, the
// product d * (1/s) is taken with 1/s made 2^-21 smaller and 2^-21 larger; adding
// 1.5 * 2^23 rounds each to an integer held in the low mantissa bits.  The two
// bracket the IEEE quotient (1/s and the brackets' own roundings move them by
// less than 2^-22), so where they agree that integer is the quotient's; where
// they do not -- ties, nearly -- the quotient itself decides.  A negative s stands
// for -s with quotients for all elements (see store_rows_int4).
struct Bracket {
  float lo, hi;  // 1/s, less and more
};

__device__ __forceinline__ Bracket bracket(float inv) {
  return {inv * (1.f - 0x1p-21f), inv * (1.f + 0x1p-21f)};
}

// Nibbles of 8 words' low bytes.
__device__ __forceinline__ uint32_t pack_nibbles(const uint32_t (&k)[8]) {
  const uint32_t even = dev::prmt(dev::prmt(k[0], k[2], 0x0040u), dev::prmt(k[4], k[6], 0x0040u),
                                  0x5410u);
  const uint32_t odd = dev::prmt(dev::prmt(k[1], k[3], 0x0040u), dev::prmt(k[5], k[7], 0x0040u),
                                 0x5410u);
  return odd * 16u + even;
}

// Both 16-bit halves of w less z, each rounded once to float32.
template <bool kBf16>
__device__ __forceinline__ float2 sub2(uint32_t w, float z) {
  float2 d;
  if constexpr (kBf16)
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; sub.rn.f32.bf16 %0, l, %3; sub.rn.f32.bf16 %1, h, %3;}"
        : "=f"(d.x), "=f"(d.y) : "r"(w), "f"(z));
  else
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; sub.rn.f32.f16 %0, l, %3; sub.rn.f32.f16 %1, h, %3;}"
        : "=f"(d.x), "=f"(d.y) : "r"(w), "f"(z));
  return d;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t quantise8_u4(const uint4& raw, float s, float z, Bracket b) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const uint64_t magic2 = dev::f2pack(kMagic, kMagic);
  const uint64_t lo2 = dev::f2pack(b.lo, b.lo), hi2 = dev::f2pack(b.hi, b.hi);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const uint64_t minus2 = dev::f2pack(-1.f, -1.f);
  uint32_t k[8];
  uint64_t more2[4], sum2 = 0;  // n - m >= 0: 1 where the brackets do not agree
  float d[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 du = sub2<kBf16>(w[i], z);
    const uint64_t d2 = dev::f2pack(du.x, du.y);
    const float2 mu = dev::f2unpack(dev::ffma2(d2, lo2, magic2));
    more2[i] = dev::ffma2(dev::f2pack(mu.x, mu.y), minus2, dev::ffma2(d2, hi2, magic2));
    sum2 = dev::fadd2(sum2, more2[i]);
    d[2 * i] = du.x;
    d[2 * i + 1] = du.y;
    k[2 * i] = __float_as_uint(mu.x);
    k[2 * i + 1] = __float_as_uint(mu.y);
  }
  const float2 sum = dev::f2unpack(sum2);
  if (sum.x + sum.y > 0.f || s < 0.f) {
    const bool slow = s < 0.f;
    const float sa = fabsf(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 u = dev::f2unpack(more2[e / 2]);
      if ((e % 2 == 0 ? u.x : u.y) > 0.f || slow)
        k[e] = __float_as_uint(kMagic + fminf(rintf(__fdiv_rn(d[e], sa)), 15.f));
    }
  }
  return pack_nibbles(k);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t min8(const uint4& r) {
  return min2<kBf16>(min2<kBf16>(r.x, r.y), min2<kBf16>(r.z, r.w));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t max8(const uint4& r) {
  return max2<kBf16>(max2<kBf16>(r.x, r.y), max2<kBf16>(r.z, r.w));
}

// Smallest and largest of a row's groups over this lane's chunks: of group 0 in
// the low half, of group 1 in the high one.
template <bool kBf16, int D>
__device__ __forceinline__ void row_range(const RowPair& r, const LaneChunks& k, uint32_t& lo,
                                          uint32_t& hi) {
  uint32_t mna = min8<kBf16>(r.a), mnb = min8<kBf16>(r.b);
  uint32_t mxa = max8<kBf16>(r.a), mxb = max8<kBf16>(r.b);
  if constexpr (D == 64) {
    lo = min2<kBf16>(mna, mnb);
    hi = max2<kBf16>(mxa, mxb);
    lo = min2<kBf16>(lo, __byte_perm(lo, lo, 0x1032));
    hi = max2<kBf16>(hi, __byte_perm(hi, hi, 0x1032));
  } else {
    constexpr uint32_t kInf = (kBf16 ? 0x7f80u : 0x7c00u) * 0x10001u, kSign = 0x80008000u;
    mna = min2<kBf16>(mna, __byte_perm(mna, mna, 0x1032));
    mnb = min2<kBf16>(mnb, __byte_perm(mnb, mnb, 0x1032));
    mxa = max2<kBf16>(mxa, __byte_perm(mxa, mxa, 0x1032));
    mxb = max2<kBf16>(mxb, __byte_perm(mxb, mxb, 0x1032));
    const uint32_t in_a = (k.a * 8 < 64) ? 0x0000ffffu : 0xffff0000u;
    const uint32_t in_b = (k.b * 8 < 64) ? 0x0000ffffu : 0xffff0000u;
    lo = min2<kBf16>((mna & in_a) | (kInf & ~in_a), (mnb & in_b) | (kInf & ~in_b));
    hi = max2<kBf16>((mxa & in_a) | ((kInf | kSign) & ~in_a),
                     (mxb & in_b) | ((kInf | kSign) & ~in_b));
  }
}

// Quantise a K and a V row, shared by the D / 16 lanes whose `c` count from 0, and
// write codes and (scale, zero) pairs.  All lanes of the warp call it; `store`
// tells whether this lane's rows exist.  The rows have 2 D / 64 groups, and the
// divisions for a group -- the scale and its reciprocal -- are done by one lane
// each and passed round.
template <bool kBf16, int D>
__device__ __forceinline__ void store_rows_int4(const RowPair& x, const RowPair& y,
                                                const LaneChunks& k, int c, bool store,
                                                const RowParams& p, size_t srow) {
  constexpr int L = D / 16, kG = D / 64;
  uint32_t lo[2], hi[2];  // K, V
  row_range<kBf16, D>(x, k, lo[0], hi[0]);
  row_range<kBf16, D>(y, k, lo[1], hi[1]);
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[i] = min2<kBf16>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = max2<kBf16>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  }
  // lane c: group c % kG of K (c / kG even) or V
  const bool of_v = (c / kG) % 2 != 0, high = kG == 2 && c % 2 != 0;
  const uint32_t my_lo = of_v ? lo[1] : lo[0], my_hi = of_v ? hi[1] : hi[0];
  const float2 zz = dev::unpack2<kBf16>(my_lo), tt = dev::unpack2<kBf16>(my_hi);
  const float range = high ? __fsub_rn(tt.y, zz.y) : __fsub_rn(tt.x, zz.x);
  const uint32_t sp = dev::pack2<kBf16>(__fdiv_rn(range, 15.f), 0.f);
  const float s = dev::unpack2<kBf16>(sp).x;
  // Below the 16-bit type's normal range the scale's own rounding can push codes
  // past 15, and outside [2^-126, 2^126] the brackets do not hold: such groups
  // take the quotients (a negative scale is passed round).
  const bool fits = s >= (kBf16 ? 0x1p-126f : 0x1p-14f) && s <= 0x1p126f;
  const float inv = fits ? __fdiv_rn(1.f, s) : 0.f;
  const float signed_s = fits ? s : -s;
  if (store && c < 2 * kG) {
    const uint32_t pair = __byte_perm(sp, my_lo, high ? 0x7610 : 0x5410);
    (of_v ? p.v_sz : p.k_sz)[srow * kG + c % kG] = pair;
  }
  const int base = (threadIdx.x & 31) - c;
  const int ga = kG == 2 && k.a * 8 >= 64 ? 1 : 0, gb = kG == 2 && k.b * 8 >= 64 ? 1 : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // K and V, chunks a and b
    const int g = i % 2 == 0 ? ga : gb;
    const float2 z = dev::unpack2<kBf16>(lo[i / 2]);
    const float in = __shfl_sync(0xffffffffu, inv, base + i / 2 * kG + g);
    const float sc = __shfl_sync(0xffffffffu, signed_s, base + i / 2 * kG + g);
    const RowPair& r = i < 2 ? x : y;
    const uint32_t word =
        quantise8_u4<kBf16>(i % 2 == 0 ? r.a : r.b, sc, g ? z.y : z.x, bracket(in));
    uint8_t* codes = static_cast<uint8_t*>(i < 2 ? p.k_cache : p.v_cache) + srow * (D / 2);
    if (store) *reinterpret_cast<uint32_t*>(codes + (i % 2 == 0 ? k.a : k.b) * 4) = word;
  }
}

// cos and sin of the 4 pairs from `first` on (a lane's run of pairs).
__device__ __forceinline__ void load_angles(const RowParams& p, const int (&pos)[4], int first,
                                            float* cs, float* sn) {
  const int half = p.rotary_dim / 2;
  auto row = [&](int i) {
    const int at = i < p.axis_end[0] ? pos[0]
                   : i < p.axis_end[1] ? pos[1]
                   : i < p.axis_end[2] ? pos[2]
                                       : pos[3];
    return p.cos_sin + static_cast<size_t>(at) * p.rotary_dim + i;
  };
  if (p.sections_by_4) {  // the 4 pairs lie on one axis
    const float* a = row(first);
    const float4 c4 = *reinterpret_cast<const float4*>(a);
    const float4 s4 = *reinterpret_cast<const float4*>(a + half);
    cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
    sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* a = row(first + j);
      cs[j] = a[0];
      sn[j] = a[half];
    }
  }
}

// One CTA: kRowThreads / L row slots (L = D / 16 lanes each), row_lanes = 2^row_shift
// of them on one token.  A slot takes the token's units r, r + step, ...:
// query rows first, then (K, V) row pairs of the kv heads; gridDim.y CTAs share a
// token's units.
template <bool kBf16, int D, bool kRope, bool kInt4>
__global__ void __launch_bounds__(kRowThreads, kRope ? 6 : 8) row_kernel(const RowParams p) {
  constexpr int L = D / 16;
  constexpr int kSlots = kRowThreads / L;
  constexpr int kWarpRows = 32 / L;  // row slots of a warp
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int c = threadIdx.x % L;
  const int rs = threadIdx.x / L;
  const int row_lanes = 1 << p.row_shift;
  const long long t =
      static_cast<long long>(blockIdx.x) * (kSlots >> p.row_shift) + (rs >> p.row_shift);
  const bool there = t < p.num_tokens;
  const long long tt = there ? t : 0;
  const int unit0 = blockIdx.y * row_lanes + (rs & (row_lanes - 1));
  const int step = gridDim.y * row_lanes;
  const int nq = kRope ? p.num_q_heads : 0;
  const LaneChunks k = lane_chunks<D, kRope>(p, c);

  // The slot, the positions and the first rows set out together (the rows of a
  // padding token for nothing): 8191 tokens of 64 + 8 heads 54.6 -> 53.4 us, a step
  // of 64 tokens 3.0 -> 2.7.  Not where the quantiser follows: there the rows it
  // holds back spill (140 -> 154 us).
  constexpr bool kAhead = !kInt4;
  constexpr int U = kRope ? 4 : 2;  // rows in flight per lane
  const uint16_t* q = p.q + tt * p.q_stride;
  const uint16_t* kr = p.key + tt * p.k_stride;
  const uint16_t* vr = p.value + tt * p.v_stride;
  RowPair x[U];  // query rows, or a K and a V row
  auto load_queries = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * step < nq) x[u] = load_pair(q + (r + u * step) * D, k.a, k.b);
  };
  if (kAhead && unit0 < nq) {
    load_queries(unit0);
  } else if (kAhead) {
    const int h = min(unit0 - nq, p.num_kv_heads - 1);
    x[0] = load_pair(kr + h * D, k.a, k.b);
    x[1] = load_pair(vr + h * D, k.a, k.b);
  }
  int pos[4] = {0, 0, 0, 0};
  if constexpr (kRope) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (a < p.num_axes) pos[a] = p.positions[static_cast<size_t>(a) * p.num_tokens + tt];
  }
  // (a warp can hold several tokens and shares its lanes' sums: it goes on while
  // one of them is live)
  const int slot = there ? p.slots[tt] : -1;
  bool live = slot >= 0;  // not a padding token
  if (!__any_sync(0xffffffffu, live)) return;

  bool bad = slot >= p.num_slots;
  float cs[8], sn[8];
  if constexpr (kRope) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (live && a < p.num_axes) bad |= pos[a] < 0 || pos[a] >= p.max_position;
    if (live && !bad) {
      if (k.rot_a) load_angles(p, pos, p.interleaved ? 4 * k.a : 8 * c, cs, sn);
      if (k.rot_b) load_angles(p, pos, p.interleaved ? 4 * k.b : 8 * c + 4, cs + 4, sn + 4);
    }
  }
  if (bad) {
    if (unit0 == 0 && c == 0) dev::set_status(p.status, kErrBadBlock);
    if constexpr (kRope) {
      RowPair zero;
      zero.a = zero.b = make_uint4(0u, 0u, 0u, 0u);
      for (int r = unit0; r < nq; r += step)
        store_pair(p.q_out + t * p.q_out_stride + r * D, k.a, k.b, zero);
    }
    live = false;
  }

  int r = unit0;
  // this lane's slot among those of its token in the warp
  const int lead = rs & (min(row_lanes, kWarpRows) - 1);
  if constexpr (kRope) {
    uint16_t* qo = p.q_out + tt * p.q_out_stride;
    while (live && r < nq) {
      if (!kAhead) load_queries(r);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u * step < nq) {
          rotate<kBf16>(x[u], k, p.interleaved != 0, cs, sn);
          store_pair(qo + (r + u * step) * D, k.a, k.b, x[u]);
        }
      }
      r += U * step;
      if (kAhead) load_queries(r);
    }
    // back to the first unit at which one of the token's slots in this warp is past
    // the query rows
    const int last = unit0 - lead + min(row_lanes, kWarpRows) - 1;
    r = last >= nq ? unit0 : unit0 + (nq - last + step - 1) / step * step;
  }
  // K and V rows.  All lanes of the warp come here together; the loop runs until
  // the first slots are done.  (Lanes without a row redo one.)
  for (; r - lead < nq + p.num_kv_heads; r += step) {
    const int h = r - nq;
    const bool store = live && h >= 0 && h < p.num_kv_heads;
    RowPair kx, vx;
    if (kAhead) kx = x[0], vx = x[1];
    if (!kAhead || r != unit0) {
      const int hc = min(max(h, 0), p.num_kv_heads - 1);
      kx = load_pair(kr + hc * D, k.a, k.b);
      vx = load_pair(vr + hc * D, k.a, k.b);
    }
    if constexpr (kRope) rotate<kBf16>(kx, k, p.interleaved != 0, cs, sn);
    const size_t srow =
        (static_cast<size_t>(slot / kBlockSize) * p.num_kv_heads + h) * kBlockSize +
        slot % kBlockSize;
    if constexpr (kInt4) {
      store_rows_int4<kBf16, D>(kx, vx, k, c, store, p, srow);
    } else if (store) {
      store_pair(static_cast<uint16_t*>(p.k_cache) + srow * D, k.a, k.b, kx);
      store_pair(static_cast<uint16_t*>(p.v_cache) + srow * D, k.a, k.b, vx);
    }
  }
}

// Values of 8 codes with their (scale, zero) pair, as a 16-byte chunk.  A code
// moved to the bottom of a word under the exponent of 2^23 is 2^23 + c; s * c is
// exact in float32 (11 + 4 bits), so the FMA rounds s * c + z once to float32
// before the 16-bit rounding.
template <bool kBf16>
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t sz) {
  const float2 f = dev::unpack2<kBf16>(sz);
  const uint64_t s2 = dev::f2pack(f.x, f.x), z2 = dev::f2pack(f.y, f.y);
  const uint64_t base2 = dev::f2pack(-8388608.f, -8388608.f);
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = __uint_as_float(((w >> (8 * e)) & 15u) | 0x4b000000u);
    const float b = __uint_as_float(((w >> (8 * e + 4)) & 15u) | 0x4b000000u);
    const float2 x = dev::f2unpack(dev::ffma2(dev::fadd2(dev::f2pack(a, b), base2), s2, z2));
    v[e] = dev::pack2<kBf16>(x.x, x.y);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// A warp per 512 / D rows: of one token and as many heads, or, with fewer heads,
// `heads` (a power of two) of each of several tokens.  L = D / 16 lanes share a
// row; lane c writes the 16-byte chunks c and c + L of K and of V, so that a store
// covers whole sectors (32 bytes a lane in a row instead: 128 us where this takes
// 110).
template <bool kBf16, int D>
__global__ void __launch_bounds__(128) read_int4_kernel(
    uint4* __restrict__ key, uint4* __restrict__ value, const uint8_t* __restrict__ kc,
    const uint8_t* __restrict__ vc, const uint32_t* __restrict__ ksz,
    const uint32_t* __restrict__ vsz, const int32_t* __restrict__ slots, int num_tokens,
    int num_kv_heads, int heads, int num_slots, int32_t* status) {
  constexpr int L = D / 16, kRows = 32 / L;
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int lane = threadIdx.x & 31, c = lane % L;
  const int row = lane / L, h = blockIdx.y * heads + (row & (heads - 1));
  const int shift = 31 - __clz(heads);
  const long long t = (static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5)) *
                          (kRows >> shift) +
                      (row >> shift);
  if (t >= num_tokens) return;
  const int slot = slots[t];
  if (slot < 0) return;  // padding token: the rows are left as they are
  const bool bad = slot >= num_slots;
  if (bad && h == 0 && c == 0) dev::set_status(status, kErrBadBlock);
  const size_t row0 =
      bad ? 0
          : static_cast<size_t>(slot / kBlockSize) * num_kv_heads * kBlockSize + slot % kBlockSize;
  uint4* ko = key + t * num_kv_heads * (D / 8) + c;
  uint4* vo = value + t * num_kv_heads * (D / 8) + c;
  if (h < num_kv_heads) {
    uint4 k2[2], v2[2];
    if (bad) {
      k2[0] = k2[1] = v2[0] = v2[1] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const size_t srow = row0 + static_cast<size_t>(h) * kBlockSize;
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(kc + srow * (D / 2)) + c;
      const uint32_t* vw = reinterpret_cast<const uint32_t*>(vc + srow * (D / 2)) + c;
      const uint32_t w[4] = {kw[0], kw[L], vw[0], vw[L]};
      uint2 kp, vp;  // pairs of chunk c and of chunk c + L
      if constexpr (D == 128) {
        kp = *reinterpret_cast<const uint2*>(ksz + srow * 2);
        vp = *reinterpret_cast<const uint2*>(vsz + srow * 2);
      } else {
        kp.x = kp.y = ksz[srow];
        vp.x = vp.y = vsz[srow];
      }
      k2[0] = dequant8<kBf16>(w[0], kp.x);
      k2[1] = dequant8<kBf16>(w[1], kp.y);
      v2[0] = dequant8<kBf16>(w[2], vp.x);
      v2[1] = dequant8<kBf16>(w[3], vp.y);
    }
    ko[h * (D / 8)] = k2[0];
    ko[h * (D / 8) + L] = k2[1];
    vo[h * (D / 8)] = v2[0];
    vo[h * (D / 8) + L] = v2[1];
  }
}

template <bool kBf16, int D, bool kRope, bool kInt4>
cudaError_t launch_rows(RowParams p, cudaStream_t s) {
  constexpr int kSlots = kRowThreads / (D / 16);
  const long long units = (kRope ? p.num_q_heads : 0) + p.num_kv_heads;
  // Few tokens: all of a CTA's slots on one token, and CTAs side by side.  The step
  // lies where four CTAs per SM have work: rotation of 64 + 8 heads of 128 into 4
  // bits, 128 tokens 6.5 and 5.0 us (many, few), 256 tokens 6.5 and 6.8, 4096
  // tokens 31 and 59; 16 + 8 heads of 64, 512 tokens 5.2 and 4.7, 1024 tokens 5.3
  // and 6.9.
  // Many: up to 8 slots per token.  A rotating slot takes 9 of the token's units,
  // for it reads the token's angles, as many bytes as a row, and has 4 rows in
  // flight: 29843 tokens of 7 + 1 heads with 1 slot 27 us, with 2 30, with 8 65;
  // but with less than 1.5 CTAs per SM slots go before (1024 tokens of 16 + 8
  // heads, 4 slots 7.0 us, 8 slots 5.2).
  const bool many = p.num_tokens * units >= 152 * 4 * kSlots;
  const long long most = std::min<long long>(units, many ? 8 : kSlots);
  const long long want = many && kRope ? std::min((units + 8) / 9, most) : most;
  p.row_shift = 0;
  const long long tokens = p.num_tokens;
  while (1 << p.row_shift < want ||
         (1 << p.row_shift < most && tokens << p.row_shift < 152 * 3 / 2 * kSlots))
    ++p.row_shift;
  const int row_lanes = 1 << p.row_shift;
  const long long per_cta = kSlots / row_lanes;
  const dim3 grid(static_cast<unsigned>((p.num_tokens + per_cta - 1) / per_cta),
                  many ? 1u : static_cast<unsigned>((units + row_lanes - 1) / row_lanes));
  return launch_pdl(row_kernel<kBf16, D, kRope, kInt4>, grid, dim3(kRowThreads), 0, s, p);
}

template <bool kRope, bool kInt4>
cudaError_t launch_rows_typed(const RowParams& p, bool bf16, int head_dim, cudaStream_t s) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (bf16 && head_dim == 64) return launch_rows<true, 64, kRope, kInt4>(p, s);
  if (bf16 && head_dim == 128) return launch_rows<true, 128, kRope, kInt4>(p, s);
  if (!bf16 && head_dim == 64) return launch_rows<false, 64, kRope, kInt4>(p, s);
  if (!bf16 && head_dim == 128) return launch_rows<false, 128, kRope, kInt4>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_append_int4(const RowParams& p, bool bf16, int head_dim, cudaStream_t s) {
  return launch_rows_typed<false, true>(p, bf16, head_dim, s);
}

cudaError_t launch_rope_append(const RowParams& p, bool bf16, int head_dim, bool int4,
                               cudaStream_t s) {
  return int4 ? launch_rows_typed<true, true>(p, bf16, head_dim, s)
              : launch_rows_typed<true, false>(p, bf16, head_dim, s);
}

cudaError_t launch_read_int4(void* key, void* value, bool bf16, const uint8_t* kc,
                             const uint8_t* vc, const void* ksz, const void* vsz,
                             const int32_t* slots, int num_tokens, const kvp_cache_desc& c,
                             int32_t* status, cudaStream_t s) {
  if (num_tokens == 0) return cudaSuccess;
  const int rows = 512 / c.head_dim;  // of a warp
  int heads = 1;
  while (heads < c.num_kv_heads && heads < rows) heads *= 2;
  const int tokens = 4 * (rows / heads);  // of a CTA
  const dim3 grid(static_cast<unsigned>((num_tokens - 1) / tokens + 1),
                  static_cast<unsigned>((c.num_kv_heads + heads - 1) / heads));
  const int nslots = c.num_blocks * kBlockSize;
#define KVP_READ_CASE(BF, DD)                                                                   \
  if (bf16 == BF && c.head_dim == DD)                                                           \
    return launch_pdl(read_int4_kernel<BF, DD>, grid, dim3(128), 0, s, static_cast<uint4*>(key), \
                      static_cast<uint4*>(value), kc, vc, static_cast<const uint32_t*>(ksz),    \
                      static_cast<const uint32_t*>(vsz), slots, num_tokens, c.num_kv_heads,     \
                      heads, nslots, status);
  KVP_READ_CASE(false, 64)
  KVP_READ_CASE(false, 128)
  KVP_READ_CASE(true, 64)
  KVP_READ_CASE(true, 128)
#undef KVP_READ_CASE
  return cudaErrorInvalidValue;
}

}  // namespace kvp
