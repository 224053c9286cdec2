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
// of the token it works on.
#include "kvp_device.cuh"
#include "kvp_internal.h"

namespace kvp {
namespace {

constexpr int kRowThreads = 256;

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
// FMA d * (1/s) + 1.5 * 2^23 rounds the quotient once to an integer held in the
// low mantissa bits.  d * (1/s) is within 15 * 2^-22 of the IEEE quotient, so
// both round alike unless the fraction is within 1e-4 of a half; such an
// element takes the quotient itself.  So does every element when s or 1/s
// leaves the normal range (`exact`), where that bound does not hold.
__device__ __forceinline__ uint32_t quantise8_u4(const float (&x)[8], float s, float z) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  constexpr float kBand = 0.5f - 1.0e-4f;
  const bool exact = s > 0.f && !(s >= 1.17549435e-38f && s <= 8.5070592e37f);
  const float inv = (s > 0.f && !exact) ? __frcp_rn(s) : 0.f;
  uint32_t word = 0u - 0x4b400000u * 0x11111111u;  // minus every element's magic bits
  float far = 0.f;
  uint32_t k[8];
  float d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    d[e] = __fsub_rn(x[e], z);
    const float m = __fmaf_rn(d[e], inv, kMagic);
    far = fmaxf(far, fabsf(__fmaf_rn(d[e], inv, kMagic - m)));
    k[e] = __float_as_uint(fminf(m, kMagic + 15.f));
  }
  if (far > kBand || exact) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      k[e] = __float_as_uint(__fadd_rn(kMagic, fminf(rintf(__fdiv_rn(d[e], s)), 15.f)));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) word += k[e] << (4 * e);
  return word;
}

// Quantise the row shared by the D / 16 lanes of `mask` and write its codes and
// (scale, zero) pairs.
template <bool kBf16, int D>
__device__ __forceinline__ void store_row_int4(const RowPair& r, const LaneChunks& k, int c,
                                               uint32_t mask, uint8_t* codes, uint32_t* sz) {
  constexpr int L = D / 16;
  uint32_t mna = min2<kBf16>(min2<kBf16>(r.a.x, r.a.y), min2<kBf16>(r.a.z, r.a.w));
  uint32_t mnb = min2<kBf16>(min2<kBf16>(r.b.x, r.b.y), min2<kBf16>(r.b.z, r.b.w));
  uint32_t mxa = max2<kBf16>(max2<kBf16>(r.a.x, r.a.y), max2<kBf16>(r.a.z, r.a.w));
  uint32_t mxb = max2<kBf16>(max2<kBf16>(r.b.x, r.b.y), max2<kBf16>(r.b.z, r.b.w));
  uint32_t lo, hi;  // smallest and largest: of group 0 in the low half, of group 1 in the high
  if constexpr (D == 64) {
    lo = min2<kBf16>(mna, mnb);
    hi = max2<kBf16>(mxa, mxb);
    lo = min2<kBf16>(lo, __byte_perm(lo, lo, 0x1032));
    hi = max2<kBf16>(hi, __byte_perm(hi, hi, 0x1032));
  } else {
    constexpr uint32_t kInf = kBf16 ? 0x7f80u : 0x7c00u;
    mna = min2<kBf16>(mna, __byte_perm(mna, mna, 0x1032));
    mnb = min2<kBf16>(mnb, __byte_perm(mnb, mnb, 0x1032));
    mxa = max2<kBf16>(mxa, __byte_perm(mxa, mxa, 0x1032));
    mxb = max2<kBf16>(mxb, __byte_perm(mxb, mxb, 0x1032));
    const uint32_t in_a = (k.a * 8 < 64) ? 0x0000ffffu : 0xffff0000u;
    const uint32_t in_b = (k.b * 8 < 64) ? 0x0000ffffu : 0xffff0000u;
    lo = min2<kBf16>((mna & in_a) | ((kInf * 0x10001u) & ~in_a),
                     (mnb & in_b) | ((kInf * 0x10001u) & ~in_b));
    hi = max2<kBf16>((mxa & in_a) | (((kInf | 0x8000u) * 0x10001u) & ~in_a),
                     (mxb & in_b) | (((kInf | 0x8000u) * 0x10001u) & ~in_b));
  }
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) {
    lo = min2<kBf16>(lo, __shfl_xor_sync(mask, lo, o));
    hi = max2<kBf16>(hi, __shfl_xor_sync(mask, hi, o));
  }
  const float2 z = dev::unpack2<kBf16>(lo), top = dev::unpack2<kBf16>(hi);
  const uint32_t sp = dev::pack2<kBf16>(__fdiv_rn(__fsub_rn(top.x, z.x), 15.f),
                                        __fdiv_rn(__fsub_rn(top.y, z.y), 15.f));
  const float2 s = dev::unpack2<kBf16>(sp);
  float x[8];
  const bool ga = D > 64 && k.a * 8 >= 64, gb = D > 64 && k.b * 8 >= 64;
  unpack8<kBf16>(r.a, x);
  *reinterpret_cast<uint32_t*>(codes + k.a * 4) = quantise8_u4(x, ga ? s.y : s.x, ga ? z.y : z.x);
  unpack8<kBf16>(r.b, x);
  *reinterpret_cast<uint32_t*>(codes + k.b * 4) = quantise8_u4(x, gb ? s.y : s.x, gb ? z.y : z.x);
  if (c == 0) {
    if constexpr (D == 64) {
      sz[0] = __byte_perm(sp, lo, 0x5410);
    } else {
      *reinterpret_cast<uint2*>(sz) =
          make_uint2(__byte_perm(sp, lo, 0x5410), __byte_perm(sp, lo, 0x7632));
    }
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

// One CTA: 256 / L row slots (L = D / 16 lanes each), row_lanes of them on one
// token.  A slot takes the token's units r, r + step, ...: query rows first,
// then (K, V) row pairs of the kv heads; gridDim.y CTAs share a token's units.
template <bool kBf16, int D, bool kRope, bool kInt4>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const RowParams p) {
  constexpr int L = D / 16;
  constexpr int kSlots = kRowThreads / L;
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int c = threadIdx.x % L;
  const int rs = threadIdx.x / L;
  const long long t =
      static_cast<long long>(blockIdx.x) * (kSlots / p.row_lanes) + rs / p.row_lanes;
  if (t >= p.num_tokens) return;
  const int slot = p.slots[t];
  if (slot < 0) return;  // padding token
  const int unit0 = blockIdx.y * p.row_lanes + rs % p.row_lanes;
  const int step = gridDim.y * p.row_lanes;
  const int nq = kRope ? p.num_q_heads : 0;

  const LaneChunks k = lane_chunks<D, kRope>(p, c);
  bool bad = slot >= p.num_slots;
  float cs[8], sn[8];
  if constexpr (kRope) {
    int pos[4] = {0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a < p.num_axes) {
        pos[a] = p.positions[static_cast<size_t>(a) * p.num_tokens + t];
        bad |= pos[a] < 0 || pos[a] >= p.max_position;
      }
    }
    if (!bad) {
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
    return;
  }

  int r = unit0;
  if constexpr (kRope) {
    constexpr int U = 4;  // rows in flight per lane
    const uint16_t* q = p.q + t * p.q_stride;
    uint16_t* qo = p.q_out + t * p.q_out_stride;
    for (; r < nq; r += U * step) {
      RowPair x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + u * step < nq) x[u] = load_pair(q + (r + u * step) * D, k.a, k.b);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u * step < nq) {
          rotate<kBf16>(x[u], k, p.interleaved != 0, cs, sn);
          store_pair(qo + (r + u * step) * D, k.a, k.b, x[u]);
        }
      }
    }
    // back to this slot's first unit at or past the query rows
    r = unit0 >= nq ? unit0 : unit0 + (nq - unit0 + step - 1) / step * step;
  }
  const uint32_t mask = ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
  const uint16_t* kr = p.key + t * p.k_stride;
  const uint16_t* vr = p.value + t * p.v_stride;
  for (; r < nq + p.num_kv_heads; r += step) {
    const int h = r - nq;
    RowPair x = load_pair(kr + h * D, k.a, k.b);
    const RowPair y = load_pair(vr + h * D, k.a, k.b);
    if constexpr (kRope) rotate<kBf16>(x, k, p.interleaved != 0, cs, sn);
    const size_t srow =
        (static_cast<size_t>(slot / kBlockSize) * p.num_kv_heads + h) * kBlockSize +
        slot % kBlockSize;
    if constexpr (kInt4) {
      store_row_int4<kBf16, D>(x, k, c, mask, static_cast<uint8_t*>(p.k_cache) + srow * (D / 2),
                               p.k_sz + srow * (D / 64));
      store_row_int4<kBf16, D>(y, k, c, mask, static_cast<uint8_t*>(p.v_cache) + srow * (D / 2),
                               p.v_sz + srow * (D / 64));
    } else {
      store_pair(static_cast<uint16_t*>(p.k_cache) + srow * D, k.a, k.b, x);
      store_pair(static_cast<uint16_t*>(p.v_cache) + srow * D, k.a, k.b, y);
    }
  }
}

// Values of 16 codes (8 bytes) with one (scale, zero) pair, as two 16-byte
// chunks: s * c is exact in float32 (11 + 4 bits), so the FMA rounds s * c + z
// once to float32 before the 16-bit rounding.
template <bool kBf16>
__device__ __forceinline__ void dequant16(uint2 w, uint32_t sz, uint4 (&out)[2]) {
  const float2 f = dev::unpack2<kBf16>(sz);
  const uint32_t word[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = __fmaf_rn(f.x, static_cast<float>((word[i] >> (4 * e)) & 15u), f.y);
    out[i] = pack8<kBf16>(x);
  }
}

// One lane per 16 elements of a row of K and of V: grid.x over tokens, the
// heads of a token over its lanes.
template <bool kBf16, int D>
__global__ void __launch_bounds__(256) read_int4_kernel(
    uint4* __restrict__ key, uint4* __restrict__ value, const uint8_t* __restrict__ kc,
    const uint8_t* __restrict__ vc, const uint32_t* __restrict__ ksz,
    const uint32_t* __restrict__ vsz, const int32_t* __restrict__ slots, int num_tokens,
    int num_kv_heads, int num_slots, int32_t* status) {
  constexpr int L = D / 16;
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long row = i / L;  // token * Hkv + head
  const int c = static_cast<int>(i % L);
  const long long t = row / num_kv_heads;
  const int h = static_cast<int>(row % num_kv_heads);
  if (t >= num_tokens) return;
  const int slot = slots[t];
  if (slot < 0) return;  // padding token: the row is left as it is
  uint4 k2[2], v2[2];
  if (slot >= num_slots) {
    if (h == 0 && c == 0) dev::set_status(status, kErrBadBlock);
    k2[0] = k2[1] = v2[0] = v2[1] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    const size_t srow = (static_cast<size_t>(slot / kBlockSize) * num_kv_heads + h) * kBlockSize +
                        slot % kBlockSize;
    const int g = c / 4;  // 64 elements are 4 lanes
    dequant16<kBf16>(*reinterpret_cast<const uint2*>(kc + srow * (D / 2) + c * 8),
                     ksz[srow * (D / 64) + g], k2);
    dequant16<kBf16>(*reinterpret_cast<const uint2*>(vc + srow * (D / 2) + c * 8),
                     vsz[srow * (D / 64) + g], v2);
  }
  uint4* ko = key + static_cast<size_t>(row) * (D / 8) + c * 2;
  uint4* vo = value + static_cast<size_t>(row) * (D / 8) + c * 2;
  ko[0] = k2[0];
  ko[1] = k2[1];
  vo[0] = v2[0];
  vo[1] = v2[1];
}

template <bool kBf16, int D, bool kRope, bool kInt4>
cudaError_t launch_rows(RowParams p, cudaStream_t s) {
  constexpr int kSlots = kRowThreads / (D / 16);
  const long long units = (kRope ? p.num_q_heads : 0) + p.num_kv_heads;
  // Many tokens: 8 slots per token, so a lane uses its angles for several
  // heads.  Few: all of a CTA's slots on one token, and CTAs side by side.
  const bool many = p.num_tokens * units >= 152 * 4 * kSlots;
  p.row_lanes = many ? 8 : kSlots;
  const long long per_cta = kSlots / p.row_lanes;
  const dim3 grid(static_cast<unsigned>((p.num_tokens + per_cta - 1) / per_cta),
                  many ? 1u : static_cast<unsigned>((units + kSlots - 1) / kSlots));
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
  const long long lanes = static_cast<long long>(num_tokens) * c.num_kv_heads * (c.head_dim / 16);
  const dim3 grid(static_cast<unsigned>((lanes + 255) / 256));
  const int nslots = c.num_blocks * kBlockSize;
#define KVP_READ_CASE(BF, DD)                                                                   \
  if (bf16 == BF && c.head_dim == DD)                                                           \
    return launch_pdl(read_int4_kernel<BF, DD>, grid, dim3(256), 0, s, static_cast<uint4*>(key), \
                      static_cast<uint4*>(value), kc, vc, static_cast<const uint32_t*>(ksz),    \
                      static_cast<const uint32_t*>(vsz), slots, num_tokens, c.num_kv_heads,     \
                      nslots, status);
  KVP_READ_CASE(false, 64)
  KVP_READ_CASE(false, 128)
  KVP_READ_CASE(true, 64)
  KVP_READ_CASE(true, 128)
#undef KVP_READ_CASE
  return cudaErrorInvalidValue;
}

}  // namespace kvp
