// kvp_decode_int4.cu -- decode attention over 4-bit pools.
//
// A K or V row of a (token, kv head) is D codes c in 0..15, two to a byte, with
// one 16-bit (s, z) pair per group of 64 elements; element d stands for
// s_g c_d + z_g.  For request b and query head h,
//   u_t = scale log2(e) [ sum_g s_tg (sum_{d in g} q_d c_td) + z_tg Q_g ],
//         Q_g = sum_{d in g} q_d,
//   out_d = sum_t p_t (s_tg c_td + z_tg) / sum_t p_t,   p_t = 2^(u_t - m).
// The work split is that of the other decodes (kvp_decode.cuh): a CTA per
// (request, kv head, up to 8 query heads, partition), 4 warps that each stream
// their own 16-token blocks through a ring of stages, states merged at the end.
//
// A block is 2 (8 D + 32 D / 64) bytes = 2304 at D = 128, little over half of
// an INT8 block, while a warp has the same 32 D codes to widen: the kernel is
// bound by issue slots before HBM, so the arithmetic is arranged to widen a
// code with less than one instruction.
//   * A code left where it lies is already a number: the fp16 bit pattern
//     0x000c is the subnormal c 2^-24 and 0x00c0 is 16 c 2^-24, both exact
//     tensor-core operands.  So one AND turns two codes into an operand pair,
//     and one shift serves the other two pairs of a word; no subtraction, no
//     convert.  The factor 16 of every second pair goes into q (before the
//     K product) and into the output (after the V product).
//   * q is scaled by a power of two kappa so that its largest element lies in
//     [2^10, 2^11): exact for fp16 and bf16 q alike (elements below 2^-24 of the
//     largest lose their last bits, 2^-35 of it), so one fp16 operand type
//     serves both and a bf16 q needs no second path.
//   * K's s multiplies a group's accumulator, z multiplies Q_g.
//   * V's s goes into the weight, a_t = p_t s_t rho, rounded to fp16 (2^-12
//     relative, independent from token to token); rho is a power of two per
//     head that keeps a within [0, 4096], moved only when a block exceeds that,
//     so the accumulators stay in the tensor core's registers and no block
//     costs a rescale.  A product with ones gives sum_t a_t of the rounded
//     weights; subtracting 7.5 times it centres the codes, so that the
//     rounding of a is weighted by c - 7.5 and not by c.
//   * The reference m of the softmax is moved in that same rare branch (when a
//     weight passes 2^16), which saves the six shuffles of a maximum per block.
//   * z's part, sum_t p_t (z_t + 7.5 s_t), is float32 on the lanes.
// Rows t of the score fragment hold tokens in the order 4 (t % 2) + t / 2 (+ 8
// in the upper half), so that the four tokens a V load touches lie in
// different shared-memory banks.
#include "kvp_decode.cuh"

namespace kvp {
namespace {

constexpr int kInt4Stages = 4;  // blocks in flight per warp

template <bool kBf16, int D>
struct Int4Path {
  static constexpr int kD = D;
  static constexpr int kHeads = 8;
  static constexpr int kElemBytes = 1;  // (no fused append)
  static constexpr int kGroups = D / 64;
  static constexpr int kCodeBytes = 16 * D / 2;      // K or V codes of a block
  static constexpr int kPairBytes = 16 * kGroups * 4;  // their (s, z) pairs
  static constexpr int kStageBytes = 2 * (kCodeBytes + kPairBytes);
  static constexpr int kS = kWarps * kInt4Stages;
  static_assert(kStageBytes % 128 == 0, "stages stay aligned for bulk copies");
  static_assert(kWarps * kHeads * (D + 2) * 4 <= kS * kStageBytes, "merge area must fit");

  struct State {
    uint32_t qb[kGroups][4][2];  // q operand per k-step
    float o[kGroups][4][4];      // 2^-24 sum a c (rows 0, 1) and 2^-20 sum a c (rows 2, 3)
    float as[kGroups][4];        // 2^-24 sum a, in every row
    float zo[kGroups][2];        // sum p (z + 7.5 s), this lane's tokens
    float qz[kGroups][2];        // scale log2(e) Q_g
    float f[2];                  // scale log2(e) 2^20 / kappa
    float m[2], l[2];            // reference and sum (this lane's tokens)
    float rho[2];
  };

  // Power of two that takes x > 0 into [2^k, 2^(k+1)), its exponent within +-100.
  __device__ __forceinline__ static float pow2_to(float x, int k) {
    const int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
    const int up = min(100, max(-100, k - e));
    return __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
  }

  __device__ __forceinline__ static void init(State& st, const DecodeParams& p, int b, int head0,
                                              int nheads, int lane) {
    const int g8 = lane >> 2, t4 = lane & 3;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                        (static_cast<size_t>(b) * p.num_q_heads + head0 + g8) * D;
    uint4 raw[kGroups][2];
    float big = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        raw[g][w] = make_uint4(0u, 0u, 0u, 0u);
        if (g8 < nheads)
          raw[g][w] = *reinterpret_cast<const uint4*>(q + 64 * g + 16 * t4 + 8 * w);
        const uint32_t r[4] = {raw[g][w].x, raw[g][w].y, raw[g][w].z, raw[g][w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = dev::unpack2<kBf16>(r[i]);
          big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
      }
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const float kappa = big > 0.f ? pow2_to(big, 10) : 1.f;
    float qs[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      qs[g] = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t r[4] = {raw[g][w].x, raw[g][w].y, raw[g][w].z, raw[g][w].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = dev::unpack2<kBf16>(r[i]);
          v[2 * i] = x.x;
          v[2 * i + 1] = x.y;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          qs[g] += v[e];
          v[e] *= kappa;
        }
        // the word's code pairs are (0, 4), 16 (1, 5), (2, 6), 16 (3, 7)
        st.qb[g][2 * w][0] = dev::pack2<false>(16.f * v[0], 16.f * v[4]);
        st.qb[g][2 * w][1] = dev::pack2<false>(v[1], v[5]);
        st.qb[g][2 * w + 1][0] = dev::pack2<false>(16.f * v[2], 16.f * v[6]);
        st.qb[g][2 * w + 1][1] = dev::pack2<false>(v[3], v[7]);
      }
      qs[g] += __shfl_xor_sync(0xffffffffu, qs[g], 1);
      qs[g] += __shfl_xor_sync(0xffffffffu, qs[g], 2);
    }
    // this lane's score columns are heads 2 t4 and 2 t4 + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = 4 * (2 * t4 + i);
      st.f[i] = p.scale_log2 * 1048576.f / __shfl_sync(0xffffffffu, kappa, src);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        st.qz[g][i] = p.scale_log2 * __shfl_sync(0xffffffffu, qs[g], src);
        st.zo[g][i] = 0.f;
      }
      st.m[i] = -INFINITY;
      st.l[i] = 0.f;
      st.rho[i] = 1.f;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st.as[g][i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) st.o[g][j][i] = 0.f;
      }
    }
  }

  // (s, z) pairs of one token, one per group.
  __device__ __forceinline__ static void load_pairs(const uint8_t* base, int tok,
                                                    float (&s)[kGroups], float (&z)[kGroups]) {
    uint32_t w[kGroups];
    if constexpr (kGroups == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(base + tok * 8);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(base + tok * 4);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float2 x = dev::unpack2<kBf16>(w[g]);
      s[g] = x.x;
      z[g] = x.y;
    }
  }

  // A block's tiles: K codes, V codes, K pairs, V pairs.
  __device__ __forceinline__ static void consume(State& st, const uint8_t* tile, int valid,
                                                 int lane) {
    constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int tok0 = 4 * (g8 & 1) + (g8 >> 1), tok1 = tok0 + 8;  // rows g8, g8 + 8
    const uint8_t* kc = tile;
    const uint8_t* vc = tile + kCodeBytes;
    const uint8_t* kp = tile + 2 * kCodeBytes;
    const uint8_t* vp = kp + kPairBytes;

    // ---- scores
    float ks0[kGroups], kz0[kGroups], ks1[kGroups], kz1[kGroups];
    load_pairs(kp, tok0, ks0, kz0);
    load_pairs(kp, tok1, ks1, kz1);
    float u[4] = {0.f, 0.f, 0.f, 0.f}, uz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint2 a = *reinterpret_cast<const uint2*>(kc + tok0 * (D / 2) + 32 * g + 8 * t4);
      const uint2 b = *reinterpret_cast<const uint2*>(kc + tok1 * (D / 2) + 32 * g + 8 * t4);
      const uint32_t wa[2] = {a.x, a.y}, wb[2] = {b.x, b.y};
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t x = wa[w], y = wb[w], xs = x >> 8, ys = y >> 8;
        dev::mma16816<false>(acc, x & kLow, y & kLow, x & kHigh, y & kHigh, st.qb[g][2 * w][0],
                             st.qb[g][2 * w][1]);
        dev::mma16816<false>(acc, xs & kLow, ys & kLow, xs & kHigh, ys & kHigh,
                             st.qb[g][2 * w + 1][0], st.qb[g][2 * w + 1][1]);
      }
      u[0] = fmaf(ks0[g], acc[0], u[0]);
      u[1] = fmaf(ks0[g], acc[1], u[1]);
      u[2] = fmaf(ks1[g], acc[2], u[2]);
      u[3] = fmaf(ks1[g], acc[3], u[3]);
      uz[0] = fmaf(kz0[g], st.qz[g][0], uz[0]);
      uz[1] = fmaf(kz0[g], st.qz[g][1], uz[1]);
      uz[2] = fmaf(kz1[g], st.qz[g][0], uz[2]);
      uz[3] = fmaf(kz1[g], st.qz[g][1], uz[3]);
    }
    u[0] = fmaf(u[0], st.f[0], uz[0]);
    u[1] = fmaf(u[1], st.f[1], uz[1]);
    u[2] = fmaf(u[2], st.f[0], uz[2]);
    u[3] = fmaf(u[3], st.f[1], uz[3]);
    float vs0[kGroups], vz0[kGroups], vs1[kGroups], vz1[kGroups];
    load_pairs(vp, tok0, vs0, vz0);
    load_pairs(vp, tok1, vs1, vz1);
    if (valid < 16) {  // slots past the context may hold anything
      const bool in0 = tok0 < valid, in1 = tok1 < valid;
      u[0] = in0 ? u[0] : -INFINITY;
      u[1] = in0 ? u[1] : -INFINITY;
      u[2] = in1 ? u[2] : -INFINITY;
      u[3] = in1 ? u[3] : -INFINITY;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        vs0[g] = in0 ? vs0[g] : 0.f;
        vz0[g] = in0 ? vz0[g] : 0.f;
        vs1[g] = in1 ? vs1[g] : 0.f;
        vz1[g] = in1 ? vz1[g] : 0.f;
      }
    }

    // ---- weights against the present reference
    float pr[4], a[kGroups][4];
    auto weights = [&] {
      pr[0] = dev::ex2_approx(u[0] - st.m[0]);
      pr[1] = dev::ex2_approx(u[1] - st.m[1]);
      pr[2] = dev::ex2_approx(u[2] - st.m[0]);
      pr[3] = dev::ex2_approx(u[3] - st.m[1]);
      const float r0 = pr[0] * st.rho[0], r1 = pr[1] * st.rho[1];
      const float r2 = pr[2] * st.rho[0], r3 = pr[3] * st.rho[1];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        a[g][0] = r0 * vs0[g];
        a[g][1] = r1 * vs0[g];
        a[g][2] = r2 * vs1[g];
        a[g][3] = r3 * vs1[g];
      }
    };
    weights();
    float amax = fmaxf(fmaxf(a[0][0], a[0][1]), fmaxf(a[0][2], a[0][3]));
    if constexpr (kGroups == 2)
      amax = fmaxf(amax, fmaxf(fmaxf(a[1][0], a[1][1]), fmaxf(a[1][2], a[1][3])));
    const float pmax = fmaxf(fmaxf(pr[0], pr[1]), fmaxf(pr[2], pr[3]));
    if (__any_sync(0xffffffffu, amax > 4096.f || pmax > 65536.f || st.m[0] == -INFINITY)) {
      // ---- rare: move the reference to the block's maximum and rho to its weights
      float mx0 = fmaxf(u[0], u[2]), mx1 = fmaxf(u[1], u[3]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float mn0 = fmaxf(st.m[0], mx0), mn1 = fmaxf(st.m[1], mx1);
      const float al[2] = {dev::ex2_approx(st.m[0] - mn0), dev::ex2_approx(st.m[1] - mn1)};
      st.m[0] = mn0;
      st.m[1] = mn1;
      const float old[2] = {st.rho[0], st.rho[1]};
      st.rho[0] = st.rho[1] = 1.f;
      weights();
      float ax[2] = {fmaxf(a[0][0], a[0][2]), fmaxf(a[0][1], a[0][3])};
      if constexpr (kGroups == 2) {
        ax[0] = fmaxf(ax[0], fmaxf(a[1][0], a[1][2]));
        ax[1] = fmaxf(ax[1], fmaxf(a[1][1], a[1][3]));
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        ax[0] = fmaxf(ax[0], __shfl_xor_sync(0xffffffffu, ax[0], o));
        ax[1] = fmaxf(ax[1], __shfl_xor_sync(0xffffffffu, ax[1], o));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // no weight yet (constant rows): the largest rho, until one exceeds it
        st.rho[i] = ax[i] > 0.f ? pow2_to(ax[i], 3) : 1.2676506e30f;  // 2^100
        const int e = (static_cast<int>(__float_as_uint(st.rho[i])) -
                       static_cast<int>(__float_as_uint(old[i]))) >> 23;
        const float ratio =
            al[i] * __uint_as_float(static_cast<uint32_t>(127 + min(126, max(-126, e))) << 23);
        st.l[i] *= al[i];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          st.zo[g][i] *= al[i];
          st.as[g][i] *= ratio;
          st.as[g][i + 2] *= ratio;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            st.o[g][j][i] *= ratio;
            st.o[g][j][i + 2] *= ratio;
          }
        }
      }
      weights();
    }
    st.l[0] += pr[0] + pr[2];
    st.l[1] += pr[1] + pr[3];

    // ---- values
    const uint8_t* vrow = vc + t4 * (D / 2) + 4 * g8;  // token t4, this lane's 8 codes
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float z0 = fmaf(7.5f, vs0[g], vz0[g]), z1 = fmaf(7.5f, vs1[g], vz1[g]);
      st.zo[g][0] = fmaf(pr[0], z0, fmaf(pr[2], z1, st.zo[g][0]));
      st.zo[g][1] = fmaf(pr[1], z0, fmaf(pr[3], z1, st.zo[g][1]));
      const uint32_t b0 = dev::movm_t(dev::pack2<false>(a[g][0], a[g][1]));
      const uint32_t b1 = dev::movm_t(dev::pack2<false>(a[g][2], a[g][3]));
      const uint32_t wa = *reinterpret_cast<const uint32_t*>(vrow + 32 * g);
      const uint32_t wb = *reinterpret_cast<const uint32_t*>(vrow + 32 * g + 4 * (D / 2));
      const uint32_t wc = *reinterpret_cast<const uint32_t*>(vrow + 32 * g + 8 * (D / 2));
      const uint32_t wd = *reinterpret_cast<const uint32_t*>(vrow + 32 * g + 12 * (D / 2));
      dev::mma16816<false>(st.as[g], 0x00010001u, 0x00010001u, 0x00010001u, 0x00010001u, b0, b1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // codes 0-3, then 4-7, of each token's word
        const uint32_t x = dev::prmt(wa, wb, h == 0 ? 0x5410u : 0x7632u);
        const uint32_t y = dev::prmt(wc, wd, h == 0 ? 0x5410u : 0x7632u);
        const uint32_t xs = x >> 8, ys = y >> 8;
        dev::mma16816<false>(st.o[g][2 * h], x & kLow, x & kHigh, y & kLow, y & kHigh, b0, b1);
        dev::mma16816<false>(st.o[g][2 * h + 1], xs & kLow, xs & kHigh, ys & kLow, ys & kHigh, b0,
                             b1);
      }
    }
  }

  __device__ __forceinline__ static void finalize(State& st, float* mo, float* mm, float* ml,
                                                  int lane) {
    const int g8 = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = st.l[i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const float un = 16777216.f / st.rho[i];  // 2^24 / rho
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float z = st.zo[g][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        const float mid = 7.5f * st.as[g][i];
        float* row = mo + (2 * t4 + i) * D + 64 * g + 8 * g8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          row[2 * j] = fmaf(st.o[g][j][i] - mid, un, z);
          row[2 * j + 1] = fmaf(fmaf(st.o[g][j][i + 2], 0.0625f, -mid), un, z);
        }
      }
      if (g8 == 0) {
        mm[2 * t4 + i] = st.m[i];
        ml[2 * t4 + i] = l;
      }
    }
  }
};

template <class Path>
constexpr size_t int4_smem_for(int part_blocks) {
  return 1024 + static_cast<size_t>(Path::kS) * Path::kStageBytes + Path::kS * 8 +
         static_cast<size_t>(part_blocks) * 4 + 16;
}

template <class Path>
__global__ void __launch_bounds__(kWarps * 32) decode_int4_kernel(const DecodeParams p) {
  using namespace dev;
  constexpr int S = Path::kS;
  constexpr int kCB = Path::kCodeBytes, kPB = Path::kPairBytes, kSB = Path::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  DecodeSmem sm;
  sm.stages = align1024(smem_raw);
  sm.scales = nullptr;
  sm.bars = reinterpret_cast<uint64_t*>(sm.stages + S * kSB);
  sm.tbl = reinterpret_cast<int32_t*>(sm.bars + S);
  __shared__ int cta_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  DecodeCta c;
  bool any_bad = false;
  if (!decode_prologue<Path>(p, sm, c, &any_bad, [&] {
        cta_flag = 0;
#pragma unroll
        for (int s = 0; s < S; ++s) mbar_init(smem_addr(sm.bars + s), 1);
      }))
    return;

  // lanes 0-3 of the warp: fetch the warp's j-th block, one copy each
  const uint8_t* src = static_cast<const uint8_t*>(
      lane == 0 ? p.k_pool : lane == 1 ? p.v_pool : lane == 2 ? p.k_sz : p.v_sz);
  const uint32_t bytes = lane < 2 ? kCB : kPB;
  const uint32_t at = lane < 2 ? lane * kCB : 2 * kCB + (lane - 2) * kPB;
  auto issue = [&](int j) {
    const int stage = warp * kInt4Stages + (j % kInt4Stages);
    const uint32_t bar = smem_addr(sm.bars + stage);
    const size_t tile = static_cast<size_t>(sm.tbl[warp + j * kWarps]) * p.num_kv_heads + c.kvh;
    if (lane == 0) mbar_arrive_expect_tx(bar, kSB);
    __syncwarp();
    if (lane < 4) bulk_load(smem_addr(sm.stages + stage * kSB) + at, src + tile * bytes, bytes, bar);
  };

  typename Path::State st;
  bool ok = !any_bad;
  if (ok) {
    Path::init(st, p, c.b, c.head0, c.nheads, lane);
    const int my_blocks = c.nb > warp ? (c.nb - warp + kWarps - 1) / kWarps : 0;
    const int prologue = my_blocks < kInt4Stages ? my_blocks : kInt4Stages;
    for (int j = 0; j < prologue; ++j) issue(j);
    int issued = prologue;
    int j = 0;
    for (; j < my_blocks; ++j) {
      const int stage = warp * kInt4Stages + (j % kInt4Stages);
      const bool landed = mbar_wait_bounded(smem_addr(sm.bars + stage), (j / kInt4Stages) & 1);
      if (!__all_sync(0xffffffffu, landed)) {
        ok = false;
        break;
      }
      const int i = warp + j * kWarps;
      const int valid = (c.last_part && i == c.nb - 1) ? c.tail_valid : kBlockSize;
      Path::consume(st, sm.stages + stage * kSB, valid, lane);
      __syncwarp();
      if (j + kInt4Stages < my_blocks) {
        fence_proxy_async_smem();
        issue(j + kInt4Stages);
        ++issued;
      }
    }
    if (!ok) {
      // A transfer did not land in time: wait (bounded) for this warp's copies
      // still in flight so no copy outlives the CTA, then report.
      if (lane == 0) {
        for (int jj = j; jj < issued; ++jj) {
          const int stage = warp * kInt4Stages + (jj % kInt4Stages);
          mbar_wait_bounded(smem_addr(sm.bars + stage), (jj / kInt4Stages) & 1);
        }
        set_status(p.status, kErrTimeout);
        atomicExch(&cta_flag, 1);
      }
    }
  } else if (threadIdx.x == 0) {
    set_status(p.status, kErrBadBlock);
  }

  launch_dependents();
  __syncthreads();
  decode_epilogue<Path>(p, sm, c, st, any_bad || cta_flag != 0);
}

template <class Path>
cudaError_t launch_int4(const DecodeParams& p, int grid_x, cudaStream_t s) {
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&decode_int4_kernel<Path>),
                                         int4_smem_for<Path>(kMaxPartBlocks));
  if (e != cudaSuccess) return e;
  const dim3 grid(grid_x, p.num_kv_heads * p.qgroups, p.batch);
  return launch_pdl(decode_int4_kernel<Path>, grid, dim3(kWarps * 32),
                    int4_smem_for<Path>(p.part_blocks), s, p);
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams& p, int grid_x, cudaStream_t s) {
  const bool bf = p.q_bf16 != 0;
  if (!bf && p.head_dim == 64) return launch_int4<Int4Path<false, 64>>(p, grid_x, s);
  if (!bf && p.head_dim == 128) return launch_int4<Int4Path<false, 128>>(p, grid_x, s);
  if (bf && p.head_dim == 64) return launch_int4<Int4Path<true, 64>>(p, grid_x, s);
  if (bf && p.head_dim == 128) return launch_int4<Int4Path<true, 128>>(p, grid_x, s);
  return cudaErrorInvalidValue;
}

}  // namespace kvp
