// kvp_decode_int4.cu -- decode attention over 4-bit pools.
//
// A K or V row of a (token, kv head) is D codes c in 0..15, two to a byte, with
// one 16-bit (s, z) pair per group of 64 elements; element d stands for
// s_g c_d + z_g.  For request b and query head h,
//   u_t = scale log2(e) [ sum_g s_tg (sum_{d in g} q_d c_td) + z_tg Q_g ],
//         Q_g = sum_{d in g} q_d,
//   out_d = sum_t p_t (s_tg c_td + z_tg) / sum_t p_t,   p_t = 2^(u_t - m).
// A CTA walks blocks of one kv head for up to 8 of its query heads: each of its
// 4 warps (its only one where there are many short runs) streams its own 16-token
// blocks, a few at a time, through a ring of stages, and the warps' states are
// merged at the end of a context.  Which blocks a CTA walks: a whole context
// where tables are short, else a piece of all contexts together (see Walk), or a
// partition of the size the caller asks for.
//
// A block is 2 (8 D + 32 D / 64) bytes = 2304 at D = 128, little over half of
// an INT8 block, while a warp has the same 32 D codes to widen: unlike the 8-bit
// decodes the kernel fills over half of the issue slots at HBM's pace, so
// everything here saves instructions (263 a block, a run's start and end among
// them).  Measured, D = 128: 57 contexts of 9200 tokens, 8 kv heads, 103 us (0.87 of
// the measured copy bandwidth), 32 of 4096 with 32 kv heads 111 us (0.80), 64 of 512
// to 8192 67 us (0.65: a start of about 6 us, a refill of the ring at every run, the
// merge's 3 us); its ring alone, without the arithmetic, takes 91 us of the 103.
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
//   * V's s goes into the weight, a_t = P_t s_t with P_t = 2^(u_t - r), rounded
//     to fp16 (2^-12 relative on average, independent from token to token).  The
//     reference r is not the maximum: it is set so that the largest a of a block
//     lies in [8, 16) and moved only when an a passes 4096, so a block costs
//     neither a maximum over its tokens nor a rescale.  Weights 2^-28 of the
//     largest are the smallest that count, as for any fp16 weight.
//   * That ties r to the size of V, which the sums of P and P z bear only so far:
//     fp16 scales (of the weights that count) from 2^-21 to 2^28, bf16 from 2^-23 to
//     2^18, both groups of a row within 2^6 of one another.  A run that meets other
//     values goes on in a loop of its own (any_size), whose r follows the scores
//     alone and whose a has a factor for each group: V of any size, 57 contexts of
//     9200 tokens 115 us instead of 103.
//   * A product with ones gives sum_t a_t of the rounded weights; subtracting
//     7.5 times it centres the codes, so that the rounding of a is weighted by
//     c - 7.5 and not by c.  (The ones are 1.0: with the subnormal 2^-24 in
//     their place the sum came out 1e-6 too small, as if products were cut off
//     where a normal operand's would be, and that is 5e-4 of the centred output
//     at 4096 tokens per warp.)
//   * The sums stay in the tensor core's accumulators, which truncate: every
//     product takes up to a step of its size off a sum, always towards zero, and
//     over a long context that adds up.  So every 8 steps the centre is taken out
//     of the sums twice over: they go to the other side of zero and come back,
//     and what truncation takes on one side it gives on the other.  (The first
//     step's sums go to -4 times themselves, half of what 8 steps add.)  Against
//     float64, root mean square over the output, fp16, four contexts of 131072
//     tokens: 3.07e-4, of which the output's own rounding is 2.1e-4 and that of a
//     the same again; 3.2e-4 with sums taken back to zero only, and 4.4e-4
//     against 3.5e-4 for a million tokens.  (The rest of a in a second product
//     would be 8 more tensor instructions a block to the 18.)
//   * z's part, sum_t P_t (z_t + 7.5 s_t), is float32 on the lanes.
//   * Blocks come by cp.async, 16 bytes per lane (5 instructions a block at
//     D = 128 where an elected lane's bulk copies, barriers and fences took 64),
//     each warp through a ring of its own that needs no barrier at all.
//   * The matrix loads (ldmatrix) bring a group's 64 codes of 16 tokens in one
//     instruction, K as it lies and V transposed: for V that also sets the codes
//     of two tokens side by side as the product wants them.
#include "kvp_decode.cuh"
#include "kvp_serve.h"

namespace kvp {
namespace {

constexpr int kBuf = 2;       // steps per warp: one in use, one on the way
constexpr int kCentre = 8;    // steps between two centrings of the sums
constexpr int kTable = 512;   // table entries of a segment
constexpr int kSms = 152;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  const __half2 r =
      __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Byte that 16-byte piece c of token row r takes in a block's code tile: the
// pieces of a row change places so that one piece of 8 rows lies in 8 different
// groups of banks (a matrix load reads just that).
template <int D>
__device__ __forceinline__ int code_piece(int r, int c) {
  const int swap = D == 128 ? (r >> 1) & 3 : (r >> 2) & 1;
  return r * (D / 2) + ((c ^ swap) << 4);
}

template <bool kBf16, int D>
struct Int4Path {
  static constexpr int kD = D;
  static constexpr int kHeads = 8;
  static constexpr int kCtas = int4_ctas_per_sm(D);
  // Blocks a warp takes at a time: as many as the registers hold, for every
  // product and table look-up waits on few others (D = 128, 32 x 32 heads of 4096
  // tokens: one block 121 us, two 110, three 114, spilling; D = 64, four contexts
  // of 131072: two blocks 69 us, three 66, four 66, spilling).
  static constexpr int kStep = D == 128 ? 2 : 3;
  static constexpr int kStages = kStep * kBuf;  // blocks
  static constexpr int kGroups = D / 64;
  static constexpr int kCodeBytes = 16 * D / 2;        // K or V codes of a block
  static constexpr int kPairBytes = 16 * kGroups * 4;  // their (s, z) pairs
  static constexpr int kStageBytes = 2 * (kCodeBytes + kPairBytes);
  static_assert(kStageBytes % 128 == 0, "stages stay aligned for 16-byte copies");

  static constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;  // code pairs of a word
  static constexpr uint32_t kOnes = 0x3c003c00u;

  struct State {
    float o[kGroups][4][4];      // 2^-24 sum a c (0, 1) and 2^-20 sum a c (2, 3), centred
                                 // but for the a in `as`
    float as[kGroups][4];        // sum a less what was taken out, in every row
    float zo[kGroups][2];        // sum P (z + 7.5 s), this lane's tokens
    float qz[kGroups][2];        // scale log2(e) Q_g
    float f[2];                  // scale log2(e) 2^20 / kappa
    float r[2], l[2];            // reference and sum of P (this lane's tokens)
  };

  // Power of two that takes x > 0 into [2^k, 2^(k+1)), 2^126 at most.
  __device__ __forceinline__ static float pow2_to(float x, int k) {
    const int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
    const int up = min(126, max(-126, k - e));
    return __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
  }

  // This lane's 16 elements per group of query head g8: 64 g + 32 w + 8 t4 ...
  struct Query {
    uint4 raw[kGroups][2];
  };

  __device__ __forceinline__ static void load_query(Query& x, const Int4DecodeParams& p, int b,
                                                    int head0, int nheads, int lane) {
    const int g8 = lane >> 2, t4 = lane & 3;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                        (static_cast<size_t>(b) * p.num_q_heads + head0 + g8) * D;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        x.raw[g][w] = make_uint4(0u, 0u, 0u, 0u);
        if (g8 < nheads)
          x.raw[g][w] = *reinterpret_cast<const uint4*>(q + 64 * g + 32 * w + 8 * t4);
      }
    }
  }

  // A lane's sum of P stays below this, so that no sum of P z over lanes, warps and
  // pieces passes the largest value: bf16 zeros have float32's range, for fp16 ones
  // there is room.
  static constexpr float kMostWeight = kBf16 ? 0x1p-14f : 0x1p60f;
  // P is that small with bf16 pairs because s comes 2^48 times larger.
  static constexpr int kLiftBy = 48;
  static constexpr float kLift = kBf16 ? static_cast<float>(1ll << kLiftBy) : 1.f;

  // The query operand of the K product lives in shared memory, a copy per warp:
  // for each group and pair of k-steps 4 words per lane.  (In registers it took
  // the step loop over the 168 that three CTAs leave.)
  static constexpr int kQueryBytes = kGroups * 2 * 32 * 16;
  // ... and behind it the factors E of the warp's sums (see any_size), one for each
  // group and head.
  static constexpr int kWarpBytes = kQueryBytes + kGroups * 8 * 4;
  __device__ __forceinline__ static float* factors(uint4* qs, int g, int i, int lane) {
    return reinterpret_cast<float*>(qs + kQueryBytes / 16) + 8 * g + 2 * (lane & 3) + i;
  }

  __device__ __forceinline__ static void init(State& st, const Query& x, float scale_log2,
                                              uint4* qs, int lane) {
    const int t4 = lane & 3;
    float big = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t r[4] = {x.raw[g][w].x, x.raw[g][w].y, x.raw[g][w].z, x.raw[g][w].w};
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
    float qsum[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      qsum[g] = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t r[4] = {x.raw[g][w].x, x.raw[g][w].y, x.raw[g][w].z, x.raw[g][w].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = dev::unpack2<kBf16>(r[i]);
          v[2 * i] = y.x;
          v[2 * i + 1] = y.y;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          qsum[g] += v[e];
          v[e] *= kappa;
        }
        // the word's code pairs are (0, 4), 16 (1, 5), (2, 6), 16 (3, 7)
        qs[(2 * g + w) * 32 + lane] =
            make_uint4(dev::pack2<false>(16.f * v[0], 16.f * v[4]), dev::pack2<false>(v[1], v[5]),
                       dev::pack2<false>(16.f * v[2], 16.f * v[6]), dev::pack2<false>(v[3], v[7]));
      }
      qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], 1);
      qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], 2);
    }
    // this lane's score columns are heads 2 t4 and 2 t4 + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = 4 * (2 * t4 + i);
      st.f[i] = scale_log2 * 1048576.f / __shfl_sync(0xffffffffu, kappa, src);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        st.qz[g][i] = scale_log2 * __shfl_sync(0xffffffffu, qsum[g], src);
        st.zo[g][i] = 0.f;
      }
      st.r[i] = 0.f;
      st.l[i] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      st.as[g][0] = st.as[g][1] = st.as[g][2] = st.as[g][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) st.o[g][j][i] = 0.f;
      }
    }
  }

  // (s, z) pairs of one token, one per group.  kLifted: s kLift, by an addition to the
  // exponent in the instruction that widens a bf16 (0 becomes 2^(48 - 127), and s from
  // 2^(128 - 48) on an infinity, a NaN or negative: too_large and reference see those).
  template <bool kLifted>
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
      s[g] = kLifted && kBf16 ? __uint_as_float(w[g] * 65536u + (uint32_t{kLiftBy} << 23)) : x.x;
      z[g] = x.y;
    }
  }

  // The row this lane addresses when the warp loads a group's codes of a tile as
  // four 8 x 16-byte matrices: tokens 0-7 and 8-15 of its first piece, then of
  // its second.
  __device__ __forceinline__ static uint32_t matrix_at(int g, int lane) {
    return code_piece<D>(lane & 15, 2 * g + (lane >> 4));
  }

  // Scores of a step's blocks relative to the present reference (v = u - r) of
  // this lane's rows g8, g8 + 8 and heads 2 t4, 2 t4 + 1, and V's pairs of those
  // tokens.  kTail: only the first `valid` tokens count (other slots may hold
  // anything).
  template <bool kTail, bool kLifted>
  __device__ __forceinline__ static void scores(const State& st, const uint4* qs,
                                                const uint8_t* tile, int valid, int lane,
                                                float (&v)[kStep][4], float (&s0)[kStep][kGroups],
                                                float (&z0)[kStep][kGroups],
                                                float (&s1)[kStep][kGroups],
                                                float (&z1)[kStep][kGroups]) {
    const int tok0 = lane >> 2, tok1 = tok0 + 8;
    float acc[kStep][kGroups][4];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      // of tokens g8 and g8 + 8: elements 64 g + 32 w + 8 t4 ...
      uint32_t wa[kStep][2], wb[kStep][2];
#pragma unroll
      for (int b = 0; b < kStep; ++b) {
        dev::ldsm_x4(dev::smem_addr(tile + b * kStageBytes) + matrix_at(g, lane), wa[b][0], wb[b][0],
                     wa[b][1], wb[b][1]);
        acc[b][g][0] = acc[b][g][1] = acc[b][g][2] = acc[b][g][3] = 0.f;
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4 q = qs[(2 * g + w) * 32 + lane];
#pragma unroll
        for (int b = 0; b < kStep; ++b) {
          const uint32_t x = wa[b][w], y = wb[b][w], xs = x >> 8, ys = y >> 8;
          dev::mma16816<false>(acc[b][g], x & kLow, y & kLow, x & kHigh, y & kHigh, q.x, q.y);
          dev::mma16816<false>(acc[b][g], xs & kLow, ys & kLow, xs & kHigh, ys & kHigh, q.z, q.w);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kStep; ++b) {
      const uint8_t* pairs = tile + b * kStageBytes + 2 * kCodeBytes;
      float ks0[kGroups], kz0[kGroups], ks1[kGroups], kz1[kGroups];
      load_pairs<false>(pairs, tok0, ks0, kz0);
      load_pairs<false>(pairs, tok1, ks1, kz1);
      float us[4] = {0.f, 0.f, 0.f, 0.f};
      v[b][0] = v[b][2] = -st.r[0];
      v[b][1] = v[b][3] = -st.r[1];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        us[0] = fmaf(ks0[g], acc[b][g][0], us[0]);
        us[1] = fmaf(ks0[g], acc[b][g][1], us[1]);
        us[2] = fmaf(ks1[g], acc[b][g][2], us[2]);
        us[3] = fmaf(ks1[g], acc[b][g][3], us[3]);
        v[b][0] = fmaf(kz0[g], st.qz[g][0], v[b][0]);
        v[b][1] = fmaf(kz0[g], st.qz[g][1], v[b][1]);
        v[b][2] = fmaf(kz1[g], st.qz[g][0], v[b][2]);
        v[b][3] = fmaf(kz1[g], st.qz[g][1], v[b][3]);
      }
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        if constexpr (D == 64) {  // (as add_weights)
          const float2 x = dev::f2unpack(dev::ffma2(dev::f2pack(us[i], us[i + 1]),
                                                    dev::f2pack(st.f[0], st.f[1]),
                                                    dev::f2pack(v[b][i], v[b][i + 1])));
          v[b][i] = x.x;
          v[b][i + 1] = x.y;
        } else {
          v[b][i] = fmaf(us[i], st.f[0], v[b][i]);
          v[b][i + 1] = fmaf(us[i + 1], st.f[1], v[b][i + 1]);
        }
      }
      load_pairs<kLifted>(pairs + kPairBytes, tok0, s0[b], z0[b]);
      load_pairs<kLifted>(pairs + kPairBytes, tok1, s1[b], z1[b]);
      if constexpr (kTail) {
        const bool in0 = tok0 < valid - 16 * b, in1 = tok1 < valid - 16 * b;
        v[b][0] = in0 ? v[b][0] : -INFINITY;
        v[b][1] = in0 ? v[b][1] : -INFINITY;
        v[b][2] = in1 ? v[b][2] : -INFINITY;
        v[b][3] = in1 ? v[b][3] : -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          s0[b][g] = in0 ? s0[b][g] : 0.f;
          z0[b][g] = in0 ? z0[b][g] : 0.f;
          s1[b][g] = in1 ? s1[b][g] : 0.f;
          z1[b][g] = in1 ? z1[b][g] : 0.f;
        }
      }
    }
  }

  // Sums of P, a block further.  D = 64 adds two heads at a time, and takes the last
  // product of their scores so: 32 x 32 heads of 4096 72.3 -> 70.3 us (D = 128 gains
  // nothing, 112.4 and 112.3).
  __device__ __forceinline__ static void add_weights(float& l0, float& l1, const float (&pr)[4]) {
    if constexpr (D == 64) {
      const float2 l = dev::f2unpack(dev::fadd2(
          dev::f2pack(l0, l1), dev::fadd2(dev::f2pack(pr[0], pr[1]), dev::f2pack(pr[2], pr[3]))));
      l0 = l.x;
      l1 = l.y;
    } else {
      l0 += pr[0] + pr[2];
      l1 += pr[1] + pr[3];
    }
  }

  // A step's sums with z (mid: 7.5, for the s that were loaded).
  __device__ __forceinline__ static void add_zeros(State& st, const float (&pr)[kStep][4],
                                                   const float (&s0)[kStep][kGroups],
                                                   const float (&z0)[kStep][kGroups],
                                                   const float (&s1)[kStep][kGroups],
                                                   const float (&z1)[kStep][kGroups], float mid) {
#pragma unroll
    for (int b = 0; b < kStep; ++b) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float c0 = fmaf(mid, s0[b][g], z0[b][g]), c1 = fmaf(mid, s1[b][g], z1[b][g]);
        st.zo[g][0] = fmaf(pr[b][0], c0, fmaf(pr[b][2], c1, st.zo[g][0]));
        st.zo[g][1] = fmaf(pr[b][1], c0, fmaf(pr[b][3], c1, st.zo[g][1]));
      }
    }
  }

  // Whether an a is above 4096 (0x6c00) or an infinity; in bf16 or negative or NaN
  // (see load_pairs), by a comparison of integers.
  __device__ __forceinline__ static bool too_large(const uint32_t (&ap)[kStep][kGroups][2]) {
    uint32_t top = 0u;
#pragma unroll
    for (int b = 0; b < kStep; ++b) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if constexpr (kBf16)
          top = __vimax3_u16x2(top, ap[b][g][0], ap[b][g][1]);
        else
          top = max_half2(top, max_half2(ap[b][g][0], ap[b][g][1]));
      }
    }
    const uint32_t above = (top & 0x7fff7fffu) + 0x13ff13ffu;
    return ((kBf16 ? above | top : above) & 0x80008000u) != 0u;
  }

  // A step's blocks, kStageBytes apart (each: K codes, V codes, K pairs, V pairs).
  // kTail: only the first `valid` of their tokens count.  first: the warp's first
  // step, which sets the reference.  False (for the whole warp) where the sizes of the
  // values are not for this path: then the step has not been taken.
  template <bool kTail>
  __device__ __forceinline__ static bool consume(State& st, const uint4* qs, const uint8_t* tile,
                                                 int valid, bool first, int lane) {
    float v[kStep][4], s0[kStep][kGroups], z0[kStep][kGroups], s1[kStep][kGroups], z1[kStep][kGroups];
    scores<kTail, true>(st, qs, tile, valid, lane, v, s0, z0, s1, z1);

    // ---- weights
    float pr[kStep][4], l0, l1;
    uint32_t ap[kStep][kGroups][2];  // a of rows g8 and g8 + 8, two heads each
    auto weights = [&] {
      l0 = st.l[0];
      l1 = st.l[1];
#pragma unroll
      for (int b = 0; b < kStep; ++b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[b][i] = dev::ex2_approx(v[b][i]);
        add_weights(l0, l1, pr[b]);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          ap[b][g][0] = dev::pack2<false>(pr[b][0] * s0[b][g], pr[b][1] * s0[b][g]);
          ap[b][g][1] = dev::pack2<false>(pr[b][2] * s1[b][g], pr[b][3] * s1[b][g]);
        }
      }
    };
    weights();
    const bool move = too_large(ap) || !(fmaxf(l0, l1) <= kMostWeight);
    if (__any_sync(0xffffffffu, move || first)) {
      if (!reference(st, v, s0, s1, first)) return false;
      weights();
    }
    st.l[0] = l0;
    st.l[1] = l1;
    add_zeros(st, pr, s0, z0, s1, z1, 7.5f / kLift);
    add_values(st, ap, tile, lane);
    return true;
  }

  // The blocks' products of a and V's codes, straight into the sums.
  __device__ __forceinline__ static void add_values(State& st,
                                                    const uint32_t (&ap)[kStep][kGroups][2],
                                                    const uint8_t* tile, int lane) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int b = 0; b < kStep; ++b) {
        const uint32_t b0 = dev::movm_t(ap[b][g][0]);
        const uint32_t b1 = dev::movm_t(ap[b][g][1]);
        // transposed, a lane gets 4 codes, 64 g + 32 h + 4 g8 ..., of tokens 2 t4
        // and 2 t4 + 1 (x), 2 t4 + 8 and 2 t4 + 9 (y): the product's operand pairs
        uint32_t x[2], y[2];
        dev::ldsm_x4_t(dev::smem_addr(tile + b * kStageBytes + kCodeBytes) + matrix_at(g, lane), x[0],
                       y[0], x[1], y[1]);
        dev::mma16816<false>(st.as[g], kOnes, kOnes, kOnes, kOnes, b0, b1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t xs = x[h] >> 8, ys = y[h] >> 8;
          dev::mma16816<false>(st.o[g][2 * h], x[h] & kLow, x[h] & kHigh, y[h] & kLow, y[h] & kHigh,
                               b0, b1);
          dev::mma16816<false>(st.o[g][2 * h + 1], xs & kLow, xs & kHigh, ys & kLow, ys & kHigh, b0,
                               b1);
        }
      }
    }
  }

  // Take the centre out of the sums, and `back` times more of it (see above).
  __device__ __forceinline__ static void centre(State& st, float back) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float even = -7.5f * 5.9604645e-8f * (1.f + back) * st.as[g][i], odd = 16.f * even;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          st.o[g][j][i] += even;
          st.o[g][j][i + 2] += odd;
        }
        st.as[g][i] = st.as[g][i + 2] = -back * st.as[g][i];
      }
    }
  }

  // Exponent of x >= 0 (-127 for 0 and below the normal range).
  __device__ __forceinline__ static int exponent(float x) {
    return static_cast<int>(__float_as_uint(x) >> 23) - 127;
  }
  // 2^x, 0 below the normal range.
  __device__ __forceinline__ static float pow2(int x) {
    return x < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(x + 127) << 23);
  }
  // Largest x over the warp's rows, for this lane's head.
  __device__ __forceinline__ static float over_rows(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  }
  // Largest score, rounded up, and largest P s of each group for that reference; v
  // becomes the scores themselves.
  __device__ __forceinline__ static float sizes(const State& st, float (&v)[kStep][4],
                                                const float (&s0)[kStep][kGroups],
                                                const float (&s1)[kStep][kGroups], int i,
                                                float (&big)[kGroups]) {
    float mx = -1e30f;
#pragma unroll
    for (int b = 0; b < kStep; ++b) {
      v[b][i] += st.r[i];
      v[b][i + 2] += st.r[i];
      mx = fmaxf(mx, fmaxf(v[b][i], v[b][i + 2]));
    }
    mx = ceilf(over_rows(mx));
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      big[g] = 0.f;
#pragma unroll
      for (int b = 0; b < kStep; ++b)
        big[g] = fmaxf(big[g], fmaxf(dev::ex2_approx(v[b][i] - mx) * s0[b][g],
                                     dev::ex2_approx(v[b][i + 2] - mx) * s1[b][g]));
      big[g] = over_rows(big[g]);
    }
    return mx;
  }

  // Rare: move the reference so that the step's largest a lies in [8, 16), never
  // down.  v is relative to the old one on entry, to the new one on exit.  False, and
  // nothing has changed, where the values are outside the sizes above.
  __device__ __forceinline__ static bool reference(State& st, float (&v)[kStep][4],
                                                   const float (&s0)[kStep][kGroups],
                                                   const float (&s1)[kStep][kGroups], bool first) {
    float now[2];
    bool fits = true;
#pragma unroll
    for (int b = 0; b < kStep; ++b) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) fits = fits && s0[b][g] >= 0.f && s1[b][g] >= 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float big[kGroups];
      const float mx = sizes(st, v, s0, s1, i, big);
      const float top = kGroups == 2 ? fmaxf(big[0], big[1]) : big[0];
      const float low = kGroups == 2 ? fminf(big[0], big[1]) : big[0];
      fits = fits && top >= (kBf16 ? 0x1p25f : 0x1p-21f) && top < (kBf16 ? 0x1p66f : 0x1p28f) &&
             low >= 0x1p-6f * top && st.l[i] <= 0.25f * kMostWeight;
      now[i] = mx + static_cast<float>(exponent(top) - 3);
      if (!first) now[i] = fmaxf(st.r[i], now[i]);
    }
    if (!__all_sync(0xffffffffu, fits)) return false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float al = first ? 0.f : dev::ex2_approx(st.r[i] - now[i]);
      st.r[i] = now[i];
#pragma unroll
      for (int b = 0; b < kStep; ++b) {
        v[b][i] -= now[i];
        v[b][i + 2] -= now[i];
      }
      st.l[i] *= al;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        st.zo[g][i] *= al;
        st.as[g][i] *= al;
        st.as[g][i + 2] *= al;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          st.o[g][j][i] *= al;
          st.o[g][j][i + 2] *= al;
        }
      }
    }
    return true;
  }

  // A step of values of any size.  The reference follows the scores alone: P is 2^-20
  // at most where it is set, and moves on when a lane's sum passes 2^-14.  a = P s E
  // has a power of two E for each head and group that takes the step's largest a of
  // that group into [8, 16).  Neither r nor 2^r / E, what an a of 1 stands for, ever
  // goes down.  So sums of P lose only what float32 does, sums of P (z + 7.5 s) never
  // pass the largest value, and what an a loses is small beside its own group.
  // enter: the steps before were `consume`'s.
  __device__ __forceinline__ static void any_size(State& st, uint4* qs, const uint8_t* tile,
                                                  int valid, bool first, bool enter, int lane) {
    float v[kStep][4], s0[kStep][kGroups], z0[kStep][kGroups], s1[kStep][kGroups], z1[kStep][kGroups];
    scores<true, false>(st, qs, tile, valid, lane, v, s0, z0, s1, z1);
    float pr[kStep][4], l0, l1;
    uint32_t ap[kStep][kGroups][2];
    auto weights = [&] {
      l0 = st.l[0];
      l1 = st.l[1];
#pragma unroll
      for (int b = 0; b < kStep; ++b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[b][i] = dev::ex2_approx(v[b][i]);
        add_weights(l0, l1, pr[b]);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float e0 = *factors(qs, g, 0, lane), e1 = *factors(qs, g, 1, lane);
          ap[b][g][0] = dev::pack2<false>(pr[b][0] * e0 * s0[b][g], pr[b][1] * e1 * s0[b][g]);
          ap[b][g][1] = dev::pack2<false>(pr[b][2] * e0 * s1[b][g], pr[b][3] * e1 * s1[b][g]);
        }
      }
    };
    if (enter) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *factors(qs, g, i, lane) = kLift;
      }
      __syncwarp();
    }
    weights();
    const bool move = first || enter || too_large(ap) || fmaxf(l0, l1) > 0x1p-14f;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float big[kGroups];
        const float mx = sizes(st, v, s0, s1, i, big), sum = over_rows(st.l[i]);
        float now = mx + 20.f;
        if (!first) now = fmaxf(now, st.r[i] + static_cast<float>(max(exponent(sum) + 20, 0)));
        const int up = first ? 0 : static_cast<int>(fminf(now - st.r[i], 400.f));
        const int past = static_cast<int>(fminf(now - mx, 400.f));
        const float al = pow2(-up);
        st.r[i] = now;
        st.l[i] *= al;
#pragma unroll
        for (int b = 0; b < kStep; ++b) {
          v[b][i] -= now;
          v[b][i + 2] -= now;
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          float* e = factors(qs, g, i, lane);
          const int was = exponent(*e);
          // (without a row with a scale: as large as it gets)
          const int want = big[g] > 0.f ? min(126, 3 + past - exponent(big[g])) : 126;
          const int to = max(-126, first ? want : min(want, was + up));
          const float keep = first ? 0.f : pow2(to - was - up);
          __syncwarp();  // the old factor is read
          *e = pow2(to);
          st.zo[g][i] *= al;
          st.as[g][i] *= keep;
          st.as[g][i + 2] *= keep;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            st.o[g][j][i] *= keep;
            st.o[g][j][i + 2] *= keep;
          }
        }
      }
      __syncwarp();
      weights();
    }
    st.l[0] = l0;
    st.l[1] = l1;
    add_zeros(st, pr, s0, z0, s1, z1, 7.5f);
    add_values(st, ap, tile, lane);
  }

  // The warp's state for the merge: per (group, head parity i) and lane, outputs
  // 64 g + 32 h + 4 g8 ... + 3 of head 2 t4 + i, a 16-byte word for each h, at a
  // place of its own for all 32 lanes (no two in a bank).
  static constexpr int kParts = 2 * kGroups;  // (group, parity) pairs
  // It lies in the last step's place of the warp's ring.
  static constexpr int kMergeAt = (kBuf - 1) * kStep * kStageBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static_assert((kParts * 256 + 16) * 4 <= kStep * kStageBytes, "the state fits a step's place");

  // kFactors: the sums have them (see any_size).
  template <bool kFactors>
  __device__ __forceinline__ static void finalize(State& st, uint4* qs, uint8_t* ring, int lane) {
    const int g8 = lane >> 2, t4 = lane & 3;
    float* mine = reinterpret_cast<float*>(ring + kMergeAt);
    float* ml = mine + kParts * 256;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = st.l[i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float z = st.zo[g][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        constexpr float kUnit = kFactors ? 1.f : 1.f / kLift;
        const float mid = 7.5f * kUnit * st.as[g][i];
        const float per = kFactors ? pow2(-exponent(*factors(qs, g, i, lane))) : 1.f;
        auto value = [&](float o, float step) {  // o steps of a code
          const float x = fmaf(o, step * kUnit, -mid);
          return kFactors ? fmaf(x, per, z) : x + z;
        };
        float4* at = reinterpret_cast<float4*>(mine + (2 * g + i) * 256) + lane;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          at[32 * h] = make_float4(value(st.o[g][2 * h][i], 16777216.f),
                                   value(st.o[g][2 * h][i + 2], 1048576.f),
                                   value(st.o[g][2 * h + 1][i], 16777216.f),
                                   value(st.o[g][2 * h + 1][i + 2], 1048576.f));
      }
      if (g8 == 0) {
        ml[2 * t4 + i] = st.r[i];
        ml[8 + 2 * t4 + i] = l;
      }
    }
  }

  // Thread `tid` of the first 32 kParts merges 8 outputs of one head, d ... d + 3
  // and d + 32 ... d + 35: their unnormalised sum, the reference M and the weight
  // L (0 without tokens).
  template <int W>
  __device__ __forceinline__ static void merge8(const uint8_t* rings, int tid, float (&o)[8],
                                                float& M, float& L, int& head, int& d) {
    const int part = tid >> 5, lane = tid & 31;
    head = 2 * (lane & 3) + (part & 1);
    d = 64 * (part >> 1) + 4 * (lane >> 2);
    M = -INFINITY;
    L = 0.f;
    const float* of[W];  // a warp's state
#pragma unroll
    for (int w = 0; w < W; ++w) {
      of[w] = reinterpret_cast<const float*>(rings + w * kRingBytes + kMergeAt);
      if (of[w][kParts * 256 + 8 + head] > 0.f) M = fmaxf(M, of[w][kParts * 256 + head]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float l = of[w][kParts * 256 + 8 + head];
      const float f = l > 0.f ? exp2f(of[w][kParts * 256 + head] - M) : 0.f;
      L = fmaf(f, l, L);
      const float4* at = reinterpret_cast<const float4*>(of[w] + part * 256) + lane;
      const float4 x = at[0], y = at[32];
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(f, v[e], o[e]);
    }
  }
};

// What a CTA walks: segments of up to kTable blocks of one context.  A run (the
// CTA's share of a context) is one segment or several.
enum : int {
  kInit = 1,      // a run's first segment
  kMerge = 2,     // a run's last
  kWhole = 4,     // the run is a whole context: its rows are final
  kStart = 8,     // the run starts a context that later pieces end
  kLater = 16     // not the CTA's first run
};
struct Segment {
  int b, blk0, nb;  // request, its blocks blk0 ... blk0 + nb - 1 (nb = 0: no more)
  int tail;         // valid tokens of the last one
  int flags;
  int runs;         // kStart: pieces the context spans
};

// Where a balanced CTA's runs lie.  The requests' blocks are laid end to end and
// cut into equal pieces, and each (piece, unit) is a CTA, a unit being a kv head
// and a group of its query heads, so that ragged contexts load the SMs evenly: a
// CTA walks the end of one context, whole ones, and the start of another.  The
// CTAs of a piece's units are neighbours and walk the same blocks at the same
// time, which keeps the tiles of a block's kv heads together on their way
// through the DRAM (with the units one after the other in one line, contexts of
// 512 to 8192 tokens and 64 x 8 heads took 99 us instead of the 82 of that time).  Only a piece's
// first and last run can be partial; their states go to the CTA's two workspace
// slots, and the CTA that starts a cut context leaves a note for the merge.
struct Walk {
  long long pos, end, size;  // blocks: next, the piece's end, per piece
  int index;                 // of the piece
  int b, n, nblk, blk0;      // context, its tokens and blocks, the next block
  int left;                  // blocks of the present run
  int flags, runs;
};

__device__ __forceinline__ int blocks_of(const Int4DecodeParams& p, int n) {
  return n <= 0 || (n - 1) / kBlockSize >= p.max_blocks ? 0 : (n - 1) / kBlockSize + 1;
}

// Exclusive prefix sum over the CTA's threads; the whole in *total.
template <class T>
__device__ __forceinline__ T prefix_sum(T mine, T* total) {
  __shared__ T part[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) part[warp] = sum;
  __syncthreads();
  T at = sum - mine;
  *total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += part[w];
    *total += part[w];
  }
  return at;
}

// Sets the walk of piece `index` of `pieces`; false when it has no blocks.
__device__ __forceinline__ bool find_piece(const Int4DecodeParams& p, int index, int pieces,
                                           Walk& walk) {
  const int per = (p.batch + kWarps * 32 - 1) / (kWarps * 32);
  const int b0 = min(p.batch, static_cast<int>(threadIdx.x) * per), b1 = min(p.batch, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += blocks_of(p, p.context_lens[b]);
  long long total;
  long long at = prefix_sum(mine, &total);
  const Cut cut = cut_contexts(total, p.batch, pieces);
  if (cut.aligned) {
    const int size = static_cast<int>(cut.size);
    int runs = 0;
    for (int b = b0; b < b1; ++b) runs += (blocks_of(p, p.context_lens[b]) + size - 1) / size;
    int all;
    int first = prefix_sum(runs, &all);
    if (index >= all) return false;
    if (first <= index && index < first + runs) {
      int b = b0, n;
      while (index >= first + (n = (blocks_of(p, p.context_lens[b]) + size - 1) / size)) {
        first += n;
        ++b;
      }
      walk.b = b;
      walk.n = p.context_lens[b];
      walk.nblk = blocks_of(p, walk.n);
      walk.blk0 = (index - first) * size;
      walk.pos = 0;  // (so that the context's pieces are counted from this one)
      walk.end = min(size, walk.nblk - walk.blk0);
      walk.size = size;
      walk.index = walk.left = walk.flags = walk.runs = 0;
    }
    __syncthreads();
    return true;
  }
  const long long size = cut.size, pos = index * size;
  if (pos >= total) return false;
  if (at <= pos && pos < at + mine) {  // one thread's requests hold the piece's start
    int b = b0, nblk;
    while (pos >= at + (nblk = blocks_of(p, p.context_lens[b]))) {
      at += nblk;
      ++b;
    }
    walk.pos = pos;
    walk.end = min(total, pos + size);
    walk.size = size;
    walk.index = index;
    walk.b = b;
    walk.n = p.context_lens[b];
    walk.nblk = nblk;
    walk.blk0 = static_cast<int>(pos - at);
    walk.left = walk.flags = walk.runs = 0;
  }
  __syncthreads();
  return true;
}

// One thread: the walk's next segment.  `ahead` is the length of the context
// behind walk.b, fetched by the call before.
__device__ __forceinline__ void next_segment(const Int4DecodeParams& p, Walk& walk, Segment& seg,
                                             int& ahead) {
  int flags = walk.flags & ~kInit;
  if (walk.left == 0) {
    if (walk.pos >= walk.end) {
      seg.nb = 0;
      return;
    }
    flags = (flags & kLater) | kInit;
    if (walk.blk0 == walk.nblk) {
      walk.n = ahead;
      walk.nblk = blocks_of(p, ahead);
      ++walk.b;
      while (walk.nblk == 0) {
        walk.n = p.context_lens[++walk.b];
        walk.nblk = blocks_of(p, walk.n);
      }
      walk.blk0 = 0;
      ahead = p.context_lens[min(walk.b + 1, p.batch - 1)];
    }
    walk.left = static_cast<int>(
        min(static_cast<long long>(walk.nblk - walk.blk0), walk.end - walk.pos));
    if (walk.blk0 == 0) {
      if (walk.left == walk.nblk) {
        flags |= kWhole;
      } else {
        flags |= kStart;
        walk.runs = static_cast<int>((walk.pos + walk.nblk - 1) / walk.size) - walk.index + 1;
      }
    }
  }
  seg.b = walk.b;
  seg.blk0 = walk.blk0;
  seg.nb = min(walk.left, kTable);
  seg.runs = walk.runs;
  walk.left -= seg.nb;
  walk.blk0 += seg.nb;
  walk.pos += seg.nb;
  seg.tail = walk.blk0 == walk.nblk ? walk.n - (walk.nblk - 1) * kBlockSize : kBlockSize;
  seg.flags = flags | (walk.left == 0 ? kMerge : 0);
  walk.flags = walk.left == 0 ? kLater : flags;
}

template <class Path, int W>
constexpr size_t int4_smem() {
  return static_cast<size_t>(W) * (Path::kRingBytes + Path::kWarpBytes) +
         2 * kTable * sizeof(int32_t);
}

// part_blocks > 0: grid (partitions, units, requests), one run per CTA.
// part_blocks == 0: balanced, grid units * pieces.
// W: warps, 4 or (short runs, see launch_int4) 1.
template <class Path, int W>
__global__ void __launch_bounds__(W * 32, Path::kCtas * (kWarps / W))
    decode_int4_kernel(const Int4DecodeParams p) {
  constexpr int D = Path::kD, H = Path::kHeads;
  constexpr int kCB = Path::kCodeBytes, kPB = Path::kPairBytes, kSB = Path::kStageBytes;
  constexpr int kPieces = kCB / 16;  // 16-byte pieces of a block's K (or V) codes
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* qs = reinterpret_cast<uint4*>(smem + W * Path::kRingBytes);
  int32_t* tables = reinterpret_cast<int32_t*>(qs + W * (Path::kWarpBytes / 16));
  qs += threadIdx.x / 32 * (Path::kWarpBytes / 16);
  __shared__ Walk walk;
  __shared__ Segment segs[4];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool balanced = W == kWarps && p.part_blocks == 0;
  const int units = p.num_kv_heads * p.qgroups;
  const int unit = balanced ? blockIdx.x % units : blockIdx.y;
  const int kvh = unit / p.qgroups;
  const int head0 = kvh * p.group + unit % p.qgroups * p.heads_per_cta;
  const int nheads = min(p.heads_per_cta, p.group - unit % p.qgroups * p.heads_per_cta);

  dev::grid_dependency_wait();
  if (balanced) {
    // requests without tokens, or with a bad length
    const int pieces = gridDim.x / units, index = blockIdx.x / units;
    for (int b = index; b < p.batch; b += pieces) {
      const int n = p.context_lens[b];
      if (blocks_of(p, n) == 0) {
        zero_rows<D>(p, b, head0, nheads);
        if (n != 0 && threadIdx.x == 0) dev::set_status(p.status, kErrBadBlock);
      }
    }
    if (threadIdx.x == 0) p.notes[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (!find_piece(p, index, pieces, walk)) return;
  } else {
    // The table's slice comes beside the length, entries behind the context
    // included (nothing looks at those): one trip to memory less, 0.5 us of 5.
    const int b = blockIdx.z, blk0 = blockIdx.x * p.part_blocks;
    const int32_t* row = p.block_tables + static_cast<size_t>(b) * p.max_blocks + blk0;
    const int most = min(min(p.part_blocks, kTable), p.max_blocks - blk0);
    for (int i = threadIdx.x; i < most; i += blockDim.x)
      cp_async4(dev::smem_addr(tables) + i * 4, row + i);
    cp_async_commit();
    const int n = p.context_lens[b], nblk = blocks_of(p, n);
    if (nblk == 0 && blk0 == 0) {
      zero_rows<D>(p, b, head0, nheads);
      if (n != 0 && threadIdx.x == 0) dev::set_status(p.status, kErrBadBlock);
    }
    if (blk0 >= nblk) {
      cp_async_wait<0>();
      return;
    }
    if (threadIdx.x == 0) {
      walk.pos = 0;
      walk.end = min(p.part_blocks, nblk - blk0);
      walk.size = 1;
      walk.b = b;
      walk.n = n;
      walk.nblk = nblk;
      walk.blk0 = blk0;
      walk.index = walk.left = walk.flags = walk.runs = 0;
    }
  }
  int ahead = 0;
  if (threadIdx.x == 0) {
    ahead = p.context_lens[min(walk.b + 1, p.batch - 1)];
    next_segment(p, walk, segs[0], ahead);
    next_segment(p, walk, segs[1], ahead);
  }
  __syncthreads();

  // This lane's pieces of a block: K and V codes lane, lane + 32, ..., and one
  // of the pairs' pieces on the first lanes.
  constexpr int kPairPieces = kPB / 16;
  const bool is_v = lane >= kPairPieces;
  uint8_t* ring = smem + warp * Path::kStages * kSB;
  constexpr int kRowPieces = D / 32;
  const uint32_t code_at =
      dev::smem_addr(ring) + code_piece<D>(lane / kRowPieces, lane % kRowPieces);
  const uint32_t pair_at = dev::smem_addr(ring) + 2 * kCB + lane * 16;
  const uint8_t* kc = static_cast<const uint8_t*>(p.k_pool) + lane * 16;
  const uint8_t* vc = static_cast<const uint8_t*>(p.v_pool) + lane * 16;
  const uint8_t* pairs = static_cast<const uint8_t*>(is_v ? p.v_sz : p.k_sz) +
                         (lane - (is_v ? kPairPieces : 0)) * 16;
  constexpr int kStep = Path::kStep, kStride = kStep * W, kStepBytes = kStep * kSB;

  // A segment's slice of the block table comes on chip during the segment
  // before ("踩坑一"), entry by entry; each thread checks those it fetched.
  auto fetch_table = [&](int s) {
    const Segment& seg = segs[s & 3];
    const int32_t* row =
        p.block_tables + static_cast<size_t>(seg.b) * p.max_blocks + seg.blk0;
    const uint32_t to = dev::smem_addr(tables + (s & 1) * kTable);
    for (int i = threadIdx.x; i < seg.nb; i += blockDim.x) cp_async4(to + i * 4, row + i);
  };
  auto table_bad = [&](int s) {
    bool bad = false;
    for (int i = threadIdx.x; i < segs[s & 3].nb; i += blockDim.x) {
      const int id = tables[(s & 1) * kTable + i];
      bad |= id < 0 || id >= p.num_blocks;
    }
    return bad;
  };

  if (balanced) {
    fetch_table(0);
    cp_async_commit();
  }
  cp_async_wait<0>();
  bool bad = __syncthreads_or(table_bad(0)) != 0;  // of this segment's table
  bool run_bad = false;                            // of the run
  typename Path::State st;
  bool plain = true;                               // no any_size in this run (of this warp)
  int done_flags = 0, done_b = 0, done_runs = 0;   // of the segment before
  for (int s = 0;; ++s) {
    const Segment& seg = segs[s & 3];
    const int nb = seg.nb;
    const int32_t* tbl = tables + (s & 1) * kTable;
    auto issue_step = [&](int i, int at) {  // table entries i, i + W ... to byte `at` of the ring
#pragma unroll
      for (int b = 0; b < kStep; ++b) {
        if (i + b * W < nb) {
          const uint32_t tile = static_cast<uint32_t>(tbl[i + b * W]) * p.num_kv_heads + kvh;
          const uint8_t* ks = kc + static_cast<uint64_t>(tile) * kCB;
          const uint8_t* vs = vc + static_cast<uint64_t>(tile) * kCB;
#pragma unroll
          for (int x = 0; x < kPieces; x += 32) {  // (32 pieces on: 8 rows, the same swap)
            cp_async16(code_at + at + b * kSB + x * 16, ks + x * 16);
            cp_async16(code_at + at + b * kSB + kCB + x * 16, vs + x * 16);
          }
          if (lane < 2 * kPairPieces)
            cp_async16(pair_at + at + b * kSB, pairs + static_cast<uint64_t>(tile) * kPB);
        }
      }
      cp_async_commit();
    };
    // ---- the first blocks, the next table and the query set out ...
    typename Path::Query query;
    if (nb > 0) {
      fetch_table(s + 1);
      if (!bad) {
#pragma unroll
        for (int b = 0; b < kBuf - 1; ++b) issue_step(warp + b * kStride, b * kStepBytes);
      } else {
        cp_async_commit();
      }
      if (seg.flags & kInit) Path::load_query(query, p, seg.b, head0, nheads, lane);
    }
    // ---- ... while the run before is merged over the warps
    if (done_flags & kMerge) {
      const size_t row0 = static_cast<size_t>(done_b) * p.num_q_heads + head0;
      for (int t = threadIdx.x; t < 32 * Path::kParts; t += 32 * W) {
        float o[8], M, L;
        int hh, d;
        Path::template merge8<W>(smem, t, o, M, L, hh, d);
        if (run_bad) L = -1.f;  // marks a failed run
        if (hh >= nheads) {
          // (a column without a query head)
        } else if (done_flags & kWhole) {
          const float inv = L > 0.f ? 1.f / L : 0.f;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = L > 0.f ? o[2 * e] * inv : 0.f, y = L > 0.f ? o[2 * e + 1] * inv : 0.f;
            w[e] = p.q_bf16 ? dev::pack2<true>(x, y) : dev::pack2<false>(x, y);
          }
          uint2* to = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row0 + hh) * D + d);
          to[0] = make_uint2(w[0], w[1]);
          to[8] = make_uint2(w[2], w[3]);
        } else {
          const size_t prow =
              balanced ? (static_cast<size_t>(blockIdx.x) * 2 + (done_flags & kLater ? 1 : 0)) * H +
                             hh
                       : (row0 + hh) * p.max_parts + blockIdx.x;
          float4* to = reinterpret_cast<float4*>(p.ws_o + prow * D + d);
          to[0] = make_float4(o[0], o[1], o[2], o[3]);
          to[8] = make_float4(o[4], o[5], o[6], o[7]);
          if (d == 0) *reinterpret_cast<float2*>(p.ws_ml + 2 * prow) = make_float2(M, L);
        }
      }
      if (balanced && (done_flags & kStart) && threadIdx.x == 0)
        p.notes[blockIdx.x] =
            make_int4(static_cast<int>(row0), nheads, done_runs, done_flags & kLater ? 1 : 0);
      run_bad = false;
      __syncthreads();  // the merged states are read: their place is free
    }
    if (nb == 0) break;
    if (threadIdx.x == 0) next_segment(p, walk, segs[(s + 2) & 3], ahead);
    if (seg.flags & kInit) {
      Path::init(st, query, p.scale_log2, qs, lane);
      plain = true;
    }

    // ---- the segment's blocks
    run_bad |= bad;
    if (!bad) {
      const int tail = seg.tail;
      const bool init = (seg.flags & kInit) != 0;
      int i = warp, at = 0, next = (kBuf - 1) * kStepBytes;
      auto fetch = [&] {
        cp_async_wait<kBuf - 2>();
        __syncwarp();  // the step has landed; its predecessor's stages are read
        issue_step(i + (kBuf - 1) * kStride, next);
      };
      auto tokens = [&] {
        const int have = min(kStep, (nb - i + W - 1) / W);
        return kBlockSize * have + (i + (have - 1) * W == nb - 1 ? tail - kBlockSize : 0);
      };
      auto advance = [&](bool first) {
        if (i / kStride % kCentre == 0) Path::centre(st, first ? kCentre / 2 : 1);
        at = at == (kBuf - 1) * kStepBytes ? 0 : at + kStepBytes;
        next = next == (kBuf - 1) * kStepBytes ? 0 : next + kStepBytes;
        i += kStride;
      };
      bool leave = false;
      if (plain) {
        while (i < nb) {
          fetch();
          const int valid = tokens();
          const bool first = init && i == warp;
          leave = !(valid == kBlockSize * kStep
                        ? Path::template consume<false>(st, qs, ring + at, valid, first, lane)
                        : Path::template consume<true>(st, qs, ring + at, valid, first, lane));
          if (leave) break;
          advance(first);
        }
        plain = !leave;
      }
      if (!plain) {
        while (i < nb) {
          if (!leave) fetch();
          const bool first = init && i == warp;
          Path::any_size(st, qs, ring + at, tokens(), first, leave, lane);
          leave = false;
          advance(first);
        }
      }
    } else if (threadIdx.x == 0) {
      dev::set_status(p.status, kErrBadBlock);
    }
    done_flags = seg.flags;
    done_b = seg.b;
    done_runs = seg.runs;
    cp_async_wait<0>();
    if (done_flags & kMerge) {
      __syncwarp();  // the ring is read
      if (plain)
        Path::template finalize<false>(st, qs, ring, lane);
      else
        Path::template finalize<true>(st, qs, ring, lane);
    }
    bad = __syncthreads_or(table_bad(s + 1)) != 0;
  }
  dev::launch_dependents();
}

// One row of a merge: a head's partial states combined run by run.
template <int E>
struct Merge {
  float M, L, o[E];
  bool bad;

  __device__ __forceinline__ void clear() {
    M = -INFINITY;
    L = 0.f;
    bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
  }
  // Workspace row `prow`, this lane's E outputs; L < 0 marks a failed run.
  __device__ __forceinline__ void add(const Int4DecodeParams& p, size_t prow, int lane) {
    const float2 v = *reinterpret_cast<const float2*>(p.ws_ml + 2 * prow);
    float x[E];
    if constexpr (E == 4) {
      const float4 t = *reinterpret_cast<const float4*>(p.ws_o + prow * (32 * E) + lane * E);
      x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
    } else {
      const float2 t = *reinterpret_cast<const float2*>(p.ws_o + prow * (32 * E) + lane * E);
      x[0] = t.x, x[1] = t.y;
    }
    bad |= v.y < 0.f;
    const float mn = fmaxf(M, v.x);
    const float f0 = exp2f(M - mn), f1 = exp2f(v.x - mn);
    M = mn;
    L = fmaf(L, f0, f1 * v.y);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f0, f1 * x[e]);
  }
  template <bool kBf16Out>
  __device__ __forceinline__ void store(const Int4DecodeParams& p, size_t row, int lane) const {
    const float inv = !bad && L > 0.f ? 1.f / L : 0.f;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
      w[e] = inv > 0.f ? dev::pack2<kBf16Out>(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
    uint16_t* out = static_cast<uint16_t*>(p.out) + row * (32 * E) + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(out) = w[0];
  }
};

// Merge of the cut contexts, many of them with few runs each: block i takes the
// one that CTA i started, a warp per head; the rest of it are the first runs
// (slot 0) of the unit's next pieces.  note: first output row, heads, runs, slot
// of the first run.
template <int D, bool kBf16Out>
__global__ void __launch_bounds__(256) merge_noted_kernel(const Int4DecodeParams p) {
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int4 note = p.notes[blockIdx.x];
  const int lane = threadIdx.x & 31, hh = threadIdx.x >> 5;
  if (note.x < 0 || hh >= note.y) return;
  const int units = p.num_kv_heads * p.qgroups;
  Merge<D / 32> m;
  m.clear();
#pragma unroll 4
  for (int i = 0; i < note.z; ++i)
    m.add(p, (static_cast<size_t>(blockIdx.x + i * units) * 2 + (i == 0 ? note.w : 0)) * 8 + hh,
          lane);
  m.template store<kBf16Out>(p, static_cast<size_t>(note.x) + hh, lane);
}

// The same for few contexts with many runs each: a block per (query head of a
// unit, unit, request) and 16 warps over the runs.  The request's place among
// the pieces is found from the lengths again (pieces / 12 of them at most).
template <int D, bool kBf16Out>
__global__ void __launch_bounds__(512) merge_long_kernel(const Int4DecodeParams p, int pieces) {
  constexpr int E = D / 32, W = 16;
  __shared__ __align__(16) float s_o[W][D];
  __shared__ float2 s_ml[W];
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = p.num_kv_heads * p.qgroups;
  const int hh = blockIdx.x, unit = blockIdx.y, b = blockIdx.z;
  const int head = unit % p.qgroups * p.heads_per_cta;
  if (head + hh >= p.group) return;
  long long total = 0, start = 0;
  for (int i = lane; i < p.batch; i += 32) {
    const int nblk = blocks_of(p, p.context_lens[i]);
    total += nblk;
    if (i < b) start += nblk;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    start += __shfl_xor_sync(0xffffffffu, start, o);
  }
  const int nblk = blocks_of(p, p.context_lens[b]);
  const Cut cut = cut_contexts(total, p.batch, pieces);
  int first = static_cast<int>(start / cut.size);
  int runs = static_cast<int>((start + nblk - 1) / cut.size) - first + 1;
  bool later = start % cut.size != 0;  // the first run is its CTA's second
  if (cut.aligned) {
    first = 0;
    for (int i = lane; i < b; i += 32)
      first += static_cast<int>((blocks_of(p, p.context_lens[i]) + cut.size - 1) / cut.size);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
    runs = static_cast<int>((nblk + cut.size - 1) / cut.size);
    later = false;
  }
  if (nblk == 0 || runs <= 1) return;  // its rows are final
  Merge<E> m;
  m.clear();
#pragma unroll 4
  for (int i = warp; i < runs; i += W)
    m.add(p,
          (static_cast<size_t>((first + i) * units + unit) * 2 + (i == 0 && later ? 1 : 0)) * 8 +
              hh,
          lane);
  if (lane == 0) s_ml[warp] = make_float2(m.M, m.bad ? -1.f : m.L);
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = m.o[e];
  __syncthreads();
  if (warp != 0) return;
  // one warp's state per lane
  const float2 v = lane < W ? s_ml[lane] : make_float2(-INFINITY, 0.f);
  m.clear();
  m.bad = __any_sync(0xffffffffu, v.y < 0.f);
  const float M = dev::warp_max(v.y > 0.f ? v.x : -INFINITY);
  const float f = v.y > 0.f ? exp2f(v.x - M) : 0.f;
  m.L = dev::warp_sum(f * v.y);
  const int warps = min(runs, W);
  for (int w = 0; w < warps; ++w) {
    const float fw = __shfl_sync(0xffffffffu, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) m.o[e] = fmaf(fw, s_o[w][lane * E + e], m.o[e]);
  }
  m.template store<kBf16Out>(
      p, static_cast<size_t>(b) * p.num_q_heads + unit / p.qgroups * p.group + head + hh, lane);
}

template <class Path, int W>
cudaError_t launch_warps(const Int4DecodeParams& p, dim3 grid, cudaStream_t s) {
  constexpr size_t smem = int4_smem<Path, W>();
  const cudaError_t e =
      ensure_smem_attr(reinterpret_cast<const void*>(&decode_int4_kernel<Path, W>), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_int4_kernel<Path, W>, grid, dim3(W * 32), smem, s, p);
}

template <class Path>
cudaError_t launch_int4(const Int4DecodeParams& p, int grid_x, cudaStream_t s) {
  if (p.part_blocks == 0) return launch_warps<Path, kWarps>(p, dim3(grid_x), s);
  // More runs than CTAs of four warps fit the GPU, all of them short: a warp for
  // each, which keeps as many warps resident but four times the runs, and no warp
  // waits for another.  One warp and four, head_dim 128, 1024 runs: of 1 block 6.3
  // and 13.2 us, of 16 14.0 and 19.9, of 32 21.6 and 26.2; 2048 runs of 32 43.4
  // and 43.6, of 64 73.7 and 66.5; 512 runs of 16 10.3 and 11.6, of 32 18.1 and
  // 17.4; 256 runs (one wave) of 1 5.3 and 5.2, of 16 9.8 and 6.7.  head_dim 64,
  // runs of 64 blocks: 1024 25.2 and 24.6, 2048 38.6 and 44.2, 4096 64.7 and 81.1.
  // (At its edge the rule costs up to 4%: 512 runs of 32, 1024 of 64.)
  constexpr int kOneWarpBlocks = Path::kD == 64 ? 64 : 32;
  const dim3 grid(grid_x, p.num_kv_heads * p.qgroups, p.batch);
  const long long runs = static_cast<long long>(grid.x) * grid.y * grid.z;
  return runs > kSms * Path::kCtas && p.part_blocks <= kOneWarpBlocks
             ? launch_warps<Path, 1>(p, grid, s)
             : launch_warps<Path, kWarps>(p, grid, s);
}

}  // namespace

cudaError_t launch_decode_int4(const Int4DecodeParams& p, int grid_x, cudaStream_t s) {
  const bool bf = p.q_bf16 != 0;
  if (!bf && p.head_dim == 64) return launch_int4<Int4Path<false, 64>>(p, grid_x, s);
  if (!bf && p.head_dim == 128) return launch_int4<Int4Path<false, 128>>(p, grid_x, s);
  if (bf && p.head_dim == 64) return launch_int4<Int4Path<true, 64>>(p, grid_x, s);
  if (bf && p.head_dim == 128) return launch_int4<Int4Path<true, 128>>(p, grid_x, s);
  return cudaErrorInvalidValue;
}

template <int D, bool kBf16Out>
static cudaError_t launch_merge(const Int4DecodeParams& p, int grid_x, cudaStream_t s) {
  // A context spans pieces / batch runs when all are alike.  A block per head
  // against a warp per head, in us: 114 runs 5 and 23 (4 contexts of one kv head),
  // 57 runs 4 and 11 (one context, 8 kv heads), 14 runs 3.8 and 5.4; 11 runs 6 and
  // 4 (40 contexts of one kv head), 7 runs 6.5 and 4.4, one or two runs 30 and 3.
  const int units = p.num_kv_heads * p.qgroups, pieces = grid_x / units;
  if (pieces >= 12 * p.batch)
    return launch_pdl(merge_long_kernel<D, kBf16Out>, dim3(p.heads_per_cta, units, p.batch),
                      dim3(512), 0, s, p, pieces);
  return launch_pdl(merge_noted_kernel<D, kBf16Out>, dim3(grid_x), dim3(256), 0, s, p);
}

cudaError_t launch_decode_int4_merge(const Int4DecodeParams& p, int grid_x, cudaStream_t s) {
  if (p.head_dim == 64)
    return p.q_bf16 ? launch_merge<64, true>(p, grid_x, s) : launch_merge<64, false>(p, grid_x, s);
  return p.q_bf16 ? launch_merge<128, true>(p, grid_x, s) : launch_merge<128, false>(p, grid_x, s);
}

}  // namespace kvp
