// kvp_matmul_fp8.cu -- matrix product of E4M3 codes with a float32 scale for every 128
// elements of a row of A and for every 128 x 128 elements of B (a weight):
//   out[m, n] = sum_g sa[m, g] sb[n / 128, g] sum_{k in g} a[m, k] b[n, k].
//
// The tensor cores (tcgen05, kind::f8f6f4) form each group's inner sum in TMEM; the
// scales differ from group to group, so every group's sum is read into registers and
// added there in float32: acc = fma(t, sa sb, acc).
//
// Here for few rows of A: the weight's 128 rows are the M side of the instruction (a TMEM
// lane each), kTokens rows of A its N side.  Bound by the weight's bytes, which a ring of
// TMA copies keeps on the way, and by the start and end of a CTA (2.6 us).  Warps: those
// that scale and add, one each that fetches tiles, issues products and stages scales.  The
// products of kBatch groups are handed over at a time, in one of two TMEM buffers: a
// hand-over takes about 1000 cycles (two barriers, the read), more than the bytes of a
// group.  TMEM is read in pieces of 16 rows, whose lanes hold two columns in eight: with a
// row to a lane every lane needs every token's scale, and those broadcasts took as many
// cycles of shared memory as the operands (64 x 10240 x 8192 2.1 us more).  Where few
// tiles meet many SMs, the CTAs of a cluster share a tile's K and add their sums through
// distributed shared memory, in the order of their ranks.  (kvp_matmul_fp8_pair.cu: many
// rows.)
//
// Measured (us, calls back to back; at HBM's measured rate the bytes alone take): 1 x 768 x
// 512 2.9 (0.1), 1 x 10240 x 8192 16.7 (12.6), 64 x 10240 x 8192 19.4 (12.9), 64 x 4096 x 4096
// 7.5 (2.6), 33 x 32000 x 4096 with 32-bit results 24.7 (20.4), 128 x 10240 x 8192 27.7 (13.1).
#include "kvp_matmul.cuh"
#include "kvp_umma.cuh"

namespace kvp {

namespace {

constexpr uint32_t kTileB = kRowsB * 128;    // bytes of a stage's weight tile
constexpr int kSpan = 16;                    // groups whose scales are staged at a time
constexpr int kSpans = 2;
constexpr int kSumPitch = kRowsB + 4;        // floats from one token's sums to the next's

template <int kTokens>
struct Shape {
  static constexpr int kCols = kTokens < 32 ? kTokens : 32;   // tokens of an adding thread
  static constexpr int kAddWarps = 4 * kTokens / kCols;
  static constexpr int kThreads = (kAddWarps + 3) * 32;
  static constexpr uint32_t kTileA = kTokens * 128;
  static constexpr uint32_t kStage = kTileB + kTileA;
  // two CTAs per SM up to 64 tokens
  static constexpr int kCtas = kTokens <= 64 ? 2 : 1;
  static constexpr int kStages = kTokens <= 64 ? 98304 / kStage : 6;
  static constexpr int kBatch = kTokens == 16 ? 8 : kTokens == 32 ? 4 : 2;
  static constexpr int kPitch = kTokens + 4;  // floats from one group's scales to the next's
  static constexpr uint32_t kScaleOff = kStages * kStage;
  static constexpr uint32_t kBarOff = kScaleOff + kSpans * kSpan * kPitch * 4;
  static constexpr uint32_t kSmem = 1024 + kBarOff + (2 * kStages + 5 + 2 * kSpans) * 8 + 16;
  static constexpr uint32_t kTmem = 2 * kBatch * kTokens;
  static_assert(kSmem * kCtas <= (kCtas == 2 ? 226 : 227) * 1024, "shared memory of an SM");
  static_assert(kTmem * kCtas <= 512 && kSpan % kBatch == 0, "TMEM, spans of whole batches");
  static_assert(kStages * kStage >= kTokens * kSumPitch * 4, "the sums lie in the ring");
};

// 16 rows x 8 kReps columns of TMEM: lane l holds columns 8 j + 2 (l % 4) and the next of rows
// l / 4 (registers 4 j, 4 j + 1) and l / 4 + 8 (4 j + 2, 4 j + 3).
template <int kReps>
__device__ __forceinline__ void load_16(uint32_t taddr, uint32_t (&r)[4 * kReps]) {
  static_assert(kReps == 2 || kReps == 4, "repetitions");
  if constexpr (kReps == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
  }
}

// Results of tokens begin, begin + kWarps, ... < end of the tile: a warp takes a token, a lane
// four weight rows; the sums of the CTAs of the cluster (at most kSplits) are added in the
// order of their ranks, kAtOnce tokens at a time.
template <int kAtOnce, int kSplits, int kWarps>
__device__ __forceinline__ void write_sums(const MatmulParams& p, const float* mine, int splits,
                                           int begin, int end, int m0, int n0, bool bad) {
  const int n4 = n0 + 4 * static_cast<int>(threadIdx.x % 32);
  const uint32_t from = dev::smem_addr(mine + 4 * (threadIdx.x % 32));
  const bool whole = n4 + 4 <= p.n && p.out_stride % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(p.out) % (p.out_type == KVP_F32 ? 16 : 8) == 0;
  for (int j0 = begin; j0 < end; j0 += kWarps * kAtOnce) {
    float4 v[kAtOnce][kSplits];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int r = 0; r < kSplits; ++r)
        if (r < splits && j0 + u * kWarps < end) {
          const int at = (j0 + u * kWarps) * kSumPitch;
          if constexpr (kSplits == 1)
            v[u][r] = *reinterpret_cast<const float4*>(mine + at + 4 * (threadIdx.x % 32));
          else
            v[u][r] = mm::load_remote4(mm::at_rank(from + 4 * at, r));
        }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int j = j0 + u * kWarps;
      if (j >= end) continue;
      float4 x = v[u][0];
#pragma unroll
      for (int r = 1; r < kSplits; ++r) {
        if (r < splits) {
          x.x += v[u][r].x;
          x.y += v[u][r].y;
          x.z += v[u][r].z;
          x.w += v[u][r].w;
        }
      }
      if (bad) x = make_float4(0.f, 0.f, 0.f, 0.f);
      const long long at = static_cast<long long>(m0 + j) * p.out_stride + n4;
      if (whole) {
        mm::store_out4(p, at, x);
      } else {
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n4 + i < p.n) mm::store_out(p, at + i, y[i]);
      }
    }
  }
}

// grid.x = (token tile, weight tile, rank of the cluster), the last running fastest.  Tiles
// of one CTA (not kCluster) have a kernel of their own: less code to fetch.
template <int kTokens, bool kCluster>
__global__ void __launch_bounds__(Shape<kTokens>::kThreads, Shape<kTokens>::kCtas)
    matmul_fp8_kernel(const MatmulParams p, int ctas, const __grid_constant__ CUtensorMap ta,
                      const __grid_constant__ CUtensorMap tb) {
  using namespace dev;
  const int splits = kCluster ? ctas : 1;
  using S = Shape<kTokens>;
  constexpr int kAddWarps = S::kAddWarps;
  constexpr uint32_t kInstr = umma::instr_desc_f16(kRowsB, kTokens, false, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(sm + S::kScaleOff);   // [kSpans][kSpan][kPitch]
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBarOff);
  uint64_t* empty = full + S::kStages;
  uint64_t* sums = empty + S::kStages;     // [2] a TMEM buffer holds a batch's sums
  uint64_t* taken = sums + 2;              // [2] they are in registers
  uint64_t* scaled = taken + 2;            // [kSpans] scales are there
  uint64_t* used = scaled + kSpans;        // [kSpans] they have been read
  uint64_t* done = used + kSpans;          // every product of the CTA complete
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  __shared__ volatile int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = kCluster ? mm::cluster_rank() : 0;
  const long long tile = blockIdx.x / splits;
  const int tiles_n = (p.n + kRowsB - 1) / kRowsB;
  const int n0 = static_cast<int>(tile % tiles_n) * kRowsB;
  const int m0 = static_cast<int>(tile / tiles_n) * kTokens;
  const int first = static_cast<int>(static_cast<long long>(p.groups) * rank / splits);
  const int end_group = static_cast<int>(static_cast<long long>(p.groups) * (rank + 1) / splits);
  const int count = end_group - first;
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_addr(full + i), 1);
      mbar_init(smem_addr(empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(sums + i), 1);
      mbar_init(smem_addr(taken + i), kAddWarps);
    }
    for (int i = 0; i < kSpans; ++i) {
      mbar_init(smem_addr(scaled + i), 1);
      mbar_init(smem_addr(used + i), kAddWarps);
    }
    mbar_init(smem_addr(done), 1);
    prefetch_tensormap(&ta);
    prefetch_tensormap(&tb);
    fence_barrier_init();
  }
  // (as many columns as all resident CTAs together find: no CTA waits for another's)
  if (warp == kAddWarps + 1) umma::alloc(smem_addr(tslot), S::kTmem);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot;
  grid_dependency_wait();

  bool ok = true;
  if (warp == kAddWarps) {
    // ---- fetch: a stage is free again once its products are complete
    mm::Ring<S::kStages> ring;
    int fetched = 0;
    for (int k = 0; k < count && ok; ++k, ring.next()) {
      ok = mm::wait(smem_addr(empty + ring.at), ring.flip ^ 1);
      if (ok && elect_one()) {
        const uint32_t bar = smem_addr(full + ring.at), at = smem_addr(sm + ring.at * S::kStage);
        mbar_arrive_expect_tx(bar, S::kStage);
        tma_load_2d(at, &tb, (first + k) * 128, n0, bar);
        tma_load_2d(at + kTileB, &ta, (first + k) * 128, m0, bar);
      }
      __syncwarp();
      fetched += ok;
    }
    // no copy may land after the exit
    for (int k = max(0, fetched - S::kStages); k < fetched; ++k)
      ok = mm::wait(smem_addr(full + k % S::kStages), (k / S::kStages) & 1) && ok;
  } else if (warp == kAddWarps + 1) {
    // ---- products: 4 x K = 32 of a stage for a group, kBatch groups to a TMEM buffer; two
    // stages are waited for at a time
    mm::Ring<S::kStages> ring;
    mm::Ring<2> buffer;
    for (int k = 0; k < count && ok; k += 2) {
      const int in = k % S::kBatch;
      const bool two = k + 1 < count;
      const bool last = in == S::kBatch - 2 || k + 2 >= count;
      mm::Ring<S::kStages> second = ring;
      second.next();
      bool ready = mbar_try_wait(smem_addr(full + ring.at), ring.flip);
      if (two) ready &= mbar_try_wait(smem_addr(full + second.at), second.flip);
      if (in == 0) ready &= mbar_try_wait(smem_addr(taken + buffer.at), buffer.flip ^ 1);
      if (!ready)
        ok = mm::wait(smem_addr(full + ring.at), ring.flip) &&
             (!two || mm::wait(smem_addr(full + second.at), second.flip)) &&
             (in != 0 || mm::wait(smem_addr(taken + buffer.at), buffer.flip ^ 1));
      umma::fence_after_sync();
      if (ok && elect_one()) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1 && !two) break;
          const int st = q == 0 ? ring.at : second.at;
          const uint32_t at = smem_addr(sm + st * S::kStage);
          const uint64_t b = umma::smem_desc_sw128(at, 16, 1024);
          const uint64_t a = umma::smem_desc_sw128(at + kTileB, 16, 1024);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma::mma_f8(tmem + (buffer.at * S::kBatch + in + q) * kTokens, b + 2 * s, a + 2 * s,
                         kInstr, s > 0);
          umma::commit(smem_addr(empty + st));
        }
        if (last) umma::commit(smem_addr(sums + buffer.at));
      }
      __syncwarp();
      if (last) buffer.next();
      ring = second;
      ring.next();
    }
    if (elect_one()) umma::commit(smem_addr(done));
    __syncwarp();
    ok = mm::wait(smem_addr(done), 0) && ok;
  } else if (warp == kAddWarps + 2) {
    // ---- scales sa sb of the tile, spans of 16 groups, 16 lanes to a token
    mm::Ring<kSpans> ring;
    const float* sb = p.b_scale + static_cast<long long>(n0 / kScaleGroup) * p.groups + first;
    for (int k = 0; k < count && ok; k += kSpan, ring.next()) {
      float* to = scales + (ring.at * kSpan + lane % kSpan) * S::kPitch + lane / kSpan;
      const int g = k + lane % kSpan;
      const float b = g < count ? sb[g] : 0.f;
      const float* sa = p.a_scale + first + g;
      constexpr int kLoads = kTokens / 2 < 16 ? kTokens / 2 : 16;   // on the way at a time
#pragma unroll 1
      for (int t = 0; t < kTokens; t += 2 * kLoads) {
        float v[kLoads];
#pragma unroll
        for (int r = 0; r < kLoads; ++r) {
          const long long m = m0 + t + 2 * r + lane / kSpan;
          v[r] = g < count && m < p.m ? sa[m * p.groups] : 0.f;
        }
        if (t == 0) ok = mm::wait(smem_addr(used + ring.at), ring.flip ^ 1);
#pragma unroll
        for (int r = 0; r < kLoads; ++r) to[t + 2 * r] = __fmul_rn(v[r], b);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(scaled + ring.at));
    }
  }

  // ---- scale and add: weight rows 32 (warp % 4) + lane / 4 + 8 i (i < 4), tokens
  // col + 8 j + 2 (lane % 4) and the next: so a lane needs a quarter of the scales only
  constexpr int kCols = S::kCols;
  constexpr int kReps = kCols / 8;
  const int col = warp / 4 * kCols;
  uint64_t acc[4][kReps];
  if (warp < kAddWarps) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kReps; ++j) acc[i][j] = 0;
    const uint32_t at = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) + col;
    mm::Ring<2> buffer;
    mm::Ring<kSpans> spans;
    for (int k0 = 0; k0 < count; k0 += S::kBatch, buffer.next()) {
      if (k0 % kSpan == 0 && ok) ok = mm::wait(smem_addr(scaled + spans.at), spans.flip);
      const float* sc = scales + (spans.at * kSpan + k0 % kSpan) * S::kPitch + col + 2 * (lane % 4);
      if (ok) ok = mm::wait(smem_addr(sums + buffer.at), buffer.flip);
      umma::fence_after_sync();
      const int batch = min(S::kBatch, count - k0);
#pragma unroll 1
      for (int g = 0; g < batch; ++g) {
        uint32_t t[2][4 * kReps];
        const uint32_t from = at + (buffer.at * S::kBatch + g) * kTokens;
        load_16<kReps>(from, t[0]);
        load_16<kReps>(from + (16u << 16), t[1]);
        uint64_t s2[kReps];
#pragma unroll
        for (int j = 0; j < kReps; ++j)
          s2[j] = *reinterpret_cast<const uint64_t*>(sc + g * S::kPitch + 8 * j);
        umma::wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < kReps; ++j) {
            const uint32_t* v = t[i / 2] + 4 * j + 2 * (i % 2);
            acc[i][j] =
                ffma2(f2pack(__uint_as_float(v[0]), __uint_as_float(v[1])), s2[j], acc[i][j]);
          }
      }
      umma::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(taken + buffer.at));
      if ((k0 + S::kBatch) % kSpan == 0) {
        if (lane == 0) mbar_arrive(smem_addr(used + spans.at));
        spans.next();
      }
    }
  }
  if (!ok) failed = 1;
  umma::fence_before_sync();
  __syncthreads();
  launch_dependents();
  if (warp == kAddWarps + 1) umma::dealloc(tmem, S::kTmem);
  bool bad = failed != 0;
  if (bad && tid == 0) set_status(p.status, kErrTimeout);

  // ---- the sums go through shared memory, a cluster's to all of its CTAs: each adds and
  // writes its share of the tokens
  float* mine = reinterpret_cast<float*>(sm);   // [kTokens][kSumPitch]
  if (warp < kAddWarps) {
    float* to = mine + (col + 2 * (lane % 4)) * kSumPitch + warp % 4 * 32 + lane / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kReps; ++j) {
        const float2 v = f2unpack(acc[i][j]);
        to[8 * j * kSumPitch + 8 * i] = v.x;
        to[(8 * j + 1) * kSumPitch + 8 * i] = v.y;
      }
  }
  if constexpr (kCluster) {
    if (bad && tid < splits)
      mm::store_remote(mm::at_rank(smem_addr(const_cast<int*>(&failed)), tid), 1);
    mm::cluster_sync();
    bad = failed != 0;
  } else {
    __syncthreads();
  }
  if (warp < kAddWarps) {
    const int begin = static_cast<int>(kTokens * rank / splits) + warp;
    const int end = min(static_cast<int>(kTokens * (rank + 1) / splits), p.m - m0);
    constexpr int kAtOnce = kCluster ? (kTokens == 64 ? 1 : 2) : 4;
    write_sums<kAtOnce, kCluster ? kMaxSplits : 1, kAddWarps>(p, mine, splits, begin, end, m0, n0,
                                                              bad);
  }
  if constexpr (kCluster) mm::cluster_sync();
}

template <int kTokens, bool kCluster>
cudaError_t launch_kernel(const MatmulParams& p, int splits, const CUtensorMap& ta,
                          const CUtensorMap& tb, cudaStream_t s) {
  using S = Shape<kTokens>;
  auto kernel = matmul_fp8_kernel<kTokens, kCluster>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), S::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((p.n + kRowsB - 1) / kRowsB) *
                          ((p.m + kTokens - 1) / kTokens);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, splits, ta, tb);
}

template <int kTokens>
cudaError_t launch(const MatmulParams& p, int splits, const CUtensorMap& ta, const CUtensorMap& tb,
                   cudaStream_t s) {
  return splits > 1 ? launch_kernel<kTokens, true>(p, splits, ta, tb, s)
                    : launch_kernel<kTokens, false>(p, splits, ta, tb, s);
}

}  // namespace

cudaError_t launch_matmul_fp8(const MatmulParams& p, const MatmulPlan& plan, const CUtensorMap& ta,
                              const CUtensorMap& tb, cudaStream_t s) {
  switch (plan.tokens) {
    case 256: return launch_matmul_fp8_pair(p, ta, tb, s);
    case 16: return launch<16>(p, plan.splits, ta, tb, s);
    case 32: return launch<32>(p, plan.splits, ta, tb, s);
    case 64: return launch<64>(p, plan.splits, ta, tb, s);
    case 128: return launch<128>(p, plan.splits, ta, tb, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvp
