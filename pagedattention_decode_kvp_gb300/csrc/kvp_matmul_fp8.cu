// kvp_matmul_fp8.cu -- matrix product of E4M3 codes with a float32 scale for every 128
// elements of a row of A and for every 128 x 128 elements of B (a weight):
//   out[m, n] = sum_g sa[m, g] sb[n / 128, g] sum_{k in g} a[m, k] b[n, k].
//
// The tensor cores (tcgen05, kind::f8f6f4) form each group's inner sum in TMEM; the
// scales differ from group to group, so every group's sum is read into registers and
// added there in float32: acc = fma(t, sa sb, acc).
//
// The weight's 128 rows are the M side of the instruction (a TMEM lane and a thread
// each), kTokens rows of A its N side.  Warps: four that scale and add, one that
// fetches tiles of 128 bytes of K by TMA, one that issues the products; two TMEM
// buffers, so that a group is scaled while the next is multiplied.  Where few tiles
// meet many SMs, the CTAs of a cluster share a tile's K and add their sums through
// distributed shared memory, in the order of their ranks.
#include "kvp_matmul.cuh"

namespace kvp {

namespace {

constexpr int kRowsB = 128;                  // weight rows of a tile
constexpr uint32_t kTileB = kRowsB * 128;    // bytes of a stage's weight tile
constexpr int kThreads = 192;
constexpr int kAddWarps = 4;
constexpr int kScaleSpan = 32;               // groups whose scales are staged at a time

template <int kTokens>
struct Shape {
  static constexpr uint32_t kTileA = kTokens * 128;
  static constexpr uint32_t kStage = kTileB + kTileA;
  // two CTAs per SM up to 64 tokens; at 128 the sums take the registers of one
  static constexpr int kCtas = kTokens <= 64 ? 2 : 1;
  static constexpr int kStages = kTokens <= 64 ? 98304 / kStage : 6;
  static constexpr uint32_t kScaleOff = kStages * kStage;
  static constexpr uint32_t kBarOff = kScaleOff + kTokens * kScaleSpan * 4;
  static constexpr uint32_t kSmem = 1024 + kBarOff + (2 * kStages + 5) * 8 + 16;
  static constexpr uint32_t kTmem = 2 * kTokens < 32 ? 32 : 2 * kTokens;
  static_assert(kStages * kStage >= kTokens * kRowsB * 4, "the sums are exchanged in the ring");
};

// grid.x = (token tile, weight tile, rank of the cluster), the last running fastest.
template <int kTokens>
__global__ void __launch_bounds__(kThreads, Shape<kTokens>::kCtas)
    matmul_fp8_kernel(const MatmulParams p, int splits, const __grid_constant__ CUtensorMap ta,
                      const __grid_constant__ CUtensorMap tb) {
  using namespace dev;
  using S = Shape<kTokens>;
  constexpr uint32_t kInstr = umma::instr_desc_f16(kRowsB, kTokens, false, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(sm + S::kScaleOff);   // [kScaleSpan][kTokens]
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBarOff);
  uint64_t* empty = full + S::kStages;
  uint64_t* sums = empty + S::kStages;     // [2] a TMEM buffer holds a group's sums
  uint64_t* taken = sums + 2;              // [2] they are in registers
  uint64_t* done = taken + 2;              // every product of the CTA complete
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  __shared__ int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = splits > 1 ? mm::cluster_rank() : 0;
  const long long tile = blockIdx.x / splits;
  const int tiles_n = (p.n + kRowsB - 1) / kRowsB;
  const int n0 = static_cast<int>(tile % tiles_n) * kRowsB;
  const int m0 = static_cast<int>(tile / tiles_n) * kTokens;
  const int first = static_cast<int>(static_cast<long long>(p.groups) * rank / splits);
  const int count = static_cast<int>(static_cast<long long>(p.groups) * (rank + 1) / splits) - first;
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
    mbar_init(smem_addr(done), 1);
    prefetch_tensormap(&ta);
    prefetch_tensormap(&tb);
    fence_barrier_init();
  }
  if (warp == kAddWarps + 1) umma::alloc(smem_addr(tslot), S::kTmem);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot;
  grid_dependency_wait();

  bool ok = true;
  if (warp == kAddWarps) {
    // ---- fetch: a stage is free again once its products are complete
    int fetched = 0;
    for (int k = 0; k < count && ok; ++k) {
      const int st = k % S::kStages;
      if (k >= S::kStages) ok = mbar_wait_bounded(smem_addr(empty + st), (k / S::kStages - 1) & 1);
      if (ok && elect_one()) {
        const uint32_t bar = smem_addr(full + st), at = smem_addr(sm + st * S::kStage);
        mbar_arrive_expect_tx(bar, S::kStage);
        tma_load_2d(at, &tb, (first + k) * 128, n0, bar);
        tma_load_2d(at + kTileB, &ta, (first + k) * 128, m0, bar);
      }
      __syncwarp();
      fetched += ok;
    }
    // no copy may land after the exit
    for (int k = max(0, fetched - S::kStages); k < fetched; ++k)
      ok = mbar_wait_bounded(smem_addr(full + k % S::kStages), (k / S::kStages) & 1) && ok;
  } else if (warp == kAddWarps + 1) {
    // ---- products: 4 x K = 32 of a stage into TMEM buffer k % 2
    for (int k = 0; k < count && ok; ++k) {
      const int st = k % S::kStages, buf = k & 1;
      ok = mbar_wait_bounded(smem_addr(full + st), (k / S::kStages) & 1);
      if (ok && k >= 2) ok = mbar_wait_bounded(smem_addr(taken + buf), (k / 2 - 1) & 1);
      umma::fence_after_sync();
      if (ok && elect_one()) {
        const uint32_t at = smem_addr(sm + st * S::kStage);
        const uint64_t b = umma::smem_desc_sw128(at, 16, 1024);
        const uint64_t a = umma::smem_desc_sw128(at + kTileB, 16, 1024);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mm::mma_f8<1>(tmem + buf * kTokens, b + 2 * s, a + 2 * s, kInstr, s > 0);
        umma::commit(smem_addr(empty + st));
        umma::commit(smem_addr(sums + buf));
      }
      __syncwarp();
    }
    if (elect_one()) umma::commit(smem_addr(done));
    __syncwarp();
    ok = mbar_wait_bounded(smem_addr(done), 0) && ok;
  }

  uint64_t acc[kTokens / 2];   // token pairs of this thread's weight row
  if (warp < kAddWarps) {
#pragma unroll
    for (int j = 0; j < kTokens / 2; ++j) acc[j] = 0;
    const uint32_t at = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (int k = 0; k < count; ++k) {
      if (k % kScaleSpan == 0) {
        // sa sb of the next groups, [group][token]; a thread takes one token's groups
        constexpr int kPer = kAddWarps * 32 / kTokens;
        if (k > 0) named_bar_sync(1, kAddWarps * 32);
        const int m = m0 + tid % kTokens;
        const int span = min(kScaleSpan, count - k);
        const float* sb = p.b_scale + static_cast<long long>(n0 / kScaleGroup) * p.groups + first + k;
        const float* sa = p.a_scale + static_cast<long long>(m) * p.groups + first + k;
        for (int g = tid / kTokens; g < span; g += kPer)
          scales[g * kTokens + tid % kTokens] = m < p.m ? __fmul_rn(sa[g], sb[g]) : 0.f;
        named_bar_sync(1, kAddWarps * 32);
      }
      const int buf = k & 1;
      if (ok) ok = mbar_wait_bounded(smem_addr(sums + buf), (k >> 1) & 1);
      umma::fence_after_sync();
      const float* sc = scales + (k % kScaleSpan) * kTokens;
#pragma unroll
      for (int j = 0; j < kTokens; j += 16) {
        float t[16];
        umma::ld16(at + buf * kTokens + j, t);
        umma::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const ulonglong2 s2 = *reinterpret_cast<const ulonglong2*>(sc + j + i);
          acc[(j + i) / 2] = ffma2(f2pack(t[i], t[i + 1]), s2.x, acc[(j + i) / 2]);
          acc[(j + i) / 2 + 1] = ffma2(f2pack(t[i + 2], t[i + 3]), s2.y, acc[(j + i) / 2 + 1]);
        }
      }
      umma::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(taken + buf));
    }
  }
  if (!ok) atomicExch(&failed, 1);
  umma::fence_before_sync();
  __syncthreads();
  launch_dependents();
  if (warp == kAddWarps + 1) umma::dealloc(tmem, S::kTmem);
  bool bad = failed != 0;
  if (bad && tid == 0) set_status(p.status, kErrTimeout);

  const int n = n0 + tid;
  if (splits == 1) {
    if (warp >= kAddWarps || n >= p.n) return;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const float2 v = f2unpack(acc[j / 2]);
      if (m0 + j < p.m)
        mm::store_out(p, static_cast<long long>(m0 + j) * p.out_stride + n, bad ? 0.f : j & 1 ? v.y : v.x);
    }
    return;
  }
  // ---- the cluster's sums: every CTA adds and writes its share of the tokens
  float* mine = reinterpret_cast<float*>(sm);   // [kTokens][128]
  if (warp < kAddWarps) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const float2 v = f2unpack(acc[j / 2]);
      mine[j * kRowsB + tid] = j & 1 ? v.y : v.x;
    }
  }
  mm::cluster_sync();
  for (int r = 0; r < splits; ++r) bad = mm::load_remote(mm::at_rank(smem_addr(&failed), r)) != 0 || bad;
  if (warp < kAddWarps && n < p.n) {
    const int end = min(static_cast<int>(kTokens * (rank + 1) / splits), p.m - m0);
    for (int j = kTokens * rank / splits; j < end; ++j) {
      float v = 0.f;
      for (int r = 0; r < splits; ++r)
        v += __uint_as_float(mm::load_remote(mm::at_rank(smem_addr(mine + j * kRowsB + tid), r)));
      mm::store_out(p, static_cast<long long>(m0 + j) * p.out_stride + n, bad ? 0.f : v);
    }
  }
  mm::cluster_sync();
}

template <int kTokens>
cudaError_t launch(const MatmulParams& p, int splits, const CUtensorMap& ta, const CUtensorMap& tb,
                   cudaStream_t s) {
  using S = Shape<kTokens>;
  auto kernel = matmul_fp8_kernel<kTokens>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), S::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((p.n + kRowsB - 1) / kRowsB) *
                          ((p.m + kTokens - 1) / kTokens);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
  cfg.blockDim = dim3(kThreads);
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
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, splits, ta, tb);
}

}  // namespace

MatmulPlan matmul_plan(int m, int n, int groups) {
  MatmulPlan plan;
  plan.tokens = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const long long tiles = static_cast<long long>((n + kRowsB - 1) / kRowsB) *
                          ((m + plan.tokens - 1) / plan.tokens);
  plan.splits = 1;
  // pairs where their tiles are enough for the SMs
  if (m > 128 && static_cast<long long>((m + 255) / 256) * ((n + 255) / 256) >= kNumSms / 2) {
    plan.tokens = 256;
    return plan;
  }
  while (plan.splits < 8 && tiles * plan.splits * 2 <= 304 && plan.splits * 4 <= groups)
    plan.splits *= 2;
  return plan;
}

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
