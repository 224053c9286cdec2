// kvp_matmul_fp8_pair.cu -- the block-scaled product of kvp_matmul_fp8 for many rows:
// pairs of CTAs on tiles of 256 x 256.
//
// A pair's tcgen05.mma (cta_group::2, M = N = 256) takes half of A's rows and half of
// B's from each CTA's shared memory, so that a byte fetched serves 256 rows; each CTA
// holds the sums of 128 rows in its TMEM: two buffers of 256 columns, all of it.  Eight
// warps read a group's sums, a thread 128 columns of one row, and add them, scaled, to
// float32 sums in registers (whose columns share one scale of B, and whose row one of
// A) while the tensor cores form the next group's.  Persistent: a pair walks the tiles,
// and the fetching warps run on into the next one.
#include "kvp_matmul.cuh"

namespace kvp {

namespace {

constexpr int kTile = 256;                    // rows and columns of a pair's tile
constexpr uint32_t kHalf = 128 * 128;         // bytes of a CTA's half of A or B per stage
constexpr uint32_t kStage = 2 * kHalf;
constexpr int kStages = 6;
constexpr int kAddWarps = 8;
constexpr int kThreads = (kAddWarps + 4) * 32;   // three warpgroups; two warps are idle
// Registers: the launch's 168 a thread are split anew, 2 * 128 * 232 + 128 * 40 = 384 * 168.
constexpr int kAddRegs = 232;
constexpr int kOtherRegs = 40;
static_assert(kAddWarps * 32 * kAddRegs + 128 * kOtherRegs <= kThreads * 168, "registers");
constexpr uint32_t kWarpBytes = 4096;         // each adding warp's: scales, then results
constexpr uint32_t kWarpOff = kStages * kStage;
constexpr uint32_t kBarOff = kWarpOff + kAddWarps * kWarpBytes;
constexpr uint32_t kSmem = 1024 + kBarOff + (2 * kStages + 5) * 8 + 16;
constexpr uint32_t kTmem = 512;
constexpr int kSpan = 32;                     // groups whose scales are staged at a time
constexpr int kBand = 8;                      // row tiles that are walked together
static_assert(kSmem <= 232448, "shared memory of a CTA");

// A tile of codes, at this CTA's `dst`; completes on the pair's first CTA's `bar`.
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrive on both CTAs' barrier at `bar` once the products issued so far are complete.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t there) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(there)
               : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
               "r"(kTmem)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmem)
               : "memory");
}

// acc += t s; volatile, so that the sums of one read of TMEM are done before the next's
// registers are needed.
__device__ __forceinline__ void add_scaled(uint64_t& acc, float t0, float t1, uint64_t s2) {
  asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(dev::f2pack(t0, t1)), "l"(s2));
}

// Tile number -> row and column tile: bands of kBand row tiles, walked column by
// column, so that the pairs at work at one time share rows of A and of B in L2.
struct Walk {
  int tiles_m, tiles_n;
  __device__ __forceinline__ void at(long long i, int* m, int* n) const {
    const long long per = static_cast<long long>(kBand) * tiles_n;
    const int band = static_cast<int>(i / per);
    const int in = static_cast<int>(i - band * per);
    const int height = min(kBand, tiles_m - band * kBand);
    *n = in / height;
    *m = band * kBand + in % height;
  }
};

// A ring's place and how often it has wrapped (mod 2): what is waited for is the phase
// `flip` of a full place, and `flip ^ 1` of a free one (a new barrier's passes).
template <int kPlaces>
struct Ring {
  int at = 0;
  uint32_t flip = 0;
  __device__ __forceinline__ void next() {
    if (++at == kPlaces) {
      at = 0;
      flip ^= 1;
    }
  }
};

template <int kOut>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    matmul_fp8_pair_kernel(const MatmulParams p, const __grid_constant__ CUtensorMap ta,
                           const __grid_constant__ CUtensorMap tb) {
  using namespace dev;
  constexpr uint32_t kInstr = umma::instr_desc_f16(kTile, kTile, false, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kBarOff);   // (of the first CTA)
  uint64_t* empty = full + kStages;
  uint64_t* sums = empty + kStages;   // [2] a TMEM buffer holds a group's sums
  uint64_t* taken = sums + 2;         // [2] both CTAs have them in registers (first CTA)
  uint64_t* done = taken + 2;         // every product of the pair complete
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  __shared__ int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = mm::cluster_rank();
  const Walk walk{(p.m + kTile - 1) / kTile, (p.n + kTile - 1) / kTile};
  const long long tiles = static_cast<long long>(walk.tiles_m) * walk.tiles_n;
  const long long pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(full + i), 1);
      mbar_init(smem_addr(empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(sums + i), 1);
      mbar_init(smem_addr(taken + i), 2 * kAddWarps);
    }
    mbar_init(smem_addr(done), 1);
    prefetch_tensormap(&ta);
    prefetch_tensormap(&tb);
    fence_barrier_init();
  }
  if (warp == kAddWarps + 1) alloc_pair(smem_addr(tslot));
  umma::fence_before_sync();
  __syncthreads();
  mm::cluster_sync();   // both CTAs' barriers are there
  umma::fence_after_sync();
  const uint32_t tmem = *tslot;
  grid_dependency_wait();

  bool ok = true;
  if (warp >= kAddWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kAddWarps) {
    // ---- fetch this CTA's halves; the first CTA expects the bytes of both
    Ring<kStages> ring;
    for (long long i = pair; i < tiles && ok; i += pairs) {
      int tm, tn;
      walk.at(i, &tm, &tn);
      const int m0 = tm * kTile + 128 * rank, n0 = tn * kTile + 128 * rank;
      for (int k = 0; k < p.groups && ok; ++k, ring.next()) {
        const int st = ring.at;
        ok = mm::wait(smem_addr(empty + st), ring.flip ^ 1);
        if (ok && elect_one()) {
          const uint32_t bar = mm::at_rank(smem_addr(full + st), 0);
          const uint32_t at = smem_addr(sm + st * kStage);
          if (rank == 0) mbar_arrive_expect_tx(smem_addr(full + st), 2 * kStage);
          load_pair(at, &ta, k * 128, m0, bar);
          load_pair(at + kHalf, &tb, k * 128, n0, bar);
        }
        __syncwarp();
      }
    }
    // no copy may land after the exit: the pair's last products have read every stage
    ok = mm::wait(smem_addr(done), 0) && ok;
  } else if (warp == kAddWarps + 1 && rank == 0) {
    // ---- products of the pair
    Ring<kStages> ring;
    Ring<2> buffer;
    for (long long i = pair; i < tiles && ok; i += pairs) {
      for (int k = 0; k < p.groups && ok; ++k, ring.next(), buffer.next()) {
        const int st = ring.at, buf = buffer.at;
        ok = mm::wait(smem_addr(full + st), ring.flip) &&
             mm::wait(smem_addr(taken + buf), buffer.flip ^ 1);
        umma::fence_after_sync();
        if (ok && elect_one()) {
          const uint32_t at = smem_addr(sm + st * kStage);
          const uint64_t a = umma::smem_desc_sw128(at, 16, 1024);
          const uint64_t b = umma::smem_desc_sw128(at + kHalf, 16, 1024);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mm::mma_f8<2>(tmem + buf * kTile, a + 2 * s, b + 2 * s, kInstr, s > 0);
          commit_pair(smem_addr(empty + st));
          commit_pair(smem_addr(sums + buf));
        }
        __syncwarp();
      }
    }
    if (elect_one()) commit_pair(smem_addr(done));
    __syncwarp();
    ok = mm::wait(smem_addr(done), 0) && ok;
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAddRegs));
    // ---- scale and add: row 32 (warp % 4) + lane, columns 128 (warp / 4) .. + 127
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    float* mine = reinterpret_cast<float*>(sm + kWarpOff + warp * kWarpBytes);
    const uint32_t free_bar[2] = {mm::at_rank(smem_addr(taken), 0),
                                  mm::at_rank(smem_addr(taken + 1), 0)};
    Ring<2> buffer;
    for (long long i = pair; i < tiles; i += pairs) {
      int tm, tn;
      walk.at(i, &tm, &tn);
      const int m0 = tm * kTile + 128 * static_cast<int>(rank) + 32 * quarter;
      const int n0 = tn * kTile + 128 * half;
      const bool live = n0 < p.n;
      const float* sb = p.b_scale + static_cast<long long>(live ? n0 / kScaleGroup : 0) * p.groups;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0;
      for (int k = 0; k < p.groups; ++k, buffer.next()) {
        if (k % kSpan == 0) {
          // sa sb of the warp's 32 rows and the next 32 groups: fetched with a lane per
          // group, read with a lane per row; (row, group) at 32 row + (group ^ row)
          const int g = k + lane;
          const float b = g < p.groups ? sb[g] : 0.f;
          __syncwarp();
#pragma unroll 8
          for (int r = 0; r < 32; ++r) {
            const float a = m0 + r < p.m && g < p.groups
                                ? p.a_scale[static_cast<long long>(m0 + r) * p.groups + g] : 0.f;
            mine[32 * r + (lane ^ r)] = __fmul_rn(a, b);
          }
          __syncwarp();
        }
        const int buf = buffer.at;
        const float s = mine[32 * lane + ((k % kSpan) ^ lane)];
        const uint64_t s2 = f2pack(s, s);
        if (ok) ok = mm::wait(smem_addr(sums + buf), buffer.flip);
        umma::fence_after_sync();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float t[32];
          umma::ld32(at + buf * kTile + 32 * j, t);
          umma::wait_ld();
          if (j == 3) {
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_remote(free_bar[buf]);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c)
            add_scaled(acc[16 * j + c], t[2 * c], t[2 * c + 1], s2);
        }
      }
      // ---- the warp's 32 rows, 128 bytes at a time through its shared memory
      __syncwarp();
      constexpr int kElem = kOut == KVP_F32 ? 4 : 2;
      constexpr int kCols = 128 / kElem;           // columns of a piece
      const bool wide = p.out_stride * kElem % 16 == 0 &&
                        (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
      uint4* piece = reinterpret_cast<uint4*>(mine);
      // unrolled: acc is indexed by constants
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += kCols) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {              // 16 bytes of this lane's row
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kOut == KVP_F32) {
              const float2 f = f2unpack(acc[(c0 + 4 * q + e) / 2]);
              w[e] = __float_as_uint((c0 + 4 * q + e) & 1 ? f.y : f.x);
            } else {
              const float2 f = f2unpack(acc[(c0 + 8 * q + 2 * e) / 2]);
              w[e] = pack2<kOut == KVP_BF16>(f.x, f.y);
            }
            if (!ok) w[e] = 0;
          }
          piece[8 * lane + (q ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int n = n0 + c0;
        if (wide && n + kCols <= p.n) {
#pragma unroll
          for (int r = 0; r < 32; r += 4) {
            const int row = r + lane / 8, q = lane & 7;
            const uint4 v = piece[8 * row + (q ^ (row & 7))];
            if (m0 + row < p.m)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                        ((m0 + row) * p.out_stride + n) * kElem + 16 * q) = v;
          }
        } else {
          for (int r = 0; r < 32 && m0 + r < p.m; ++r) {
            for (int c = lane; c < kCols && n + c < p.n; c += 32) {
              const int q = c * kElem / 16;
              const void* from = reinterpret_cast<const uint8_t*>(piece) +
                                 16 * (8 * r + (q ^ (r & 7))) + c * kElem % 16;
              const long long to = (m0 + r) * p.out_stride + n + c;
              if constexpr (kOut == KVP_F32)
                static_cast<float*>(p.out)[to] = *static_cast<const float*>(from);
              else
                static_cast<uint16_t*>(p.out)[to] = *static_cast<const uint16_t*>(from);
            }
          }
        }
        __syncwarp();
      }
    }
  }
  if (!ok) atomicExch(&failed, 1);
  launch_dependents();
  umma::fence_before_sync();
  __syncthreads();
  // neither CTA leaves, or gives up its TMEM, while the other's work may reach it
  mm::cluster_sync();
  if (warp == kAddWarps + 1) dealloc_pair(tmem);
  if (tid == 0 && failed != 0) set_status(p.status, kErrTimeout);
}

template <int kOut>
cudaError_t launch(const MatmulParams& p, const CUtensorMap& ta, const CUtensorMap& tb,
                   cudaStream_t s) {
  auto kernel = matmul_fp8_pair_kernel<kOut>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((p.m + kTile - 1) / kTile) *
                          ((p.n + kTile - 1) / kTile);
  const long long pairs = tiles < kNumSms / 2 ? tiles : kNumSms / 2;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), kSmem, s, p, ta,
                    tb);
}

}  // namespace

cudaError_t launch_matmul_fp8_pair(const MatmulParams& p, const CUtensorMap& ta,
                                   const CUtensorMap& tb, cudaStream_t s) {
  switch (p.out_type) {
    case KVP_F16: return launch<KVP_F16>(p, ta, tb, s);
    case KVP_BF16: return launch<KVP_BF16>(p, ta, tb, s);
    case KVP_F32: return launch<KVP_F32>(p, ta, tb, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvp
