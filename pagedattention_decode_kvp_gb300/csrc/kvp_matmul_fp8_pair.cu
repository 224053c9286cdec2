// kvp_matmul_fp8_pair.cu -- the block-scaled product of kvp_matmul_fp8 for many rows:
// pairs of CTAs on tiles of 256 x 256.
//
// A pair's tcgen05.mma (cta_group::2, M = N = 256) takes half of A's rows and half of B's
// from each CTA's shared memory, so that a byte fetched serves 256 rows; each CTA holds the
// sums of 128 rows in its TMEM: two buffers of 256 columns, all of it.  Eight warps read a
// group's sums, a thread 128 columns of one row, and add them, scaled, to float32 sums in
// registers (whose columns share one scale of B, and whose row one of A) while the tensor
// cores form the next group's.  Persistent: a pair walks the tiles; the warps that fetch
// tiles and scales run on into the next one.
//
// Measured, calls back to back: 8192 x 8192 x 8192 435 us, 2530 TFLOP/s; 33098 x 12288 x 4096
// 1350 us, 2470; 8191 x 10240 x 8192 535 us, 2570; few groups a tile, 8191 x 10240 x 512, 74 us
// (its bytes take 27): a tile's results are written by the warps that add, 4.4 us a tile of
// which the four groups take 1.8.  These calls are held by the board's power (run for seconds
// 1350 W, SM clock 1640 MHz, 2300 TFLOP/s); before the clock falls, in a run of a few
// milliseconds, the first takes 395 to 420 us.  Of 395 the products alone take 240 (4600
// TFLOP/s), with the fetches 283; the rest is the way round of a TMEM buffer (product,
// commit, read, arrivals from both CTAs: 900 cycles a group where the product takes 512).
// Two words a thread are spilled (ptxas: 8 bytes).  Tried, on the first shape in such runs: 16 adding warps of 64 columns (their 104 registers
// cost moves and spills: 502 us), 16 columns a read (449), the next group's first read
// ahead of this one's last sums (501), halves of 128 columns with a warp, barriers and
// buffers each (430), tiles of 192 columns (506: a group takes as long), the issuing warp's
// loop by one lane (411), a look at the next buffer before the last sums (407).
#include "kvp_matmul.cuh"
#include "kvp_umma.cuh"

namespace kvp {

namespace {

constexpr int kTile = 256;                    // rows and columns of a pair's tile
constexpr uint32_t kHalf = 128 * 128;         // bytes of a CTA's half of A or B per stage
constexpr uint32_t kStage = 2 * kHalf;
constexpr int kStages = 5;
constexpr int kAddWarps = 8;
constexpr int kCols = 128;                    // a thread's, of one row
constexpr int kThreads = (kAddWarps + 4) * 32;   // three warpgroups
// Registers: the launch's 168 a thread are split anew, 256 * 224 + 128 * 56 = 384 * 168.
constexpr int kAddRegs = 224;
constexpr int kOtherRegs = 56;
static_assert(kAddWarps * 32 * kAddRegs + 128 * kOtherRegs <= kThreads * 168, "registers");
constexpr uint32_t kWarpBytes = 4096;         // each adding warp's, for its results
constexpr int kSpan = 8;                      // groups whose scales are staged at a time
constexpr int kSpans = 4;                     // spans that are there
constexpr int kPitch = 132;                   // floats from one group's row scales to the next's
constexpr uint32_t kSpanBytes = (kSpan * kPitch + 2 * kSpan) * 4;   // rows', then the halves' of B
constexpr uint32_t kScaleOff = kStages * kStage;
constexpr uint32_t kWarpOff = kScaleOff + kSpans * kSpanBytes;
constexpr uint32_t kBarOff = kWarpOff + kAddWarps * kWarpBytes;
constexpr int kNumBars = 2 * kStages + 5 + 2 * kSpans;
constexpr uint32_t kSmem = 1024 + kBarOff + kNumBars * 8 + 16;
constexpr uint32_t kTmem = 512;
constexpr int kBand = 8;                      // row tiles that are walked together
static_assert(kSmem <= 232448, "shared memory of a CTA");

// A tile of codes, at this CTA's `dst`; completes on the pair's first CTA's `bar`.
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* map, int32_t x,
                                          int32_t y, uint32_t bar) {
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
// Relaxed: what it announces is that TMEM was read, which tcgen05.wait::ld and the fence
// order; a release at cluster scope waits for this thread's memory accesses and made a
// group take 2200 cycles instead of 1300.
__device__ __forceinline__ void arrive_remote(uint32_t there) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(there)
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
  __device__ __forceinline__ void at(uint32_t i, int* m, int* n) const {
    const uint32_t per = static_cast<uint32_t>(kBand) * tiles_n;
    const uint32_t band = i / per, in = i - band * per;
    const uint32_t height = min(kBand, tiles_m - static_cast<int>(band) * kBand);
    *n = static_cast<int>(in / height);
    *m = static_cast<int>(band * kBand + in % height);
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
  // barriers, by their shared addresses
  const uint32_t base = smem_addr(sm);
  const uint32_t full = base + kBarOff;                // [kStages] (the first CTA's)
  const uint32_t empty = full + 8 * kStages;           // [kStages]
  const uint32_t sums = empty + 8 * kStages;           // [2] a TMEM buffer holds a group's sums
  const uint32_t taken = sums + 16;                    // [2] both CTAs have read them (first's)
  const uint32_t scaled = taken + 16;                  // [kSpans] scales are there
  const uint32_t used = scaled + 8 * kSpans;           // [kSpans] they have been read
  const uint32_t done = used + 8 * kSpans;             // every product of the pair complete
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + kBarOff + (kNumBars - 1) * 8 + 8);
  __shared__ int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = mm::cluster_rank();
  const Walk walk{(p.m + kTile - 1) / kTile, (p.n + kTile - 1) / kTile};
  const uint32_t tiles = static_cast<uint32_t>(walk.tiles_m) * walk.tiles_n;   // (below 2^31)
  const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sums + 8 * i, 1);
      mbar_init(taken + 8 * i, 2 * kAddWarps);
    }
    for (int i = 0; i < kSpans; ++i) {
      mbar_init(scaled + 8 * i, 1);
      mbar_init(used + 8 * i, kAddWarps);
    }
    mbar_init(done, 1);
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
      mm::Ring<kStages> ring;
      for (uint32_t i = pair; i < tiles && ok; i += pairs) {
        int tm, tn;
        walk.at(i, &tm, &tn);
        const int m0 = tm * kTile + 128 * rank, n0 = tn * kTile + 128 * rank;
        for (int k = 0; k < p.groups && ok; ++k, ring.next()) {
          const int st = ring.at;
          ok = mm::wait(empty + 8 * st, ring.flip ^ 1);
          if (ok && elect_one()) {
            const uint32_t bar = mm::at_rank(full + 8 * st, 0);
            const uint32_t at = base + st * kStage;
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * st, 2 * kStage);
            load_pair(at, &ta, k * 128, m0, bar);
            load_pair(at + kHalf, &tb, k * 128, n0, bar);
          }
          __syncwarp();
        }
      }
      // no copy may land after the exit: the pair's last products have read every stage
      ok = mm::wait(done, 0) && ok;
    } else if (warp == kAddWarps + 1 && rank == 0) {
      // ---- products of the pair
      mm::Ring<kStages> ring;
      mm::Ring<2> buffer;
      for (uint32_t i = pair; i < tiles && ok; i += pairs) {
        for (int k = 0; k < p.groups && ok; ++k, ring.next(), buffer.next()) {
          const int st = ring.at, buf = buffer.at;
          const uint32_t at = base + st * kStage;
          const uint64_t a = umma::smem_desc_sw128(at, 16, 1024);
          const uint64_t b = umma::smem_desc_sw128(at + kHalf, 16, 1024);
          // (two trips to shared memory at a time)
          const bool ready = mbar_try_wait(full + 8 * st, ring.flip) &
                             mbar_try_wait(taken + 8 * buf, buffer.flip ^ 1);
          if (!ready)
            ok = mm::wait(full + 8 * st, ring.flip) && mm::wait(taken + 8 * buf, buffer.flip ^ 1);
          umma::fence_after_sync();
          if (ok && elect_one()) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              umma::mma_f8<2>(tmem + buf * kTile, a + 2 * s, b + 2 * s, kInstr, s > 0);
            commit_pair(sums + 8 * buf);
            commit_pair(empty + 8 * st);
          }
          __syncwarp();
        }
      }
      if (elect_one()) commit_pair(done);
      __syncwarp();
      ok = mm::wait(done, 0) && ok;
    } else if (warp == kAddWarps + 3) {
      // ---- scales of the CTA's 128 rows and of the tile's two halves, spans of 8 groups: 8
      // lanes take a row's, so that its 32 bytes are one sector
      mm::Ring<kSpans> ring;
      for (uint32_t i = pair; i < tiles && ok; i += pairs) {
        int tm, tn;
        walk.at(i, &tm, &tn);
        const int m0 = tm * kTile + 128 * static_cast<int>(rank) + lane / 8;
        const int n0 = tn * kTile;
        for (int k = 0; k < p.groups && ok; k += kSpan, ring.next()) {
          float* to = reinterpret_cast<float*>(sm + kScaleOff + ring.at * kSpanBytes);
          const int g = k + lane % 8;
          const bool in = g < p.groups;
          const float* from = p.a_scale + static_cast<long long>(m0) * p.groups + g;
          const int n = n0 + lane / 8 * kScaleGroup;
          const long long block = n / kScaleGroup;
          const float b = in && lane < 16 && n < p.n ? p.b_scale[block * p.groups + g] : 0.f;
#pragma unroll 1
          for (int h = 0; h < 32; h += 8) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
              v[r] = in && m0 + 4 * (h + r) < p.m
                         ? from[static_cast<long long>(4 * (h + r)) * p.groups] : 0.f;
            if (h == 0) ok = mm::wait(used + 8 * ring.at, ring.flip ^ 1);
#pragma unroll
            for (int r = 0; r < 8; ++r) to[lane % 8 * kPitch + lane / 8 + 4 * (h + r)] = v[r];
          }
          if (lane < 16) to[kSpan * kPitch + lane] = b;
          __syncwarp();
          if (lane == 0) mbar_arrive(scaled + 8 * ring.at);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAddRegs));
    // ---- scale and add: row 32 (warp % 4) + lane, kCols columns from kCols (warp / 4) on
    const int quarter = warp & 3, first = warp / 4 * kCols, half = first / kScaleGroup;
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + first;
    uint4* piece = reinterpret_cast<uint4*>(sm + kWarpOff + warp * kWarpBytes);
    const uint32_t free_bar = mm::at_rank(taken, 0);
    mm::Ring<2> buffer;
    mm::Ring<kSpans> spans;
    for (uint32_t i = pair; i < tiles; i += pairs) {
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
      for (int k0 = 0; k0 < p.groups; k0 += kSpan, spans.next()) {
        const float* sa = reinterpret_cast<const float*>(sm + kScaleOff + spans.at * kSpanBytes) +
                          32 * quarter + lane;
        const float* sb = sa - 32 * quarter - lane + kSpan * kPitch + kSpan * half;
        if (ok) ok = mm::wait(scaled + 8 * spans.at, spans.flip);
        const int span = min(kSpan, p.groups - k0);
#pragma unroll 1
        for (int k = 0; k < span; ++k, buffer.next()) {
          const int buf = buffer.at;
          const float s = __fmul_rn(sa[k * kPitch], sb[k]);
          const uint64_t s2 = f2pack(s, s);
          if (ok) ok = mm::wait(sums + 8 * buf, buffer.flip);
          umma::fence_after_sync();
          // 32 columns are on their way while 32 are added
          float t[2][32];
          umma::ld32(at + buf * kTile, t[0]);
#pragma unroll
          for (int j = 0; j < kCols / 32; ++j) {
            umma::wait_ld();
            if (j < kCols / 32 - 1) {
              umma::ld32(at + buf * kTile + 32 * (j + 1), t[(j + 1) & 1]);
            } else {
              umma::fence_before_sync();
              __syncwarp();
              if (lane == 0) arrive_remote(free_bar + 8 * buf);
            }
#pragma unroll
            for (int c = 0; c < 16; ++c)
              add_scaled(acc[16 * j + c], t[j & 1][2 * c], t[j & 1][2 * c + 1], s2);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(used + 8 * spans.at);
      }
      int tm, tn;
      walk.at(i, &tm, &tn);
      const int m0 = tm * kTile + 128 * static_cast<int>(rank) + 32 * quarter;
      const int n0 = tn * kTile + first;
      // ---- the warp's 32 rows, 128 bytes at a time through its shared memory
      __syncwarp();
      constexpr int kElem = kOut == KVP_F32 ? 4 : 2;
      constexpr int kPiece = 128 / kElem;          // columns of a piece
      const bool wide = p.out_stride * kElem % 16 == 0 &&
                        (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
      // unrolled: acc is indexed by constants
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += kPiece) {
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
        if (wide && n + kPiece <= p.n) {
#pragma unroll
          for (int r = 0; r < 32; r += 4) {
            const int row = r + lane / 8, q = lane & 7;
            const uint4 v = piece[8 * row + (q ^ (row & 7))];
            if (m0 + row < p.m)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                        ((m0 + row) * p.out_stride + n) * kElem + 16 * q) = v;
          }
        } else {
#pragma unroll 4
          for (int e = lane; e < 32 * kPiece; e += 32) {
            const int r = e / kPiece, c = e % kPiece;
            if (m0 + r >= p.m || n + c >= p.n) continue;
            const void* from = reinterpret_cast<const uint8_t*>(piece) +
                               16 * (8 * r + (c * kElem / 16 ^ (r & 7))) + c * kElem % 16;
            const long long to = (m0 + r) * p.out_stride + n + c;
            if constexpr (kOut == KVP_F32)
              static_cast<float*>(p.out)[to] = *static_cast<const float*>(from);
            else
              static_cast<uint16_t*>(p.out)[to] = *static_cast<const uint16_t*>(from);
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
