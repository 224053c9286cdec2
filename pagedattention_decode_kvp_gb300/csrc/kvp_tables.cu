// kvp_tables.cu -- block tables and slot maps made on the GPU from request
// lengths, so that a captured serving loop plans its own steps:
//   * extend: every request b grows from n to n + new tokens; it takes
//     ceil((n + new) / 16) - ceil(n / 16) blocks off the free stack (request
//     order, top of the stack first), and the new tokens' slots, positions and
//     query offsets are listed;
//   * release: the blocks of finished requests go back on the stack.
// Both are all-or-nothing: everything is checked before anything is written.
//
// The work is a scan over the requests and a few words per token: latency is
// all there is to save, so a call is one launch.  A cluster of up to 8 CTAs
// (a hardware barrier instead of a second launch) shares the tokens; each CTA
// scans all requests by itself -- 16 at most per thread, read from L2 -- and
// keeps the offsets in shared memory, where a token finds its request by
// bisection.  The barrier between the checks and the writes also lets lengths
// and counts be updated in place.
#include <cooperative_groups.h>

#include "kvp_device.cuh"
#include "kvp_internal.h"

namespace kvp {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kPerThread = kMaxTableBatch / kThreads;
static_assert(kMaxTableBatch % kThreads == 0, "whole requests per thread");

// Exclusive prefix sums of two counts over the CTA's threads; totals in *sum.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2* sum) {
  __shared__ longlong2 part[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  longlong2 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, s.x, o);
    const long long y = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) {
      s.x += x;
      s.y += y;
    }
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  longlong2 before = make_longlong2(0, 0), all = make_longlong2(0, 0);
  {
    longlong2 w = part[lane];  // kThreads / 32 == 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, w.x, o);
      const long long y = __shfl_up_sync(0xffffffffu, w.y, o);
      if (lane >= o) {
        w.x += x;
        w.y += y;
      }
    }
    all.x = __shfl_sync(0xffffffffu, w.x, 31);
    all.y = __shfl_sync(0xffffffffu, w.y, 31);
    const int prev = warp > 0 ? warp - 1 : 0;
    before.x = __shfl_sync(0xffffffffu, w.x, prev);
    before.y = __shfl_sync(0xffffffffu, w.y, prev);
    if (warp == 0) before = make_longlong2(0, 0);
  }
  *sum = all;
  return make_longlong2(before.x + s.x - v.x, before.y + s.y - v.y);
}

// Largest b in [0, n) with start[b] <= x (start is non-decreasing, start[0] = 0).
__device__ __forceinline__ int find_request(const int32_t* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The first error of the cluster's CTAs (0: none).  Every CTA's reads of the
// arrays a later phase rewrites are behind this barrier.
__device__ __forceinline__ int cluster_error(int mine) {
  __shared__ int err;
  cg::cluster_group cl = cg::this_cluster();
  if (threadIdx.x == 0) err = 0;
  __syncthreads();
  if (mine != 0) atomicCAS(&err, 0, mine);
  cl.sync();
  int e = 0;
  for (unsigned r = 0; r < cl.num_blocks() && e == 0; ++r) e = *cl.map_shared_rank(&err, r);
  cl.sync();  // no CTA leaves while another still reads its word
  return e;
}

__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const TableParams p) {
  extern __shared__ int32_t smem[];
  int32_t* tok0 = smem;                   // [batch] first new token
  int32_t* blk0 = smem + p.batch;         // [batch] first new block
  int32_t* len = smem + 2 * p.batch;      // [batch] tokens before
  dev::grid_dependency_wait();
  dev::launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  const int first = cl.block_rank() * kThreads + threadIdx.x;
  const int stride = cl.num_blocks() * kThreads;
  const long long most = static_cast<long long>(p.max_blocks) * kBlockSize;

  int err = 0;
  // ---- this thread's run of requests
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per;
  int n_of[kPerThread], new_of[kPerThread];
  longlong2 mine = make_longlong2(0, 0);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    n_of[i] = new_of[i] = 0;
    if (i < per && b < p.batch) {
      n_of[i] = p.context_lens[b];
      new_of[i] = p.new_lens[b];
      if (n_of[i] < 0 || new_of[i] < 0 ||
          static_cast<long long>(n_of[i]) + new_of[i] > most) {
        err = kErrBadBlock;
        n_of[i] = new_of[i] = 0;
      }
      mine.x += new_of[i];
      mine.y += (n_of[i] + new_of[i] + kBlockSize - 1) / kBlockSize -
                (n_of[i] + kBlockSize - 1) / kBlockSize;
    }
  }
  const int count = *p.free_count;
  longlong2 sum;
  longlong2 at = block_scan(mine, &sum);
  if (sum.x > p.num_tokens || count < 0 || count > p.num_blocks) err = kErrBadBlock;
  else if (sum.y > count) err = KVP_ERR_OOM;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    if (i < per && b < p.batch) {
      tok0[b] = static_cast<int32_t>(at.x);
      blk0[b] = static_cast<int32_t>(at.y);
      len[b] = n_of[i];
      at.x += new_of[i];
      at.y += (n_of[i] + new_of[i] + kBlockSize - 1) / kBlockSize -
              (n_of[i] + kBlockSize - 1) / kBlockSize;
    }
  }
  err = __syncthreads_or(err == kErrBadBlock) ? kErrBadBlock
                                              : (__syncthreads_or(err) ? KVP_ERR_OOM : 0);
  const int tokens = static_cast<int>(sum.x), blocks = static_cast<int>(sum.y);

  // ---- the ids this step will use: blocks off the stack, and the partly
  // filled block that a request's first new token goes into
  if (err == 0) {
    for (int j = first; j < blocks; j += stride) {
      const int id = p.free_blocks[count - 1 - j];
      if (id < 0 || id >= p.num_blocks) err = kErrBadBlock;
    }
    for (int b = first; b < p.batch; b += stride) {
      const int n = len[b];
      const int next = b + 1 < p.batch ? tok0[b + 1] : tokens;
      if (next > tok0[b] && n % kBlockSize != 0) {
        const int id = p.block_tables[static_cast<size_t>(b) * p.max_blocks + n / kBlockSize];
        if (id < 0 || id >= p.num_blocks) err = kErrBadBlock;
      }
    }
  }
  err = cluster_error(err);

  // ---- writes
  if (err != 0) {  // nothing changes: no tokens in this step
    if (first == 0) {
      dev::set_status(p.status, err);
      *p.free_count_out = count;
    }
    for (int b = first; b <= p.batch; b += stride) p.query_start[b] = 0;
    for (int t = first; t < p.num_tokens; t += stride) {
      p.slot_mapping[t] = -1;
      if (p.positions != nullptr) p.positions[t] = 0;
    }
    if (p.context_lens_out != p.context_lens)
      for (int b = first; b < p.batch; b += stride) p.context_lens_out[b] = p.context_lens[b];
    return;
  }
  if (first == 0) {
    *p.free_count_out = count - blocks;
    p.query_start[p.batch] = tokens;
  }
  for (int b = first; b < p.batch; b += stride) {
    const int next = b + 1 < p.batch ? tok0[b + 1] : tokens;
    p.query_start[b] = tok0[b];
    p.context_lens_out[b] = len[b] + next - tok0[b];
  }
  for (int j = first; j < blocks; j += stride) {
    const int b = find_request(blk0, p.batch, j);
    const int i = (len[b] + kBlockSize - 1) / kBlockSize + j - blk0[b];
    p.block_tables[static_cast<size_t>(b) * p.max_blocks + i] = p.free_blocks[count - 1 - j];
  }
  for (int t = first; t < p.num_tokens; t += stride) {
    int slot = -1, pos = 0;
    if (t < tokens) {
      const int b = find_request(tok0, p.batch, t);
      pos = len[b] + t - tok0[b];
      const int i = pos / kBlockSize;
      const int have = (len[b] + kBlockSize - 1) / kBlockSize;
      const int id = i < have ? p.block_tables[static_cast<size_t>(b) * p.max_blocks + i]
                              : p.free_blocks[count - 1 - (blk0[b] + i - have)];
      slot = id * kBlockSize + pos % kBlockSize;
    }
    p.slot_mapping[t] = slot;
    if (p.positions != nullptr) p.positions[t] = pos;
  }
}

__global__ void __launch_bounds__(kThreads) release_tables_kernel(const TableParams p) {
  extern __shared__ int32_t smem[];
  int32_t* blk0 = smem;  // [batch] first released block
  dev::grid_dependency_wait();
  dev::launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  const int first = cl.block_rank() * kThreads + threadIdx.x;
  const int stride = cl.num_blocks() * kThreads;
  const long long most = static_cast<long long>(p.max_blocks) * kBlockSize;

  int err = 0;
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per;
  int nb[kPerThread];
  longlong2 mine = make_longlong2(0, 0);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    nb[i] = 0;
    if (i < per && b < p.batch) {
      const int n = p.context_lens[b];
      if (n < 0 || n > most) err = kErrBadBlock;
      else if (p.finished[b] != 0) nb[i] = (n + kBlockSize - 1) / kBlockSize;
      mine.y += nb[i];
    }
  }
  const int count = *p.free_count;
  longlong2 sum;
  longlong2 at = block_scan(mine, &sum);
  if (count < 0 || count > p.num_blocks) err = kErrBadBlock;
  else if (count + sum.y > p.num_blocks && err == 0) err = KVP_ERR_REFCOUNT;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    if (i < per && b < p.batch) {
      blk0[b] = static_cast<int32_t>(at.y);
      at.y += nb[i];
    }
  }
  err = __syncthreads_or(err == kErrBadBlock) ? kErrBadBlock
                                              : (__syncthreads_or(err) ? KVP_ERR_REFCOUNT : 0);
  const int blocks = static_cast<int>(sum.y);
  auto id_of = [&](int j) {
    const int b = find_request(blk0, p.batch, j);
    return p.block_tables[static_cast<size_t>(b) * p.max_blocks + (j - blk0[b])];
  };
  if (err == 0) {
    for (int j = first; j < blocks; j += stride) {
      const int id = id_of(j);
      if (id < 0 || id >= p.num_blocks) err = kErrBadBlock;
    }
  }
  err = cluster_error(err);
  if (err != 0) {
    if (first == 0) {
      dev::set_status(p.status, err);
      *p.free_count_out = count;
    }
    if (p.context_lens_out != p.context_lens)
      for (int b = first; b < p.batch; b += stride) p.context_lens_out[b] = p.context_lens[b];
    return;
  }
  if (first == 0) *p.free_count_out = count + blocks;
  for (int j = first; j < blocks; j += stride) p.free_blocks[count + j] = id_of(j);
  for (int b = first; b < p.batch; b += stride)
    p.context_lens_out[b] = p.finished[b] != 0 ? 0 : p.context_lens[b];
}

cudaError_t launch_tables(void (*kernel)(TableParams), const TableParams& p, long long items,
                          int arrays, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(arrays) * kMaxTableBatch * sizeof(int32_t);
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  // one CTA up to two items a thread, then as many as the items fill, up to
  // the 8 of a portable cluster
  unsigned ctas = 1;
  while (ctas < 8 && items > static_cast<long long>(ctas) * 2 * kThreads) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(arrays) * p.batch * sizeof(int32_t);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_extend_tables(const TableParams& p, cudaStream_t s) {
  return launch_tables(&extend_tables_kernel, p,
                       static_cast<long long>(p.num_tokens) + p.batch, 3, s);
}

cudaError_t launch_release_tables(const TableParams& p, cudaStream_t s) {
  // the blocks that come back are only known on the device; a quarter of the
  // requests at a quarter of the table's width is a busy step
  return launch_tables(&release_tables_kernel, p,
                       static_cast<long long>(p.batch) * (1 + p.max_blocks / 16), 1, s);
}

}  // namespace kvp
