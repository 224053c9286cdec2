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
// all there is to save.  One launch of one CTA does a decode step; above 2048
// words of work it is a cluster of up to 8 (a hardware barrier instead of a
// second launch) whose CTAs each scan all requests -- 16 at most per thread, read
// from L2 -- and share the rest.  The offsets lie in shared
// memory, where a token finds its request by bisection.  The barrier between the
// checks and the writes also lets lengths and counts be updated in place.  Above
// 16384 tokens the slots are written by a second launch that fills the GPU, from
// the first one's outputs alone (tables, lengths and query offsets).
// Measured, a release and an extend together: 64 requests of one token each 8.8 to
// 9.7 us, 1000 of them 13, 1024 requests with prompts, 524291 slots, 20 (37 with the
// slots in the cluster's launch; 64 requests with 64003 slots 13.6 against 12.9, and
// a second launch for 1000 slots costs 5); 16384 requests 131.
#include <cooperative_groups.h>

#include "kvp_device.cuh"
#include "kvp_serve.h"

namespace kvp {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;                         // of a CTA of the first launch
constexpr int kFillThreads = 256, kFillTokens = 1024;  // of the second launch
constexpr int kFusedTokens = 16384;                    // slots the first launch writes itself

// Exclusive prefix sums of two counts over the CTA's threads; totals in *sum.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2* sum) {
  constexpr int kW = kThreads / 32;
  __shared__ longlong2 part[kW];
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
  longlong2 w = lane < kW ? part[lane] : make_longlong2(0, 0);
#pragma unroll
  for (int o = 1; o < kW; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, w.x, o);
    const long long y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  sum->x = __shfl_sync(0xffffffffu, w.x, kW - 1);
  sum->y = __shfl_sync(0xffffffffu, w.y, kW - 1);
  const int prev = warp > 0 ? warp - 1 : 0;
  const long long bx = __shfl_sync(0xffffffffu, w.x, prev);
  const long long by = __shfl_sync(0xffffffffu, w.y, prev);
  return make_longlong2((warp > 0 ? bx : 0) + s.x - v.x, (warp > 0 ? by : 0) + s.y - v.y);
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

// Largest b in [0, n) with start[b] <= x, by a warp: 32 places a round.
__device__ __forceinline__ int warp_find_request(const int32_t* start, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const unsigned at = __ballot_sync(0xffffffffu, i < n && start[lo + i] <= x);
    const int k = __popc(at) - 1;  // lane 0's place always is
    lo += k * step;
    n = min(step, n - k * step);
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
  if (cl.num_blocks() == 1) {
    __syncthreads();
    return err;
  }
  cl.sync();
  int e = 0;
  for (unsigned r = 0; r < cl.num_blocks() && e == 0; ++r) e = *cl.map_shared_rank(&err, r);
  cl.sync();  // no CTA leaves while another still reads its word
  return e;
}

// Blocks that hold n tokens.
__device__ __forceinline__ int blocks_for(int n) { return (n + kBlockSize - 1) / kBlockSize; }

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
  // ---- this thread's run of requests, read once for the sums and once more
  // (from L1) for the offsets
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, static_cast<int>(threadIdx.x) * per), b1 = min(p.batch, b0 + per);
  const int count = *p.free_count;
  longlong2 mine = make_longlong2(0, 0);
  for (int b = b0; b < b1; ++b) {
    const int n = p.context_lens[b], k = p.new_lens[b];
    if (n < 0 || k < 0 || static_cast<long long>(n) + k > most) {
      err = kErrBadBlock;
    } else {
      mine.x += k;
      mine.y += blocks_for(n + k) - blocks_for(n);
    }
  }
  longlong2 sum;
  longlong2 at = block_scan(mine, &sum);
  for (int b = b0; b < b1; ++b) {  // (wrong lengths give wrong offsets, which nothing uses)
    const int n = p.context_lens[b], k = p.new_lens[b];
    tok0[b] = static_cast<int32_t>(at.x);
    blk0[b] = static_cast<int32_t>(at.y);
    len[b] = n;
    at.x += k;
    at.y += blocks_for(n + k) - blocks_for(n);
  }
  if (__syncthreads_or(err) || sum.x > p.num_tokens || count < 0 || count > p.num_blocks)
    err = kErrBadBlock;
  else if (sum.y > count)
    err = KVP_ERR_OOM;
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
    for (int t = first; t < (p.num_tokens > kFusedTokens ? 0 : p.num_tokens); t += stride) {
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
    const int i = blocks_for(len[b]) + j - blk0[b];
    p.block_tables[static_cast<size_t>(b) * p.max_blocks + i] = p.free_blocks[count - 1 - j];
  }
  if (p.num_tokens > kFusedTokens) return;
  for (int t = first; t < p.num_tokens; t += stride) {
    int slot = -1, pos = 0;
    if (t < tokens) {
      const int b = find_request(tok0, p.batch, t);
      pos = len[b] + t - tok0[b];
      const int i = pos / kBlockSize, have = blocks_for(len[b]);
      const int id = i < have ? p.block_tables[static_cast<size_t>(b) * p.max_blocks + i]
                              : p.free_blocks[count - 1 - (blk0[b] + i - have)];
      slot = id * kBlockSize + pos % kBlockSize;
    }
    p.slot_mapping[t] = slot;
    if (p.positions != nullptr) p.positions[t] = pos;
  }
}

// Slots and positions of many tokens, from what the first launch wrote: request
// b's new tokens are query_start[b] .. query_start[b + 1] - 1, the last ones of
// its context_lens_out[b].  A CTA takes kFillTokens of them; its first and last
// request are found by two warps, and the offsets between them come on chip.
__global__ void __launch_bounds__(kFillThreads) fill_slots_kernel(const TableParams p) {
  __shared__ int32_t start[kFillTokens + 1], before[kFillTokens];
  __shared__ int range[2];
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int t0 = blockIdx.x * kFillTokens, t1 = min(t0 + kFillTokens, p.num_tokens);
  const int tokens = p.query_start[p.batch];
  const int warp = threadIdx.x >> 5;
  if (t0 < tokens && warp < 2) {
    const int b = warp_find_request(p.query_start, p.batch,
                                    warp == 0 ? t0 : min(t1, tokens) - 1);
    if ((threadIdx.x & 31) == 0) range[warp] = b;
  }
  __syncthreads();
  int b0 = 0, n = 0;
  if (t0 < tokens) {
    b0 = range[0];
    n = range[1] - b0 + 1;
  }
  // (requests without new tokens can make the range longer than the tokens)
  const bool on_chip = n <= kFillTokens;
  if (on_chip) {
    for (int i = threadIdx.x; i < n; i += kFillThreads) {
      const int s = p.query_start[b0 + i];
      start[i] = s;
      before[i] = p.context_lens_out[b0 + i] - (p.query_start[b0 + i + 1] - s);
    }
  }
  __syncthreads();
  for (int t = t0 + threadIdx.x; t < t1; t += kFillThreads) {
    int slot = -1, pos = 0;
    if (t < tokens) {
      int b;
      if (on_chip) {
        const int i = find_request(start, n, t);
        b = b0 + i;
        pos = before[i] + t - start[i];
      } else {
        b = b0 + find_request(p.query_start + b0, n, t);
        pos = p.context_lens_out[b] - (p.query_start[b + 1] - t);
      }
      slot = p.block_tables[static_cast<size_t>(b) * p.max_blocks + pos / kBlockSize] * kBlockSize +
             pos % kBlockSize;
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
  const int b0 = min(p.batch, static_cast<int>(threadIdx.x) * per), b1 = min(p.batch, b0 + per);
  const int count = *p.free_count;
  longlong2 mine = make_longlong2(0, 0);
  for (int b = b0; b < b1; ++b) {
    const int n = p.context_lens[b];
    if (n < 0 || n > most) err = kErrBadBlock;
    else if (p.finished[b] != 0) mine.y += blocks_for(n);
  }
  longlong2 sum;
  longlong2 at = block_scan(mine, &sum);
  for (int b = b0; b < b1; ++b) {
    blk0[b] = static_cast<int32_t>(at.y);
    if (p.finished[b] != 0) at.y += blocks_for(p.context_lens[b]);
  }
  if (__syncthreads_or(err) || count < 0 || count > p.num_blocks) err = kErrBadBlock;
  else if (count + sum.y > p.num_blocks) err = KVP_ERR_REFCOUNT;
  const int blocks = static_cast<int>(sum.y);
  auto id_of = [&](int j) {
    const int b = find_request(blk0, p.batch, j);
    return p.block_tables[static_cast<size_t>(b) * p.max_blocks + (j - blk0[b])];
  };
  int mine0 = 0;  // this thread's first id, mostly its only one
  if (err == 0) {
    for (int j = first; j < blocks; j += stride) {
      const int id = id_of(j);
      if (id < 0 || id >= p.num_blocks) err = kErrBadBlock;
      if (j == first) mine0 = id;
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
  for (int j = first; j < blocks; j += stride)
    p.free_blocks[count + j] = j == first ? mine0 : id_of(j);
  for (int b = first; b < p.batch; b += stride)
    p.context_lens_out[b] = p.finished[b] != 0 ? 0 : p.context_lens[b];
}

// One launch for about `items` words of work, with `arrays` words per request in
// shared memory: one CTA up to two items a thread, then a cluster of as many as
// the items fill, up to the portable 8.
cudaError_t launch_tables(void (*kernel)(TableParams), const TableParams& p, long long items,
                          int arrays, cudaStream_t s) {
  const cudaError_t e =
      ensure_smem_attr(reinterpret_cast<const void*>(kernel),
                       static_cast<size_t>(arrays) * kMaxTableBatch * sizeof(int32_t));
  if (e != cudaSuccess) return e;
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
  const bool fused = p.num_tokens <= kFusedTokens;
  const long long items =
      p.batch + (fused ? p.num_tokens : p.num_tokens / kBlockSize);  // slots, or table entries
  const cudaError_t e = launch_tables(&extend_tables_kernel, p, items, 3, s);
  if (e != cudaSuccess || fused) return e;
  return launch_pdl(fill_slots_kernel, dim3((p.num_tokens - 1) / kFillTokens + 1),
                    dim3(kFillThreads), 0, s, p);
}

cudaError_t launch_release_tables(const TableParams& p, cudaStream_t s) {
  // the blocks that come back are only known on the device; an eighth of the
  // requests at a quarter of the table's width is a busy step
  const long long items = static_cast<long long>(p.batch) * (1 + p.max_blocks / 32);
  return launch_tables(&release_tables_kernel, p, items, 1, s);
}

}  // namespace kvp
