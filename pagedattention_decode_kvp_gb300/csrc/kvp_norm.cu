// kvp_norm.cu -- root-mean-square norms and E4M3 quantisers of 16-bit rows.
//
// Norm of a row x of D elements with weight w:
//   h = x, or RN16(x + residual) (float32 sum, rounded once and given back),
//   y_i = h_i * r * w_i,  r = 1 / sqrt(sum h^2 / D + eps),
// in float32; y is rounded once to the 16-bit type, or held as E4M3 codes.
//
// Codes of a group of 128 elements y (of a row, or of 128 rows of a weight):
//   a = max |y|,  b = max(a, 2^-100),  scale = b / 448 (1 where a = 0),
//   code = E4M3(y * (448 / b)),  each operation rounded to float32 by itself.
// The bound 2^-100 keeps 448 / b finite.
//
// A lane holds whole 16-byte chunks of 8 elements, a row's chunks lie on consecutive
// lanes, so that 16 lanes hold a group.  Bound by HBM for prompts and by one launch for a
// step.  Measured (calls back to back; shares of the measured copy bandwidth): norm in codes
// with a residual, 33098 rows of 4096, 138 us (1.03); norm with a residual, 8191 rows of 8192,
// 78 us (1.03); norm of 8191 x 64 heads of 128, 45 us (0.90, held by its instructions: 77 % of
// the issue slots; one row a slot 67 us, four 47, a factor worked out once a row 44, a look
// whether a row is out of range 0.6 more); 8191 rows of 8192 in codes 31 us (0.97; 8 elements
// a lane and float maxima 63); a weight of 10240 x 8192 in codes 39 us (0.96; float maxima
// 48); a step of 64 tokens of 8192 2.5 us, in codes 2.7.
#include "kvp_device.cuh"
#include "kvp_project.h"

namespace kvp {

namespace {

constexpr float kLargest = 448.0f;   // of E4M3

__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

template <bool kBf16>
__device__ __forceinline__ void widen(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = dev::unpack2<kBf16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool kBf16>
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(dev::pack2<kBf16>(x[0], x[1]), dev::pack2<kBf16>(x[2], x[3]),
                    dev::pack2<kBf16>(x[4], x[5]), dev::pack2<kBf16>(x[6], x[7]));
}

__device__ __forceinline__ float absmax8(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}

// Scale of a group whose largest magnitude is `most`, and what its elements are
// multiplied by.
__device__ __forceinline__ float group_scale(float most, float* up) {
  const float b = fmaxf(most, 0x1p-100f);
  *up = __fdiv_rn(kLargest, b);
  return most > 0.f ? __fdiv_rn(b, kLargest) : 1.0f;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float up) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = dev::f32x2_to_e4m3x2(__fmul_rn(x[2 * i], up), __fmul_rn(x[2 * i + 1], up));
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Largest of the values of `kLanes` neighbouring lanes.
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum of the values of a row's `kThreads` neighbouring threads (part: kThreads / 32 floats
// where they are a CTA).
template <int kThreads>
__device__ __forceinline__ float row_sum(float sum, float* part) {
#pragma unroll
  for (int o = (kThreads < 32 ? kThreads : 32) / 2; o > 0; o >>= 1)
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (kThreads > 32) {
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum += part[i];
  }
  return sum;
}

__device__ __forceinline__ float mean_square(float sum, int dim, float eps) {
  return __fadd_rn(__fdiv_rn(sum, static_cast<float>(dim)), eps);
}

__device__ __forceinline__ uint4 load_weight(const NormParams& p, int at) {
  return at < p.dim ? load16(p.weight + at) : make_uint4(0u, 0u, 0u, 0u);
}

// Results of 8 elements x of a row: token t, `at` elements behind the row's start, which is
// col elements behind the token's; r: the row's factor; weight: that of the elements.  Lanes
// that hold none (not `mine`) only take part in a group's maximum.
template <bool kBf16, bool kFp8, int kThreads>
__device__ __forceinline__ void put_results(const NormParams& p, uint32_t t, uint32_t col, int at,
                                            bool mine, float (&x)[8], float r,
                                            const uint4& weight) {
  float w[8];
  widen<kBf16>(weight, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  if constexpr (kFp8) {
    const float most = lanes_max<(kThreads < 16 ? kThreads : 16)>(mine ? absmax8(x) : 0.f);
    float up;
    const float scale = group_scale(most, &up);
    if (mine) {
      *reinterpret_cast<uint2*>(p.codes + t * p.codes_stride + at) = codes8(x, up);
      if (at % kScaleGroup == 0)
        p.scales[static_cast<size_t>(t) * ((p.dim + kScaleGroup - 1) / kScaleGroup) +
                 at / kScaleGroup] = scale;
    }
  } else if (mine) {
    *reinterpret_cast<uint4*>(p.out + t * p.out_stride + col + at) = narrow<kBf16>(x);
  }
}

// Whether a row's mean square does not give its factor: bf16 elements reach from 2^-133 to
// 2^128, their squares leave float32 (at 2^-100 those that vanish do not count any more).
__device__ __forceinline__ bool out_of_range(float mean) {
  constexpr uint32_t kLow = 27u << 23;   // 2^-100
  return __float_as_uint(mean) - kLow >= (255u << 23) - kLow;
}

// A row of bf16 beside, or itself, one that is out of range: read once more (with a
// residual, the sum that this thread wrote) and scaled by a power of two, a large one, its
// elements up to 2^128, by 2^-80, a small one, all of it below 2^-40, by 2^100.  Of a large
// row's factor half of the power stays with the elements, so that neither leaves float32.
// A row in range gets the bits that it has elsewhere.
template <bool kFp8, int kThreads, int kChunks>
__device__ __forceinline__ void put_far_row(const NormParams& p, uint32_t t, uint32_t col, bool in,
                                            float mean, float* part) {
  const int lane = static_cast<int>(threadIdx.x) % kThreads;
  const uint16_t* h = p.residual != nullptr ? p.residual_out + t * p.residual_out_stride
                                            : p.x + t * p.x_stride + col;
  float up = 1.f, more = 1.f;
  if (out_of_range(mean)) up = mean < 1.f ? 0x1p100f : 0x1p-40f;
  if (up < 1.f) more = up;
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < kChunks; ++c) {
    const int at = 8 * (lane + c * kThreads);
    float x[8];
    widen<true>(in && at < p.dim ? load16(h + at) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i] * up * more, x[i] * up * more, sum);
  }
  if constexpr (kThreads > 32) __syncthreads();   // (part has been read)
  sum = row_sum<kThreads>(sum, part);
  const float r =
      __frsqrt_rn(mean_square(sum, p.dim, p.eps * (up * more) * (up * more))) * more;
#pragma unroll 1
  for (int c = 0; c < kChunks; ++c) {
    const int at = 8 * (lane + c * kThreads);
    float x[8];
    widen<true>(in && at < p.dim ? load16(h + at) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= up;
    put_results<true, kFp8, kThreads>(p, t, col, at, in && at < p.dim, x, r,
                                      load_weight(p, at));
  }
}

// kThreads threads hold a row, kChunks chunks each; up to 32 of them: 128 / kThreads slots
// to a CTA, kRows rows a slot, fetched together; more: a CTA to a row.  kAhead: the weight is
// fetched beside the row.  Its registers cost a prompt's kernels warps (8191 rows of 8192 with
// a residual 78 us, 85 so), a step's CTAs, one to an SM, nothing (64 such rows 2.5 us, 2.3).
template <bool kBf16, bool kFp8, int kThreads, int kChunks, int kRows, bool kAhead>
__global__ void __launch_bounds__(kThreads < 128 ? 128 : kThreads) rms_norm_kernel(NormParams p) {
  constexpr int kSlots = kThreads < 128 ? 128 / kThreads : 1;
  __shared__ float part[kThreads > 32 ? kThreads / 32 : 1];
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kThreads;
  const uint32_t rows = static_cast<uint32_t>(p.num_tokens) * static_cast<uint32_t>(p.num_heads);
  uint4 raw[kRows][kChunks], other[kRows][kChunks];
  bool in[kRows];
  uint32_t t[kRows], col[kRows];   // token, and where the row lies within it
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const uint32_t row = (blockIdx.x * kRows + j) * kSlots + threadIdx.x / kThreads;
    in[j] = row < rows;
    t[j] = p.num_heads == 1 ? row : row / static_cast<uint32_t>(p.num_heads);
    col[j] = (row - t[j] * static_cast<uint32_t>(p.num_heads)) * static_cast<uint32_t>(p.dim);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int at = 8 * (lane + c * kThreads);
      raw[j][c] = other[j][c] = make_uint4(0u, 0u, 0u, 0u);
      if (in[j] && at < p.dim) {
        raw[j][c] = load16(p.x + t[j] * p.x_stride + col[j] + at);
        if (p.residual != nullptr)
          other[j][c] = load16(p.residual + t[j] * p.residual_stride + at);
      }
    }
  }
  uint4 weight[kAhead ? kChunks : 1];
  if constexpr (kAhead) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) weight[c] = load_weight(p, 8 * (lane + c * kThreads));
  }
  float sums[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float x[8];
      widen<kBf16>(raw[j][c], x);
      if (p.residual != nullptr) {
        float r[8];
        widen<kBf16>(other[j][c], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += r[i];
        raw[j][c] = narrow<kBf16>(x);
        widen<kBf16>(raw[j][c], x);
        const int at = 8 * (lane + c * kThreads);
        if (in[j] && at < p.dim)
          *reinterpret_cast<uint4*>(p.residual_out + t[j] * p.residual_out_stride + at) = raw[j][c];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    }
    sums[j] = row_sum<kThreads>(sum, part);
  }
  // lane j % kRows of a row's lanes works out row j's factor for all of them
  float mine_r = sums[0];
#pragma unroll
  for (int j = 1; j < kRows; ++j) mine_r = lane % kRows == j ? sums[j] : mine_r;
  mine_r = mean_square(mine_r, p.dim, p.eps);
  // (a vote of the warp: its rows stay together; of a CTA with one row all threads agree)
  if constexpr (kBf16) {
    if (__any_sync(0xffffffffu, out_of_range(mine_r))) {
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        put_far_row<kFp8, kThreads, kChunks>(p, t[j], col[j], in[j],
                                             mean_square(sums[j], p.dim, p.eps), part);
      return;
    }
  }
  mine_r = __frsqrt_rn(mine_r);
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float r = mine_r;
    if constexpr (kRows > 1) r = __shfl_sync(0xffffffffu, mine_r, j, kThreads < 32 ? kThreads : 32);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int at = 8 * (lane + c * kThreads);
      float x[8];
      widen<kBf16>(raw[j][c], x);
      put_results<kBf16, kFp8, kThreads>(p, t[j], col[j], at, in[j] && at < p.dim, x, r,
                                         kAhead ? weight[c] : load_weight(p, at));
    }
  }
}

// Largest magnitude of two 16-byte chunks, by pairs of 16-bit values (exact).
template <bool kBf16>
__device__ __forceinline__ uint32_t absmax_pair(const uint4& a, const uint4& b) {
  using dev::absmax2;
  return absmax2<kBf16>(absmax2<kBf16>(absmax2<kBf16>(a.x, a.y), absmax2<kBf16>(a.z, a.w)),
                        absmax2<kBf16>(absmax2<kBf16>(b.x, b.y), absmax2<kBf16>(b.z, b.w)));
}

// Rows by themselves: 8 lanes take a group, 16 elements each, kUnits groups fetched
// together.
constexpr int kQuantUnits = 4;
constexpr int kQuantSlots = 32;   // groups that a CTA of 256 threads works on at a time
template <bool kBf16>
__global__ void __launch_bounds__(256) quantise_rows_kernel(QuantiseParams p, uint32_t groups) {
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const int sub = threadIdx.x % 8;
  const uint32_t units = static_cast<uint32_t>(p.rows) * groups;
  const uint32_t first = blockIdx.x * (kQuantSlots * kQuantUnits) + threadIdx.x / 8;
  uint4 raw[kQuantUnits][2];
  uint32_t row[kQuantUnits];
  int at[kQuantUnits];
#pragma unroll
  for (int j = 0; j < kQuantUnits; ++j) {
    const uint32_t u = first + j * kQuantSlots;
    row[j] = u / groups;
    at[j] = static_cast<int>(u - row[j] * groups) * kScaleGroup + 16 * sub;
    if (u >= units || at[j] >= p.cols) at[j] = -1;
    raw[j][0] = raw[j][1] = make_uint4(0u, 0u, 0u, 0u);
    if (at[j] >= 0) {
      const uint16_t* x = p.x + row[j] * p.x_stride + at[j];
      raw[j][0] = load16(x);
      raw[j][1] = load16(x + 8);
    }
  }
#pragma unroll
  for (int j = 0; j < kQuantUnits; ++j) {
    uint32_t m = absmax_pair<kBf16>(raw[j][0], raw[j][1]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      m = dev::absmax2<kBf16>(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float2 two = dev::unpack2<kBf16>(m);
    float x[8], y[8], up;
    const float scale = group_scale(fmaxf(two.x, two.y), &up);
    if (at[j] < 0) continue;
    widen<kBf16>(raw[j][0], x);
    widen<kBf16>(raw[j][1], y);
    const uint2 a = codes8(x, up), b = codes8(y, up);
    *reinterpret_cast<uint4*>(p.codes + row[j] * p.codes_stride + at[j]) =
        make_uint4(a.x, a.y, b.x, b.y);
    if (sub == 0) p.scales[static_cast<size_t>(row[j]) * groups + at[j] / kScaleGroup] = scale;
  }
}

// A CTA takes 128 rows of 128 columns: 8 chunks a thread.
template <bool kBf16>
__global__ void __launch_bounds__(256) quantise_blocks_kernel(QuantiseParams p, int groups) {
  dev::grid_dependency_wait();
  dev::launch_dependents();
  const long long block = blockIdx.x / groups;
  const int group = blockIdx.x % groups;
  const int at = group * kScaleGroup + 8 * (threadIdx.x % 16);
  uint4 raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long row = block * kScaleGroup + threadIdx.x / 16 + 16 * j;
    raw[j] = row < p.rows && at < p.cols ? load16(p.x + row * p.x_stride + at)
                                         : make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    m = dev::absmax2<kBf16>(m, absmax_pair<kBf16>(raw[j], raw[j + 1]));
  const float2 two = dev::unpack2<kBf16>(m);
  float most = fmaxf(two.x, two.y);
  most = dev::warp_max(most);
  __shared__ float part[8];
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, part[i]);
  float up;
  const float scale = group_scale(most, &up);
  if (threadIdx.x == 0) p.scales[block * groups + group] = scale;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long row = block * kScaleGroup + threadIdx.x / 16 + 16 * j;
    if (row >= p.rows || at >= p.cols) continue;
    float x[8];
    widen<kBf16>(raw[j], x);
    *reinterpret_cast<uint2*>(p.codes + row * p.codes_stride + at) = codes8(x, up);
  }
}

template <bool kBf16, bool kFp8>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.num_tokens) * p.num_heads;
  const int chunks = p.dim / 8;
#define KVP_NORM(T, C, R)                                                               \
  {                                                                                     \
    constexpr int kPer = R * (T < 128 ? 128 / T : 1);                                   \
    auto kernel = rms_norm_kernel<kBf16, kFp8, T, C, R, false>;                         \
    if constexpr (T >= 128) {                                                           \
      if (rows <= kNumSms) kernel = rms_norm_kernel<kBf16, kFp8, T, C, R, true>;        \
    }                                                                                   \
    return launch_pdl(kernel, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)),    \
                      dim3(T < 128 ? 128 : T), 0, s, p);                                \
  }
  if (chunks <= 8) KVP_NORM(8, 1, 4)
  if (chunks <= 16) KVP_NORM(16, 1, 4)
  if (chunks <= 32) KVP_NORM(32, 1, 4)
  if (chunks <= 64) KVP_NORM(32, 2, 2)
  if (chunks <= 128) KVP_NORM(128, 1, 1)
  if (chunks <= 256) KVP_NORM(128, 2, 1)
  if (chunks <= 512) KVP_NORM(256, 2, 1)
  if (chunks <= 1024) KVP_NORM(512, 2, 1)
  if (chunks <= 2048) KVP_NORM(1024, 2, 1)
  if (chunks <= 4096) KVP_NORM(1024, 4, 1)
#undef KVP_NORM
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t s) {
  if (p.out == nullptr)
    return bf16 ? launch_norm<true, true>(p, s) : launch_norm<false, true>(p, s);
  return bf16 ? launch_norm<true, false>(p, s) : launch_norm<false, false>(p, s);
}

cudaError_t launch_quantise_fp8(const QuantiseParams& p, bool bf16, cudaStream_t s) {
  const int groups = (p.cols + kScaleGroup - 1) / kScaleGroup;
  if (p.block_rows == 1) {
    const long long units = static_cast<long long>(p.rows) * groups;
    constexpr int kPer = kQuantSlots * kQuantUnits;
    const dim3 grid(static_cast<unsigned>((units + kPer - 1) / kPer));
    return launch_pdl(bf16 ? quantise_rows_kernel<true> : quantise_rows_kernel<false>, grid,
                      dim3(256), 0, s, p, static_cast<uint32_t>(groups));
  }
  const long long blocks = (static_cast<long long>(p.rows) + kScaleGroup - 1) / kScaleGroup;
  const dim3 grid(static_cast<unsigned>(blocks * groups));
  return launch_pdl(bf16 ? quantise_blocks_kernel<true> : quantise_blocks_kernel<false>, grid,
                    dim3(256), 0, s, p, groups);
}

}  // namespace kvp
