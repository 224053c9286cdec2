// kvp_project.h -- internal interface between the C ABI and the kernels of a layer's
// projections: norms, E4M3 quantisers and the block-scaled matrix product.
#pragma once

#include "kvp_internal.h"
#include "kvp_matmul_plan.h"

namespace kvp {

constexpr int kScaleGroup = 128;       // elements of a row, and rows of a weight, per scale
constexpr int kMaxNormDim = 32768;     // elements of a row that a CTA holds in registers

// Rows of a norm: token t's head h starts at x + t * x_stride + h * dim (elements).
struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;   // nullable (one head only)
  uint16_t* residual_out;
  const uint16_t* weight;     // [dim]
  uint16_t* out;              // 16-bit rows, or null:
  uint8_t* codes;             // E4M3 rows, codes_stride bytes apart
  float* scales;              // [T, ceil(dim / 128)]
  long long x_stride, residual_stride, residual_out_stride, out_stride, codes_stride;
  int32_t num_tokens, num_heads, dim;
  float eps;
};

struct QuantiseParams {
  const uint16_t* x;          // rows x_stride elements apart
  uint8_t* codes;             // rows codes_stride bytes apart
  float* scales;              // [ceil(rows / block_rows), ceil(cols / 128)]
  long long x_stride, codes_stride;
  int32_t rows, cols, block_rows;
};

// out[m, n] = sum_g a_scale[m, g] b_scale[n / 128, g] sum_{k in g} a[m, k] b[n, k].
struct MatmulParams {
  void* out;                  // [M, N], rows out_stride elements apart
  const float* a_scale;       // [M, groups]
  const float* b_scale;       // [ceil(N / 128), groups]
  int32_t* status;            // nullable
  long long out_stride;
  int32_t m, n, groups;       // groups = ceil(K / 128)
  int32_t out_type;           // a kvp_dtype
};

cudaError_t launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t s);
cudaError_t launch_quantise_fp8(const QuantiseParams& p, bool bf16, cudaStream_t s);
// ta, tb: K-major maps of a and b with boxes of 128 bytes x plan.box() (a) and 128 rows (b).
cudaError_t launch_matmul_fp8(const MatmulParams& p, const MatmulPlan& plan, const CUtensorMap& ta,
                              const CUtensorMap& tb, cudaStream_t s);
cudaError_t launch_matmul_fp8_pair(const MatmulParams& p, const CUtensorMap& ta,
                                   const CUtensorMap& tb, cudaStream_t s);

}  // namespace kvp
