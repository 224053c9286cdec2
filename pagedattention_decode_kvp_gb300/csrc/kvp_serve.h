// kvp_serve.h -- internal interface between the C ABI and the kernels of the 4-bit
// cache, the rotary append and the device-side block tables.
#pragma once

#include "kvp_internal.h"

namespace kvp {

// A decode over 4-bit pools: codes in k_pool / v_pool (no tensor maps, no scale
// pools), with
struct Int4DecodeParams : DecodeParams {
  const void* k_sz;             // (scale, zero) pairs [NB, Hkv, bs, D / 64, 2]
  const void* v_sz;
  int4* notes;                  // balanced decode (part_blocks == 0): one per CTA
};

// Resident CTAs of the 4-bit decode per SM: its step loop takes 168 registers at
// head_dim 128 (with 128 it spills: 119 us against 107 for 57 contexts of 9200
// tokens) and 128 at head_dim 64 (4 CTAs 70 us, 3 CTAs 76, 32 x 32 heads of 4096).
constexpr int int4_ctas_per_sm(int head_dim) { return head_dim == 128 ? 3 : 4; }

// How a balanced decode cuts `batch` contexts of `total` blocks together into at
// most `pieces` pieces: equal ones, contexts laid end to end -- or, where that
// makes the pieces longer by kAlign blocks at most, every context by itself into
// pieces of one size, so that no CTA has the end of one context and the start of
// another (sum of ceil(n / size) <= total / size + batch <= pieces).  By itself
// and end to end, in us: 8 contexts of 1000 to 2000 tokens, 8 kv heads, 12.9 and
// 14.8 (3 blocks longer); 100 of 200 to 3000, one kv head, 14.8 and 17.2 (8); 4 of
// 32768, 8 kv heads, 38.7 and 36.9 (11); 4 of 131072, 113 and 107 (43).
struct Cut {
  long long size;  // blocks of a piece
  bool aligned;    // every context by itself
};
constexpr int kMinRun = 8;  // blocks of a piece at least: two for every warp
constexpr int kAlign = 8;
__host__ __device__ inline Cut cut_contexts(long long total, int batch, int pieces) {
  const long long spare = pieces - batch;
  Cut c;
  c.aligned = batch > 1 && spare > 0 && total * batch <= kAlign * pieces * spare;
  const long long n = c.aligned ? spare : pieces;
  c.size = (total + n - 1) / n;
  if (c.size < kMinRun) c.size = kMinRun;
  return c;
}

// Heads of a token (query heads included) that the row kernels take: 32-bit
// offsets within its rows.
constexpr int kMaxRowHeads = 65535;

// Everything the row kernels (rotary positions, 4-bit quantisation, scatter)
// need.  Strides are elements from one token to the next.
struct RowParams {
  const uint16_t* q;            // [T, Hq, D] rows (rotary only)
  uint16_t* q_out;
  const uint16_t* key;          // [T, Hkv, D] rows
  const uint16_t* value;
  long long q_stride, q_out_stride, k_stride, v_stride;
  void* k_cache;                // 16-bit rows, or packed 4-bit codes
  void* v_cache;
  uint32_t* k_sz;               // 4-bit pools: (scale, zero) pairs
  uint32_t* v_sz;
  const float* cos_sin;         // [max_position, R]: R / 2 cosines, R / 2 sines
  const int32_t* positions;     // [num_axes, T]
  const int32_t* slots;         // [T]
  int32_t* status;              // nullable
  int32_t num_tokens, num_q_heads, num_kv_heads, num_slots, max_position;
  int32_t rotary_dim;           // R, a multiple of 16
  int32_t num_axes;
  int32_t axis_end[3];          // first pair past axis 0, 1, 2
  int32_t interleaved;          // pairs (2i, 2i + 1), else (i, i + R / 2)
  int32_t sections_by_4;        // every section is a multiple of 4 pairs
  int32_t row_shift;            // log2 of the rows of one token a CTA works on at a time (set
                                // at launch)
};

// Requests one table call handles (its offsets live in shared memory), and slots
// it lists (their indexes stay clear of 2^31 by a CTA's share).
constexpr int kMaxTableBatch = 16384;
constexpr int kMaxTableTokens = 1 << 30;

// Device-side block tables: extend (all fields) and release (no new_lens,
// slot_mapping, query_start, positions).
struct TableParams {
  int32_t* block_tables;        // [B, MB]
  const int32_t* context_lens;  // [B]
  const int32_t* new_lens;      // [B]
  const int32_t* finished;      // [B]
  int32_t* free_blocks;         // [num_blocks], the lowest *free_count are free
  const int32_t* free_count;
  int32_t* context_lens_out;    // may be context_lens
  int32_t* free_count_out;      // may be free_count
  int32_t* slot_mapping;        // [T]
  int32_t* query_start;         // [B + 1]
  int32_t* positions;           // [T], nullable
  int32_t* status;              // nullable
  int32_t batch, max_blocks, num_blocks, num_tokens;
};

// 4-bit pools (codes in k_pool / v_pool, pairs in k_sz / v_sz); part_blocks == 0:
// balanced over grid_x CTAs, whose cut units the second launch merges.
cudaError_t launch_decode_int4(const Int4DecodeParams& p, int grid_x, cudaStream_t s);
cudaError_t launch_decode_int4_merge(const Int4DecodeParams& p, int grid_x, cudaStream_t s);

cudaError_t launch_copy_blocks_int4(void* k_cache, void* v_cache, void* k_sz, void* v_sz,
                                    const int32_t* pairs, int num_pairs, const kvp_cache_desc& c,
                                    int32_t* status, cudaStream_t s);
cudaError_t launch_append_int4(const RowParams& p, bool bf16, int head_dim, cudaStream_t s);
cudaError_t launch_rope_append(const RowParams& p, bool bf16, int head_dim, bool int4,
                               cudaStream_t s);
cudaError_t launch_read_int4(void* key, void* value, bool bf16, const uint8_t* kc,
                             const uint8_t* vc, const void* ksz, const void* vsz,
                             const int32_t* slots, int num_tokens, const kvp_cache_desc& c,
                             int32_t* status, cudaStream_t s);
cudaError_t launch_extend_tables(const TableParams& p, cudaStream_t s);
cudaError_t launch_release_tables(const TableParams& p, cudaStream_t s);

}  // namespace kvp
