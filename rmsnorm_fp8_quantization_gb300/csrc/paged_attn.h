// Parameter block and launchers of the paged attention's kernels.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "gbnorm.h"

namespace gbn {

struct AttnParams {
  const void* q;       // [tokens, hq, d]
  const void* k;       // cache
  const void* v;
  void* out;           // [tokens, hq, d]
  float* lse;          // [tokens, hq] or null
  const int32_t* cu;       // [batches + 1]
  const int32_t* kv_lens;  // [batches]
  const int32_t* table;
  const float* k_scale_inv;  // E4M3 caches
  const float* v_scale_inv;
  float* part_o;       // [splits][tokens * hq][d] fp32
  float2* part_ml;     // [tokens * hq][splits]: (reference in log2 units, sum)
  int64_t qt, qh;      // element strides of q
  int64_t ot, oh;      // of out
  int64_t kp, ks, kh;  // of the caches: page, slot, head
  int64_t vp, vs, vh;
  int64_t table_stride;
  int64_t num_pages;
  int tokens, batches;
  int hq, hkv, group;  // group = hq / hkv
  int d;
  int page_shift, table_pages;
  int max_q, max_kv;
  int causal, window;
  int row_tiles;       // row tiles per (sequence, kv head)
  int splits;
  int split_len;
  int cluster;         // the splits of a row tile are a thread-block cluster and merge themselves
  float scale_log2;    // scale * log2(e)
};

// Tensor map of a cache as [pages][slots][heads][d]: boxes of `inner` elements of
// one head in min(page, rows) slots, in the 128-byte (64-byte, where a row is no
// longer) swizzle or plain.  False if the driver refuses it.
bool make_cache_map(CUtensorMap* map, const void* base, int esize, bool bf16, int inner, int rows,
                    bool swizzle, const AttnParams& p, int64_t sp, int64_t ss, int64_t sh);

// The tcgen05 kernel for many rows per kv head (two-byte caches and E4M3,
// head sizes up to 128).
cudaError_t launch_paged_prefill(const AttnParams& p, gbn_dtype dtype, gbn_dtype cache_dtype,
                                 cudaStream_t stream);
cudaError_t read_prefill_error(unsigned int* v, bool clear);
cudaError_t read_attention_error(unsigned int* v, bool clear);
cudaError_t read_rope_error(unsigned int* v, bool clear);

constexpr int kPrefillRows = 256;  // rows (token x head of the group) per CTA of that kernel
constexpr int kPrefillKeys = 128;  // keys per tile of it

}  // namespace gbn
