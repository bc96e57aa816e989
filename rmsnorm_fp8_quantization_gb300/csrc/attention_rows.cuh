// Parameters, masks and the key-by-key gradients of the attention's backward pass.
//
// With p_ij = 2^(scale log2(e) q_i.k_j - lse_i log2(e)) (kept pairs), dp_ij = dout_i.v_j
// and delta_i = dout_i.out_i:
//     ds_ij = p_ij (dp_ij - delta_i),
//     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
// the sums for a key over the queries of every head of its group.
#pragma once

#include "paged_rows.cuh"

namespace gbn {

struct AttnBwdParams {
  const void *q, *k, *v, *out, *dout;
  const float* lse;         // [tokens, hq]
  const int32_t *cu, *cu_k;  // [batches + 1], or null: max_q, max_k rows each
  void *dq, *dk, *dv;
  float* nlse;    // [hq][stat_stride]: -lse log2(e) (+ kWeightLog2), sequences 16-byte aligned
  float* ndelta;  // [hq][stat_stride]: -delta
  float* q_norms;  // f16: [hq][q_norm_stride], largest squared norms of kStatTokens rows of dout
  float* v_norms;  // and [hkv][v_norm_stride] of v
  int64_t qt, qh, kt, kh, vt, vh, ot, oh, gt, gh;  // element strides: token, head (g: dout)
  int64_t dqt, dqh, dkt, dkh, dvt, dvh;
  int64_t stat_stride, q_norm_stride, v_norm_stride;
  int tokens, keys, batches, hq, hkv, group, d, max_q, max_k;
  int causal, window;
  float *kv_part, *q_part;  // sums in parts: [kv_splits][dk, dv][keys][hkv][d], [q_splits][tokens][hq][d]
  int kv_splits, q_splits;         // CTAs that share a tile's steps
  int kv_each, q_each;             // heads that a CTA takes one after another
  int kv_join_blocks, join_blocks;
  int kv_blocks, q_blocks;         // CTAs for dk and dv, and for dq
  int q_stat_blocks, stat_blocks;  // of the row statistics: for q's rows, and with v's
  float scale, scale_log2;
};

constexpr int kBwdTile = 128;   // queries and keys of a tile
constexpr int kStatTokens = 16;  // rows that share a norm

// f16 ends at 2^-14 (2^-24 with fewer bits) where fp32 and bf16 go on, and probabilities
// reach that with a few thousand keys: f16 ones are taken 2^12 larger (at most 2^12 then,
// with room for a score's rounding), so they keep their 11 bits down to 2^-26.
template <typename T>
constexpr int kWeightLog2 = Elem<T>::kDt == DT_F16 ? 12 : 0;

// Where sequence b's row statistics begin: a multiple of 4 (16 bytes, for bulk copies), and
// at least its rows before the next sequence's.
__device__ __forceinline__ int64_t stat_base(int q0, int b) {
  return (static_cast<int64_t>(q0) + 3 * static_cast<int64_t>(b) + 3) & ~int64_t(3);
}

// Where the norms of sequence b's rows begin (its first row: `first`).
__device__ __forceinline__ int64_t norm_base(int first, int b) { return first / kStatTokens + b; }

__device__ __forceinline__ SeqRange bwd_range(const AttnBwdParams& p, int b, bool flag) {
  return packed_range(p.cu, p.cu_k, b, p.tokens, p.keys, p.max_q, p.max_k, flag);
}

// Keys [first, end) of query i, queries [first, end) of key j.  (64 bits: a window near
// 2^31 must not wrap.)
__device__ __forceinline__ int key_end(const AttnBwdParams& p, const SeqRange& s, int i) {
  return p.causal ? min(max(s.off + i + 1, 0), s.kv) : s.kv;
}
__device__ __forceinline__ int key_first(const AttnBwdParams& p, const SeqRange& s, int i) {
  if (p.window <= 0) return 0;
  const int64_t l = static_cast<int64_t>(s.off) + i - p.window + 1;
  return l > 0 ? static_cast<int>(min(l, static_cast<int64_t>(s.kv))) : 0;
}
__device__ __forceinline__ int query_first(const AttnBwdParams& p, const SeqRange& s, int j) {
  return p.causal ? min(max(j - s.off, 0), s.qlen) : 0;
}
__device__ __forceinline__ int query_end(const AttnBwdParams& p, const SeqRange& s, int j) {
  if (p.window <= 0) return s.qlen;
  const int64_t e = static_cast<int64_t>(j) - s.off + p.window;
  return e > 0 ? static_cast<int>(min(e, static_cast<int64_t>(s.qlen))) : 0;
}

template <typename T>
__device__ __forceinline__ void eight(const void* base, int64_t at, float* f) {
  const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
  const uint32_t h[4] = {w.x, w.y, w.z, w.w};
  unpack<T, 8>(h, f);
}
template <typename T>
__device__ __forceinline__ float row_dot(const void* a, int64_t at, const void* b, int64_t bt, int d) {
  float s = 0.f;
  for (int c = 0; c < d; c += 8) {
    float x[8], y[8];
    eight<T>(a, at + c, x);
    eight<T>(b, bt + c, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
  }
  return s;
}
// Bit e: f[e] is NaN.
__device__ __forceinline__ uint32_t nan_bits(const float* f) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) r |= f[e] != f[e] ? 1u << e : 0u;
  return r;
}

// (p, ds) of one kept pair: query i of `head`, key j of kv head h; p 2^kWeightLog2 larger.
template <typename T>
__device__ __forceinline__ float2 pair_again(const AttnBwdParams& p, const SeqRange& s, int64_t stat,
                                             int head, int h, int i, int j) {
  const int64_t qi = s.q0 + i, kj = s.k0 + j;
  const float z = row_dot<T>(p.q, qi * p.qt + head * p.qh, p.k, kj * p.kt + h * p.kh, p.d);
  const float w = ex2(fmaf(z, p.scale_log2, p.nlse[head * p.stat_stride + stat + i]));
  const float dp = row_dot<T>(p.dout, qi * p.gt + head * p.gh, p.v, kj * p.vt + h * p.vh, p.d);
  return make_float2(w, w * (dp + p.ndelta[head * p.stat_stride + stat + i]));
}

// Eight columns of one row's gradient, f: dq of query `row` (of q head `head`), or dk (WHICH 1)
// and dv (2) of key `row` of kv head h.  The products of whole tiles give a pair that is not
// kept the weight 0, and 0 times an infinity or NaN is NaN: columns that came out NaN next to
// such pairs are computed here pair by pair, where those do not enter.  Rare, and slow; a NaN that
// belongs there (a kept gradient's, its row's delta, or what an infinite delta makes of its row) is
// looked for first, and ends it (4096 tokens, 8 / 2 heads of 128, f16: one such gradient 31 ms a call, an
// infinity in every seventh 62).
template <typename T, int WHICH>
__device__ __noinline__ void grad_again(const AttnBwdParams& p, const SeqRange& s, int b, int head,
                                        int h, int row, int col, float* f) {
  const uint32_t need = nan_bits(f);
  const int64_t stat = stat_base(s.q0, b);
  const int lo = WHICH ? query_first(p, s, row) : key_first(p, s, row);
  const int hi = WHICH ? query_end(p, s, row) : key_end(p, s, row);
  const int heads = WHICH ? p.group : 1;
  uint32_t sure = 0;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int g = 0; g < heads; ++g) {
    const int n = WHICH ? h * p.group + g : head;
#pragma unroll 1
    for (int o = lo; o < (WHICH ? hi : min(hi, lo + 1)); ++o) {
      const int i = WHICH ? o : row;
      if (WHICH != 2) {
        const float nd = p.ndelta[n * p.stat_stride + stat + i];
        if (nd != nd) return;
        if (WHICH == 1 && fabsf(nd) == INFINITY) {
          // (what these pairs alone make NaN, the whole sum has NaN)
          const float2 w = pair_again<T>(p, s, stat, n, h, i, row);
          float x[8];
          eight<T>(p.q, (s.q0 + static_cast<int64_t>(i)) * p.qt + n * p.qh + col, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(w.y, x[e], acc[e]);
          if ((need & ~nan_bits(acc)) == 0u) return;
        }
      } else {
        float x[8];
        eight<T>(p.dout, (s.q0 + static_cast<int64_t>(i)) * p.gt + n * p.gh + col, x);
        sure |= nan_bits(x);
        if ((need & ~sure) == 0u) return;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int g = 0; g < heads; ++g) {
    const int n = WHICH ? h * p.group + g : head;
#pragma unroll 1
    for (int o = lo; o < hi; ++o) {
      const int i = WHICH ? o : row, j = WHICH ? row : o;
      const float2 w = pair_again<T>(p, s, stat, n, h, i, j);
      float x[8];
      if (WHICH == 0) eight<T>(p.k, (s.k0 + static_cast<int64_t>(j)) * p.kt + h * p.kh + col, x);
      if (WHICH == 1) eight<T>(p.q, (s.q0 + static_cast<int64_t>(i)) * p.qt + n * p.qh + col, x);
      if (WHICH == 2) eight<T>(p.dout, (s.q0 + static_cast<int64_t>(i)) * p.gt + n * p.gh + col, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(WHICH == 2 ? w.x : w.y, x[e], acc[e]);
      if ((need & ~nan_bits(acc)) == 0u) return;  // (nothing that is added changes that)
    }
  }
  const float factor = ex2(-static_cast<float>(kWeightLog2<T>)) * (WHICH == 2 ? 1.f : p.scale);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (need & (1u << e)) f[e] = acc[e] * factor;
}

cudaError_t launch_attention_bwd_bf16(const AttnBwdParams& p, cudaStream_t stream);
cudaError_t launch_attention_bwd_f16(const AttnBwdParams& p, cudaStream_t stream);
cudaError_t read_attention_bwd_bf16_error(unsigned int* v, bool clear);
cudaError_t read_attention_bwd_f16_error(unsigned int* v, bool clear);

}  // namespace gbn
