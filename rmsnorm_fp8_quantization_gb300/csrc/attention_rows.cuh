// Parameters, masks and the gradients pair by pair of the attention's backward pass.
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

// Four elements; beyond the head 0.
template <typename T>
__device__ __forceinline__ uint2 four_words(const T* row, int col, int d) {
  return col < d ? *reinterpret_cast<const uint2*>(row + col) : make_uint2(0u, 0u);
}
template <typename T>
__device__ __forceinline__ void four_floats(uint2 w, float* f) {
  const uint32_t a[2] = {w.x, w.y};
  unpack<T, 4>(a, f);
}

// The columns from `first` on of one row's gradient that came out NaN, by a whole warp: dq of query x (WHICH 0,
// of q head `head`), or dk (1) and dv (2) of key x of kv head h; dst: the row.
//
// The products of whole tiles give a pair that is not kept the weight 0, and 0 times an infinity or NaN
// is NaN.  So a NaN either belongs there or comes from a row of the other side that x's tiles hold and
// x dropped; then the sum is taken again pair by pair, over the kept pairs alone.  That costs a pass over
// the range for a row, so what can be told from less is told from less:
//  * a query's -lse or -delta that is NaN makes every kept pair's share NaN;
//  * the rows that x dropped, at most two tiles of them, hold nothing infinite or NaN (queries: their lse and
//    delta are numbers; lse is not where a kept score is not, delta is not where dout is not): it belongs;
//  * kept pairs whose share is infinite or NaN alone decide the sum, if there are any: dk and dv take them
//    first, dq looks for columns of kept keys that are not finite (lse is, so their weight is 0, and 0
//    times them NaN).
// A lane takes four columns; every sum in a fixed order.  (2 x 4096 tokens, 32 / 8 heads of 128, causal, 0.61 ms
// without such values: a NaN in a gradient, inside a tile, 26 ms; infinities of either sign in every seventh 1.1;
// nothing but one infinity 105, where no share decides.)
template <typename T, int WHICH>
__device__ __noinline__ void grad_again(const AttnBwdParams& p, const SeqRange& s, int b, int head, int h, int x,
                                        int first, int columns, T* dst) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  constexpr bool kv = WHICH != 0;
  constexpr int kAtOnce = 8;  // pairs under way
  const int lane = threadIdx.x & 31, col = lane * 4;
  const int heads = kv ? p.group : 1;
  const int lo = kv ? query_first(p, s, x) : key_first(p, s, x);
  const int hi = kv ? query_end(p, s, x) : key_end(p, s, x);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t need = 0;  // bit e: column col + e
  if (col >= first && col < min(first + columns, p.d)) {
    float f[4];
    four_floats<T>(four_words(dst, col, p.d), f);
#pragma unroll
    for (int e = 0; e < 4; ++e) need |= f[e] != f[e] ? 1u << e : 0u;
  }
  if (!__any_sync(kAll, need != 0u)) return;
  auto write = [&](uint32_t which) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((which >> e) & 1u)
        reinterpret_cast<uint16_t*>(dst)[col + e] = static_cast<uint16_t>(narrow2<T>(p2(acc[e], acc[e])));
  };
  if (hi <= lo) return write(need);

  const int64_t stat = stat_base(s.q0, b) + static_cast<int64_t>(kv ? h * p.group : head) * p.stat_stride;
  const float* const nlse = p.nlse + stat;
  const float* const ndelta = p.ndelta + stat;
  float own_nl = 0.f, own_nd = 0.f;
  if constexpr (!kv) {
    own_nl = nlse[x];
    own_nd = ndelta[x];
    if (own_nl != own_nl || own_nd != own_nd) return;
  }
  // Rows of the other side, this lane's columns: q or k, dout or v.  (What a row needs, out of the
  // parameters once: read there for every row it is what the passes below wait for.)
  const bool has = col < p.d;
  const int64_t row0 = kv ? s.q0 : s.k0, step1 = kv ? p.qt : p.kt, step2 = kv ? p.gt : p.vt;
  const int64_t head1 = kv ? p.qh : p.kh, head2 = kv ? p.gh : p.vh, stats = p.stat_stride;
  const T* const base1 = static_cast<const T*>(kv ? p.q : p.k) + row0 * step1 + (kv ? h * p.group : h) * head1 + col;
  const T* const base2 = static_cast<const T*>(kv ? p.dout : p.v) + row0 * step2 + (kv ? h * p.group : h) * head2 + col;
  const float scale_log2 = p.scale_log2;
  auto four = [&](const T* at) { return has ? *reinterpret_cast<const uint2*>(at) : make_uint2(0u, 0u); };
  auto not_finite = [&](int y) {  // of k's columns (dq)
    float f[4];
    four_floats<T>(four(base1 + y * step1), f);
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) r |= finite32(f[e]) ? 0u : 1u << e;
    return r;
  };

  // The rows of x's tiles that x dropped.
  {
    const int x0 = x & ~(kBwdTile - 1), last = min(x0 + kBwdTile, kv ? s.kv : s.qlen) - 1;
    const int from = (kv ? query_first(p, s, x0) : key_first(p, s, x0)) & ~(kBwdTile - 1);
    const int end = kv ? query_end(p, s, last) : key_end(p, s, last);
    const int to = min((end + kBwdTile - 1) & ~(kBwdTile - 1), kv ? s.qlen : s.kv);
    const int count = to - from - (hi - lo);
    auto dropped = [&](int o) { return from + o < lo ? from + o : from + o + hi - lo; };
    if constexpr (kv) {
      bool any = false;
      for (int g = 0; g < heads && !any; ++g) {
        const float* const nl = nlse + g * stats;
        const float* const nd = ndelta + g * stats;
        bool bad = false;
#pragma unroll 4
        for (int o = lane; o < count; o += 32) bad |= !finite32(nl[dropped(o)]) || !finite32(nd[dropped(o)]);
        any = __any_sync(kAll, bad);
      }
      if (!any) return;
    } else {
      uint32_t bad = 0;
#pragma unroll 8
      for (int o = 0; o < count; ++o) bad |= not_finite(dropped(o));
      need &= bad;
      if (!__any_sync(kAll, need != 0u)) return;
    }
  }

  float a[4], c[4];  // x's own row: k or q, v or dout
  {
    const int64_t row = static_cast<int64_t>(kv ? s.k0 : s.q0) + x;
    four_floats<T>(four_words(static_cast<const T*>(kv ? p.k : p.q) + (kv ? row * p.kt + h * p.kh : row * p.qt + head * p.qh),
                              col, p.d), a);
    four_floats<T>(four_words(static_cast<const T*>(kv ? p.v : p.dout) + (kv ? row * p.vt + h * p.vh : row * p.gt + head * p.gh),
                              col, p.d), c);
  }
  // Adds the shares of the pairs with rows y[0 ..] of the group's head g (negative: none).
  auto add = [&](int g, const int* y) {
    uint2 w1[kAtOnce], w2[kAtOnce];
    // The pair whose weight this lane computes.
    const int which = lane / (32 / kAtOnce);
    int mine = -1;
    const T* const from1 = base1 + g * head1;
    const T* const from2 = base2 + g * head2;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      w1[i] = w2[i] = make_uint2(0u, 0u);
      if (i == which) mine = y[i];
      if (y[i] < 0) continue;
      w1[i] = four(from1 + y[i] * step1);
      w2[i] = four(from2 + y[i] * step2);
    }
    float nl = own_nl, nd = own_nd, z[kAtOnce], dp[kAtOnce];
    if (kv && mine >= 0) {
      nl = nlse[g * stats + mine];
      nd = ndelta[g * stats + mine];
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      float f[4];
      four_floats<T>(w1[i], f);
      z[i] = fmaf(a[3], f[3], fmaf(a[2], f[2], fmaf(a[1], f[1], a[0] * f[0])));
      four_floats<T>(w2[i], f);
      dp[i] = fmaf(c[3], f[3], fmaf(c[2], f[2], fmaf(c[1], f[1], c[0] * f[0])));
    }
    const float zs = sum_of_pairs<kAtOnce>(z), dps = WHICH == 2 ? 0.f : sum_of_pairs<kAtOnce>(dp);
    const float w = ex2(fmaf(zs, scale_log2, nl));
    const float weight = mine < 0 ? 0.f : WHICH == 2 ? w : w * (dps + nd);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      float f[4];
      four_floats<T>(WHICH == 2 ? w2[i] : w1[i], f);
      const float v = __shfl_sync(kAll, weight, i * (32 / kAtOnce));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(v, f[e], acc[e]);
    }
  };
  // Nothing that is added changes what is NaN already.
  auto settled = [&] {
    uint32_t nan = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) nan |= acc[e] != acc[e] ? 1u << e : 0u;
    return __all_sync(kAll, (need & ~nan) == 0u);
  };

  if constexpr (kv) {
    bool some = false;
#pragma unroll 1
    for (int g = 0; g < heads; ++g)
#pragma unroll 1
      for (int o = lo; o < hi; o += 32) {
        float nl = 0.f, nd = 0.f;
        if (o + lane < hi) {
          nl = nlse[g * stats + o + lane];
          nd = ndelta[g * stats + o + lane];
        }
        if (__any_sync(kAll, nl != nl || (WHICH == 1 && nd != nd))) return;
        uint32_t bad = __ballot_sync(kAll, !finite32(nl) || !finite32(nd));
        if (!bad) continue;
        some = true;
#pragma unroll 1
        while (bad) {
          int y[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            y[i] = bad ? o + __ffs(bad) - 1 : -1;
            bad &= bad - 1;  // (0 stays 0)
          }
          add(g, y);
        }
        if (settled()) return;
      }
    if (some) {
      uint32_t nan = 0, inf = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        nan |= acc[e] != acc[e] ? 1u << e : 0u;
        inf |= fabsf(acc[e]) == INFINITY ? 1u << e : 0u;
      }
      write(need & inf);
      need &= ~(nan | inf);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = 0.f;
    }
  } else if (finite32(own_nl)) {
    uint32_t bad = 0;
#pragma unroll 8
    for (int o = lo; o < hi; ++o) bad |= not_finite(o);
    need &= ~bad;
  }
  if (!__any_sync(kAll, need != 0u)) return;

#pragma unroll 1
  for (int g = 0; g < heads; ++g)
#pragma unroll 1
    for (int o = lo; o < hi; o += kAtOnce) {
      int y[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) y[i] = o + i < hi ? o + i : -1;
      add(g, y);
      if ((o - lo) % 64 == 0 && settled()) return;
    }
  const float factor = ex2(-static_cast<float>(kWeightLog2<T>)) * (WHICH == 2 ? 1.f : p.scale);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] *= factor;
  write(need);
}

cudaError_t launch_attention_bwd_bf16(const AttnBwdParams& p, cudaStream_t stream);
cudaError_t launch_attention_bwd_f16(const AttnBwdParams& p, cudaStream_t stream);
cudaError_t read_attention_bwd_bf16_error(unsigned int* v, bool clear);
cudaError_t read_attention_bwd_f16_error(unsigned int* v, bool clear);

}  // namespace gbn
