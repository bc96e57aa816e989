// Rows, masks and key ranges of the paged attention.
//
// The rows of one (sequence, kv head) are its new tokens times the group's
// query heads: row r is token r / group, head kvh * group + r % group, so
// the heads that share keys share a tile and the keys are read once for all
// of them.  Token i stands at key position off + i (off = kv_len - q_len) and
// keeps the keys j in [low(i), high(i)):
//   high = off + i + 1 (causal) or kv_len, low = off + i - window + 1 or 0.
#pragma once

#include <atomic>

#include "paged.cuh"
#include "paged_attn.h"

namespace gbn {

// Raises a kernel's limit of dynamic shared memory, once per kernel and device
// (`done`: one bit per device; the setting lasts as long as the context).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

struct SeqRange {
  int q0;    // first token
  int qlen;  // new tokens
  int kv;    // keys with them
  int off;   // kv - qlen (negative: the first tokens keep nothing)
};

// Sequence b's lengths, bounded by the buffers whatever the values are; what
// does not fit is flagged.
__device__ __forceinline__ SeqRange seq_range(const AttnParams& p, int b, bool flag) {
  SeqRange s;
  const int c0 = p.cu[b], c1 = p.cu[b + 1], kv = p.kv_lens[b];
  s.q0 = min(max(c0, 0), p.tokens);
  s.qlen = min(max(c1, s.q0), p.tokens) - s.q0;
  const int64_t room = static_cast<int64_t>(p.table_pages) << p.page_shift;
  s.kv = static_cast<int>(min(static_cast<int64_t>(min(max(kv, 0), p.max_kv)), room));
  s.off = s.kv - s.qlen;
  if (flag && (s.q0 != c0 || s.q0 + s.qlen != c1 || s.kv != kv || s.qlen > p.max_q))
    flag_bad_index();
  return s;
}

__device__ __forceinline__ int row_high(const AttnParams& p, const SeqRange& s, int i) {
  return p.causal ? min(max(s.off + i + 1, 0), s.kv) : s.kv;
}
__device__ __forceinline__ int row_low(const AttnParams& p, const SeqRange& s, int i) {
  // 64-bit: a window near 2^31 must not wrap.
  if (p.window <= 0) return 0;
  const int64_t l = static_cast<int64_t>(s.off) + i - p.window + 1;
  return l > 0 ? static_cast<int>(min(l, static_cast<int64_t>(s.kv))) : 0;
}

__device__ __forceinline__ float ex2(float a) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
// The reference that a row's probabilities 2^(s - reference) are taken against, from
// its maximum m (log2 units; -inf stays).  bf16: m itself.  f16 ends at 2^-14 (2^-24
// with fewer bits) where fp32 and bf16 go on: against m, 262144 keys 18 nats below one
// that dominates would all vanish from the product with the values and stay in the
// sum.  So f16 takes a reference 2^H lower, which the division by the sum takes out
// again; not for maxima whose own spacing (2^-3 from 2^20 on) would blur it.
template <typename T, int H>
__device__ __forceinline__ float reference(float m) {
  if constexpr (Elem<T>::kDt == DT_F16) return fabsf(m) < 1048576.f ? m - H : m;
  else return m;
}
// 16 bytes into shared memory, zeros where not `live` (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
// One box of a tensor map into shared memory, reported as transactions on `bar`.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                        int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// Two E4M3 codes (low 16 bits) to a pair of f16, exact; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(c));
  return r;
}

// Eight elements of a q row (T) to f16 in place, next to E4M3 keys.  bf16 rows
// are scaled by the power of two that brings the row's largest magnitude into
// [2^8, 2^9); returns what undoes it.  The row's chunks are in C neighbouring
// lanes (a power of two), all of which call this together.
template <typename T, int C>
__device__ __forceinline__ float q_to_f16(uint4& w) {
  if constexpr (Elem<T>::kDt == DT_F16) {
    return 1.f;
  } else {
    float f[8];
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    unpack<T, 8>(in, f);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
    for (int o = C / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    // 2^(8 - exponent), the exponent within what keeps both factors normal.
    const int ex = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -110), 127);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - ex) << 23);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = narrow2<__half>(p2(f[2 * e] * up, f[2 * e + 1] * up));
    w = make_uint4(o[0], o[1], o[2], o[3]);
    return __uint_as_float(static_cast<uint32_t>(127 - 8 + ex) << 23);
  }
}

// Eight cache elements from element offset `at`.
template <typename T, bool FP8>
__device__ __forceinline__ void cache_values(const void* cache, int64_t at, float* f) {
  if constexpr (FP8) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at);
    const uint32_t h[4] = {e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16),
                           e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16)};
    unpack<__half, 8>(h, f);
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const T*>(cache) + at);
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
    unpack<T, 8>(h, f);
  }
}

// Eight output columns of one row again, key by key, over j in [lo, hi) alone:
// l times the mean of v_j with the weights 2^(scale q.k_j), l the row's sum.  The
// products of whole tiles give a dropped key the weight 0, and 0 times an infinity
// or NaN among its values is NaN; a row that dropped keys of its tiles and came out
// NaN is computed here, where dropped keys do not enter (a NaN that belongs there
// comes out again).  Against its own maximum and sum: of large scores the rounding,
// which goes by the order of summation, exceeds one.  Rare, and slow.
template <typename T, bool FP8>
__device__ __noinline__ void row_again(const AttnParams& p, int b, int h, const T* q, float scale,
                                       float l, int lo, int hi, int col, float* acc) {
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass)
    for (int j = lo; j < hi; ++j) {
      const int pg = p.table[b * p.table_stride + (j >> p.page_shift)];
      if (pg < 0 || pg >= p.num_pages) continue;
      const int slot = j & ((1 << p.page_shift) - 1);
      const int64_t ko = pg * p.kp + slot * p.ks + h * p.kh, vo = pg * p.vp + slot * p.vs + h * p.vh;
      float s = 0.f;
      for (int c = 0; c < p.d; c += 8) {
        float qf[8], kf[8];
        const uint4 w = *reinterpret_cast<const uint4*>(q + c);
        const uint32_t qw[4] = {w.x, w.y, w.z, w.w};
        unpack<T, 8>(qw, qf);
        cache_values<T, FP8>(p.k, ko + c, kf);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(qf[e], kf[e], s);
      }
      s = __fmul_rn(s, scale);  // (not into the subtraction below: its rounding is the maximum's)
      if (pass == 0) {
        top = fmaxf(top, s);
        continue;
      }
      const float w = ex2(s - (top == -INFINITY ? 0.f : top));
      sum += w;
      float vf[8];
      cache_values<T, FP8>(p.v, vo + col, vf);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, vf[e], acc[e]);
    }
  const float back = sum == 0.f ? 0.f : l / sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] *= back;
}

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kAttnLog2e = 1.4426950408889634f;

}  // namespace gbn
