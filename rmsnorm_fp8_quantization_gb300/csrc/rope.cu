// Rotary positions, and the append of new keys and values to a paged cache
// with the rotation applied on the way.
//
// A pair (a, b) of a head's elements at position p turns by the angle
// p * inv_freq[i]:   a' = m (a cos - b sin),   b' = m (a sin + b cos),
// m the caller's mscale; the backward is the transpose (angle negated).
//
// Angles.  A position's angle matters modulo one turn only, so it is kept as
// a 64-bit fixed-point fraction of a turn: inv_freq / (2 pi) * 2^64 times the
// position in wrapping integer arithmetic is exact modulo one turn up to the
// fraction's own error for each position (2^-64 of a turn, and 2^-66 of the frequency
// from 64 bits of 2 / pi: another word of it, for frequencies beyond 4, cost registers
// and 15 % of the fp32 kernel's time), where the product in fp32 would have no
// fraction left at far positions.  (The leading bits of 2 / pi: after Payne and
// Hanek's reduction.)  What is left after
// taking off the nearest quarter turn converts to fp32 with a relative error
// of 2^-24, and cos and sin of it come from sincospif.  No 64-bit
// floating-point arithmetic: its rate on this chip is about 1/64 of fp32's.
//
// Shape of the work.  The kernels are bound by HBM (each element read once
// and written once).  A unit is one pair of vectors: V elements a and the V
// elements b they turn with (16 bytes each; 8 bytes or single elements where
// the sizes, strides or pointers do not allow it).  A CTA of 256 threads
// takes up to 4 units a thread -- whole tokens while they fit, else a range
// of a token's heads -- and issues all its loads before it computes the
// cosines of its tokens (one per token and pair, into shared memory, read by
// every head), so that the loads' latency covers the arithmetic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"
#include "gbn_internal.h"

namespace gbn {
namespace {

// What a caller in another language lays out by hand.
static_assert(sizeof(gbn_rope_args) == 6 * 8 + 19 * 8 + 4 * 4, "");
static_assert(sizeof(gbn_paged_append_args) == 12 * 8 + 24 * 8 + 4 * 4, "");

constexpr int kRopeThreads = 256;
constexpr int kRopeUnits = 4;                       // units per thread
constexpr int kRopeItems = kRopeThreads * kRopeUnits;
constexpr int kRopeMaxTokens = 64;                  // tokens per CTA
constexpr int kRopeTrig = 2048;                     // (cos, sin) pairs per CTA (16 KB)

struct Strided {  // element strides
  int64_t b, s, h;
};

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;          // append only
  void* q_out;
  void* k_out;            // append: the key cache
  void* v_out;            // append: the value cache
  Strided qs, ks, vs, qo, ko, vo;  // append: ko / vo = (page, slot, head) of the caches
  const double* inv_freq;
  const void* positions;  // rope: int32 or int64, or null for 0, 1, ...
  int64_t pos_stride;     // between batches
  int pos_bytes;
  int64_t seq;
  int64_t tokens;
  int hq, hk, hv;
  int d, rot;
  int units;              // per head row
  uint32_t units_mul;     // ceil(2^32 / units)
  int rows_per_cta;       // head rows (q, then k, then v) per CTA
  uint32_t rows_mul;
  int tokens_per_cta;
  int row_chunks;
  int layout;             // gbn_rope_layout
  float mscale;
  float sign;             // -1: backward
  // append
  const int32_t* cu;
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t table_stride;
  int batches;
  int table_pages;        // entries per row
  int64_t num_pages;
  int page_shift;
  bool each;              // a lane for each sequence
  const float* k_scale;
  const float* v_scale;
};

// n / d for n * d < 2^32, given mul = ceil(2^32 / d) (0 for d == 1).
__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t mul) {
  return mul ? __umulhi(n, mul) : n;
}

// inv_freq / (2 pi) as a fraction of a turn in units of 2^-64, modulo one
// turn.  With x = m 2^e (m the 53-bit significand) and C = 2^66 / (2 pi):
// m C 2^(e - 2), the 128-bit product shifted.
__device__ __forceinline__ uint64_t turn_fraction(double x) {
  constexpr uint64_t kC = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi)) = floor(2^64 * 2 / pi)
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  const int ex = static_cast<int>((u >> 52) & 0x7FFu);
  if (ex == 0) return 0ull;  // zero and subnormal: no turn
  const uint64_t m = (u & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const int s = 2 - (ex - 1075);  // right shift of m * C
  const uint64_t hi = __umul64hi(m, kC), lo = m * kC;
  uint64_t f;
  if (s <= 0) f = s > -64 ? lo << -s : 0ull;
  else if (s < 64) f = (hi << (64 - s)) | (lo >> s);
  else f = s < 128 ? hi >> (s - 64) : 0ull;
  return (u >> 63) ? 0ull - f : f;
}

// mscale * (cos, sign * sin) of pos * inv_freq; NaN where inv_freq is not finite.
__device__ __forceinline__ float2 turn(double inv_freq, int64_t pos, float mscale, float sign) {
  const uint64_t t = turn_fraction(inv_freq) * static_cast<uint64_t>(pos);
  const uint32_t quarter = static_cast<uint32_t>((t + (1ull << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(t - (static_cast<uint64_t>(quarter) << 62));
  // The high word of an infinite or NaN double is a NaN as a float, that of any below 2^1017
  // a finite one: 0 times it is NaN, or 0.  (A comparison and a selection took the fp32
  // backward from 11.8 to 12.7 us.)
  mscale = fmaf(__int_as_float(__double2hiint(inv_freq)), 0.f, mscale);
  float s, c;
  sincospif(static_cast<float>(rest) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
  const float c2 = quarter & 1 ? -s : c, s2 = quarter & 1 ? c : s;
  const bool neg = (quarter & 2) != 0;
  return make_float2(mscale * (neg ? -c2 : c2), mscale * sign * (neg ? -s2 : s2));
}

// V elements of T, raw.
template <typename T, int V>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16) {
      const uint4 r = *reinterpret_cast<const uint4*>(p);
      w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
    } else if constexpr (kBytes == 8) {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      w[0] = r.x; w[1] = r.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void floats(float* f) const {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 4) f[0] = __uint_as_float(w[0]);
      else {
        float t[2];
        unpack<T, 2>(w, t);
        f[0] = t[0];
      }
    } else {
      unpack<T, V>(w, f);
    }
  }
};

// Stores V floats as T (round to nearest even), or as E4M3 codes after the scale.
template <typename T, int V, bool FP8>
__device__ __forceinline__ void put(void* base, int64_t at, const float* f, float scale) {
  if constexpr (FP8) {
    uint8_t* p = reinterpret_cast<uint8_t*>(base) + at;
    if constexpr (V == 1) {
      *p = e4m3(f[0] * scale);
    } else {
      uint32_t c[V / 4];
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        c[i] = e4m3x2(f[4 * i] * scale, f[4 * i + 1] * scale) |
               (e4m3x2(f[4 * i + 2] * scale, f[4 * i + 3] * scale) << 16);
      st_words<V / 4>(p, c);
    }
  } else {
    T* p = reinterpret_cast<T*>(base) + at;
    if constexpr (V == 1) {
      st_scalar<T>(p, 0, f[0]);
    } else {
      uint64_t pr[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) pr[i] = p2(f[2 * i], f[2 * i + 1]);
      uint32_t w[Words<T, V>::n];
      narrow_pairs<T, V>(pr, w);
      st_words<Words<T, V>::n>(p, w);
    }
  }
}

// V: elements per vector.  APPEND: k and v go to the paged cache, tokens are
// rows of a packed batch.  FP8 (append): the cache holds E4M3 codes.  EACH (append):
// up to 31 sequences, which the lanes of a warp hold to look a token up.
template <typename T, int V, bool APPEND, bool FP8, bool EACH>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  pdl_begin();
  // cos and sin of each token's pairs, in the order in which they are read: W
  // consecutive pairs of a unit side by side, then the same of the next unit, so
  // that neighbouring lanes read neighbouring vectors.
  constexpr int W = V < 4 ? V : 4, K = V / W;
  __shared__ __align__(16) float trig[2 * kRopeTrig];
  __shared__ int64_t s_pos[kRopeMaxTokens];   // APPEND: position, or -1: leave the token alone
  __shared__ int64_t s_page[kRopeMaxTokens];  // APPEND: page
  const int tid = threadIdx.x;
  const int64_t block = blockIdx.x / p.row_chunks;
  const int chunk = static_cast<int>(blockIdx.x - block * p.row_chunks);
  const int64_t t0 = block * p.tokens_per_cta;
  const int row0 = chunk * p.rows_per_cta;
  const int rows = min(p.rows_per_cta, p.hq + p.hk + p.hv - row0);
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.tokens_per_cta), p.tokens - t0));
  const int nrot = p.rot / (2 * V);  // units that turn
  const int half = p.layout == GBN_ROPE_HALF ? p.rot / 2 : 0;

  // Batch and place of the CTA's first token: one division, in 32 bits where it
  // fits (64 bits take a hundred instructions).
  int64_t b0 = 0, s0 = t0;
  if (!APPEND && p.seq != p.tokens) {
    b0 = p.tokens <= INT32_MAX
             ? static_cast<int64_t>(static_cast<uint32_t>(t0) / static_cast<uint32_t>(p.seq))
             : t0 / p.seq;
    s0 = t0 - b0 * p.seq;
  }
  auto place_of = [&](int tok, int64_t& bi, int64_t& si) {
    bi = b0;
    si = s0 + tok;
    if (!APPEND && si >= p.seq) {
      if (p.seq >= kRopeMaxTokens) {
        ++bi;
        si -= p.seq;
      } else {
        const uint32_t n = static_cast<uint32_t>(si) / static_cast<uint32_t>(p.seq);
        bi += n;
        si -= static_cast<int64_t>(n) * p.seq;
      }
    }
  };
  // Element offsets of a unit's two vectors within its head.
  auto places = [&](int u, int& a, int& b) {
    if (u < nrot) {
      a = half ? u * V : 2 * u * V;
      b = half ? half + u * V : a + V;
    } else {
      a = p.rot + (u - nrot) * 2 * V;
      b = a + V;
    }
  };

  float ksc = 1.f, vsc = 1.f;
  if constexpr (FP8) {
    ksc = *p.k_scale;
    vsc = *p.v_scale;
  }

  // Token (6 bits), head row (14) and unit of this thread's items; -1: none.
  int code[kRopeUnits];
  Raw<T, V> va[kRopeUnits], vb[kRopeUnits];
#pragma unroll
  for (int i = 0; i < kRopeUnits; ++i) {
    const uint32_t item = tid + i * kRopeThreads;
    const uint32_t r = div_by(item, p.units_mul);
    const int u = static_cast<int>(item - r * p.units);
    const int tok = static_cast<int>(div_by(r, p.rows_mul));
    int row = static_cast<int>(r) - tok * p.rows_per_cta;
    code[i] = -1;
    if (tok >= ntok || row >= rows) continue;
    row += row0;
    code[i] = tok | (row << 6) | (u << 20);
    int a, b;
    places(u, a, b);
    int64_t bi, si;
    place_of(tok, bi, si);
    const bool is_q = row < p.hq;
    const bool is_v = APPEND && row >= p.hq + p.hk;
    const Strided& st = is_q ? p.qs : is_v ? p.vs : p.ks;
    const int h = is_q ? row : is_v ? row - p.hq - p.hk : row - p.hq;
    const T* src = reinterpret_cast<const T*>(is_q ? p.q : is_v ? p.v : p.k) + si * st.s + h * st.h;
    if (!APPEND) src += bi * st.b;
    va[i].load(src + a);
    if (b < p.d) vb[i].load(src + b);
  }

  if constexpr (APPEND) {
    // Sequence, position and page of each token, one warp per token.
    const int lane = tid & 31;
    const int cl = EACH && lane <= p.batches ? p.cu[lane] : INT32_MAX;
    const int kl = EACH && lane < p.batches ? p.kv_lens[lane] : 0;
    for (int tok = tid >> 5; tok < ntok; tok += kRopeThreads / 32) {
      const int64_t t = t0 + tok;
      const int b = EACH ? __popc(__ballot_sync(0xFFFFFFFFu, lane > 0 && lane <= p.batches && cl <= t))
                        : warp_find_sequence(p.cu, p.batches, t);
      int64_t c0, c1, kv;
      if (EACH) {  // (past the last sequence: unused)
        c0 = __shfl_sync(0xFFFFFFFFu, cl, b);
        c1 = __shfl_sync(0xFFFFFFFFu, cl, b + 1);
        kv = __shfl_sync(0xFFFFFFFFu, kl, b);
      } else {
        const int i = min(b, p.batches - 1);
        c0 = p.cu[i];
        c1 = p.cu[i + 1];
        kv = p.kv_lens[i];
      }
      int64_t pos = -1, page = -1;
      // Rows before the first and behind the last sequence are padding.
      if (b < p.batches && !(b == 0 && t < c0)) {
        pos = kv - (c1 - c0) + (t - c0);
        const int64_t e = pos >> p.page_shift;
        if (t < c0 || pos < 0 || e >= p.table_pages) {
          pos = -1;
        } else {
          page = p.table[b * p.table_stride + e];
          if (page < 0 || page >= p.num_pages) pos = -1;
        }
        if (pos < 0 && (tid & 31) == 0) flag_bad_index();
      }
      if ((tid & 31) == 0) {
        s_pos[tok] = pos;
        s_page[tok] = page;
      }
    }
    __syncthreads();
  }

  const int pairs = p.rot / 2;
  if (p.inv_freq != nullptr) {
    for (int i = tid; i < ntok * pairs; i += kRopeThreads) {
      const int tok = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(pairs));
      const int pr = i - tok * pairs;
      int64_t pos;
      if constexpr (APPEND) {
        pos = s_pos[tok];
      } else {
        int64_t bi, si;
        place_of(tok, bi, si);
        if (p.positions == nullptr) pos = si;
        else if (p.pos_bytes == 8)
          pos = reinterpret_cast<const int64_t*>(p.positions)[bi * p.pos_stride + si];
        else
          pos = reinterpret_cast<const int32_t*>(p.positions)[bi * p.pos_stride + si];
      }
      const float2 cs = turn(p.inv_freq[pr], pos, p.mscale, p.sign);
      const int u = pr / V, e = pr % V;
      float* at = trig + ((tok * 2 * K + e / W) * nrot + u) * W + e % W;
      at[0] = cs.x;
      at[K * nrot * W] = cs.y;
    }
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < kRopeUnits; ++i) {
    if (code[i] < 0) continue;
    const int tok = code[i] & 63, row = (code[i] >> 6) & 0x3FFF, u = code[i] >> 20;
    if constexpr (APPEND) {
      if (s_pos[tok] < 0) continue;
    }
    int a, b;
    places(u, a, b);
    float fa[V], fb[V];
    va[i].floats(fa);
    if (b < p.d) vb[i].floats(fb);
    if (u < nrot && row < p.hq + p.hk && p.inv_freq != nullptr) {
      float c[V], sn[V];
      const float* at = trig + (tok * 2 * K * nrot + u) * W;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          c[k * W + e] = at[k * nrot * W + e];
          sn[k * W + e] = at[(K + k) * nrot * W + e];
        }
      if (half || V == 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x = fa[e], y = fb[e];
          fa[e] = x * c[e] - y * sn[e];
          fb[e] = x * sn[e] + y * c[e];
        }
      } else {
        // 2 V elements from 2 u V: V pairs side by side.
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float x = fa[2 * e], y = fa[2 * e + 1];
          fa[2 * e] = x * c[e] - y * sn[e];
          fa[2 * e + 1] = x * sn[e] + y * c[e];
          const float z = fb[2 * e], w = fb[2 * e + 1];
          fb[2 * e] = z * c[V / 2 + e] - w * sn[V / 2 + e];
          fb[2 * e + 1] = z * sn[V / 2 + e] + w * c[V / 2 + e];
        }
      }
    }
    if constexpr (APPEND) {
      if (row < p.hq) {
        const int64_t at = (t0 + tok) * p.qo.s + row * p.qo.h;
        put<T, V, false>(p.q_out, at + a, fa, 1.f);
        if (b < p.d) put<T, V, false>(p.q_out, at + b, fb, 1.f);
      } else {
        const int64_t slot = s_pos[tok] & ((int64_t(1) << p.page_shift) - 1);
        const bool is_k = row < p.hq + p.hk;
        const Strided& st = is_k ? p.ko : p.vo;
        void* dst = is_k ? p.k_out : p.v_out;
        const int h = row - p.hq - (is_k ? 0 : p.hk);
        const float sc = is_k ? ksc : vsc;
        const int64_t at = s_page[tok] * st.b + slot * st.s + h * st.h;
        put<T, V, FP8>(dst, at + a, fa, sc);
        if (b < p.d) put<T, V, FP8>(dst, at + b, fb, sc);
      }
    } else {
      int64_t bi, si;
      place_of(tok, bi, si);
      const bool is_q = row < p.hq;
      const Strided& st = is_q ? p.qo : p.ko;
      void* dst = is_q ? p.q_out : p.k_out;
      const int64_t at = bi * st.b + si * st.s + (is_q ? row : row - p.hq) * st.h;
      put<T, V, false>(dst, at + a, fa, 1.f);
      if (b < p.d) put<T, V, false>(dst, at + b, fb, 1.f);
    }
  }
}

// ---- host side

uint32_t div_mul(uint32_t d) {
  return d == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + d - 1) / d);
}

// Whether vectors of `bytes` at every multiple of the strides are aligned.
bool vec_ok(const void* p, const Strided& s, int esize, int bytes, int64_t nb, int64_t ns,
            int64_t nh) {
  if (reinterpret_cast<uintptr_t>(p) % bytes) return false;
  return (nb <= 1 || s.b * esize % bytes == 0) && (ns <= 1 || s.s * esize % bytes == 0) &&
         (nh <= 1 || s.h * esize % bytes == 0);
}

// Grid geometry of p for V-element vectors; false if the sizes do not fit.
bool rope_geometry(RopeParams& p, int v, int sms, int64_t* grid) {
  const int rows = p.hq + p.hk + p.hv;
  p.units = (p.d + 2 * v - 1) / (2 * v);
  if (p.units > kRopeItems) return false;
  const int pairs = p.rot / 2;
  const int fit = kRopeItems / p.units;  // head rows per CTA
  // Small calls: a CTA per token and head range of one unit a thread, so
  // that the latency of one round of loads is all there is.
  const bool small = p.tokens * rows * p.units <= int64_t(kRopeItems) * sms;
  const int want = small ? (kRopeThreads / p.units > 0 ? kRopeThreads / p.units : 1) : fit;
  if (rows > want) {
    p.row_chunks = (rows + want - 1) / want;
    p.rows_per_cta = (rows + p.row_chunks - 1) / p.row_chunks;
    p.row_chunks = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
    p.tokens_per_cta = 1;
  } else {
    p.row_chunks = 1;
    p.rows_per_cta = rows;
    int t = want / rows;
    if (t > kRopeMaxTokens) t = kRopeMaxTokens;
    if (pairs > 0 && t > kRopeTrig / pairs) t = kRopeTrig / pairs;
    if (t < 1) t = 1;
    p.tokens_per_cta = t;
  }
  // Append: up to 31 sequences are looked up with a lane for each, one read instead of a
  // search, where a CTA waits for the look-up: in small calls (31 tokens 2.6 us against
  // 2.9) and where it has many tokens (10 of them, 5200 in all: 12.2 us against 13.0; 5:
  // 17.2 against 17.5).  Where it has few it waits for their loads, and the search is ahead
  // (one, 9300 in all: 72.4 us against 77.0; two: 43.5 against 44.9; four: 30.7 against
  // 31.3).  Two-byte and E4M3 caches alike.
  p.each = p.batches < 32 && (small || p.tokens_per_cta > 4);
  p.units_mul = div_mul(p.units);
  p.rows_mul = div_mul(p.rows_per_cta);
  const int64_t blocks = (p.tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
  *grid = blocks * p.row_chunks;
  return *grid <= 0x7FFFFFFF;
}

// The largest vector (16 bytes, 8 bytes, one element) that the sizes allow.
template <typename T>
int rope_vector(const RopeParams& p, bool append, bool fp8) {
  for (int bytes = 16; bytes >= 8; bytes /= 2) {
    const int v = bytes / (int)sizeof(T);
    if (v < 2 || (fp8 && v < 4)) break;
    if (p.d % v || p.rot % (2 * v)) continue;
    const int64_t nb = append ? 1 : p.tokens / p.seq, ns = append ? p.tokens : p.seq;
    if (p.hq && !(vec_ok(p.q, p.qs, sizeof(T), bytes, nb, ns, p.hq) &&
                  vec_ok(p.q_out, p.qo, sizeof(T), bytes, nb, ns, p.hq)))
      continue;
    const int ce = fp8 ? 1 : (int)sizeof(T);
    const int64_t ob = append ? p.num_pages : nb;
    const int64_t os = append ? int64_t(1) << p.page_shift : ns;
    if (p.hk && !(vec_ok(p.k, p.ks, sizeof(T), bytes, nb, ns, p.hk) &&
                  vec_ok(p.k_out, p.ko, ce, v * ce, ob, os, p.hk)))
      continue;
    if (p.hv && !(vec_ok(p.v, p.vs, sizeof(T), bytes, nb, ns, p.hv) &&
                  vec_ok(p.v_out, p.vo, ce, v * ce, ob, os, p.hv)))
      continue;
    return v;
  }
  return 1;
}

template <typename T, bool APPEND, bool FP8, bool EACH>
cudaError_t rope_launch_v(const RopeParams& p, int v, int64_t grid, cudaStream_t stream) {
  const dim3 g(static_cast<unsigned>(grid)), b(kRopeThreads);
  constexpr int kV16 = 16 / (int)sizeof(T), kV8 = 8 / (int)sizeof(T);
  if (v == kV16) return launch_pdl(rope_kernel<T, kV16, APPEND, FP8, EACH>, g, b, 0, stream, p);
  if (v == kV8) {
    if constexpr (FP8 && kV8 < 4) return cudaErrorInvalidValue;
    else return launch_pdl(rope_kernel<T, kV8, APPEND, FP8, EACH>, g, b, 0, stream, p);
  }
  return launch_pdl(rope_kernel<T, 1, APPEND, FP8, EACH>, g, b, 0, stream, p);
}

template <typename T, bool APPEND, bool FP8>
gbn_status rope_launch(RopeParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GBN_ERR_CUDA;
  const int v = rope_vector<T>(p, APPEND, FP8);
  int64_t grid = 0;
  if (!rope_geometry(p, v, sms, &grid)) return GBN_ERR_SHAPE;
  cudaError_t e;
  if constexpr (APPEND)
    e = p.each ? rope_launch_v<T, true, FP8, true>(p, v, grid, stream)
               : rope_launch_v<T, true, FP8, false>(p, v, grid, stream);
  else
    e = rope_launch_v<T, false, false, false>(p, v, grid, stream);
  return e == cudaSuccess ? GBN_OK : GBN_ERR_CUDA;
}

Strided strides3(const int64_t* s) { return {s[0], s[1], s[2]}; }
Strided strides2(const int64_t* s) { return {0, s[0], s[1]}; }

gbn_status rope_call(const gbn_rope_args* a, float sign, cudaStream_t stream) {
  if (!a) return GBN_ERR_NULL;
  const int dtype = a->dtype, layout = a->layout;
  const int64_t batches = a->batches, seq = a->seq, q_heads = a->q_heads, k_heads = a->k_heads,
                head_dim = a->head_dim, rotary_dim = a->rotary_dim;
  if (dtype != GBN_F32 && dtype != GBN_BF16 && dtype != GBN_F16) return GBN_ERR_DTYPE;
  if (layout != GBN_ROPE_HALF && layout != GBN_ROPE_INTERLEAVED) return GBN_ERR_ENUM;
  if (a->position_bytes != 4 && a->position_bytes != 8) return GBN_ERR_DTYPE;
  if (batches < 0 || seq < 0 || q_heads < 0 || k_heads < 0 || q_heads > 4096 || k_heads > 4096 ||
      head_dim < 1 || head_dim > GBN_ROPE_MAX_DIM || rotary_dim < 0 || rotary_dim > head_dim ||
      rotary_dim % 2)
    return GBN_ERR_SHAPE;
  if (seq && batches > INT64_MAX / seq) return GBN_ERR_SHAPE;
  RopeParams p = {};
  p.tokens = batches * seq;
  if (p.tokens == 0 || q_heads + k_heads == 0) return GBN_OK;
  if ((q_heads && (!a->q || !a->q_out)) || (k_heads && (!a->k || !a->k_out)) ||
      (rotary_dim && !a->inv_freq))
    return GBN_ERR_NULL;
  p.q = a->q;
  p.k = a->k;
  p.q_out = a->q_out;
  p.k_out = a->k_out;
  p.qs = strides3(a->q_strides);
  p.ks = strides3(a->k_strides);
  p.qo = strides3(a->q_out_strides);
  p.ko = strides3(a->k_out_strides);
  p.inv_freq = rotary_dim ? a->inv_freq : nullptr;
  p.positions = a->positions;
  p.pos_stride = a->position_stride;
  p.pos_bytes = a->position_bytes;
  p.seq = seq;
  p.hq = static_cast<int>(q_heads);
  p.hk = static_cast<int>(k_heads);
  p.d = static_cast<int>(head_dim);
  p.rot = static_cast<int>(rotary_dim);
  p.layout = layout;
  p.mscale = a->mscale;
  p.sign = sign;
  if (dtype == GBN_F32) return rope_launch<float, false, false>(p, stream);
  if (dtype == GBN_BF16) return rope_launch<__nv_bfloat16, false, false>(p, stream);
  return rope_launch<__half, false, false>(p, stream);
}

}  // namespace

cudaError_t read_rope_error(unsigned int* v, bool clear) { return read_paged_error(v, clear); }

}  // namespace gbn

using namespace gbn;

extern "C" {

gbn_status gbn_rope_fwd(const gbn_rope_args* args, cudaStream_t stream) {
  return rope_call(args, 1.f, stream);
}

gbn_status gbn_rope_bwd(const gbn_rope_args* args, cudaStream_t stream) {
  return rope_call(args, -1.f, stream);
}

gbn_status gbn_paged_append(const gbn_paged_append_args* a, cudaStream_t stream) {
  if (!a) return GBN_ERR_NULL;
  const int dtype = a->dtype, cache_dtype = a->cache_dtype, layout = a->layout;
  const int64_t page_size = a->page_size, rot = a->rotary_dim;
  if (dtype != GBN_BF16 && dtype != GBN_F16) return GBN_ERR_DTYPE;
  if (cache_dtype != dtype && cache_dtype != GBN_E4M3) return GBN_ERR_DTYPE;
  if (layout != GBN_ROPE_HALF && layout != GBN_ROPE_INTERLEAVED) return GBN_ERR_ENUM;
  if (a->tokens < 0 || a->tokens > INT32_MAX || a->batches < 0 ||
      a->batches > GBN_PAGED_MAX_BATCHES || a->q_heads < 0 || a->q_heads > 4096 ||
      a->kv_heads < 1 || a->kv_heads > 4096 || a->head_dim < 1 ||
      a->head_dim > GBN_ROPE_MAX_DIM || rot < 0 || rot > a->head_dim || rot % 2 ||
      a->num_pages < 0 || a->num_pages > INT32_MAX || page_size < 1 ||
      page_size > GBN_PAGED_MAX_PAGE || (page_size & (page_size - 1)) || a->table_pages < 0 ||
      a->table_pages > INT32_MAX || a->table_stride < 0)
    return GBN_ERR_SHAPE;
  if (a->tokens == 0 || a->batches == 0) return GBN_OK;
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->cu_seqlens || !a->kv_lens ||
      !a->block_table || (a->q_heads && (!a->q || !a->q_out)) || (rot && !a->inv_freq))
    return GBN_ERR_NULL;
  const bool fp8 = cache_dtype == GBN_E4M3;
  if (fp8 && (!a->k_scale || !a->v_scale)) return GBN_ERR_NULL;
  RopeParams p = {};
  p.tokens = a->tokens;
  p.seq = a->tokens;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_out = a->q_out;
  p.k_out = a->k_cache;
  p.v_out = a->v_cache;
  p.qs = strides2(a->q_strides);
  p.ks = strides2(a->k_strides);
  p.vs = strides2(a->v_strides);
  p.qo = strides2(a->q_out_strides);
  p.ko = strides3(a->k_cache_strides);
  p.vo = strides3(a->v_cache_strides);
  p.inv_freq = rot ? a->inv_freq : nullptr;
  p.hq = static_cast<int>(a->q_heads);
  p.hk = p.hv = static_cast<int>(a->kv_heads);
  p.d = static_cast<int>(a->head_dim);
  p.rot = static_cast<int>(rot);
  p.layout = layout;
  p.mscale = a->mscale;
  p.sign = 1.f;
  p.cu = a->cu_seqlens;
  p.kv_lens = a->kv_lens;
  p.table = a->block_table;
  p.table_stride = a->table_stride;
  p.batches = static_cast<int>(a->batches);
  p.table_pages = static_cast<int>(a->table_pages);
  p.num_pages = a->num_pages;
  while ((int64_t(1) << p.page_shift) < page_size) ++p.page_shift;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  if (dtype == GBN_BF16)
    return fp8 ? rope_launch<__nv_bfloat16, true, true>(p, stream)
               : rope_launch<__nv_bfloat16, true, false>(p, stream);
  return fp8 ? rope_launch<__half, true, true>(p, stream)
             : rope_launch<__half, true, false>(p, stream);
}

}  // extern "C"
