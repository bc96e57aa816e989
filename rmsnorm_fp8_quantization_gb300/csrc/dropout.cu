// Dropout whose mask is never stored, with the residual's addition.
//
// Element e of the n in row-major order takes word e % 4 of Philox 4x32-10 (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) of the
// counter (e / 4, offset) under the key `seed`, two 64-bit numbers each; it is dropped
// where word < p 2^32.  A mask is a function of (seed, offset, e) alone: the backward
// computes it again, whatever the launch shape or alignment of either.
//
//     out = (kept ? x / (1 - p) : 0) + residual
//
// 16384 x 4096 elements: fp32 and bf16 with a residual are bound by memory (6600 GB/s,
// 60.7 us bf16); bf16 alone by the generator's twenty 32-bit products for four elements,
// which the multiplier takes four cycles each for (54 us, 40 from memory; as separate low and
// high products 62).
#include <cmath>
#include <cstdint>

#include "gbn_device.cuh"
#include "gbnorm.h"

namespace gbn {
namespace {

struct DropoutParams {
  const void* x;
  const void* residual;  // or null
  void* out;
  const uint64_t* rng;  // seed, offset
  int64_t n;
  uint32_t least;  // of the words that keep their element
  float scale;     // 1 / (1 - p)
};

// kDraw: as above; kKeep, kDrop: p so close to 0 or 1 that every word keeps or drops.
enum Mode { kDraw, kKeep, kDrop };

constexpr int kThreads = 256;
constexpr int kBytes = 32;  // of x a thread takes (two 16-byte vectors)

__device__ __forceinline__ void wide(uint32_t a, uint32_t b, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b64 t;\n\tmul.wide.u32 t, %2, %3;\n\tmov.b64 {%0, %1}, t;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(a), "r"(b));
}
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                        uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    uint32_t alo, ahi, blo, bhi;
    wide(c0, 0xD2511F53u, &alo, &ahi);
    wide(c2, 0xCD9E8D57u, &blo, &bhi);
    c0 = bhi ^ c1 ^ k0;
    c1 = blo;
    c2 = ahi ^ c3 ^ k1;
    c3 = alo;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

template <typename T>
__device__ __forceinline__ T narrow(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (Elem<T>::kDt == DT_BF16) return __float2bfloat16_rn(v);
  else return __float2half_rn(v);
}

// 16 bytes that are used once, by a coherent load: out may be x or residual, and what a kernel
// writes must not be read on the read-only path, not even each thread its own bytes before it
// writes them (half a sector is another thread's).
__device__ __forceinline__ uint4 ld_once16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// VEC: pointers on 16 bytes; else element by element, four (one draw) at a time.
template <typename T, int MODE, bool ADD, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p) {
  constexpr int kElems = VEC ? 16 / (int)sizeof(T) : 4;      // of a vector
  constexpr int kVecs = VEC ? kBytes / 16 : 2;               // a thread
  constexpr int kDraws = kElems / 4;                         // a vector
  pdl_begin();
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kVecs) + threadIdx.x;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  T* out = static_cast<T*>(p.out);
  uint64_t seed = 0, offset = 0;
  if constexpr (MODE == kDraw) {
    seed = p.rng[0];
    offset = p.rng[1];
  }
  // A block's draws share their counter's high half (their number divides 2^32).
  const uint32_t high = static_cast<uint32_t>(
      (static_cast<int64_t>(blockIdx.x) * (kThreads * kVecs * kDraws)) >> 32);
  uint4 xw[kVecs], rw[kVecs];
  if constexpr (VEC) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int64_t e0 = (v0 + u * kThreads) * kElems;
      if (e0 + kElems > p.n) continue;
      if (MODE != kDrop) xw[u] = ld_once16(x + e0);
      if (ADD) rw[u] = ld_once16(res + e0);
    }
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int64_t v = v0 + u * kThreads, e0 = v * kElems;
    if (e0 >= p.n) break;
    bool keep[kElems];
#pragma unroll
    for (int d = 0; d < kDraws; ++d) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (MODE == kDraw)
        w = philox(static_cast<uint32_t>(v * kDraws + d), high, static_cast<uint32_t>(offset),
                   static_cast<uint32_t>(offset >> 32), static_cast<uint32_t>(seed),
                   static_cast<uint32_t>(seed >> 32));
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        keep[d * 4 + e] = MODE == kKeep || (MODE == kDraw && words[e] >= p.least);
    }
    if (VEC && e0 + kElems <= p.n) {
      float f[kElems] = {}, r[kElems];
      if (MODE != kDrop) {
        const uint32_t h[4] = {xw[u].x, xw[u].y, xw[u].z, xw[u].w};
        unpack<T, kElems>(h, f);
      }
      if (ADD) {
        const uint32_t h[4] = {rw[u].x, rw[u].y, rw[u].z, rw[u].w};
        unpack<T, kElems>(h, r);
      }
      uint64_t o[kElems / 2];
#pragma unroll
      for (int e = 0; e < kElems; e += 2) {
        const float2 y = u2(mul2(p2(f[e], f[e + 1]), p2(p.scale, p.scale)));
        o[e / 2] = p2(keep[e] ? y.x : 0.f, keep[e + 1] ? y.y : 0.f);
        if (ADD) o[e / 2] = add2(o[e / 2], p2(r[e], r[e + 1]));
      }
      uint32_t w[4];
      narrow_pairs<T, kElems>(o, w);
      *reinterpret_cast<uint4*>(out + e0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < kElems; ++e) {
        if (e0 + e >= p.n) break;
        const float a = MODE != kDrop && keep[e] ? Elem<T>::to_f(x[e0 + e]) * p.scale : 0.f;
        out[e0 + e] = narrow<T>(ADD ? a + Elem<T>::to_f(res[e0 + e]) : a);
      }
    }
  }
}

template <typename T, int MODE, bool ADD>
cudaError_t launch_add(const DropoutParams& p, cudaStream_t st) {
  auto on16 = [](const void* a) { return (reinterpret_cast<uintptr_t>(a) & 15u) == 0; };
  const bool vec = on16(p.x) && on16(p.out) && (!ADD || on16(p.residual));
  const int64_t each = vec ? kBytes / static_cast<int>(sizeof(T)) : 8;  // elements a thread
  const int64_t blocks = (p.n + kThreads * each - 1) / (kThreads * each);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  return vec ? launch_pdl(dropout_kernel<T, MODE, ADD, true>, grid, dim3(kThreads), 0, st, p)
             : launch_pdl(dropout_kernel<T, MODE, ADD, false>, grid, dim3(kThreads), 0, st, p);
}
template <typename T, int MODE>
cudaError_t launch_mode(const DropoutParams& p, cudaStream_t st) {
  return p.residual ? launch_add<T, MODE, true>(p, st) : launch_add<T, MODE, false>(p, st);
}
template <typename T>
cudaError_t launch(const DropoutParams& p, int mode, cudaStream_t st) {
  return mode == kDraw   ? launch_mode<T, kDraw>(p, st)
         : mode == kKeep ? launch_mode<T, kKeep>(p, st)
                         : launch_mode<T, kDrop>(p, st);
}

gbn_status run(const void* x, const void* residual, void* out, const int64_t* rng, int64_t n, double prob,
               gbn_dtype dtype, cudaStream_t stream) {
  if (dtype != GBN_F32 && dtype != GBN_BF16 && dtype != GBN_F16) return GBN_ERR_DTYPE;
  if (n < 0 || n > GBN_DROPOUT_MAX_ELEMENTS || !(prob >= 0.0 && prob <= 1.0)) return GBN_ERR_SHAPE;
  if (n == 0) return GBN_OK;
  if (!x || !out || !rng) return GBN_ERR_NULL;
  const uintptr_t odd = dtype == GBN_F32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) |
        reinterpret_cast<uintptr_t>(residual)) & odd) != 0 ||
      (reinterpret_cast<uintptr_t>(rng) & 7u) != 0)
    return GBN_ERR_ALIGNMENT;
  const double least = std::ceil(prob * 4294967296.0);
  const int mode = least == 0.0 ? kKeep : least >= 4294967296.0 ? kDrop : kDraw;
  DropoutParams p = {};
  p.x = x;
  p.residual = residual;
  p.out = out;
  p.rng = reinterpret_cast<const uint64_t*>(rng);
  p.n = n;
  p.least = mode == kDraw ? static_cast<uint32_t>(least) : 0u;
  p.scale = mode == kDrop ? 0.f : static_cast<float>(1.0 / (1.0 - prob));
  const cudaError_t e = dtype == GBN_F32    ? launch<float>(p, mode, stream)
                        : dtype == GBN_BF16 ? launch<__nv_bfloat16>(p, mode, stream)
                                            : launch<__half>(p, mode, stream);
  return e == cudaSuccess ? GBN_OK : GBN_ERR_CUDA;
}

}  // namespace
}  // namespace gbn

extern "C" {

gbn_status gbn_dropout_fwd(const void* x, const void* residual, void* out, const int64_t* rng, int64_t n,
                           double p, gbn_dtype dtype, cudaStream_t stream) {
  return gbn::run(x, residual, out, rng, n, p, dtype, stream);
}

gbn_status gbn_dropout_bwd(const void* dout, void* dx, const int64_t* rng, int64_t n, double p,
                           gbn_dtype dtype, cudaStream_t stream) {
  return gbn::run(dout, nullptr, dx, rng, n, p, dtype, stream);
}

}  // extern "C"
