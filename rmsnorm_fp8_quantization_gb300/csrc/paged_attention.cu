// Attention of new tokens over a paged key/value cache: the kernel for few
// rows per kv head (single tokens, a few tokens to verify; and any chunk with
// heads wider than 128), the merge of split key ranges, and the C entry.
//
//   s_j = scale * q . k_j over the keys the row keeps,
//   o = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m),  m the
//   running maximum: one pass over the keys, rescaling what is summed so far
//   when the maximum grows.
//
// What bounds it: with few rows each key and value is read from HBM once and
// used for a handful of rows, so the bytes of the cache.  One warp of a CTA
// fetches tiles of 64 keys into a ring in shared memory by TMA, a box per page
// (or per 64 slots of a larger one), in the 128-byte swizzle that keeps the four
// computing warps' reads free of bank conflicts; those wait on the ring's
// barriers alone.  The rows of the kv head's whole group share the tile.  With up
// to 16 rows the four warps take 16 keys each and keep maxima, sums and outputs
// of their own, merged once at the end; with 32 rows they are 2 x 2, with 64 each
// warp has its own 16 rows and all keys.  The products run on mma.sync m16n8k16:
// the tensor work per byte is far below what tcgen05 is for, and the accumulators
// stay in registers next to the softmax.  Long key ranges are split over CTAs
// so that a few sequences fill the GPU: up to eight of them are a thread-block
// cluster, whose CTAs read one another's fp32 partial outputs from shared memory
// and write the result; more leave them in the workspace for a second kernel.
//
// Pages of fewer than 8 slots are smaller than the swizzle's pattern: the same
// warp then copies them 16 bytes a lane (cp.async) into the same places.
//
// E4M3 caches: a thread reads 16 bytes of a key row and converts in
// registers.  The head elements of Q K^T may be summed in any order, and the
// columns of the output may be computed in any order, so the fragments take
// whatever elements those 16 bytes hold and no byte is shuffled between lanes.
// Keys and values become f16 (an E4M3 value is exact in it, one instruction a
// pair), the probabilities f16 next to the values, and a bf16 q becomes f16 too,
// its row scaled by the power of two that brings its largest element near 2^8:
// elements 2^-22 below that and smaller lose bits, 2^-33 of the row's largest.
// (Keys in bf16 took four instructions a pair, and the kernel 133 us instead of
// 79 us of HBM time for 262144 keys.)
#include <cmath>
#include <type_traits>

#include <cuda.h>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_rows.cuh"

namespace gbn {
namespace {

// What a caller in another language lays out by hand.
static_assert(sizeof(gbn_paged_attention_args) == 12 * 8 + 22 * 8 + 4 * 4, "");

constexpr int kStepThreads = 128;
constexpr int kStepKeys = 64;          // keys per tile
constexpr int kMaxSplits = 512;
constexpr int kMaxCluster = 8;         // splits that merge within a cluster (the portable size)
constexpr int kHeadroom = 15;          // the row's largest probability is 2^15 in f16 (at most 65504)

// Shared-memory address `a` of this CTA, in CTA `rank` of its cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles in shared memory: panels of 128 bytes a row (64 for E4M3 heads of 64) and
// 64 rows, the 16-byte chunks of a row permuted as TMA's swizzle does it.
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  if constexpr (ROW_BYTES >= 128)
    return (chunk >> 3) * (kStepKeys * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
  else
    return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

template <typename T, bool FP8, int DP>
struct StepShape {
  static constexpr int kRowBytes = DP * (FP8 ? 1 : 2);
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kTileBytes = kStepKeys * kRowBytes;  // keys or values of one tile
  // Bytes in flight: 96 KB a CTA of two-byte 128-wide heads, two CTAs an SM.
  static constexpr int kStages = kRowBytes >= 512 ? 2 : kRowBytes >= 256 ? 3 : 4;
  static constexpr int kRing = kStages * 2 * kTileBytes;
  static constexpr int kMerge = 4 * 16 * DP * 4;  // outputs of the four warps, over the ring
  // Over the ring too: this CTA's own merged rows, for its cluster.
  static constexpr int kBody = kRing > 2 * kMerge ? kRing : 2 * kMerge;
  static constexpr int kQPitch = DP * 2 + 16;
  // CTAs an SM, by shared memory and registers (E4M3 heads of 128 in three CTAs
  // of 128 registers spill: 111 us for 262144 keys against 95 in two).
  static constexpr int kResident = DP <= 64 ? 3 : DP <= 128 ? 2 : 1;
  static constexpr int smem(int mt) {
    return kBody + 16 * mt * kQPitch + 4 * 16 * 8 + 16 * mt * (4 + 8) + 2 * kStages * 8;
  }
};

// T: q's type.  MT: 16-row tiles (1, 2, 4).
template <typename T, bool FP8, int DP, int MT>
__global__ void __launch_bounds__(kStepThreads + 32, MT <= 2 ? StepShape<T, FP8, DP>::kResident : 1)
    paged_step_kernel(const __grid_constant__ AttnParams p,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using Shape = StepShape<T, FP8, DP>;
  constexpr int WN = 4 / MT;                 // warps over the keys
  constexpr int KW = kStepKeys / WN;         // keys per warp and tile
  constexpr int NT = KW / 8;                 // score tiles of 8 keys
  constexpr int DT = DP / 8;                 // output tiles of 8 columns
  constexpr int KS = DP / 16;                // steps of 16 head elements
  constexpr bool kQReg = DP <= 128;          // q's fragments stay in registers
  using TP = typename std::conditional<FP8, __half, T>::type;  // type of both products
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_q = smem + Shape::kBody;
  // Of each warp's rows (and in the workspace of each split's): the reference of its sums
  // (below the maximum next to f16 values) and the sum.
  float2* s_ml = reinterpret_cast<float2*>(s_q + 16 * MT * Shape::kQPitch);
  float* s_qs = reinterpret_cast<float*>(s_ml + 4 * 16);  // E4M3: what a q row's scores are times
  float2* s_pml = reinterpret_cast<float2*>(s_qs + 16 * MT);  // cluster: the same of each row
  uint64_t* s_full = reinterpret_cast<uint64_t*>(s_pml + 16 * MT);
  uint64_t* s_empty = s_full + Shape::kStages;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool by_tma = p.page_shift >= 3;
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < Shape::kStages; ++i) {
      mbar_init(&s_full[i], by_tma ? 1 : 32);
      mbar_init(&s_empty[i], 4);
    }
    fence_mbar_init();
  }
  if (by_tma && warp == 4 && lane < 2) prefetch_map(lane ? &vmap : &kmap);
  __syncthreads();
  pdl_begin();
  const int wm = warp / WN, wn = warp % WN;
  const int qr = lane >> 2, qc = lane & 3;
  uint32_t x = blockIdx.x;
  int split = 0;
  if (p.cluster) {  // a cluster is consecutive CTAs
    split = x % p.splits;
    x /= p.splits;
  }
  const int h = x % p.hkv;
  x /= p.hkv;
  const int rt = x % p.row_tiles;
  x /= p.row_tiles;
  if (!p.cluster) {
    split = x % p.splits;
    x /= p.splits;
  }
  const int b = x;

  const SeqRange s = seq_range(p, b, tid == 0 && split == 0 && rt == 0 && h == 0);
  const int r0 = rt * 16 * MT;
  const int rows = min(16 * MT, s.qlen * p.group - r0);
  if (rows <= 0) return;
  const int i0 = r0 / p.group, i1 = (r0 + rows - 1) / p.group;
  const int lo = row_low(p, s, i0), hi = row_high(p, s, i1);
  const int64_t start = lo + static_cast<int64_t>(split) * p.split_len;
  const int k0 = static_cast<int>(min(start, static_cast<int64_t>(max(hi, 0))));
  const int k1 = static_cast<int>(min(start + p.split_len, static_cast<int64_t>(max(hi, 0))));
  const int base = k0 & ~(kStepKeys - 1);  // first key of the tiles
  const int ntiles = k1 > k0 ? (k1 - base + kStepKeys - 1) / kStepKeys : 0;
  if (ntiles == 0 && split > 0 && !p.cluster) {
    // Nothing here: say so (the merge reads every split's maximum and sum).
    for (int r = tid; r < rows; r += kStepThreads + 32) {
      const int gr = r0 + r;
      const int64_t o = static_cast<int64_t>(s.q0 + gr / p.group) * p.hq + h * p.group + gr % p.group;
      p.part_ml[o * p.splits + split] = make_float2(-INFINITY, 0.f);
    }
    return;
  }

  // q's rows into shared memory (rows past the end and columns past d: zero), by
  // the computing warps alone: the fetch of keys does not wait for them.
  if (warp < 4) {
    constexpr int C = DP / 8;
    const T* q = reinterpret_cast<const T*>(p.q);
    for (int i = tid; i < 16 * MT * C; i += kStepThreads) {
      const int r = i / C, c = i % C;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && c * 8 < p.d) {
        const int gr = r0 + r;
        w = *reinterpret_cast<const uint4*>(q + (s.q0 + gr / p.group) * p.qt +
                                            (h * p.group + gr % p.group) * p.qh + c * 8);
      }
      if constexpr (FP8) {
        // A row's C chunks are in C neighbouring lanes.
        const float back = q_to_f16<T, C>(w);
        if (c == 0) s_qs[r] = back;
      }
      *reinterpret_cast<uint4*>(s_q + r * Shape::kQPitch + c * 16) = w;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kStepThreads) : "memory");
  }

  const uint32_t ring = smem_u32(smem);
  bool ok = true;
  if (warp == 4) {
    // ------------------------------------------------ fetch
    const int page = 1 << p.page_shift;
    const int32_t* tab = p.table + b * p.table_stride;
    const int e_last = ntiles > 0 ? (k1 - 1) >> p.page_shift : 0;
    if (by_tma) {
      const int box = min(page, kStepKeys), boxes = kStepKeys / box;  // at most 8
      const int zero_page = max(1, static_cast<int>(p.num_pages));    // one past: zeros
      // This lane's box: its table entry is read one tile ahead.
      auto wanted = [&](int t) {
        const int key = base + t * kStepKeys + lane * box;
        return lane < boxes && key < k1 && key + box > k0;
      };
      auto entry = [&](int t) {
        const int key = base + t * kStepKeys + lane * box;
        return wanted(t) ? tab[min(key >> p.page_shift, e_last)] : 0;
      };
      int cur = ntiles > 0 ? entry(0) : 0;
      int t = 0;
      for (; t < ntiles; ++t) {
        const int st = t % Shape::kStages, use = t / Shape::kStages;
        const int next = t + 1 < ntiles ? entry(t + 1) : 0;
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_empty[st], (use - 1) & 1));
        if (!ok) break;
        int pg = zero_page;
        if (wanted(t)) {
          if (cur >= 0 && cur < p.num_pages) pg = cur;
          else flag_bad_index();  // its keys read as zero
        }
        if (lane == 0) mbar_arrive_expect_tx(&s_full[st], 2 * Shape::kTileBytes);
        __syncwarp();
        if (lane < boxes) {
          const int slot = (base + t * kStepKeys + lane * box) & (page - 1);
          const uint32_t dst = ring + st * 2 * Shape::kTileBytes + lane * box * Shape::kPanelBytes;
#pragma unroll
          for (int pn = 0; pn < Shape::kPanels; ++pn) {
            const int c0 = pn * (Shape::kPanelBytes / (FP8 ? 1 : 2));
            tma_box(dst + pn * kStepKeys * 128, &kmap, c0, h, slot, pg, &s_full[st]);
            tma_box(dst + Shape::kTileBytes + pn * kStepKeys * 128, &vmap, c0, h, slot, pg,
                    &s_full[st]);
          }
        }
        cur = next;
      }
      if (!ok)  // leave no copy in flight behind
        for (int i = max(0, t - Shape::kStages); i < t; ++i)
          mbar_wait(&s_full[i % Shape::kStages], (i / Shape::kStages) & 1);
    } else {
      const uint8_t* kbase = reinterpret_cast<const uint8_t*>(p.k) + h * p.kh * (FP8 ? 1 : 2);
      const uint8_t* vbase = reinterpret_cast<const uint8_t*>(p.v) + h * p.vh * (FP8 ? 1 : 2);
      for (int t = 0; t < ntiles; ++t) {
        const int st = t % Shape::kStages, use = t / Shape::kStages;
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_empty[st], (use - 1) & 1));
        if (!ok) break;
        const uint32_t kd = ring + st * 2 * Shape::kTileBytes;
        for (int i = lane; i < kStepKeys * Shape::kChunks; i += 32) {
          const int r = i / Shape::kChunks, c = i % Shape::kChunks;
          const int j = base + t * kStepKeys + r;
          int pg = -1;
          if (j >= k0 && j < k1) {
            pg = tab[j >> p.page_shift];
            if (pg < 0 || pg >= p.num_pages) {
              flag_bad_index();
              pg = -1;
            }
          }
          const bool live = pg >= 0 && c * 16 < p.d * (FP8 ? 1 : 2);
          const int slot = j & (page - 1);
          const int64_t ko = live ? (pg * p.kp + slot * p.ks) * (FP8 ? 1 : 2) + c * 16 : 0;
          const int64_t vo = live ? (pg * p.vp + slot * p.vs) * (FP8 ? 1 : 2) + c * 16 : 0;
          const uint32_t at = tile_at<Shape::kRowBytes>(r, c);
          cp_async16(kd + at, kbase + ko, live);
          cp_async16(kd + Shape::kTileBytes + at, vbase + vo, live);
        }
        // Arrives when this lane's copies so far have landed.
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&s_full[st]))
                     : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (!ok && lane == 0) flag_wait_timeout();
  }

  // q fragments.  Two-byte caches: the standard order.  E4M3: step ks of the
  // 64-column block takes, for lane column qc, elements 16 qc + 4 (ks % 4).. + 3.
  const uint32_t qbase = smem_u32(s_q) + (wm & (MT - 1)) * 16 * Shape::kQPitch;
  auto load_q = [&](int ks, uint32_t* a) {
    if constexpr (!FP8) {
      ldsm4(a, qbase + (lane & 15) * Shape::kQPitch + ks * 32 + (lane >> 4) * 16);
    } else {
      const uint32_t col = ((ks / 4) * 64 + qc * 16 + (ks % 4) * 4) * 2;
      const uint2 u = lds8(qbase + qr * Shape::kQPitch + col);
      const uint2 w = lds8(qbase + (qr + 8) * Shape::kQPitch + col);
      a[0] = u.x;
      a[1] = w.x;
      a[2] = u.y;
      a[3] = w.y;
    }
  };
  uint32_t qf[kQReg ? KS : 1][4];
  if constexpr (kQReg) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) load_q(ks, qf[ks]);
  }

  // Key limits of this thread's two rows.
  int rlo[2], rhi[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = (wm & (MT - 1)) * 16 + qr + 8 * e;
    const int i = (r0 + min(r, rows - 1)) / p.group;
    rlo[e] = max(row_low(p, s, i), k0);
    rhi[e] = min(row_high(p, s, i), k1);
  }
  // Keys that every row of the CTA keeps need no test.
  const int all_lo = max(row_low(p, s, i1), k0), all_hi = min(row_high(p, s, i0), k1);

  float scale[2] = {p.scale_log2, p.scale_log2};
  if constexpr (FP8) {
#pragma unroll
    for (int e = 0; e < 2; ++e) scale[e] *= *p.k_scale_inv * s_qs[(wm & (MT - 1)) * 16 + qr + 8 * e];
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[DT][4];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[d][e] = 0.f;

  for (int t = 0; warp < 4 && t < ntiles; ++t) {
    const int st = t % Shape::kStages;
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[st], (t / Shape::kStages) & 1));
    if (!ok) {
      if (lane == 0) flag_wait_timeout();
      break;
    }
    const uint32_t kd = ring + st * 2 * Shape::kTileBytes;
    const uint32_t vd = kd + Shape::kTileBytes;
    const int kw = wn * KW;  // this warp's first key row in the tile
    const bool cut = base + t * kStepKeys < k0 || base + (t + 1) * kStepKeys > k1;
    if (cut) {
      // A weight of 0 times what stands in a slot outside the range must be 0.
      // (Warps that share rows all write the same zeros before they read.)
      uint8_t* v = smem + st * 2 * Shape::kTileBytes + Shape::kTileBytes;
      for (int i = lane; i < KW * Shape::kChunks; i += 32) {
        const int r = kw + i / Shape::kChunks, key = base + t * kStepKeys + r;
        if (key < k0 || key >= k1)
          *reinterpret_cast<uint4*>(v + tile_at<Shape::kRowBytes>(r, i % Shape::kChunks)) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    float sc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
    if constexpr (!FP8) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        if constexpr (!kQReg) load_q(ks, a);
        const uint32_t* af = kQReg ? qf[kQReg ? ks : 0] : a;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          const int row = kw + n * 8 + (lane & 7) + ((lane >> 4) << 3);
          const int ch = ks * 2 + ((lane >> 3) & 1);
          uint32_t kb[4];
          ldsm4(kb, kd + tile_at<Shape::kRowBytes>(row, ch));
          mma16816<TP>(sc[n], af, kb[0], kb[1]);
          mma16816<TP>(sc[n + 1], af, kb[2], kb[3]);
        }
      }
    } else {
#pragma unroll
      for (int blk = 0; blk < DP / 64; ++blk) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int row = kw + n * 8 + qr;
          const uint4 u = lds16(kd + tile_at<Shape::kRowBytes>(row, blk * 4 + qc));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int s4 = 0; s4 < 4; ++s4) {
            uint32_t a[4];
            if constexpr (!kQReg) load_q(blk * 4 + s4, a);
            const uint32_t* af = kQReg ? qf[kQReg ? blk * 4 + s4 : 0] : a;
            mma16816<TP>(sc[n], af, e4m3x2_to_f16x2(w[s4] & 0xFFFFu), e4m3x2_to_f16x2(w[s4] >> 16));
          }
        }
      }
    }

    // Scale, mask, running maximum.
    const int jbase = base + t * kStepKeys + kw;
    float mx[2] = {m[0], m[1]};
    if (jbase >= all_lo && jbase + KW <= all_hi) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[n][e] = __fmul_rn(sc[n][e], scale[e >> 1]);  // (never one with the subtraction below)
          mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
        }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = jbase + n * 8 + qc * 2 + (e & 1);
          const bool keep = j >= rlo[e >> 1] && j < rhi[e >> 1];
          sc[n][e] = keep ? __fmul_rn(sc[n][e], scale[e >> 1]) : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
        }
    }
    float base[2];  // what the scores are taken against
    bool grew = false;
    float al[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 2));
      base[e] = mx[e] == -INFINITY ? 0.f : reference<TP, kHeadroom>(mx[e]);
      al[e] = ex2(reference<TP, kHeadroom>(m[e]) - base[e]);  // m = -inf: 0, and the sums are still 0
      grew |= mx[e] != m[e];
      m[e] = mx[e];
    }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] *= al[e];
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] *= al[e >> 1];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[n][e] = ex2(sc[n][e] - base[e >> 1]);
        l[e >> 1] += sc[n][e];
      }
    // P V.  P is rounded to the values' type, the sums l keep it unrounded: at most
    // half a step relative, in f16 for weights down to 2^-29 of the row's largest so
    // far, and 2^-40 of that largest below.
#pragma unroll
    for (int kk = 0; kk < NT / 2; ++kk) {
      uint32_t a[4];
      a[0] = narrow2<TP>(p2(sc[2 * kk][0], sc[2 * kk][1]));
      a[1] = narrow2<TP>(p2(sc[2 * kk][2], sc[2 * kk][3]));
      a[2] = narrow2<TP>(p2(sc[2 * kk + 1][0], sc[2 * kk + 1][1]));
      a[3] = narrow2<TP>(p2(sc[2 * kk + 1][2], sc[2 * kk + 1][3]));
      const int kr = kw + kk * 16;
      if constexpr (!FP8) {
#pragma unroll
        for (int d = 0; d < DT; d += 2) {
          const int row = kr + (lane & 15);
          uint32_t vb[4];
          ldsm4t(vb, vd + tile_at<Shape::kRowBytes>(row, d + (lane >> 4)));
          mma16816<TP>(o[d], a, vb[0], vb[1]);
          mma16816<TP>(o[d + 1], a, vb[2], vb[3]);
        }
      } else {
        // Output tile d of a block of 128 (64) columns holds, for lane row qr,
        // column 16 qr + d (8 qr + d).
        constexpr int CB = DP >= 128 ? 16 : 8;  // bytes per load
#pragma unroll
        for (int blk = 0; blk < DP / (CB * 8); ++blk) {
          uint32_t w[4][CB / 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = kr + qc * 2 + (e & 1) + (e >> 1) * 8;
            if constexpr (CB == 16) {
              const uint4 u = lds16(vd + tile_at<Shape::kRowBytes>(row, blk * 8 + qr));
              w[e][0] = u.x; w[e][1] = u.y; w[e][2] = u.z; w[e][3] = u.w;
            } else {
              const uint2 u = lds8(vd + tile_at<Shape::kRowBytes>(row, qr >> 1) + (qr & 1) * 8);
              w[e][0] = u.x; w[e][1] = u.y;
            }
          }
#pragma unroll
          for (int i = 0; i < CB / 4; ++i) {
            const uint32_t x0 = __byte_perm(w[0][i], w[1][i], 0x5140);  // bytes 0, 1 of both keys
            const uint32_t x1 = __byte_perm(w[0][i], w[1][i], 0x7362);
            const uint32_t y0 = __byte_perm(w[2][i], w[3][i], 0x5140);
            const uint32_t y1 = __byte_perm(w[2][i], w[3][i], 0x7362);
            const int d = blk * CB + i * 4;
            mma16816<TP>(o[d], a, e4m3x2_to_f16x2(x0 & 0xFFFFu), e4m3x2_to_f16x2(y0 & 0xFFFFu));
            mma16816<TP>(o[d + 1], a, e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(y0 >> 16));
            mma16816<TP>(o[d + 2], a, e4m3x2_to_f16x2(x1 & 0xFFFFu), e4m3x2_to_f16x2(y1 & 0xFFFFu));
            mma16816<TP>(o[d + 3], a, e4m3x2_to_f16x2(x1 >> 16), e4m3x2_to_f16x2(y1 >> 16));
          }
        }
      }
    }
    if (cut) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeros, before the next copy
    __syncwarp();
    if (lane == 0)
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&s_empty[st])) : "memory");
  }

  // Merge the warps of each row tile through shared memory.
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
    l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
  }
  __syncthreads();  // the ring is free
  float* s_o = reinterpret_cast<float*>(smem) + (warp & 3) * 16 * DP;
#pragma unroll
  for (int d = 0; warp < 4 && d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = qr + 8 * (e >> 1);
      int col;
      if constexpr (!FP8) {
        col = d * 8 + qc * 2 + (e & 1);
      } else {
        constexpr int CB = DP >= 128 ? 16 : 8;
        col = (d / CB) * CB * 8 + (qc * 2 + (e & 1)) * CB + d % CB;
      }
      s_o[r * DP + col] = o[d][e];
    }
  if (warp < 4 && qc == 0) {
    s_ml[warp * 16 + qr] = make_float2(reference<TP, kHeadroom>(m[0]), l[0]);
    s_ml[warp * 16 + qr + 8] = make_float2(reference<TP, kHeadroom>(m[1]), l[1]);
  }
  __syncthreads();
  const float vscale = FP8 ? *p.v_scale_inv : 1.f;
  constexpr int Q4 = DP / 8;  // groups of 8 columns per row
  float* s_part = reinterpret_cast<float*>(smem + Shape::kMerge);
  for (int i = tid; i < rows * Q4; i += kStepThreads + 32) {
    const int r = i / Q4, c = (i % Q4) * 8;
    if (c >= p.d) continue;
    const int w0 = (r / 16) * WN;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < WN; ++w) mm = fmaxf(mm, s_ml[(w0 + w) * 16 + r % 16].x);
    const float mb = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WN; ++w) {
      const float2 ml = s_ml[(w0 + w) * 16 + r % 16];
      const float f = ex2(ml.x - mb);
      ll += ml.y * f;
      const float* src = reinterpret_cast<const float*>(smem) + ((w0 + w) * 16 + r % 16) * DP + c;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(src[e], f, acc[e]);
    }
    const int gr = r0 + r;
    const int token = s.q0 + gr / p.group, head = h * p.group + gr % p.group;
    const int64_t ro = static_cast<int64_t>(token) * p.hq + head;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) nan |= acc[e] != acc[e];
    if (nan && ll == ll) {  // (a NaN sum: a kept score is NaN, and so is the row)
      const int low = max(row_low(p, s, gr / p.group), k0), high = min(row_high(p, s, gr / p.group), k1);
      if (low > k0 || high < k1)  // it dropped keys that others of its tile keep
        row_again<T, FP8>(p, b, h, reinterpret_cast<const T*>(p.q) + token * p.qt + head * p.qh,
                          FP8 ? p.scale_log2 * *p.k_scale_inv : p.scale_log2, ll, low, high, c, acc);
    }
    if (p.cluster) {
      float* dst = s_part + r * DP + c;
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (c == 0) s_pml[r] = make_float2(mm, ll);
    } else if (p.splits > 1) {
      float* dst = p.part_o + (static_cast<int64_t>(split) * p.tokens * p.hq + ro) * p.d + c;
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (c == 0) p.part_ml[ro * p.splits + split] = make_float2(mm, ll);
    } else {
      const float inv = ll == 0.f ? 0.f : vscale / ll;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = narrow2<T>(p2(acc[2 * e] * inv, acc[2 * e + 1] * inv));
      st_words<4>(reinterpret_cast<T*>(p.out) + token * p.ot + head * p.oh + c, w);
      if (c == 0 && p.lse) p.lse[ro] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
  }
  if (p.cluster) {
    // Every CTA of the cluster merges a share of the rows from all of them, in the
    // order of the splits.
    cluster_sync();
    const uint32_t part = smem_u32(s_part), pml = smem_u32(s_pml);
    for (int i = split * (kStepThreads + 32) + tid; i < rows * Q4;
         i += p.splits * (kStepThreads + 32)) {
      const int r = i / Q4, c = (i % Q4) * 8;
      if (c >= p.d) continue;
      float2 ml[kMaxCluster];
      float m2 = -INFINITY;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (k < p.splits) {
          const uint32_t a = cluster_addr(pml + r * 8, k);
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml[k].x), "=f"(ml[k].y) : "r"(a));
        }
        m2 = fmaxf(m2, ml[k].x);
      }
      const float mb = m2 == -INFINITY ? 0.f : m2;
      float l2 = 0.f, acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      // Four splits' outputs are requested together (one at a time, with a latency
      // each, took 3500 cycles of a call's 11000).
#pragma unroll
      for (int k = 0; k < kMaxCluster; k += 4) {
        if (k >= p.splits) break;
        float v[4][8];
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const uint32_t a = cluster_addr(part + (r * DP + c) * 4, min(k + i4, p.splits - 1));
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[i4][e]), "=f"(v[i4][e + 1]), "=f"(v[i4][e + 2]), "=f"(v[i4][e + 3])
                         : "r"(a + e * 4));
        }
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          // (nothing kept there, or no such split: a weight of 0 and no value; each
          // load is waited for all the same)
          const float2 x = ml[k + i4];
          const float w = x.y == 0.f ? 0.f : ex2(x.x - mb);
          l2 += x.y * w;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(x.y == 0.f ? 0.f : v[i4][e], w, acc[e]);
        }
      }
      const int gr = r0 + r;
      const int token = s.q0 + gr / p.group, head = h * p.group + gr % p.group;
      const float inv = l2 == 0.f ? 0.f : vscale / l2;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = narrow2<T>(p2(acc[2 * e] * inv, acc[2 * e + 1] * inv));
      st_words<4>(reinterpret_cast<T*>(p.out) + token * p.ot + head * p.oh + c, w);
      if (c == 0 && p.lse)
        p.lse[static_cast<int64_t>(token) * p.hq + head] = l2 == 0.f ? -INFINITY : (m2 + log2f(l2)) * kLn2;
    }
    // Nobody leaves while its shared memory is read.  What was read has been used, and
    // nothing is handed over: no ordering, which would wait for the outputs to land.
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  }
}

// Merge of split key ranges: one CTA per (token, query head).
//   o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s
// in the order of the splits within each of the CTA's split groups, the
// groups added in order: the same bits every time.
constexpr int kMergeThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads)
    paged_merge_kernel(const __grid_constant__ AttnParams p, int fp8) {
  pdl_begin();
  __shared__ float s_w[kMaxSplits];
  __shared__ float s_red[kMergeThreads / 32];
  __shared__ float4 s_o[kMergeThreads];
  const int64_t ro = blockIdx.x;
  const int token = static_cast<int>(ro / p.hq), head = static_cast<int>(ro % p.hq);
  // Padding rows behind the last sequence are left alone.
  if (token >= p.cu[p.batches] || token < p.cu[0]) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float2* ml = p.part_ml + ro * p.splits;
  float m = -INFINITY;
  for (int s = tid; s < p.splits; s += kMergeThreads) m = fmaxf(m, ml[s].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (lane == 0) s_red[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) m = fmaxf(m, s_red[w]);
  __syncthreads();
  const float mb = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int s = tid; s < p.splits; s += kMergeThreads) {
    const float2 v = ml[s];
    // A split without a kept key wrote no partial output: weight exactly 0,
    // and its slot is skipped below.
    const float w = v.y == 0.f ? 0.f : ex2(v.x - mb);
    s_w[s] = w;
    l += v.y == 0.f ? 0.f : v.y * w;
  }
  l = warp_sum(l);
  if (lane == 0) s_red[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) l += s_red[w];

  const int cols = p.d / 4;                       // float4 columns (4 .. 64)
  const int groups = kMergeThreads / cols;        // split groups (2 .. 32)
  const int col = tid % cols, grp = tid / cols;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (grp < groups) {
    const float* src = p.part_o + ro * p.d + col * 4;
    const int64_t step = static_cast<int64_t>(p.tokens) * p.hq * p.d;
#pragma unroll 4
    for (int s = grp; s < p.splits; s += groups) {
      const float w = s_w[s];
      if (w != 0.f) {
        const float4 v = *reinterpret_cast<const float4*>(src + s * step);
        acc.x = fmaf(v.x, w, acc.x);
        acc.y = fmaf(v.y, w, acc.y);
        acc.z = fmaf(v.z, w, acc.z);
        acc.w = fmaf(v.w, w, acc.w);
      }
    }
  }
  s_o[tid] = acc;
  __syncthreads();
  if (tid < cols) {
    for (int g = 1; g < groups; ++g) {
      const float4 v = s_o[g * cols + tid];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float inv = l == 0.f ? 0.f : (fp8 ? *p.v_scale_inv : 1.f) / l;
    uint32_t w[2] = {narrow2<T>(p2(acc.x * inv, acc.y * inv)),
                     narrow2<T>(p2(acc.z * inv, acc.w * inv))};
    st_words<2>(reinterpret_cast<T*>(p.out) + token * p.ot + head * p.oh + tid * 4, w);
    if (tid == 0 && p.lse) p.lse[ro] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// ---- host side

template <typename T, bool FP8, int DP, int MT>
cudaError_t allow_step() {
  static std::atomic<uint64_t> done{0};
  return allow_smem(paged_step_kernel<T, FP8, DP, MT>, StepShape<T, FP8, DP>::smem(MT), done);
}

// Clusters of c CTAs of this kernel that device `dev` holds at once (they do not
// cross the SM groups of the chip, so fewer than its CTA slots / c); 0: unknown.
// Asked of the runtime once per device and size.
template <bool FP8, int DP, int MT>
int step_room(int c, int dev) {
  using T = __nv_bfloat16;  // the same footprint as __half
  static std::atomic<int> known[16][kMaxCluster + 1];
  if (dev < 16 && known[dev][c].load(std::memory_order_relaxed) > 0)
    return known[dev][c].load(std::memory_order_relaxed) - 1;
  int n = 0;
  if (allow_step<T, FP8, DP, MT>() != cudaSuccess) return 0;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(c);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c));
  cfg.blockDim = dim3(kStepThreads + 32);
  cfg.dynamicSmemBytes = StepShape<T, FP8, DP>::smem(MT);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, paged_step_kernel<T, FP8, DP, MT>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 16) known[dev][c].store(n + 1, std::memory_order_relaxed);
  return n;
}
template <bool FP8, int DP>
int step_room_mt(int mt, int c, int dev) {
  return mt == 1 ? step_room<FP8, DP, 1>(c, dev)
                 : mt == 2 ? step_room<FP8, DP, 2>(c, dev) : step_room<FP8, DP, 4>(c, dev);
}
template <bool FP8>
int step_room_d(int64_t d, int mt, int c, int dev) {
  return d <= 64 ? step_room_mt<FP8, 64>(mt, c, dev)
                 : d <= 128 ? step_room_mt<FP8, 128>(mt, c, dev) : step_room_mt<FP8, 256>(mt, c, dev);
}

template <typename T, bool FP8, int DP, int MT>
cudaError_t launch_step(const AttnParams& p, int64_t grid, cudaStream_t st) {
  using Shape = StepShape<T, FP8, DP>;
  constexpr int smem = Shape::smem(MT);
  auto k = paged_step_kernel<T, FP8, DP, MT>;
  const cudaError_t e = allow_step<T, FP8, DP, MT>();
  if (e != cudaSuccess) return e;
  CUtensorMap km = {}, vm = {};
  if (p.page_shift >= 3) {
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int es = FP8 ? 1 : 2;
    if (!make_cache_map(&km, p.k, es, bf16, Shape::kPanelBytes / es, kStepKeys, true, p, p.kp, p.ks,
                        p.kh) ||
        !make_cache_map(&vm, p.v, es, bf16, Shape::kPanelBytes / es, kStepKeys, true, p, p.vp, p.vs,
                        p.vh))
      return cudaErrorInvalidValue;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kStepThreads + 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 2 : 1;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, k, p, km, vm);
  return le != cudaSuccess ? le : cudaGetLastError();
}
template <typename T, bool FP8, int DP>
cudaError_t launch_step_mt(const AttnParams& p, int mt, int64_t grid, cudaStream_t st) {
  if (mt == 1) return launch_step<T, FP8, DP, 1>(p, grid, st);
  if (mt == 2) return launch_step<T, FP8, DP, 2>(p, grid, st);
  return launch_step<T, FP8, DP, 4>(p, grid, st);
}
template <typename T, bool FP8>
cudaError_t launch_step_d(const AttnParams& p, int mt, int64_t grid, cudaStream_t st) {
  if (p.d <= 64) return launch_step_mt<T, FP8, 64>(p, mt, grid, st);
  if (p.d <= 128) return launch_step_mt<T, FP8, 128>(p, mt, grid, st);
  return launch_step_mt<T, FP8, 256>(p, mt, grid, st);
}

// The same for up to 32 splits: a warp per row, a lane per split for the weights
// and D / 32 columns per lane for the outputs, nothing shared (14400 rows of two
// splits: a CTA per row took 18 us).
constexpr int kMergeRows = 4;  // rows (warps) per CTA
template <typename T>
__global__ void __launch_bounds__(32 * kMergeRows)
    paged_merge_few_kernel(const __grid_constant__ AttnParams p, int fp8) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int64_t ro = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  if (ro >= static_cast<int64_t>(p.tokens) * p.hq) return;
  const int token = static_cast<int>(ro / p.hq), head = static_cast<int>(ro - static_cast<int64_t>(token) * p.hq);
  if (token >= p.cu[p.batches] || token < p.cu[0]) return;  // padding rows
  const float2 ml = lane < p.splits ? p.part_ml[ro * p.splits + lane] : make_float2(-INFINITY, 0.f);
  float m = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float mb = m == -INFINITY ? 0.f : m;
  const float w = ml.y == 0.f ? 0.f : ex2(ml.x - mb);
  const float l = warp_sum(ml.y == 0.f ? 0.f : ml.y * w);
  const int cols = p.d / 4;  // float4 columns (4 .. 64)
  const float inv = l == 0.f ? 0.f : (fp8 ? *p.v_scale_inv : 1.f) / l;
  const int64_t step = static_cast<int64_t>(p.tokens) * p.hq * p.d;
  for (int c0 = 0; c0 < cols; c0 += 32) {
    const int col = c0 + lane;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = p.part_o + ro * p.d + col * 4;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      const float ws = __shfl_sync(0xFFFFFFFFu, w, s);
      if (ws != 0.f && col < cols) {
        const float4 v = *reinterpret_cast<const float4*>(src + s * step);
        acc.x = fmaf(v.x, ws, acc.x);
        acc.y = fmaf(v.y, ws, acc.y);
        acc.z = fmaf(v.z, ws, acc.z);
        acc.w = fmaf(v.w, ws, acc.w);
      }
    }
    if (col < cols) {
      uint32_t o[2] = {narrow2<T>(p2(acc.x * inv, acc.y * inv)), narrow2<T>(p2(acc.z * inv, acc.w * inv))};
      st_words<2>(reinterpret_cast<T*>(p.out) + token * p.ot + head * p.oh + col * 4, o);
    }
  }
  if (lane == 0 && p.lse) p.lse[ro] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const AttnParams& p, bool fp8, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.hq;
  if (p.splits <= 32 && (rows >= 256 || p.splits <= 8))
    return launch_pdl(paged_merge_few_kernel<T>,
                      dim3(static_cast<unsigned>((rows + kMergeRows - 1) / kMergeRows)),
                      dim3(32 * kMergeRows), 0, st, p, int(fp8));
  return launch_pdl(paged_merge_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(kMergeThreads), 0,
                    st, p, int(fp8));
}

// How a call is carried out: a function of sizes that the host knows.
struct AttnPlan {
  bool prefill;   // the tcgen05 kernel
  int rows;       // rows per CTA (16, 32, 64; prefill: 256)
  int row_tiles;
  int splits;
  int split_len;
  bool cluster;   // the splits merge within a cluster: no workspace, no second kernel
  int64_t ctas;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

AttnPlan attn_plan(int64_t batches, int64_t hkv, int64_t group, int64_t d, int64_t max_q,
                   int64_t max_kv, int64_t window, int causal, int page_shift, bool fp8, int sms,
                   int dev) {
  AttnPlan a;
  const int64_t r = max_q * group;
  const int64_t keys = window > 0 && causal && window + max_q < max_kv ? window + max_q : max_kv;
  // The tcgen05 kernel from the first size on that fills half a tile of it, and
  // for 33 to 64 rows of wide heads but for short sequences (48 rows, heads of 128:
  // 4 sequences of 3000-4000 keys 21 us against 34 on mma.sync, 35 of 18000-25000 470
  // against 680, E4M3 550 against 900; one of 2000 the same; 4 of 300 11.0 against
  // 10.1).  Heads of 64 gain 15 % at most and lose 40 % where sequences bring fewer
  // tokens than the longest (24 of 8 to 48 rows, 24 us against 19).  Its boxes are
  // at least 8 slots (one swizzle atom).
  a.prefill = (r > 64 || (r > 32 && d > 64 && keys > 512)) && d <= 128 && page_shift >= 3;
  // 33 to 64 rows as two tiles of 32: a step is shorter (each warp has half of
  // the keys) and the second read of the keys comes from L2.
  a.rows = a.prefill ? kPrefillRows : r <= 16 ? 16 : r <= 64 ? 32 : 64;
  a.row_tiles = static_cast<int>(ceil_div(r, a.rows));
  // Longest key range of a row tile.
  int64_t range = max_kv;
  if (window > 0 && causal) {
    const int64_t tile_tokens = ceil_div(a.rows, group) + 1;
    const int64_t w = window + (tile_tokens < max_q ? tile_tokens : max_q);
    if (w < range) range = w;
  }
  const int64_t tiles = batches * hkv * a.row_tiles;
  const int64_t step = a.prefill ? kPrefillKeys : kStepKeys;
  const int64_t slots = sms * (d <= 64 ? 3 : d <= 128 ? 2 : 1);  // CTAs of the step kernel at once
  auto room = [&](int c) {  // clusters of c CTAs at once
    return fp8 ? step_room_d<true>(d, a.rows / 16, c, dev) : step_room_d<false>(d, a.rows / 16, c, dev);
  };
  int64_t splits = 1;
  if (a.prefill) {
    // One CTA per SM: as many as fit one round, at least 256 keys each (one sequence
    // of 2000 keys, 48 rows, 8 kv heads: 12.1 us in eights, 13.8 in fours, 26 whole; 4
    // of 4000 keys: 21 us in one round, 30 in half of one, 28 in 1.5).
    splits = sms / (tiles > 0 ? tiles : 1);
    const int64_t most = ceil_div(range, 256);
    if (splits > most) splits = most;
  } else if (range > 256) {
    // One round of CTAs: the largest clusters of which there is room for all.  Up to
    // 16 sequences of 6000-8000 keys, heads of 128, one token each: 73 us against 82
    // in shares of 512 keys and a second kernel; 1000-8000 keys 54 against 59.
    // Beyond what eight CTAs do in 512 keys each, as many as fill the GPU (2 sequences
    // of 12000-16000: 26 us against 30 in one and a half rounds).  Each CTA's
    // share is limited: where sequences differ in length, the longest alone decides
    // (4 E4M3 sequences of 5000-40000 keys: 69 us in clusters, 47 in more and smaller
    // shares; two-byte caches share what the short ones leave of HBM).
    int64_t one = 0;
    if (a.row_tiles == 1 && tiles <= slots) {
      if (range > kMaxCluster * 512 && (batches == 1 || tiles * 12 <= slots)) {
        one = slots / tiles;
      } else {
        for (const int c : {8, 6, 4, 3, 2, 1}) {
          one = c;
          if (c == 1 || room(c) >= tiles) break;
        }
      }
      if (batches > 1 && range > one * (fp8 ? 1024 : 8192)) one = 0;
    }
    if (one > 0) {
      // At least 128 keys each (one sequence of 300 keys: 5.8 us in threes, 7.3 whole).
      splits = one;
      const int64_t most = ceil_div(range, 128);
      if (splits > most) splits = most;
    } else {
      // Several rounds.  Sequences may differ in length, and the long ones' CTAs are
      // then what is left: 64 sequences of 2000-16000 keys 350 us at 10 rounds, 377
      // at 3.4.  Each CTA has so many keys that it pays its start: 64 sequences
      // of 100-1000 keys 35 us whole, 66 in fives.
      const int64_t rounds2 = tiles * 4 < slots ? 3 : tiles < slots ? 8 : 20;
      splits = rounds2 * slots / (2 * (tiles > 0 ? tiles : 1));
      const int64_t most = ceil_div(range, tiles >= slots ? 1536 : tiles * 4 >= slots ? 512 : 192);
      if (splits > most) splits = most;
      // What a cluster can merge, where that leaves no more than 512 keys each.
      if (splits > kMaxCluster && range <= kMaxCluster * 512 && tiles * kMaxCluster <= slots)
        splits = kMaxCluster;
    }
    if (splits > kMaxSplits) splits = kMaxSplits;
  }
  if (splits < 1) splits = 1;
  int64_t len = ceil_div(ceil_div(range, splits), step) * step;
  if (len < 1) len = 1;
  a.split_len = static_cast<int>(len);
  a.splits = static_cast<int>(range > 0 ? ceil_div(range, len) : 1);
  // Clusters where all of them are resident at once: 4 sequences of up to 700 keys
  // 6.4 us against 7.3 with a second kernel; beyond that, clusters wait for room
  // for all their CTAs (64 sequences of 2000-16000 keys in sixes 510 us against 348;
  // 6 sequences of 4000 keys, 48 clusters of six where 46 fit, 24 us, of four 17).
  a.cluster = !a.prefill && a.splits > 1 && a.splits <= kMaxCluster && tiles * a.splits <= slots &&
              room(a.splits) >= tiles;
  a.ctas = tiles * a.splits;
  return a;
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

struct AttnSizes {
  int64_t tokens, batches, hq, hkv, d, page, table_pages, max_q, max_kv, window;
};

gbn_status check_sizes(const AttnSizes& z, gbn_dtype dtype, gbn_dtype cache_dtype) {
  if (dtype != GBN_BF16 && dtype != GBN_F16) return GBN_ERR_DTYPE;
  if (cache_dtype != dtype && cache_dtype != GBN_E4M3) return GBN_ERR_DTYPE;
  if (z.tokens < 0 || z.tokens > INT32_MAX || z.batches < 0 || z.batches > GBN_PAGED_MAX_BATCHES ||
      z.hkv < 1 || z.hkv > 4096 || z.hq < z.hkv || z.hq > 4096 || z.hq % z.hkv || z.d < 16 ||
      z.d > GBN_PAGED_MAX_DIM || z.d % 16 || z.page < 1 || z.page > GBN_PAGED_MAX_PAGE ||
      (z.page & (z.page - 1)) || z.table_pages < 0 || z.table_pages > INT32_MAX || z.max_q < 0 ||
      z.max_kv < 0 || z.max_kv > (1 << 30) || z.window < 0 ||
      z.window > INT32_MAX || z.tokens * z.hq > INT32_MAX)
    return GBN_ERR_SHAPE;
  return GBN_OK;
}

int log2_of(int64_t v) {
  int s = 0;
  while ((int64_t(1) << s) < v) ++s;
  return s;
}

gbn_status plan_for(const AttnSizes& z, int causal, bool fp8, AttnPlan* a) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GBN_ERR_CUDA;
  const int64_t room = z.table_pages * z.page;
  const int64_t kv = z.max_kv < room ? z.max_kv : room;
  const int64_t mq = z.max_q < z.tokens ? z.max_q : z.tokens;
  *a = attn_plan(z.batches, z.hkv, z.hq / z.hkv, z.d, mq, kv, z.window, causal, log2_of(z.page),
                 fp8, sms, dev);
  if (a->splits > kMaxSplits || a->ctas > 0x7FFFFFFF) return GBN_ERR_SHAPE;
  return GBN_OK;
}

size_t plan_bytes(const AttnSizes& z, const AttnPlan& a) {
  if (a.splits <= 1 || a.cluster) return 0;
  const int64_t rows = z.tokens * z.hq;
  return static_cast<size_t>(align256(rows * a.splits * 8) + rows * a.splits * z.d * 4);
}

}  // namespace

cudaError_t read_attention_error(unsigned int* v, bool clear) { return read_paged_error(v, clear); }

}  // namespace gbn

using namespace gbn;

extern "C" {

gbn_status gbn_paged_attention_workspace_size(int64_t tokens, int64_t batches, int64_t q_heads,
                                              int64_t kv_heads, int64_t head_dim,
                                              int64_t page_size, int64_t table_pages,
                                              int64_t max_q, int64_t max_kv, int64_t window,
                                              int causal, gbn_dtype dtype, gbn_dtype cache_dtype,
                                              size_t* bytes) {
  if (!bytes) return GBN_ERR_NULL;
  const AttnSizes z{tokens, batches, q_heads, kv_heads, head_dim,
                    page_size, table_pages, max_q, max_kv, window};
  gbn_status st = check_sizes(z, dtype, cache_dtype);
  if (st != GBN_OK) return st;
  *bytes = 0;
  if (tokens == 0 || batches == 0 || max_q == 0) return GBN_OK;
  AttnPlan a;
  st = plan_for(z, causal, cache_dtype == GBN_E4M3, &a);
  if (st != GBN_OK) return st;
  *bytes = plan_bytes(z, a);
  return GBN_OK;
}

gbn_status gbn_paged_attention(const gbn_paged_attention_args* args, cudaStream_t stream) {
  if (!args) return GBN_ERR_NULL;
  const gbn_paged_attention_args& c = *args;
  const gbn_dtype dtype = static_cast<gbn_dtype>(c.dtype);
  const gbn_dtype cache_dtype = static_cast<gbn_dtype>(c.cache_dtype);
  const AttnSizes z{c.tokens,    c.batches,     c.q_heads, c.kv_heads, c.head_dim,
                    c.page_size, c.table_pages, c.max_q,   c.max_kv,   c.window};
  gbn_status st = check_sizes(z, dtype, cache_dtype);
  if (st != GBN_OK) return st;
  // The kernels work with scale * log2 e, which has to be finite too.
  if (c.num_pages < 0 || c.num_pages > INT32_MAX || c.table_stride < 0 || !(c.scale > 0.f) ||
      !std::isfinite(c.scale * kAttnLog2e))
    return GBN_ERR_SHAPE;
  if (c.tokens == 0 || c.batches == 0 || c.max_q == 0) return GBN_OK;
  if (!c.q || !c.k_cache || !c.v_cache || !c.cu_seqlens || !c.kv_lens || !c.block_table || !c.out)
    return GBN_ERR_NULL;
  const bool fp8 = cache_dtype == GBN_E4M3;
  if (fp8 && (!c.k_scale_inv || !c.v_scale_inv)) return GBN_ERR_NULL;
  const int ce = fp8 ? 1 : 2;
  auto aligned = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; };
  auto off = [](int64_t extent, int64_t stride, int esize) {
    return extent > 1 && stride * esize % 16 != 0;
  };
  if (!aligned(c.q) || !aligned(c.out) || !aligned(c.k_cache) || !aligned(c.v_cache) ||
      off(c.tokens, c.q_strides[0], 2) || off(c.tokens, c.out_strides[0], 2) ||
      off(c.q_heads, c.q_strides[1], 2) || off(c.q_heads, c.out_strides[1], 2) ||
      off(c.num_pages, c.k_cache_strides[0], ce) || off(c.num_pages, c.v_cache_strides[0], ce) ||
      off(c.page_size, c.k_cache_strides[1], ce) || off(c.page_size, c.v_cache_strides[1], ce) ||
      off(c.kv_heads, c.k_cache_strides[2], ce) || off(c.kv_heads, c.v_cache_strides[2], ce))
    return GBN_ERR_ALIGNMENT;
  // What a tensor map takes: cache strides in (0, 2^40) bytes.
  auto far = [&](int64_t extent, int64_t stride) {
    return extent > 1 && (stride <= 0 || stride >= (int64_t(1) << 40) / ce);
  };
  if (far(c.num_pages, c.k_cache_strides[0]) || far(c.num_pages, c.v_cache_strides[0]) ||
      far(c.page_size, c.k_cache_strides[1]) || far(c.page_size, c.v_cache_strides[1]) ||
      far(c.kv_heads, c.k_cache_strides[2]) || far(c.kv_heads, c.v_cache_strides[2]))
    return GBN_ERR_SHAPE;
  AttnPlan a;
  st = plan_for(z, c.causal, fp8, &a);
  if (st != GBN_OK) return st;
  if (plan_bytes(z, a) > 0 &&
      (!c.workspace || c.workspace_bytes < plan_bytes(z, a) || !aligned(c.workspace)))
    return GBN_ERR_WORKSPACE;

  AttnParams p = {};
  p.q = c.q;
  p.k = c.k_cache;
  p.v = c.v_cache;
  p.out = c.out;
  p.lse = c.lse;
  p.cu = c.cu_seqlens;
  p.kv_lens = c.kv_lens;
  p.table = c.block_table;
  p.k_scale_inv = c.k_scale_inv;
  p.v_scale_inv = c.v_scale_inv;
  p.part_ml = reinterpret_cast<float2*>(c.workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(c.workspace) +
                                      align256(c.tokens * c.q_heads * a.splits * 8));
  p.qt = c.q_strides[0];
  p.qh = c.q_strides[1];
  p.ot = c.out_strides[0];
  p.oh = c.out_strides[1];
  p.kp = c.k_cache_strides[0];
  p.ks = c.k_cache_strides[1];
  p.kh = c.k_cache_strides[2];
  p.vp = c.v_cache_strides[0];
  p.vs = c.v_cache_strides[1];
  p.vh = c.v_cache_strides[2];
  p.table_stride = c.table_stride;
  p.num_pages = c.num_pages;
  p.tokens = static_cast<int>(c.tokens);
  p.batches = static_cast<int>(c.batches);
  p.hq = static_cast<int>(c.q_heads);
  p.hkv = static_cast<int>(c.kv_heads);
  p.group = p.hq / p.hkv;
  p.d = static_cast<int>(c.head_dim);
  p.page_shift = log2_of(c.page_size);
  p.table_pages = static_cast<int>(c.table_pages);
  p.max_q = static_cast<int>(c.max_q < c.tokens ? c.max_q : c.tokens);
  p.max_kv = static_cast<int>(c.max_kv);
  p.causal = c.causal != 0;
  p.window = static_cast<int>(c.window);
  p.row_tiles = a.row_tiles;
  p.splits = a.splits;
  p.split_len = a.split_len;
  p.cluster = a.cluster;
  p.scale_log2 = c.scale * kAttnLog2e;

  const int mt = a.rows / 16;
  cudaError_t e;
  if (a.prefill)
    e = launch_paged_prefill(p, dtype, cache_dtype, stream);
  else if (dtype == GBN_BF16)
    e = fp8 ? launch_step_d<__nv_bfloat16, true>(p, mt, a.ctas, stream)
            : launch_step_d<__nv_bfloat16, false>(p, mt, a.ctas, stream);
  else
    e = fp8 ? launch_step_d<__half, true>(p, mt, a.ctas, stream)
            : launch_step_d<__half, false>(p, mt, a.ctas, stream);
  if (e != cudaSuccess) return GBN_ERR_CUDA;
  if (a.splits > 1 && !a.cluster) {
    e = dtype == GBN_BF16 ? launch_merge<__nv_bfloat16>(p, fp8, stream)
                          : launch_merge<__half>(p, fp8, stream);
    if (e != cudaSuccess) return GBN_ERR_CUDA;
  }
  return GBN_OK;
}

}  // extern "C"
