// Paged attention for many rows per kv head: prompts and chunks of prompts on
// the 5th-generation tensor cores.  Same mathematics as the kernel for few
// rows (paged_attention.cu); here the matrix products bound it: 4 d flops per
// kept (row, key) against the bytes of a key shared by 256 rows.
//
// A CTA holds two tiles of 128 rows (token x head of the kv head's group) and
// streams tiles of 128 keys past both.  Roles:
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one thread per row
//   warps 8, 9       issue the tcgen05.mma of row tile 0 and 1 (one thread each)
//   warp 10          issues the TMA loads, one lane per page box
//   warp 11          zeroes the values of slots outside the key range
//   warps 12-15      E4M3 caches (instead of 11): convert the loaded codes to f16
// Tensor memory (512 columns): scores S0, S1 (128 fp32 columns each) and
// outputs O0, O1.  S = Q K^T reads both operands from shared memory; the
// probabilities go back into S's columns as 16-bit pairs and are the A operand
// of O += P V straight from tensor memory, so they never pass through shared
// memory.  While the tensor core works on one row tile (P V of a key tile, then
// Q K^T of the next), the other's softmax runs: the two alternate.  The softmax
// hands P over in halves of 64 keys, and the first half's product runs while it
// computes the second.  (Scores in halves too, with four steps under way, were
// slower: N = 64 makes Q K^T read 192 bytes of shared memory a cycle, more than
// there are, 547 us against 468 for a prompt of 8192 tokens.)
//
// The outputs stay in tensor memory for the whole key range.  A row's
// reference maximum moves only when the running maximum has grown by more
// than 2^8 over it (bf16; f16: 2^6): until then the probabilities lose nothing in
// fp32 sums or 16-bit mantissas, and O is not touched; when it moves the
// row's own thread rescales O (a few times per row, mostly in the first
// tiles).  f16 holds probabilities from 2^-14 on with all its bits: they are taken
// 2^9 larger there, so those down to 2^-23 of the row's largest so far keep
// 2^-11 relative and smaller ones lose at most 2^-34 of that largest.
//
// K and V tiles: [128 keys][64 elements] panels with 128-byte rows in the
// 128-byte swizzle, written by TMA boxes of one page (or 128 slots of a larger
// one) each; K is read K-major, V MN-major from the same layout.  A box whose
// keys all lie outside the range is fetched from the page index one past the
// cache, which TMA fills with zeros: the byte count stays the same and nothing
// is read.  Rows of a box that the range cuts are zeroed in shared memory for
// V (a weight of 0 times what stands in such a slot must be 0); for K the mask
// replaces the score.
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "packed_tiles.cuh"
#include "paged_rows.cuh"
#include "tensor_core.cuh"

namespace gbn {
namespace {

constexpr int kRowsT = 128;                // rows per tile
constexpr int kKeys = kPrefillKeys;        // keys per tile
constexpr int kHalf = kKeys / 2;           // keys per step of the tensor core and the softmax
constexpr int kPanel = kKeys * 128;        // bytes of [128][64] 16-bit elements
constexpr int kMmaWarp = 8, kLoadWarp = 10, kZeroWarp = 11, kConvertWarp = 12;
constexpr int kLoaders = 128;              // E4M3 caches: threads of warps 12-15
constexpr int kStaging = 4;                // E4M3 caches: at most so many tiles of codes
constexpr int kSortBatches = 256;          // up to so many sequences are taken by length
// log2 growth of a row's maximum before its reference moves, and how far below the
// maximum the reference stands (f16 values): 2^(6 + 9) fits f16.  (4 + 11 hold smaller
// probabilities, and move the reference oftener: E4M3 prompts 468 us against 462, f16 heads of
// 64 335 against 330.)
template <typename TP>
constexpr float kRescale = std::is_same<TP, __half>::value ? 6.f : 8.f;
constexpr int kHeadroom = 9;
constexpr float kLargeScore = 268435456.f;  // 2^28: see large_factor

struct Barriers {
  // p_full, o_full: [row tile][half of the keys]
  uint64_t full[8], empty[8], s_full[2], p_full[2][2], o_full[2][2], q_full, cut, zeroed, turn[2];
  uint64_t raw_full[kStaging], raw_empty[kStaging];  // E4M3 caches
  float q_scale[2][kRowsT];  // E4M3 caches: what a q row's scores are times
  uint32_t tmem;
  int sequence;  // of this CTA
};

template <bool FP8, int DP>
struct PrefillShape {
  static constexpr int kPanels = DP / 64;
  static constexpr int kSlot = kPanels * kPanel;   // one K or V tile
  // Ring slots (K and V alternate); E4M3 caches: and tiles of codes on their way
  // to the conversion.
  static constexpr int kSlots = DP == 128 ? (FP8 ? 4 : 5) : (FP8 ? 6 : 8);
  static constexpr int kRaw = FP8 ? kKeys * DP : 0;
  static constexpr int kRaws = FP8 ? (DP == 128 ? 2 : 4) : 0;
  static_assert(kRaws <= kStaging, "");
  static constexpr int kQ = 2 * kSlot;
  static constexpr int kBody = kQ + kSlots * kSlot + kRaws * kRaw;
  static constexpr int kSmem = kBody + (int)sizeof(Barriers);
  static_assert(kSmem <= 232448, "");
  static constexpr int kThreads = FP8 ? 512 : 384;
  // Registers a thread: launched with 65536 / kThreads (128, 168), moved from
  // the other warps to the softmax.  256 x softmax + the rest x other =
  // kThreads x launch, exactly.
  static constexpr int kRegsLaunch = FP8 ? 128 : 168;
  static constexpr int kRegsSoftmax = FP8 ? 184 : 208;
  static constexpr int kRegsOther = FP8 ? 72 : 88;
  static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther == kThreads * kRegsLaunch, "");
};

// The factor of a row whose largest score is beyond 2^28 (log2 units) in magnitude: the power
// of two at or below the row's own, with which products are exact.  Any other rounds them by up
// to 8 and more there, and taken against the rounded maximum the largest key's probability
// would be 0 or infinite.  Scores so large are 16 powers of two apart or equal: with a
// factor up to half as large the largest still has the weight.
__device__ __forceinline__ float large_factor(float scale) {
  return __uint_as_float(__float_as_uint(scale) & 0xFF800000u);
}

// A row's columns that came out NaN (bad: bit c: among 8 c .. 8 c + 7), after it has been written, in 32 bits
// where it is a part of several (see columns_to_sum; l = 0: nothing has a weight, and they are 0).  By the row's
// thread: the rows of a warp go through the same keys, and read them once.  Whole warps that took one row after
// another were slower (34 ms against 23: 2 x 4096 tokens, 32 / 8 heads of 128, causal, with a NaN among the values of
// one token), and a call of all lanes together costs every call of this kernel 3 %.
template <typename T, bool FP8, bool PACKED>
__device__ __noinline__ void columns_again(const AttnParams& p, int b, int first, int h, const T* q, float scale,
                                           float l, float inv, int k0, int k1, int lo, int hi, uint32_t bad,
                                           uint8_t* row) {
  const Keys<T, FP8, PACKED> keys = {p, b, first, h};
  auto write = [&](int col, float f) {
    if (p.splits > 1) reinterpret_cast<float*>(row)[col] = f;
    else reinterpret_cast<uint16_t*>(row)[col] = static_cast<uint16_t>(narrow2<T>(p2(f * inv, f * inv)));
  };
  float top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int group = 0; group < p.d; group += 32) {
    uint32_t open = 0;  // bit e: column group + e
#pragma unroll 1
    for (int c = 0; c < 32 && group + c < p.d; c += 8) {
      if (!((bad >> ((group + c) / 8)) & 1u)) continue;
      uint32_t up = 0, down = 0, zero = 0;
      if (l != 0.f) open |= columns_to_sum(keys, q, scale, k0, k1, lo, hi, group + c, &up, &down) << c;
      else zero = 0xFFu;
      for (int e = 0; e < 8; ++e)
        if (((up | down | zero) >> e) & 1u) write(group + c + e, (up >> e) & 1u ? INFINITY : (down >> e) & 1u ? -INFINITY : 0.f);
    }
    if (open == 0u) continue;
    if (sum == 0.f) {
#pragma unroll 1
      for (int j = lo; j < hi; ++j) {
        float s;
        if (!keys.score(q, scale, j, &s) || s == -INFINITY) continue;
        if (s > top) sum = top == -INFINITY ? 0.f : sum * ex2(top - s);
        top = fmaxf(top, s);
        sum += ex2(s - top);
      }
    }
    float acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int j = lo; j < hi; ++j) {
      float s;
      if (!keys.score(q, scale, j, &s)) continue;
      const float w = ex2(s - (top == -INFINITY ? 0.f : top));
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (((open >> c) & 0xFFu) != 0u) keys.value(j, group + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c + e] = fmaf(w, f[e], acc[c + e]);
      }
    }
    const float back = sum == 0.f ? 0.f : l / sum;
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if ((open >> e) & 1u) write(group + e, acc[e] * back);
  }
}

template <typename T, bool FP8, int DP, bool PACKED>
__global__ void __launch_bounds__(PrefillShape<FP8, DP>::kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ AttnParams p,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  using Shape = PrefillShape<FP8, DP>;
  using TP = typename std::conditional<FP8, __half, T>::type;
  constexpr int kType = std::is_same<TP, __half>::value ? 0 : 1;  // of both products
  extern __shared__ __align__(1024) uint8_t raw[];
  Barriers& bars = *reinterpret_cast<Barriers*>(raw + Shape::kBody);

  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The longest work first, so that the last CTAs to start are short: sequences
  // by their keys, a sequence's row blocks from the last one down (causal rows
  // late in it have the most keys).
  uint32_t x = blockIdx.x;
  const int h = x % p.hkv;
  x /= p.hkv;
  int split = 0, rt, b;
  SeqRange s;
  if constexpr (PACKED) {
    // Lengths that do not fit are flagged a sequence by a thread.
    auto range = [&](int i, bool flag) {
      return packed_range(p.cu, p.cu_k, i, p.tokens, p.keys, p.max_q, p.max_kv, flag);
    };
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * Shape::kThreads + tid;
    if ((p.cu || p.cu_k) && mine < p.batches) range(static_cast<int>(mine), true);
    const TilePlace place = find_tile<Shape::kThreads>(p.cu, p.cu_k, p.batches, p.max_q, p.max_kv, p.group,
                                                       kPrefillRows, static_cast<int>(x), raw);
    if (place.tile < 0) return;
    b = place.sequence;
    rt = place.tiles - 1 - place.tile;
    s = range(b, false);
  } else {
    split = x % p.splits;
    x /= p.splits;
    rt = p.row_tiles - 1 - static_cast<int>(x % p.row_tiles);
    b = x / p.row_tiles;
    if (p.batches > 1 && p.batches <= kSortBatches) {
      // The sequence with b longer ones.  Every CTA counts for itself: a few hundred
      // cycles against a second launch.
      for (int i = tid; i < p.batches; i += Shape::kThreads) {
        const int mine = p.kv_lens[i];
        int before = 0;
#pragma unroll 8
        for (int j = 0; j < p.batches; ++j) {
          const int kv = p.kv_lens[j];
          before += kv > mine || (kv == mine && j < i);
        }
        if (before == b) bars.sequence = i;
      }
      __syncthreads();
      b = bars.sequence;
    }
    s = seq_range(p, b, tid == 0 && split == 0 && rt == 0 && h == 0);
  }
  const int r0 = rt * kPrefillRows;
  const int rows = min(kPrefillRows, s.qlen * p.group - r0);
  if (rows <= 0) return;

  // Key range of this CTA [k0, k1), first key of its tiles, tiles per row tile.
  const int i_last = (r0 + rows - 1) / p.group;
  const int lo = row_low(p, s, r0 / p.group), hi = row_high(p, s, i_last);
  const int64_t start = lo + static_cast<int64_t>(split) * p.split_len;
  const int k0 = static_cast<int>(min(start, static_cast<int64_t>(hi)));
  const int k1 = static_cast<int>(min(start + p.split_len, static_cast<int64_t>(hi)));
  const int base = k0 & ~(kKeys - 1);
  int nt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(r0 + kRowsT * (t + 1), r0 + rows) - 1;  // last row of the tile
    const int end = last < r0 + kRowsT * t ? 0 : min(row_high(p, s, last / p.group), k1);
    nt[t] = k1 > k0 && end > base ? (end - base + kKeys - 1) / kKeys : 0;
  }
  const int nmax = max(nt[0], nt[1]);

  const uint32_t qs = smem_u32(raw), ring = qs + Shape::kQ;
  uint8_t* const gen0 = raw;  // the same, generic
  if (qs & 1023u) {  // the swizzle goes by address bits; the compiler's alignment holds
    if (tid == 0) flag_wait_timeout();
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < Shape::kSlots; ++i) {
      mbar_init(&bars.full[i], FP8 ? kLoaders / 32 : 1);
      mbar_init(&bars.empty[i], 2);  // one arrival for each row tile
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.turn[t], 1);
      for (int hf = 0; hf < 2; ++hf) {
        mbar_init(&bars.p_full[t][hf], 4);  // one arrival per warp
        mbar_init(&bars.o_full[t][hf], 1);
      }
    }
    for (int i = 0; i < Shape::kRaws; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], kLoaders / 32);
    }
    mbar_init(&bars.q_full, 8);
    mbar_init(&bars.cut, 2);
    mbar_init(&bars.zeroed, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc_alloc(&bars.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  bool ok = true;

  float kscale = 1.f, vscale = 1.f;
  if constexpr (FP8) {
    kscale = *p.k_scale_inv;
    vscale = *p.v_scale_inv;
  }

  // Key tiles with slots outside [k0, k1) (only the first and the last can be).
  const bool cut_first = nmax > 0 && base < k0;
  const bool cut_last = nmax > 0 && base + nmax * kKeys > k1 && !(nmax == 1 && cut_first);

  if (warp >= kMmaWarp) {
    set_regs_dec<Shape::kRegsOther>();
    if (warp < kMmaWarp + 2) {
      // ------------------------------------------------ tensor core issue
      constexpr uint32_t kIdQK = instr_desc(kType, kRowsT, kKeys, 0);
      constexpr uint32_t kIdPV = instr_desc(kType, kRowsT, DP, 1);
      // Uniform across the warp, and known to be.
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t q_lo = __shfl_sync(0xFFFFFFFFu, desc_lo(qs, 16), 0);
      const uint32_t k_lo = __shfl_sync(0xFFFFFFFFu, desc_lo(ring, 16), 0);
      const uint32_t v_lo = __shfl_sync(0xFFFFFFFFu, desc_lo(ring, kPanel), 0);
      // One thread per row tile, nothing collective.  The tensor core's queue is
      // short: an issuing thread is held until the step before its own has
      // begun, so what it does between two products -- a wait on a barrier that
      // is complete already costs about 100 cycles -- leaves the tensor core
      // idle.  With a thread per tile one waits while the other's products run.
      // They take turns (P V of a key tile, Q K^T of the next): left to themselves
      // both tiles' products interleave, both softmaxes then run at once and the
      // tensor core waits (600 us for a prompt of 8192 tokens instead of the 500
      // of one thread for both).  The turn passes two steps before its end, so
      // that it arrives in time.
      if (nmax > 0 && elect_one()) {
        const int t = warp - kMmaWarp, n = nt[t];
        const uint32_t ts = tm + t * 128, to = tm + 256 + t * 128;
        const uint32_t qt = q_lo + t * (Shape::kSlot >> 4);
        constexpr int kSteps = DP / 16;
        auto qk = [&](int slot) {
          const uint32_t kt = k_lo + slot * (Shape::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
            if (kk == kSteps - 2) mbar_arrive(&bars.turn[t ^ 1]);
            const uint32_t at = ((kk / 4) * kPanel + (kk % 4) * 32) >> 4;
            tc_mma_ss(ts, qt + at, kt + at, kDescHi, kIdQK, kk > 0);
          }
          tc_commit(&bars.s_full[t]);
        };
        // This thread's turns: tile 1's i-th follows tile 0's i-th.
        uint32_t turns = 0;
        auto my_turn = [&]() {
          const uint32_t i = turns++;
          return t == 0 ? i == 0 || mbar_wait(&bars.turn[0], (i - 1) & 1)
                        : mbar_wait(&bars.turn[1], i & 1);
        };
        uint32_t zeros = 0;  // waits for zeroed slots so far
        ok = mbar_wait(&bars.q_full, 0) && mbar_wait(&bars.full[0], 0) && my_turn();
        if (ok) {
          tc_fence_after();
          if (n > 0) {
            qk(0);
            tc_commit(&bars.empty[0]);
          } else {
            // Each tile arrives once per use of a slot, in order: also one that
            // does not read it waits until it is full.
            mbar_arrive(&bars.turn[t ^ 1]);
            mbar_arrive(&bars.empty[0]);
          }
        }
        int vs = 1, vph = 0;  // V's slot in the ring and its phase
        for (int j = 0; ok && j < nmax; ++j) {
          int ks = vs + 1, kph = vph;
          if (ks == Shape::kSlots) ks = 0, kph ^= 1;
          const bool more = j + 1 < nmax, cut = (j == 0 && cut_first) || (j == nmax - 1 && cut_last);
          ok = mbar_wait(&bars.full[vs], vph) && (!more || mbar_wait(&bars.full[ks], kph));
          if (!FP8 && ok && cut) {
            mbar_arrive(&bars.cut);  // its values are here: zero what lies outside
            if (j < n) ok = mbar_wait(&bars.zeroed, zeros++ & 1);
          }
          if (ok && j < n) ok = mbar_wait(&bars.p_full[t][0], j & 1);
          ok = ok && my_turn();
          if (!ok) break;
          if (j < n) {
            const bool next = j + 1 < n;
            const uint32_t vt = v_lo + vs * (Shape::kSlot >> 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              if (hf == 1) ok = mbar_wait(&bars.p_full[t][1], j & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = hf * 4; kk < hf * 4 + 4; ++kk) {
                if (kk == 6 && !next) mbar_arrive(&bars.turn[t ^ 1]);
                tc_mma_ts(to, ts + hf * kHalf + (kk - hf * 4) * 8, vt + kk * (2048 >> 4), kDescHi, kIdPV,
                          kk > 0 ? 1u : static_cast<uint32_t>(j > 0));
              }
              tc_commit(&bars.o_full[t][hf]);
            }
            if (!ok) break;
            tc_commit(&bars.empty[vs]);
            if (next) {
              qk(ks);
              tc_commit(&bars.empty[ks]);
            } else if (more) {
              mbar_arrive(&bars.empty[ks]);
            }
          } else {
            // The other tile's key tiles go on.
            mbar_arrive(&bars.turn[t ^ 1]);
            mbar_arrive(&bars.empty[vs]);
            if (more) mbar_arrive(&bars.empty[ks]);
          }
          vs = ks + 1;
          vph = kph;
          if (vs == Shape::kSlots) vs = 0, vph ^= 1;
        }
        // The last arrivals have landed before the CTA ends.
        if (ok) {
          const int last = 2 * nmax - 1;
          ok = mbar_wait(&bars.empty[last % Shape::kSlots], (last / Shape::kSlots) & 1);
        }
      }
      __syncwarp();
    } else if (!FP8 && warp == kZeroWarp) {
      // ------------------------------------------------ slots outside the range
      // Values of slots outside [k0, k1) become zero (a weight of 0 times what
      // stands there must be 0).
      uint32_t event = 0;
      for (int e = 0; e < 2; ++e) {
        if (e == 0 ? !cut_first : !cut_last) continue;
        const int j = e == 0 ? 0 : nmax - 1, slot = (2 * j + 1) % Shape::kSlots;
        // (a whole key range may lie before the last tile's turn: a longer limit)
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_for(&bars.cut, event++ & 1, 30 * kWaitLimitNs));
        if (!ok) break;
        const int tb = base + j * kKeys;
        const int za = max(0, k0 - tb), zb = min(kKeys, k1 - tb);
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        const int outside = za + kKeys - zb;
        for (int i = lane; i < outside * 8 * Shape::kPanels; i += 32) {
          const int c = i & 7, pr = i >> 3;
          const int pn = pr % Shape::kPanels, o = pr / Shape::kPanels;
          const int r = o < za ? o : zb + (o - za);
          *reinterpret_cast<uint4*>(gen0 + Shape::kQ + slot * Shape::kSlot + pn * kPanel +
                                    r * 128 + c * 16) = z;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.zeroed);
      }
    } else if (warp == kLoadWarp) {
      // ------------------------------------------------ TMA loads
      const int page = PACKED ? kKeys : 1 << p.page_shift;
      const int box = min(page, kKeys);           // keys per box
      const int boxes = kKeys / box;              // per panel, at most 16
      const int32_t* tab = p.table + b * p.table_stride;
      const int e_last = k1 > 0 ? (k1 - 1) >> p.page_shift : 0;
      // This lane's box of key tile j: its table entry, read one tile ahead and
      // looked at only when the tile's turn comes.
      const int zero_page = max(1, static_cast<int>(p.num_pages));  // one past: zeros
      auto wanted = [&](int j) {
        const int key = base + j * kKeys + lane * box;
        return lane < boxes && key < k1 && key + box > k0;
      };
      auto entry = [&](int j) {
        if constexpr (PACKED) return 0;
        const int key = base + j * kKeys + lane * box;
        return wanted(j) ? tab[min(key >> p.page_shift, e_last)] : 0;
      };
      // Two-byte caches: panels of 64 elements straight into the ring; E4M3:
      // whole rows of codes into the staging tiles.
      constexpr int kDeep = FP8 ? Shape::kRaws : Shape::kSlots;
      constexpr uint32_t kBytes = FP8 ? Shape::kRaw : Shape::kSlot;
      uint64_t* const full = FP8 ? bars.raw_full : bars.full;
      uint64_t* const empty = FP8 ? bars.raw_empty : bars.empty;
      const uint32_t dst0 = FP8 ? ring + Shape::kSlots * Shape::kSlot : ring;
      int issued = 0;
      int cur = nmax > 0 ? entry(0) : 0;
      for (int j = 0; ok && j < nmax; ++j) {
        const int next = j + 1 < nmax ? entry(j + 1) : 0;
        int pg = zero_page;
        if constexpr (PACKED) {
          pg = 0;  // (rows behind the sequence are the next one's, behind the last zeros)
        } else if (wanted(j)) {
          if (cur >= 0 && cur < p.num_pages) pg = cur;
          else flag_bad_index();
        }
        const int key = base + j * kKeys + lane * box;
        for (int kv = 0; kv < 2; ++kv) {
          const int it = 2 * j + kv, slot = it % kDeep, use = it / kDeep;
          if (use > 0) ok = warp_wait(&empty[slot], (use - 1) & 1);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], kBytes);
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int pn = 0; pn < (FP8 ? 1 : Shape::kPanels); ++pn)
              tma_box(dst0 + slot * kBytes + pn * kPanel + lane * box * (FP8 ? DP : 128),
                      kv ? &vmap : &kmap, pn * 64, h,
                      PACKED ? s.k0 + key : key & (page - 1), pg, &full[slot]);
          }
          issued = it + 1;
        }
        cur = next;
      }
      if (!ok) {
        // Leave no copy in flight behind.
        for (int i = max(0, issued - kDeep); i < issued; ++i)
          warp_wait(&full[i % kDeep], (i / kDeep) & 1);
      }
    } else if (FP8 && warp >= kConvertWarp) {
      // ------------------------------------------------ E4M3: codes to f16
      if constexpr (FP8) {
        constexpr int kChunks = DP / 16;               // 16-byte chunks per key
        constexpr int kRowsStep = kLoaders / kChunks;  // key rows per step
        constexpr int kSteps = kKeys / kRowsStep;
        const int lt = tid - 32 * kConvertWarp;
        const int c = lt % kChunks, row0 = lt / kChunks;
        for (int it = 0; ok && it < 2 * nmax; ++it) {
          const int rs = it % Shape::kRaws, slot = it % Shape::kSlots, use = it / Shape::kSlots;
          ok = warp_wait(&bars.raw_full[rs], (it / Shape::kRaws) & 1);
          if (!ok) break;
          const uint8_t* src = gen0 + Shape::kQ + Shape::kSlots * Shape::kSlot + rs * Shape::kRaw;
          const int tb = base + (it >> 1) * kKeys;
          uint4 w[kSteps];
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const int r = st * kRowsStep + row0;
            w[st] = *reinterpret_cast<const uint4*>(src + r * DP + c * 16);
            // What stands outside the range must not enter.
            if (tb + r < k0 || tb + r >= k1) w[st] = make_uint4(0u, 0u, 0u, 0u);
          }
          if (use > 0) ok = warp_wait(&bars.empty[slot], (use - 1) & 1);
          if (!ok) break;
          uint8_t* dst = gen0 + Shape::kQ + slot * Shape::kSlot + (c / 4) * kPanel;
          const int c2 = (c % 4) * 2;
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const uint32_t a[4] = {w[st].x, w[st].y, w[st].z, w[st].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[2 * e] = e4m3x2_to_f16x2(a[e] & 0xFFFFu);
              o[2 * e + 1] = e4m3x2_to_f16x2(a[e] >> 16);
            }
            const int r = st * kRowsStep + row0;
            *reinterpret_cast<uint4*>(dst + r * 128 + ((c2 ^ (r & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + r * 128 + (((c2 + 1) ^ (r & 7)) << 4)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.raw_empty[rs]);
            mbar_arrive(&bars.full[slot]);
          }
        }
      }
    }
  } else {
    // -------------------------------------------------- softmax
    set_regs_inc<Shape::kRegsSoftmax>();
    const int t = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const int gr = r0 + t * kRowsT + r;          // row of the (sequence, kv head)
    const bool live = t * kRowsT + r < rows;
    const int token_i = live ? gr / p.group : i_last;
    const int head = h * p.group + (live ? gr - token_i * p.group : 0);
    // q's rows, by whole warps: a row's 16-byte chunks by neighbouring lanes, its
    // place from the lane that has divided for it.  Nothing waits before all of them
    // are under way: one load at a time took most of the 21000 cycles that a CTA
    // needed up to its first scores.
    {
      constexpr int C = DP / 8;
      const T* q = reinterpret_cast<const T*>(p.q);
      const int c = lane % C;
      const int64_t q_at = (s.q0 + token_i) * p.qt + head * p.qh;
      const bool in_d = c * 8 < p.d;
      auto place = [&](int rr) {  // of this lane's chunk of the warp's row rr, in bytes
        const int row = quad * 32 + rr;
        return t * Shape::kSlot + (c / 8) * kPanel + row * 128 + (((c & 7) ^ (row & 7)) << 4);
      };
      const int left = rows - t * kRowsT - quad * 32;  // rows of this warp that there are
      if constexpr (!FP8) {
#pragma unroll 1
        for (int i = 0; i < C; ++i) {
          const int rr = i * (32 / C) + lane / C;
          const int64_t from = __shfl_sync(0xFFFFFFFFu, q_at, rr);
          const bool on = rr < left && in_d;
          cp_async16(qs + place(rr), q + (on ? from + c * 8 : 0), on);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      } else {
        // A negative factor of the keys turns q's sign, a factor of 0 clears it:
        // what is left multiplies the scores by something positive.
        const uint32_t flip = kscale < 0.f ? 0x80008000u : 0u, keep = kscale == 0.f ? 0u : ~0u;
        uint4 ws[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int rr = i * (32 / C) + lane / C;
          const int64_t from = __shfl_sync(0xFFFFFFFFu, q_at, rr);
          ws[i] = make_uint4(0u, 0u, 0u, 0u);
          if (rr < left && in_d) ws[i] = *reinterpret_cast<const uint4*>(q + from + c * 8);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int rr = i * (32 / C) + lane / C;
          uint4& w = ws[i];
          const float back = q_to_f16<T, C>(w);
          if (c == 0) bars.q_scale[t][quad * 32 + rr] = back;
          w.x = (w.x ^ flip) & keep;
          w.y = (w.y ^ flip) & keep;
          w.z = (w.z ^ flip) & keep;
          w.w = (w.w ^ flip) & keep;
          *reinterpret_cast<uint4*>(gen0 + place(rr)) = w;
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full);
    }
    const int rlo = max(row_low(p, s, token_i), k0), rhi = min(row_high(p, s, token_i), k1);
    auto factor = [&]() {  // of the row's scores
      float f = p.scale_log2 * (kscale == 0.f ? 1.f : fabsf(kscale));
      if constexpr (FP8) f *= bars.q_scale[t][r];  // written by this warp
      return f == 0.f ? 1.4e-45f : f;  // (a product that vanished: -inf times it has to stay -inf)
    };
    float scale = factor();
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128;             // S, and P over it
    const uint32_t to = tmem + lanes + 256 + t * 128;
    float m = -INFINITY;   // the row's reference maximum (log2 units)
    float l = 0.f;
    const int n = nt[t];
    // Step i: keys 64 i .. 64 i + 63 of the range, half i % 2 of key tile i / 2.
    for (int i = 0; i < 2 * n; ++i) {
      const int hf = i & 1;
      const uint32_t th = ts + hf * kHalf;       // this half's scores, P over them
      if (hf == 0) {
        ok = warp_wait(&bars.s_full[t], (i >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      const int tb = base + i * kHalf;
      const bool cut = __any_sync(0xFFFFFFFFu, tb < rlo || tb + kHalf > rhi);
      bool done = false;
      if (i > 0 && !cut) {
        // The usual step: every key kept.  The exponentials go ahead with the
        // reference as it stands, the step's maximum beside them (another pipe);
        // where it turns out to have grown too far, the step is done again
        // below.  Bound by ex2 (4.3 to 5 cycles a warp); a path that could go
        // either way with the scores in registers would copy them.
        uint32_t sc[64], pk[32];
        tc_ld32(th, sc);
        tc_ld32(th + 32, sc + 32);
        tc_wait_ld<64>(sc);
        const float mb = m == -INFINITY ? 0.f : reference<TP, kHeadroom>(m);
        const uint64_t sc2 = p2(scale, scale), mb2 = p2(-mb, -mb);
        uint64_t l2[2] = {p2(l, 0.f), 0ull};
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float s0 = __uint_as_float(sc[2 * e]), s1 = __uint_as_float(sc[2 * e + 1]);
          const float2 a = u2(fma2(p2(s0, s1), sc2, mb2));
          mx[e & 3] = max3(mx[e & 3], s0, s1);
          const uint64_t x2 = p2(ex2(a.x), ex2(a.y));
          l2[e & 1] = add2(l2[e & 1], x2);
          pk[e] = narrow2<TP>(x2);
        }
        const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
        // -inf - -inf is not a number: no growth.
        if (!__any_sync(0xFFFFFFFFu, mt - m > kRescale<TP>)) {
          tc_st32(th, pk);
          const float2 la = u2(add2(l2[0], l2[1]));
          l = la.x + la.y;
          done = true;
        }
      }
      if (!done) {
        // The first step, one that the range or the mask cuts, and one whose
        // maximum has grown: the maximum first, then the rest.
        uint32_t sc[64], pk[32];
        tc_ld32(th, sc);
        tc_ld32(th + 32, sc + 32);
        tc_wait_ld<64>(sc);
        // Bit e: key tb + e is kept (two comparisons a key took 1000 cycles a step).
        const uint64_t kept = low_bits(rhi - tb) & ~low_bits(rlo - tb);
        const uint32_t kept_lo = static_cast<uint32_t>(kept), kept_hi = static_cast<uint32_t>(kept >> 32);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          const uint32_t bit = (e < 32 ? kept_lo : kept_hi) & (1u << (e & 31));
          sc[e] = bit ? sc[e] : 0xFF800000u;  // -inf
        }
#pragma unroll
        for (int e = 0; e < 64; e += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = max3(mx[i], __uint_as_float(sc[e + i]), __uint_as_float(sc[e + 4 + i]));
        const float raw = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), mt = raw * scale;
        if (__any_sync(0xFFFFFFFFu, mt - m > kRescale<TP>)) {
          float mn = fmaxf(m, mt);
          float al = mn == -INFINITY ? 1.f
                                     : ex2(reference<TP, kHeadroom>(m) - reference<TP, kHeadroom>(mn));
          if ((fabsf(mn) >= kLargeScore || (fabsf(m) >= kLargeScore && m != -INFINITY)) && mn != -INFINITY) {
            // Large scores, now or so far: both maxima by the row's own factor.
            const float f = factor(), was = m / scale, m0 = scale == f ? m : was * f;
            const float n0 = fmaxf(m0, raw * f);
            al = fminf(ex2(m0 - n0), 1.f);
            scale = fabsf(n0) >= kLargeScore ? large_factor(f) : f;
            mn = n0 == m0 && scale == f ? m0 : fmaxf(was, raw) * scale;
          }
          l *= al;
          m = mn;
          if (i > 0) {
            // Every product of the steps before has to be in O.
            ok = warp_wait(&bars.o_full[t][hf ^ 1], ((i - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int q2 = 0; q2 < DP / 32; ++q2) {
              uint32_t o[32];
              tc_ld32(to + q2 * 32, o);
              tc_wait_ld<32>(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tc_st32(to + q2 * 32, o);
            }
          }
        }
        const float mb = m == -INFINITY ? 0.f : reference<TP, kHeadroom>(m);
        const uint64_t sc2 = p2(scale, scale), mb2 = p2(-mb, -mb);
        uint64_t l2[2] = {p2(l, 0.f), 0ull};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 a = u2(fma2(
              p2(__uint_as_float(sc[2 * e]), __uint_as_float(sc[2 * e + 1])), sc2, mb2));
          const uint64_t x2 = p2(ex2(a.x), ex2(a.y));
          l2[e & 1] = add2(l2[e & 1], x2);
          pk[e] = narrow2<TP>(x2);
        }
        tc_st32(th, pk);
        const float2 la = u2(add2(l2[0], l2[1]));
        l = la.x + la.y;
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[t][hf]);
    }
    // Output.
    if (ok && n > 0) {
      ok = warp_wait(&bars.o_full[t][1], (n - 1) & 1);
      tc_fence_after();
    }
    if (ok) {
      const int64_t token = s.q0 + token_i;
      const int64_t ro = token * p.hq + head;
      const bool part = p.splits > 1;
      // Through shared memory (q's rows of this warp are used up), 128 bytes a row at
      // a time, so that a store writes whole lines: a lane to a row took 5400 cycles
      // a CTA, this 3900.
      uint8_t* const stage = gen0 + t * Shape::kSlot + quad * 32 * 128;
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, live && (!part || l != 0.f));
      uint8_t* const dst = part ? reinterpret_cast<uint8_t*>(p.part_o) : static_cast<uint8_t*>(p.out);
      const int64_t at = part ? (static_cast<int64_t>(split) * p.tokens * p.hq + ro) * p.d * 4
                              : (token * p.ot + head * p.oh) * 2;
      auto put = [&](int c, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(w0, w1, w2, w3);
      };
      auto flush = [&](int from, int chunks) {  // byte of the row, 16-byte chunks
        __syncwarp();
        const int c = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3);
          const int64_t row = __shfl_sync(0xFFFFFFFFu, at, rr);
          const bool on = (some >> rr) & 1;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
          if (on && c < chunks) *reinterpret_cast<uint4*>(dst + row + from + c * 16) = w;
        }
        __syncwarp();
      };
      const float inv = part ? 1.f : l == 0.f ? 0.f : vscale / l;
      const float ref = reference<TP, kHeadroom>(scale == factor() ? m : m / scale * factor());
      if (live) {
        if (part) p.part_ml[ro * p.splits + split] = make_float2(ref, l);
        else if (p.lse) p.lse[ro] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
      }
      uint32_t bad = 0;  // bit c: a NaN in columns 8 c .. 8 c + 7
      // (one copy of the code: a CTA runs it once, and fetching it is what it costs)
#pragma unroll 1
      for (int q4 = 0; q4 < DP / 32; ++q4) {
        const int col = q4 * 32;
        uint32_t o[32];
        if (n > 0) {
          tc_ld32(to + col, o);
          tc_wait_ld<32>(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          float x = __uint_as_float(o[i]);
#pragma unroll
          for (int e = 1; e < 7; e += 2)
            x = max3_nan(x, __uint_as_float(o[i + e]), __uint_as_float(o[i + e + 1]));
          x = max3_nan(x, x, __uint_as_float(o[i + 7]));
          bad |= x != x ? 1u << (q4 * 4 + i / 8) : 0u;
        }
        auto narrow = [&](float x, float y) { return narrow2<T>(mul2(p2(x, y), p2(inv, inv))); };
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i) put(i, o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = narrow(__uint_as_float(o[i + 2 * e]), __uint_as_float(o[i + 2 * e + 1]));
            put((q4 & 1) * 4 + i / 8, w[0], w[1], w[2], w[3]);
          }
        }
        if (part) flush(col * 4, (p.d - col) / 4);
        else if (q4 & 1) flush((col - 32) * 2, (p.d - (col - 32)) / 8);
        else __syncwarp();  // the loads of tensor memory take the whole warp
      }
      // NaN next to keys that the row dropped and others of its tiles keep, or where nothing has a weight.  (A NaN
      // sum: a kept score is NaN, and so is the row.)
      if (bad && ((some >> lane) & 1u) && l == l && (l == 0.f || rlo > k0 || rhi < k1))
        columns_again<T, FP8, PACKED>(p, b, s.k0, h, reinterpret_cast<const T*>(p.q) + token * p.qt + head * p.qh,
                                      FP8 ? p.scale_log2 * kscale : p.scale_log2, l, inv, k0, k1, rlo, rhi, bad,
                                      dst + at);
    }
  }

  if (!ok) flag_wait_timeout();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tc_dealloc(tmem);
}

// ---- host side

template <typename T, bool FP8, int DP, bool PACKED = false>
cudaError_t launch(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                   cudaStream_t st) {
  using Shape = PrefillShape<FP8, DP>;
  auto k = paged_prefill_kernel<T, FP8, DP, PACKED>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k, Shape::kSmem, done);
  if (e != cudaSuccess) return e;
  // (contiguous keys: row_tiles counts those of all sequences)
  const int64_t grid = int64_t(p.row_tiles) * (PACKED ? 1 : p.batches) * p.splits * p.hkv;
  return launch_pdl(k, dim3(static_cast<unsigned>(grid)), dim3(Shape::kThreads), Shape::kSmem, st, p,
                    km, vm);
}

}  // namespace

bool make_cache_map(CUtensorMap* map, const void* base, int esize, bool bf16, int inner, int rows,
                    bool swizzle, const AttnParams& p, int64_t sp, int64_t ss, int64_t sh) {
  EncodeFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t es = static_cast<cuuint64_t>(esize), page = cuuint64_t(1) << p.page_shift;
  const cuuint64_t pages = cuuint64_t(p.num_pages > 0 ? p.num_pages : 1);
  const cuuint64_t dims[4] = {cuuint64_t(p.d), cuuint64_t(p.hkv), page, pages};
  // Dimensions of one element may have any stride: give those a valid one.
  const cuuint64_t strides[3] = {p.hkv > 1 ? cuuint64_t(sh) * es : 16,
                                 page > 1 ? cuuint64_t(ss) * es : 16,
                                 pages > 1 ? cuuint64_t(sp) * es : 16};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), 1,
                             static_cast<cuuint32_t>(page < cuuint64_t(rows) ? page : rows), 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : bf16     ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle sw = !swizzle              ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : inner * esize >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                       : CU_TENSOR_MAP_SWIZZLE_64B;
  return enc(map, type, 4, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_paged_prefill(const AttnParams& p, gbn_dtype dtype, gbn_dtype cache_dtype,
                                 cudaStream_t stream) {
  const bool fp8 = cache_dtype == GBN_E4M3, bf16 = dtype == GBN_BF16;
  CUtensorMap km = {}, vm = {};
  const int esize = fp8 ? 1 : 2, dp = p.d <= 64 ? 64 : 128;
  const int inner = fp8 ? dp : 64;
  if (!make_cache_map(&km, p.k, esize, bf16, inner, kKeys, !fp8, p, p.kp, p.ks, p.kh) ||
      !make_cache_map(&vm, p.v, esize, bf16, inner, kKeys, !fp8, p, p.vp, p.vs, p.vh))
    return cudaErrorInvalidValue;
  if (p.d <= 64) {
    if (fp8)
      return bf16 ? launch<__nv_bfloat16, true, 64>(p, km, vm, stream)
                  : launch<__half, true, 64>(p, km, vm, stream);
    return bf16 ? launch<__nv_bfloat16, false, 64>(p, km, vm, stream)
                : launch<__half, false, 64>(p, km, vm, stream);
  }
  if (fp8)
    return bf16 ? launch<__nv_bfloat16, true, 128>(p, km, vm, stream)
                : launch<__half, true, 128>(p, km, vm, stream);
  return bf16 ? launch<__nv_bfloat16, false, 128>(p, km, vm, stream)
              : launch<__half, false, 128>(p, km, vm, stream);
}

cudaError_t launch_attention_fwd(const AttnParams& p, gbn_dtype dtype, cudaStream_t stream) {
  const bool bf16 = dtype == GBN_BF16;
  CUtensorMap km = {}, vm = {};
  if (!make_packed_map(&km, p.k, bf16, p.d, p.hkv, p.keys, p.ks, p.kh, kKeys) ||
      !make_packed_map(&vm, p.v, bf16, p.d, p.hkv, p.keys, p.vs, p.vh, kKeys))
    return cudaErrorInvalidValue;
  if (p.d <= 64)
    return bf16 ? launch<__nv_bfloat16, false, 64, true>(p, km, vm, stream)
                : launch<__half, false, 64, true>(p, km, vm, stream);
  return bf16 ? launch<__nv_bfloat16, false, 128, true>(p, km, vm, stream)
              : launch<__half, false, 128, true>(p, km, vm, stream);
}

cudaError_t read_prefill_error(unsigned int* v, bool clear) { return read_paged_error(v, clear); }

}  // namespace gbn
