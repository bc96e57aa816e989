// The backward pass of the attention over whole sequences: kernels and their launches, of one
// element type a translation unit.
#pragma once

#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_rows.cuh"
#include "packed_tiles.cuh"
#include "tensor_core.cuh"

namespace gbn {
namespace {

// ---- row statistics
//
// delta_i = dout_i.out_i for every query and head, and lse beside it in the form and order
// that the kernel below reads: by head, then query.  f16 besides: the largest squared norms of
// 16 rows of dout and v.  A CTA takes 16 tokens and 16 heads; a row is C lanes of 8
// elements.  It reads out and dout once (cold, 4096 tokens of 32 heads of 128: 67 MB in 19 us, 44 %
// of what memory gives); neither that nor the issue slots (57 %) are full: a warp has eight loads
// under way and 38 % of the warps a multiprocessor can hold are there.
constexpr int kStatHeads = 16, kStatThreads = 256;

template <typename T, int C>
__global__ void __launch_bounds__(kStatThreads) attention_stats_kernel(const AttnBwdParams p) {
  constexpr bool kNorms = Elem<T>::kDt == DT_F16;
  __shared__ float deltas[kStatHeads][kStatTokens + 1];
  __shared__ float norms[kStatHeads][kStatTokens + 1];
  // The gradients' kernel may begin once everything before this one is complete (its first
  // loads do not need the statistics).
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h0 = blockIdx.y * kStatHeads;
  // Lengths that do not fit are flagged here, a sequence by a thread.
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kStatThreads + tid;
  if ((p.cu || p.cu_k) && h0 == 0 && mine < p.batches) bwd_range(p, static_cast<int>(mine), true);
  const bool values = static_cast<int>(blockIdx.x) >= p.q_stat_blocks;  // f16: v's rows
  const TilePlace place =
      values ? find_tile<kStatThreads, false>(p.cu_k, nullptr, p.batches, p.max_k, 0, 1, kStatTokens,
                                              blockIdx.x - p.q_stat_blocks, nullptr)
             : find_tile<kStatThreads, false>(p.cu, nullptr, p.batches, p.max_q, 0, 1, kStatTokens, blockIdx.x,
                                              nullptr);
  if (place.tile < 0 || (values && h0 >= p.hkv)) return;
  const int b = place.sequence, i0 = place.tile * kStatTokens;
  const SeqRange s = bwd_range(p, b, false);
  const int n = values ? s.kv : s.qlen, heads = values ? p.hkv : p.hq;
  if (i0 >= n) return;  // (lengths that do not fit)
  const int c = lane % C;
  auto row_sum = [&](float v) {
#pragma unroll
    for (int o = C / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  constexpr int kStep = kStatThreads / C, kAtOnce = 4;  // rows the CTA reads at once, times 4
  const int count = min(heads - h0, kStatHeads), total = min(kStatTokens, n - i0) * count;
  for (int from = warp * (32 / C) + lane / C, first = 0; first < total; first += kAtOnce * kStep) {
    uint4 xw[kAtOnce], yw[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int r = first + u * kStep + from;
      xw[u] = yw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < total && c * 8 < p.d) {
        const int64_t at = (values ? s.k0 : s.q0) + static_cast<int64_t>(i0) + r / count, head = h0 + r % count;
        if (!values) {
          xw[u] = ld_stream16(static_cast<const T*>(p.out) + at * p.ot + head * p.oh + c * 8);
          yw[u] = ld_stream16(static_cast<const T*>(p.dout) + at * p.gt + head * p.gh + c * 8);
        } else {
          yw[u] = ld_stream16(static_cast<const T*>(p.v) + at * p.vt + head * p.vh + c * 8);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int r = first + u * kStep + from;
      const uint32_t xa[4] = {xw[u].x, xw[u].y, xw[u].z, xw[u].w}, ya[4] = {yw[u].x, yw[u].y, yw[u].z, yw[u].w};
      float x[8], y[8], sum = 0.f, square = 0.f;
      unpack<T, 8>(xa, x);
      unpack<T, 8>(ya, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(x[e], y[e], sum);
        if (kNorms) square = fmaf(y[e], y[e], square);
      }
      sum = row_sum(sum);
      if (kNorms) square = row_sum(square);
      if (c == 0 && r < total) {
        deltas[r % count][r / count] = -sum;
        if (kNorms) norms[r % count][r / count] = square;
      }
    }
  }
  __syncthreads();
  const int64_t base = stat_base(s.q0, b) + i0;
  for (int r = tid; !values && r < kStatTokens * kStatHeads; r += kStatThreads) {
    const int t = r % kStatTokens, hh = r / kStatTokens;
    if (i0 + t >= n || h0 + hh >= heads) continue;
    const int64_t at = (h0 + hh) * p.stat_stride + base + t;
    p.ndelta[at] = deltas[hh][t];
    p.nlse[at] = fmaf(p.lse[(s.q0 + static_cast<int64_t>(i0) + t) * p.hq + h0 + hh], -kAttnLog2e,
                      static_cast<float>(kWeightLog2<T>));
  }
  if (kNorms && tid < kStatHeads && h0 + tid < heads) {
    float most = 0.f;
#pragma unroll
    for (int t = 0; t < kStatTokens; ++t) most = i0 + t < n ? fmax_nan(most, norms[tid][t]) : most;
    const int64_t head = h0 + tid;
    if (values) p.v_norms[head * p.v_norm_stride + norm_base(s.k0, b) + place.tile] = most;
    else p.q_norms[head * p.q_norm_stride + norm_base(s.q0, b) + place.tile] = most;
  }
}

// ---- the gradients on the tensor cores
//
// A CTA holds one tile of 128 rows (x: keys for dk and dv, queries for dq) and streams tiles
// of 128 rows of the other side (y) past it; with x1, x2 = k, v and y1, y2 = q, dout (or the
// other way round) a step is
//     S = x1 y1^T,  dP = x2 y2^T
//     P = 2^(S scale log2(e) - lse log2(e)),  dS = P (dP - delta)
//     acc1 += dS y1 (dk, or dq),  acc2 += P y2 (dv)
// P and dS are transposed for dk and dv as they come, so neither passes through shared
// memory: they go back into the columns of S and dP as 16-bit pairs, and are the first
// operand from there.  A pass for all three gradients would need five products a step
// instead of the seven of two passes, but its dq is a sum over CTAs: in memory, by additions
// in an order that changes from run to run, and of as many bytes as the products read.  Two
// passes add everything up in the tensor core's accumulators, in a fixed order.
//
// Roles (as in the forward): warps 0-3 and 4-7 take the columns 0-63 and 64-127 of a step, a
// thread per row; warps 8 and 9 issue the tcgen05.mma (one thread each), warp 10 the TMA
// loads, warp 11 zeroes rows of y behind the sequence.  (16 warps of 32 columns were no
// faster: 694 us against 690.)  Order of the products, so that the threads' work on one is
// hidden behind the next ones:
//     dk, dv:  dv(i)  S(i+1)  |  dk(i)  dP(i+1)
//     dq:      S(i+1)  |  dq(i)  dP(i+1)
// x goes to tensor memory too where there is room (for dq, and at head_dim 64): a product
// reads 64 bytes of shared memory a cycle then instead of 128, all there are.
//
// Bound at head_dim 128 by the tensor core: 2048 (dk, dv) and 1536 (dq) cycles a step.  Two
// sequences of 4096 tokens, 32 / 8 heads: not causal 1131 us, causal 612 with the same inputs
// again and again (637 to 661 with inputs that alternate); the seven products
// run at 1700 TFLOP/s and 1570, and the same kernel without exponentials, conversions and
// reads of the statistics was 2 % faster.  At 64 by the chain from one product over the rows'
// threads to the next (2100 and 1700 cycles a step, 1230 and 870 of them products; causal 490
// us): P and dS in columns of their own, which frees S and dP earlier, took 555, and two CTAs
// a multiprocessor with steps of 64 rows 503, with ragged windows a third more.  A CTA takes
// about 9000 cycles besides its steps: up to the first scores 5500, the output 3000.  Where a
// tile has few steps a CTA takes several heads of it in rounds: the next round's x goes to its
// place, and its first products run, before the last one's output.

struct BwdBarriers {
  uint64_t full[8], empty[8], s_full, p_full[2], dp_full, ds_full[2], x_full[2], x_ready[2], acc_full;
  uint64_t turn[2], stat_full[2], stat_empty[2], cut[2], zeroed[2];
  uint32_t tmem;
  // What the rows' threads need between the steps and would hold in registers during them.
  struct {
    SeqRange range;
    int sequence, head0, rounds, x0, rows;
  } kept;
  uint32_t again[8][4];  // by warp of the rows: those with a NaN, a word a round
};

template <int DP, bool KV>
struct BwdShape {
  static constexpr int kPanel = kBwdTile * 128;  // bytes of [128][64] 16-bit elements
  static constexpr int kPanels = DP / 64;
  static constexpr int kSlot = kPanels * kPanel;
  // x goes to tensor memory where it has room (columns: S, dP 256, results 128 or 256).
  static constexpr bool kXInTmem = !KV || DP == 64;
  // y1 and y2 alternate in a ring of slots; behind it x1 and x2, which become slots of it too
  // once they are in tensor memory (at 128; dq's loads were late with 5 slots).
  static constexpr int kFirst = DP == 128 ? 5 : 8;
  static constexpr int kSlots = DP == 128 && kXInTmem ? kFirst + 2 : kFirst;
  static constexpr int kStats = (kFirst + 2) * kSlot;  // then -lse and -delta, two stages
  static constexpr int kStat = kBwdTile * 4;
  static_assert(kSlots <= 8, "");
  static constexpr int kThreads = 384;
  // 256 x softmax + 128 x other = threads x launch, exactly.
  static constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
  static_assert(256 * kRegsSoftmax + 128 * kRegsOther == kThreads * kRegsLaunch, "");
};
constexpr int kPass = 4;  // instructions before its end that a turn passes (2 and 8: 1 % slower)
template <int DP>
struct BwdShared {
  static constexpr int kBody = BwdShape<DP, true>::kStats + 4 * BwdShape<DP, true>::kStat;
  static constexpr int kSmem = kBody + (int)sizeof(BwdBarriers);
  static_assert(kSmem <= 232448, "");
};
constexpr int kBwdMmaWarp = 8, kBwdMmaWarp2 = 9, kBwdLoadWarp = 10, kBwdZeroWarp = 11;

// The largest of `n` numbers from `at` on, in `rows` rows `stride` apart (by a whole warp).
__device__ __forceinline__ float warp_largest(const float* at, int64_t stride, int rows, int n) {
  float most = 0.f;
  for (int r = 0; r < rows; ++r)
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < n; i += 32) most = fmax_nan(most, at[r * stride + i]);
  return warp_max_nan(most);
}

// What f16 ds is taken larger by: a power of two u with 2^14 <= u M < 2^15, M the largest |dout_i|
// of this CTA's queries times the largest |v_j| of the sequence.  delta is the mean of dp over
// all keys of the row, so dp - delta is 1 - p times a difference of two that are within M, and
// |ds| <= 2 M p (1 - p) <= M / 2: u |ds| stays below 2^14, a quarter of f16's range, which leaves
// what p's and delta's rounding adds (2^-11 of M, and p relative) its room.  (With the values of a
// tile's own keys alone, small ones among larger, delta passes the bound and ds is infinite.)
// Its bits end at 2^-14 / u <= 2^-28 M, half a step there is 2^-25 / u <= 2^-39 M.  ds falls with the
// number of keys and f16 ends early: without u, gradients of long sequences would be sums of
// numbers without bits.
template <typename T, bool KV>
__device__ __forceinline__ float ds_factor(const AttnBwdParams& p, const SeqRange& s, int b, int xh, int h,
                                           int x0, int rows) {
  if constexpr (Elem<T>::kDt != DT_F16) return 1.f;
  auto runs = [](int n) { return (n + kStatTokens - 1) / kStatTokens; };
  const float* q = p.q_norms + (KV ? h * p.group : xh) * p.q_norm_stride + norm_base(s.q0, b);
  const float* v = p.v_norms + h * p.v_norm_stride + norm_base(s.k0, b);
  const float mq = KV ? warp_largest(q, p.q_norm_stride, p.group, runs(s.qlen))
                      : warp_largest(q + x0 / kStatTokens, 0, 1, runs(rows));
  const float mv = warp_largest(v, 0, 1, runs(s.kv));
  const float most = sqrtf(mq) * sqrtf(mv);
  if (!(most > 0.f) || !(most < INFINITY)) return 1.f;
  const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100), 100);
  return __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
}

// Until the kernel before has completed.  Every CTA gets here before it ends, so that what comes
// after this kernel comes after the statistics too.
__device__ __forceinline__ void wait_for_stats() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The rows of a warp's gradients that have a NaN, when its outputs are written: no other role waits
// then, and what this needs in registers costs the steps nothing.
template <typename T, bool KV>
__device__ __noinline__ void tile_again(const AttnBwdParams& p, const BwdBarriers& bars) {
  const auto kept = bars.kept;
  const int warp = threadIdx.x >> 5, w = warp >> 2, half = p.d <= 64 ? 32 : 64;
  for (int round = 0; round < kept.rounds; ++round) {
    const int xh = kept.head0 + round;
    for (uint32_t todo = bars.again[warp][round]; todo; todo &= todo - 1) {
      const int x = kept.x0 + (warp & 3) * 32 + __ffs(todo) - 1;
      const int64_t row = (KV ? kept.range.k0 : kept.range.q0) + static_cast<int64_t>(x);
      if constexpr (!KV)
        grad_again<T, 0>(p, kept.range, kept.sequence, xh, xh / p.group, x, w * half, half,
                         static_cast<T*>(p.dq) + row * p.dqt + xh * p.dqh);
      else if (w == 0)
        grad_again<T, 2>(p, kept.range, kept.sequence, 0, xh, x, 0, p.d, static_cast<T*>(p.dv) + row * p.dvt + xh * p.dvh);
      else
        grad_again<T, 1>(p, kept.range, kept.sequence, 0, xh, x, 0, p.d, static_cast<T*>(p.dk) + row * p.dkt + xh * p.dkh);
    }
  }
}

// SEVERAL: a CTA may take several heads of its tile one after another, in rounds (a kernel of its
// own: with one round the code for more costs 3 to 6 % of a call).
template <typename T, int DP, bool KV, bool SEVERAL>
__device__ __forceinline__ void attention_bwd_tile(const AttnBwdParams& p, const CUtensorMap& x1map,
                                                   const CUtensorMap& x2map, const CUtensorMap& y1map,
                                                   const CUtensorMap& y2map, int block, uint8_t* raw) {
  using Shape = BwdShape<DP, KV>;
  constexpr int kType = std::is_same<T, __half>::value ? 0 : 1;
  BwdBarriers& bars = *reinterpret_cast<BwdBarriers*>(raw + BwdShared<DP>::kBody);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The longest work first: sequences by their pairs, causal keys from the first on (the most
  // queries see those), queries from the last.
  const int heads = KV ? p.hkv : p.hq, each = !SEVERAL ? 1 : KV ? p.kv_each : p.q_each;
  const int groups = (heads + each - 1) / each;
  const int xh0 = block % groups * each;        // the first of this CTA's heads,
  const int rounds = SEVERAL ? min(each, heads - xh0) : 1;  // and how many
  block /= groups;
  const int splits = KV ? p.kv_splits : p.q_splits, split = block % splits;
  block /= splits;
  const TilePlace place = KV ? find_tile<Shape::kThreads>(p.cu_k, p.cu, p.batches, p.max_k, p.max_q, 1, kBwdTile,
                                                         block, raw)
                             : find_tile<Shape::kThreads>(p.cu, p.cu_k, p.batches, p.max_q, p.max_k, 1, kBwdTile,
                                                         block, raw);
  if (place.tile < 0) return wait_for_stats();
  const int b = place.sequence, xt = KV ? place.tile : place.tiles - 1 - place.tile;
  const SeqRange s = bwd_range(p, b, false);
  const int nx = KV ? s.kv : s.qlen, ny = KV ? s.qlen : s.kv, x0 = xt * kBwdTile;
  const int rows = min(kBwdTile, nx - x0);
  if (rows <= 0) return wait_for_stats();

  // Rows of y that some row of x goes with, [y_lo, y_hi), in tiles from `base` on; for dk
  // and dv once for every head of the group.
  const int y_lo = KV ? query_first(p, s, x0) : key_first(p, s, x0);
  const int y_hi = KV ? query_end(p, s, x0 + rows - 1) : key_end(p, s, x0 + rows - 1);
  const int base = y_lo & ~(kBwdTile - 1);
  const int nt = y_hi > y_lo ? (y_hi - base + kBwdTile - 1) / kBwdTile : 0;
  // Of these steps (heads of the group times tiles) this CTA takes n from step0 on; with several
  // heads of its own, all of them for each.
  const int steps_all = nt * (KV ? p.group : 1), share = (steps_all + splits - 1) / splits;
  const int step0 = min(split * share, steps_all), n = min(share, steps_all - step0);
  const int t0 = nt > 0 ? step0 % nt : 0, g0 = nt > 0 ? step0 / nt : 0;
  // The last tile reaches beyond the sequence.
  const bool cut_last = base + nt * kBwdTile > ny;

  // A round's x1 and x2 pass through the ring ahead of its y (the first round's have a place of
  // their own) where they go on to tensor memory: the ring's positions a round.
  const int per_round = 2 * n + (Shape::kXInTmem ? 2 : 0);
  const uint32_t ring = smem_u32(raw), xs = ring + Shape::kFirst * Shape::kSlot;
  if (ring & 1023u) {  // the swizzle goes by address bits; the compiler's alignment holds
    if (tid == 0) flag_wait_timeout();
    return wait_for_stats();
  }
  // The warp of the loads sets the barriers up and goes ahead: the first tiles are on their way
  // while the others are still setting up.
  if (warp == kBwdLoadWarp && lane == 0) {
    for (int i = 0; i < Shape::kSlots; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 2);  // one arrival for each of the threads that issue
    }
    mbar_init(&bars.s_full, 1);
    mbar_init(&bars.dp_full, 1);
    mbar_init(&bars.acc_full, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.turn[i], 1);
      mbar_init(&bars.x_full[i], 1);
      mbar_init(&bars.x_ready[i], 4);
      mbar_init(&bars.p_full[i], 8);  // one arrival per warp
      mbar_init(&bars.ds_full[i], 8);
      mbar_init(&bars.cut[i], 1);
      mbar_init(&bars.zeroed[i], 1);
      mbar_init(&bars.stat_full[i], 1);
      mbar_init(&bars.stat_empty[i], 8);
    }
    fence_mbar_init();
  }
  if (tid == 0) {
    bars.kept.range = s;
    bars.kept.sequence = b;
    bars.kept.head0 = xh0;
    bars.kept.rounds = rounds;
    bars.kept.x0 = x0;
    bars.kept.rows = rows;
  }
  if (warp == kBwdMmaWarp) tc_alloc(&bars.tmem);
  uint32_t tmem = 0;
  if (warp == kBwdLoadWarp) {
    __syncwarp();
    asm volatile("barrier.cta.arrive.aligned 1, %0;" ::"n"(Shape::kThreads) : "memory");
  } else {
    tc_fence_before();
    asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(Shape::kThreads) : "memory");
    tc_fence_after();
    tmem = bars.tmem;
  }
  // Columns (S: 0); kX: x as the products' first operand, 16-bit pairs.
  constexpr uint32_t kDp = 128, kAcc2 = 256, kAcc1 = KV ? 256 + DP : 256, kX = 384;
  constexpr bool kXInTmem = Shape::kXInTmem;
  static_assert(kAcc1 + DP <= (kXInTmem ? kX : kTmemCols), "");
  bool ok = true;

  if (warp >= kBwdMmaWarp) {
    set_regs_dec<Shape::kRegsOther>();
    if (warp == kBwdMmaWarp || warp == kBwdMmaWarp2) {
      // ------------------------------------------------ tensor core issue
      constexpr uint32_t kIdXY = instr_desc(kType, kBwdTile, kBwdTile, 0);
      const bool first = warp == kBwdMmaWarp;  // the one of S (and dv), else of dP and acc1
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t x_lo = __shfl_sync(0xFFFFFFFFu, desc_lo(xs + (first ? 0 : Shape::kSlot), 16), 0);
      const uint32_t k_lo = __shfl_sync(0xFFFFFFFFu, desc_lo(ring, 16), 0);
      const uint32_t mn_lo = __shfl_sync(0xFFFFFFFFu, desc_lo(ring, Shape::kPanel), 0);
      const int steps = __shfl_sync(0xFFFFFFFFu, (p.d + 15) / 16, 0);  // of 16 elements of a head
      const uint32_t id_acc = instr_desc(kType, kBwdTile, 16 * steps, 1);
      // The tensor core's queue is short: a thread that waits on a barrier between two
      // products, also on a complete one (100 cycles), leaves it idle.  So two threads issue,
      // and each waits while the other's products run.  They take turns: turn i of the
      // first one is dv(i - 1), S(i), of the second dk or dq(i - 1), dP(i); a turn passes four
      // instructions before its end, so that it arrives in time.
      if (n > 0 && elect_one()) {
        uint64_t* const mine = &bars.turn[first ? 0 : 1];
        uint64_t* const other = &bars.turn[first ? 1 : 0];
        // D = x y^T, x from tensor memory where it has room for it
        auto product = [&](int slot, uint32_t to) {
          const uint32_t y = k_lo + slot * (Shape::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            if (kk >= steps) break;
            if (kk == max(steps - kPass, 0)) mbar_arrive(other);
            const uint32_t at = ((kk / 4) * Shape::kPanel + (kk % 4) * 32) >> 4;
            if constexpr (kXInTmem)
              tc_mma_ts(to, tm + kX + (first ? 0 : DP / 2) + kk * 8, y + at, kDescHi, kIdXY, kk > 0);
            else
              tc_mma_ss(to, x_lo + at, y + at, kDescHi, kIdXY, kk > 0);
          }
        };
        // D += (16-bit pairs in tensor memory) y, in the halves that they come in
        auto add = [&](uint32_t from, int slot, uint32_t to, bool more, bool pass, uint64_t* halves,
                       uint32_t parity) {
          const uint32_t y = mn_lo + slot * (Shape::kSlot >> 4);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            ok = ok && mbar_wait(&halves[hf], parity);
            if (!ok) return;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kk = (e >> 1) * 4 + hf * 2 + (e & 1);
              if (hf == 1 && e == 2 && pass) mbar_arrive(other);
              tc_mma_ts(to, from + (kk >> 2) * 64 + (kk & 3) * 8, y + kk * (2048 >> 4), kDescHi, id_acc,
                        hf + e > 0 ? 1u : static_cast<uint32_t>(more));
            }
          }
        };
        const int own = first ? 0 : 1;  // y1 or y2: what this thread's product reads
        int y1 = 0, y2 = 0, left = nt - t0;  // slots of the step before; tiles up to the sequence's end
        uint32_t zeros = 0, turns = 0, done = 0;  // turns, and steps of the rounds before
        int slot = 0;
        uint32_t phase = 0;
        for (int round = 0; ok && round < rounds; ++round, done += n) {
        ok = mbar_wait(kXInTmem ? &bars.x_ready[own] : &bars.x_full[own], round & 1);
        if (kXInTmem && round > 0) {
          // x1 and x2 have passed through the ring: their slots are free (two arrivals).
          for (int j = 0; j < 2; ++j) {
            if (ok && j == own) mbar_arrive(&bars.empty[slot]), mbar_arrive(&bars.empty[slot]);
            if (++slot == Shape::kSlots) slot = 0, phase ^= 1;
          }
        }
        for (int i = 0; ok && i <= n; ++i) {
          // Everything this turn needs, then the turn.
          int z1 = slot, z2 = slot;
          uint32_t ph1 = phase, ph2 = phase;
          if (++slot == Shape::kSlots) slot = 0, phase ^= 1;
          z2 = slot, ph2 = phase;
          if (++slot == Shape::kSlots) slot = 0, phase ^= 1;
          if (i == n) {
            slot = z1, phase = ph1;  // (looked at, not taken)
          } else {
            ok = mbar_wait(&bars.full[own ? z2 : z1], own ? ph2 : ph1);
            // Rows behind the sequence zeroed (a weight of 0 times what stands there must be
            // 0; v is never weighed for dq).
            if (--left == 0) {
              left = nt;
              if (ok && cut_last && (KV || first)) {
                mbar_arrive(&bars.cut[own]);
                ok = mbar_wait(&bars.zeroed[own], zeros++ & 1);
              }
            }
          }
          const uint32_t last = (done + i - 1) & 1;  // parity of the step before
          if (!KV && first && i > 0) ok = ok && mbar_wait(&bars.p_full[0], last);  // S has been read
          // (the second thread's turns follow the first one's)
          if (!first || turns > 0) ok = ok && mbar_wait(mine, (first ? turns - 1 : turns) & 1);
          ++turns;
          if (!ok) break;
          tc_fence_after();
          if (i > 0) {
            if (first) {
              if constexpr (KV) {
                add(tm, y2, tm + kAcc2, i > 1, i == n, bars.p_full, last);
                if (!ok) break;
                tc_commit(&bars.empty[y2]);
              } else if (i == n) {
                mbar_arrive(other);
              }
            } else {
              add(tm + kDp, y1, tm + kAcc1, i > 1, i == n, bars.ds_full, last);
              if (!ok) break;
              tc_commit(&bars.empty[y1]);
            }
          }
          if (i < n) {
            product(first ? z1 : z2, tm + (first ? 0 : kDp));
            tc_commit(first ? &bars.s_full : &bars.dp_full);
            tc_commit(&bars.empty[first ? z1 : z2]);
            if (!KV && !first) tc_commit(&bars.empty[z2]);  // (two arrivals a use of a slot)
            y1 = z1, y2 = z2;
          }
        }
        if (ok) tc_commit(&bars.acc_full);
        }
        if (ok) {
          // The last arrivals have landed before the CTA ends.
          const int end = (rounds - 1) * per_round + 2 * n;
          ok = mbar_wait(&bars.empty[y1], ((end - 2) / Shape::kSlots) & 1) &&
               mbar_wait(&bars.empty[y2], ((end - 1) / Shape::kSlots) & 1);
          if (first) ok = ok && mbar_wait(mine, (turns - 1) & 1);
        }
      }
      __syncwarp();
    } else if (warp == kBwdLoadWarp) {
      // ------------------------------------------------ TMA loads
      if (lane == 0 && n > 0) {
        auto tile = [&](uint32_t dst, const CUtensorMap* map, int head, int row, uint64_t* bar) {
#pragma unroll
          for (int pn = 0; pn < Shape::kPanels; ++pn)
            tma_box(dst + pn * Shape::kPanel, map, pn * 64, head, row, 0, bar);
        };
        const int xr = (KV ? s.k0 : s.q0) + x0;
        const int64_t stat = stat_base(s.q0, b) + base;
        int slot = 0, issued = 0, step = 0;
        uint32_t phase = 0;
        bool x_placed = false;  // the first round's x has left its place
        // The next slot of the ring, when it is free.
        auto fill = [&](const CUtensorMap* map, int head, int row) {
          if (issued >= Shape::kSlots) ok = mbar_wait(&bars.empty[slot], phase ^ 1);
          else if (issued >= Shape::kFirst && !x_placed)  // (only where x's room is used)
            ok = mbar_wait(&bars.x_ready[issued - Shape::kFirst], 0);
          if (!ok) return;
          mbar_arrive_expect_tx(&bars.full[slot], Shape::kSlot);
          tile(ring + slot * Shape::kSlot, map, head, row, &bars.full[slot]);
          ++issued;
          if (++slot == Shape::kSlots) slot = 0, phase ^= 1;
        };
        auto fill_x = [&](int which, int head) {  // x's own place
          mbar_arrive_expect_tx(&bars.x_full[which], Shape::kSlot);
          tile(xs + which * Shape::kSlot, which ? &x2map : &x1map, head, xr, &bars.x_full[which]);
        };
        for (int round = 0; ok && round < rounds; ++round) {
          const int xh = xh0 + round, h = KV ? xh : xh / p.group;
          if (kXInTmem && round > 0) {
            // (x_ready stays in its second phase until the second round's x is here)
            for (int j = 0; ok && !x_placed && j < 2; ++j) ok = mbar_wait(&bars.x_ready[j], 0);
            x_placed = true;
            if (ok) fill(&x1map, xh, xr);
            if (ok) fill(&x2map, xh, xr);
          }
          int t = t0, g = g0;
          for (int i = 0; ok && i < n; ++i, ++step) {
            const int yr = (KV ? s.q0 : s.k0) + base + t * kBwdTile;
            const int yh = KV ? h * p.group + g : h;
            for (int w = 0; ok && w < 2; ++w) {
              if (round == 0 && i == 0) fill_x(w, xh);  // x1 just ahead of the first y1, x2 of the first y2
              fill(w ? &y2map : &y1map, yh, yr);
              if (ok && KV && w == 0) {
                if (step == 0) wait_for_stats();
                const int st = step & 1;
                if (step >= 2) ok = mbar_wait(&bars.stat_empty[st], ((step >> 1) - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.stat_full[st], 2 * Shape::kStat);
                uint8_t* dst = raw + Shape::kStats + st * 2 * Shape::kStat;
                const int64_t from = yh * p.stat_stride + stat + t * kBwdTile;
                bulk_g2s(dst, p.nlse + from, Shape::kStat, &bars.stat_full[st]);
                bulk_g2s(dst + Shape::kStat, p.ndelta + from, Shape::kStat, &bars.stat_full[st]);
              }
            }
            if (!kXInTmem && ok && round > 0 && i == 0) {
              // x's place is free when the round before has multiplied everything.
              ok = mbar_wait(&bars.acc_full, (round - 1) & 1);
              for (int w = 0; ok && w < 2; ++w) fill_x(w, xh);
            }
            if (++t == nt) t = 0, ++g;
          }
        }
        if (!ok) {
          // Leave no copy in flight behind.
          for (int j = max(0, issued - Shape::kSlots); j < issued; ++j)
            mbar_wait(&bars.full[j % Shape::kSlots], (j / Shape::kSlots) & 1);
          if (KV)
            for (int j = max(0, step - 2); j < step; ++j) mbar_wait(&bars.stat_full[j & 1], (j >> 1) & 1);
          const uint64_t t0 = globaltimer_ns();  // (and x's, whose phase is the rows' to know)
          while (globaltimer_ns() - t0 < 1000000ull) {}
        }
      }
      __syncwarp();
    } else if (warp == kBwdZeroWarp && cut_last) {
      // ------------------------------------------------ rows of y behind the sequence
      const int ends = nt > 0 ? (step0 + n) / nt - g0 : 0;  // of the sequence among the steps
      const int events = KV ? 2 * ends : ends;
      const int from = ny - (base + (nt - 1) * kBwdTile);  // first row to zero of the last tile
      for (int e = 0; ok && e < events * rounds; ++e) {
        // (a whole range may lie before the last tile's turn: a longer limit)
        const int own = KV ? e & 1 : 0, use = KV ? e >> 1 : e;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_for(&bars.cut[own], use & 1, 30 * kWaitLimitNs));
        if (!ok) break;
        const int round = e / events, head = KV ? e % events >> 1 : e % events;
        const int64_t tile = static_cast<int64_t>(round) * per_round +
                             2 * (static_cast<int64_t>(g0 + head + 1) * nt - 1 - step0) + (KV ? e & 1 : 0);
        uint8_t* at = raw + static_cast<int>(tile % Shape::kSlots) * Shape::kSlot;
        for (int j = lane; j < (kBwdTile - from) * 8 * Shape::kPanels; j += 32)
          *reinterpret_cast<uint4*>(at + (j >> 3) % Shape::kPanels * Shape::kPanel +
                                    (from + (j >> 3) / Shape::kPanels) * 128 + (j & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.zeroed[own]);
      }
    }
  } else {
    // -------------------------------------------------- probabilities and their gradients
    set_regs_inc<Shape::kRegsSoftmax>();
    if (lane < 4) bars.again[warp][lane] = 0u;
    __syncwarp();
    const int w = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    int lo = 0, hi = 0;  // the rows of y that this thread's row goes with
    if (r < rows) {
      lo = KV ? query_first(p, s, x0 + r) : key_first(p, s, x0 + r);
      hi = KV ? query_end(p, s, x0 + r) : key_end(p, s, x0 + r);
    }
    const uint64_t sc2 = p2(p.scale_log2, p.scale_log2);
    constexpr float back = 1.f / static_cast<float>(1 << kWeightLog2<T>);  // P is 2^kWeightLog2 larger
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + w * 64;  // this warp's half of S
    // What a round takes from memory, under way before the waits for x and during the output of
    // the round before.
    float up = 1.f, nl = 0.f, nd = 0.f;  // nl, nd: dq's row's own
    // A round's steps, and after them its output, beside which the next round's first products run.
    auto between = [&](auto is_first, const int round) {  // true: another round
      constexpr bool kFirstRound = decltype(is_first)::value;
      // (everything from here to the steps anew each time: what the compiler would keep from one
      // round to the next costs registers, and the steps then time: 2000 cycles against 1760)
      int me;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(me));
      const int lane = me & 31, warp = me >> 5, w = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16, tmem = *const_cast<volatile uint32_t*>(&bars.tmem);
      const volatile auto& kept = bars.kept;
      const SeqRange s = {kept.range.q0, kept.range.qlen, kept.range.kv, kept.range.off, kept.range.k0};
      const int b = kept.sequence, xh0 = kept.head0, x = kept.x0 + r;
      const bool live = r < kept.rows;
      const bool more = kFirstRound || (SEVERAL && round < kept.rounds);
      if (!KV || kType == 0 || n == 0 || !kFirstRound) wait_for_stats();
      if (!kFirstRound && n > 0) {
        ok = warp_wait(&bars.acc_full, (round - 1) & 1);
        tc_fence_after();
      }
      const float down = p.scale / up;  // of the last round's dk or dq
      if (more) {
        const int xh = xh0 + round;
        if (!KV && live) {
          const int64_t at = xh * p.stat_stride + stat_base(s.q0, b) + x;
          nl = p.nlse[at];
          nd = p.ndelta[at];
        }
        up = ds_factor<T, KV>(p, s, b, xh, KV ? xh : xh / p.group, x - r, kept.rows);
        if (kXInTmem && n > 0) {
          // x1 (warps 0-3) or x2 into tensor memory, a row by a thread.
          const int at = round * per_round - 2 + w, slot = kFirstRound ? Shape::kFirst + w : at % Shape::kSlots;
          ok = ok && (kFirstRound ? warp_wait(&bars.x_full[w], 0)
                                  : warp_wait(&bars.full[slot], (at / Shape::kSlots) & 1));
          if (ok) {
            const uint8_t* from = raw + slot * Shape::kSlot + r * 128;
#pragma unroll
            for (int pn = 0; pn < Shape::kPanels; ++pn) {
              uint32_t v[32];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint4 q =
                    *reinterpret_cast<const uint4*>(from + pn * Shape::kPanel + ((c ^ (r & 7)) << 4));
                v[4 * c] = q.x, v[4 * c + 1] = q.y, v[4 * c + 2] = q.z, v[4 * c + 3] = q.w;
              }
              tc_st32(tmem + lanes + kX + w * (DP / 2) + pn * 32, v);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.x_ready[w]);
          }
        }
      }
      // Output: dv by the warps 0-3, dk by 4-7; or half of dq's columns by each.
      if (!kFirstRound && ok) {
        const int xh = xh0 + round - 1;
        constexpr int kCols = KV ? DP : DP / 2;
        const int col0 = KV ? 0 : w * kCols;
        const uint32_t from = tmem + lanes + (KV && w == 0 ? kAcc2 : kAcc1 + col0);
        const float factor = KV && w == 0 ? back : down;
        T* const dst = static_cast<T*>(KV ? (w == 0 ? p.dv : p.dk) : p.dq);
        const int64_t row = (KV ? s.k0 : s.q0) + static_cast<int64_t>(x);
        const int64_t at = KV ? (w == 0 ? row * p.dvt + xh * p.dvh : row * p.dkt + xh * p.dkh)
                              : row * p.dqt + xh * p.dqh;
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, live);
        bool nan = false;
        // Through shared memory, so that a store writes whole sectors, where the ring is used up; a
        // lane to a row otherwise.
        uint8_t* const stage = raw + warp * 32 * 64;
#pragma unroll 1
        for (int c = 0; c < kCols && col0 + c < p.d; c += 32) {
          uint32_t o[32];
          if (n > 0) {
            tc_ld32(from + c, o);
            tc_wait_ld<32>(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (splits > 1) {
            // A part of a sum: 32-bit, put together by attention_join_kernel.
            float* const part =
                KV ? p.kv_part + (((static_cast<int64_t>(split) * 2 + (w == 0)) * p.keys + row) * p.hkv + xh) * p.d
                   : p.q_part + ((static_cast<int64_t>(split) * p.tokens + row) * p.hq + xh) * p.d;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (live && col0 + c + e < p.d)
                *reinterpret_cast<float4*>(part + col0 + c + e) =
                    make_float4(__uint_as_float(o[e]) * factor, __uint_as_float(o[e + 1]) * factor,
                                __uint_as_float(o[e + 2]) * factor, __uint_as_float(o[e + 3]) * factor);
            continue;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float f = __uint_as_float(o[e]);
#pragma unroll
            for (int q = 1; q < 7; q += 2)
              f = max3_nan(f, __uint_as_float(o[e + q]), __uint_as_float(o[e + q + 1]));
            f = max3_nan(f, f, __uint_as_float(o[e + 7]));
            nan |= f != f;
          }
          auto put = [&](int e, const uint32_t* v) {
            if (more) {
              if (live && col0 + c + 8 * e < p.d)
                *reinterpret_cast<uint4*>(dst + at + col0 + c + 8 * e) = make_uint4(v[0], v[1], v[2], v[3]);
              return;
            }
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          };
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[q] = narrow2<T>(mul2(p2(__uint_as_float(o[8 * e + 2 * q]), __uint_as_float(o[8 * e + 2 * q + 1])),
                                     p2(factor, factor)));
            put(e, v);
          }
          __syncwarp();
          if (more) continue;
          const int e = lane & 3;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int rr = q * 8 + (lane >> 2);
            const int64_t to = __shfl_sync(0xFFFFFFFFu, at, rr);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((e ^ ((rr >> 1) & 3)) << 4));
            if (((some >> rr) & 1) && col0 + c + 8 * e < p.d)
              *reinterpret_cast<uint4*>(dst + to + col0 + c + 8 * e) = v;
          }
          __syncwarp();
        }
        if (more) tc_fence_before();  // (read before the next round's sums)
        const uint32_t again = __ballot_sync(0xFFFFFFFFu, nan && live);
        if (again != 0u && lane == 0) bars.again[warp][round - 1] = again;
      }
      return more;
    };
    auto steps_of = [&](const int round) {
      const uint32_t done = static_cast<uint32_t>(round) * n;  // steps of the rounds before
      const uint64_t up2 = p2(up * back, up * back), nl2 = p2(nl, nl), nd2 = p2(nd, nd);
      int t = t0;
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t step = done + i;
        const ulonglong2* stat =
            reinterpret_cast<const ulonglong2*>(raw + Shape::kStats + (step & 1) * 2 * Shape::kStat + w * 256);
        if (KV) ok = warp_wait(&bars.stat_full[step & 1], (step >> 1) & 1);
        ok = ok && warp_wait(&bars.s_full, step & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t sc[64];
        tc_ld32(ts, sc);
        tc_ld32(ts + 32, sc + 32);
        tc_wait_ld<64>(sc);
        if constexpr (!KV) {  // S is free again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_full[0]);
        }
        const int tb = base + t * kBwdTile + w * 64;
        if (++t == nt) t = 0;
        const bool cut = __any_sync(0xFFFFFFFFu, tb < lo || tb + 64 > hi);
        // Bit e: row tb + e of y is kept.
        const uint64_t kept = low_bits(hi - tb) & ~low_bits(lo - tb);
        const uint32_t half_kept[2] = {static_cast<uint32_t>(kept), static_cast<uint32_t>(kept >> 32)};
        uint64_t pr[32];
        // In halves of 32 columns: the tensor core begins with the first one.
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int e = hf * 16; e < hf * 16 + 16; e += 2) {
            ulonglong2 nl = make_ulonglong2(nl2, nl2);
            if (KV) nl = stat[e / 2];
            const float2 a =
                u2(fma2(p2(__uint_as_float(sc[2 * e]), __uint_as_float(sc[2 * e + 1])), sc2, nl.x));
            const float2 c =
                u2(fma2(p2(__uint_as_float(sc[2 * e + 2]), __uint_as_float(sc[2 * e + 3])), sc2, nl.y));
            pr[e] = p2(ex2(a.x), ex2(a.y));
            pr[e + 1] = p2(ex2(c.x), ex2(c.y));
          }
          if (cut) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t bits = half_kept[hf] >> (2 * e);
              const float2 a = u2(pr[hf * 16 + e]);
              pr[hf * 16 + e] = p2(bits & 1u ? a.x : 0.f, bits & 2u ? a.y : 0.f);
            }
          }
          if constexpr (KV) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = narrow2<T>(pr[hf * 16 + e]);
            tc_st16(ts + hf * 16, pk);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_full[hf]);
          }
        }
        ok = warp_wait(&bars.dp_full, step & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t td = ts + kDp;
        tc_ld32(td, sc);
        tc_ld32(td + 32, sc + 32);
        tc_wait_ld<64>(sc);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
#pragma unroll
          for (int e = hf * 16; e < hf * 16 + 16; e += 2) {
            ulonglong2 nd = make_ulonglong2(nd2, nd2);
            if (KV) nd = stat[Shape::kStat / 16 + e / 2];
            uint64_t a = add2(p2(__uint_as_float(sc[2 * e]), __uint_as_float(sc[2 * e + 1])), nd.x);
            uint64_t c = add2(p2(__uint_as_float(sc[2 * e + 2]), __uint_as_float(sc[2 * e + 3])), nd.y);
            if constexpr (kType == 0) {
              a = mul2(a, up2);
              c = mul2(c, up2);
            }
            pk[e - hf * 16] = narrow2<T>(mul2(a, pr[e]));
            pk[e - hf * 16 + 1] = narrow2<T>(mul2(c, pr[e + 1]));
          }
          if (cut) {
            // (0 times an infinity or NaN of a pair that is not kept)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t bits = half_kept[hf] >> (2 * e);
              pk[e] &= (bits & 1u ? 0xFFFFu : 0u) | (bits & 2u ? 0xFFFF0000u : 0u);
            }
          }
          tc_st16(td + hf * 16, pk);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.ds_full[hf]);
            if (KV && hf == 1) mbar_arrive(&bars.stat_empty[step & 1]);
          }
        }
      }
    };
    // (the first round apart: in one loop for all of them the compiler spends registers, and a step
    // time, on what only some rounds do: 5 % of a call with one)
    between(std::true_type(), 0);
    if (ok) steps_of(0);
#pragma unroll 1
    for (int round = 1; ok && between(std::false_type(), round) && ok; ++round) steps_of(round);
    if (splits == 1) {
      __syncwarp();
      const uint32_t* const again = bars.again[warp];
      if ((again[0] | again[1] | again[2] | again[3]) != 0u) tile_again<T, KV>(p, bars);
    }
  }

  if (!ok) flag_wait_timeout();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kBwdMmaWarp) tc_dealloc(tmem);
}

// One launch for all gradients: dk and dv's CTAs first, dq's into the room that they leave.
template <typename T, int DP, bool KV_SEVERAL, bool Q_SEVERAL>
__global__ void __launch_bounds__(BwdShape<DP, true>::kThreads, 1)
    attention_bwd_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ CUtensorMap q,
                         const __grid_constant__ CUtensorMap k, const __grid_constant__ CUtensorMap v,
                         const __grid_constant__ CUtensorMap dout) {
  extern __shared__ __align__(1024) uint8_t raw[];
  // The statistics are waited for where they are read (see wait_for_stats).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int block = blockIdx.x;
  if (block < p.kv_blocks) attention_bwd_tile<T, DP, true, KV_SEVERAL>(p, k, v, q, dout, block, raw);
  else attention_bwd_tile<T, DP, false, Q_SEVERAL>(p, q, dout, k, v, block - p.kv_blocks, raw);
}

template <typename T, int DP, bool KV_SEVERAL, bool Q_SEVERAL>
cudaError_t launch_tiles(const AttnBwdParams& p, const CUtensorMap* m, int64_t grid, cudaStream_t st) {
  auto k = attention_bwd_kernel<T, DP, KV_SEVERAL, Q_SEVERAL>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k, BwdShared<DP>::kSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 g(static_cast<unsigned>(grid)), t(BwdShape<DP, true>::kThreads);
  // (without statistics before it, it must not begin before what comes before has ended)
  if (p.stat_blocks == 0) {
    k<<<g, t, BwdShared<DP>::kSmem, st>>>(p, m[0], m[1], m[2], m[3]);
    return cudaGetLastError();
  }
  return launch_pdl(k, g, t, BwdShared<DP>::kSmem, st, p, m[0], m[1], m[2], m[3]);
}

template <typename T, int DP>
cudaError_t launch_dim(const AttnBwdParams& p, const CUtensorMap* m, int64_t grid, cudaStream_t st) {
  return p.kv_each > 1  ? launch_tiles<T, DP, true, true>(p, m, grid, st)
         : p.q_each > 1 ? launch_tiles<T, DP, false, true>(p, m, grid, st)
                        : launch_tiles<T, DP, false, false>(p, m, grid, st);
}

// ---- sums in parts
//
// Few CTAs with many steps each (few heads that share their keys, one sequence) leave most
// of the GPU idle: the steps of a tile go to several CTAs then, which write 32-bit parts,
// and this kernel adds those up in order.  A thread takes eight columns of a row; rows with a NaN
// are looked at again (grad_again).
template <typename T, int WHICH>
__device__ __forceinline__ void join_rows(const AttnBwdParams& p, int block) {
  const TilePlace place =
      WHICH ? find_tile<kStatThreads, false>(p.cu_k, nullptr, p.batches, p.max_k, 0, 1, kStatTokens, block, nullptr)
            : find_tile<kStatThreads, false>(p.cu, nullptr, p.batches, p.max_q, 0, 1, kStatTokens, block, nullptr);
  if (place.tile < 0) return;
  const int b = place.sequence, x0 = place.tile * kStatTokens;
  const SeqRange s = bwd_range(p, b, false);
  const int heads = WHICH ? p.hkv : p.hq, chunks = p.d / 8, splits = WHICH ? p.kv_splits : p.q_splits;
  const int rows = min(kStatTokens, (WHICH ? s.kv : s.qlen) - x0);
  const int64_t step = (WHICH ? 2 * static_cast<int64_t>(p.keys) * p.hkv : static_cast<int64_t>(p.tokens) * p.hq) * p.d;
  T* const dst = static_cast<T*>(WHICH == 0 ? p.dq : WHICH == 1 ? p.dk : p.dv);
  auto place_of = [&](int x, int head) {  // a row's in the output
    const int64_t row = (WHICH ? s.k0 : s.q0) + static_cast<int64_t>(x);
    return WHICH == 0 ? row * p.dqt + head * p.dqh : WHICH == 1 ? row * p.dkt + head * p.dkh : row * p.dvt + head * p.dvh;
  };
  bool nan = false;
  for (int r = threadIdx.x; r < rows * heads * chunks; r += kStatThreads) {
    const int col = r % chunks * 8, head = r / chunks % heads, x = x0 + r / chunks / heads;
    const int64_t row = (WHICH ? s.k0 : s.q0) + static_cast<int64_t>(x);
    const float* part = WHICH ? p.kv_part + (((WHICH == 1 ? 0 : 1) * static_cast<int64_t>(p.keys) + row) * p.hkv + head) * p.d + col
                              : p.q_part + (row * p.hq + head) * p.d + col;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < splits; ++i, part += step) {
      const float4 a = *reinterpret_cast<const float4*>(part), c = *reinterpret_cast<const float4*>(part + 4);
      f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
      f[4] += c.x, f[5] += c.y, f[6] += c.z, f[7] += c.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) nan |= f[e] != f[e];
    uint32_t v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = narrow2<T>(p2(f[2 * q], f[2 * q + 1]));
    *reinterpret_cast<uint4*>(dst + place_of(x, head) + col) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  if (!__syncthreads_or(nan)) return;
  for (int r = threadIdx.x >> 5; r < rows * heads; r += kStatThreads / 32) {
    const int head = r % heads, x = x0 + r / heads;
    grad_again<T, WHICH>(p, s, b, head, WHICH ? head : head / p.group, x, 0, p.d, dst + place_of(x, head));
  }
}
template <typename T>
__global__ void __launch_bounds__(kStatThreads, 2) attention_join_kernel(const AttnBwdParams p) {
  pdl_begin();
  const int block = blockIdx.x;
  if (block >= p.kv_join_blocks) {
    join_rows<T, 0>(p, block - p.kv_join_blocks);
  } else {
    join_rows<T, 1>(p, block);
    join_rows<T, 2>(p, block);
  }
}

template <typename T>
cudaError_t launch_bwd(const AttnBwdParams& p, cudaStream_t st) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  cudaError_t e = cudaSuccess;
  if (p.stat_blocks > 0) {
    const dim3 g(static_cast<unsigned>(p.stat_blocks), (p.hq + kStatHeads - 1) / kStatHeads);
    e = p.d <= 64 ? launch_pdl(attention_stats_kernel<T, 8>, g, dim3(kStatThreads), 0, st, p)
                  : launch_pdl(attention_stats_kernel<T, 16>, g, dim3(kStatThreads), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  CUtensorMap m[4] = {};
  if (!make_packed_map(&m[0], p.q, kBf16, p.d, p.hq, p.tokens, p.qt, p.qh, kBwdTile) ||
      !make_packed_map(&m[1], p.k, kBf16, p.d, p.hkv, p.keys, p.kt, p.kh, kBwdTile) ||
      !make_packed_map(&m[2], p.v, kBf16, p.d, p.hkv, p.keys, p.vt, p.vh, kBwdTile) ||
      !make_packed_map(&m[3], p.dout, kBf16, p.d, p.hq, p.tokens, p.gt, p.gh, kBwdTile))
    return cudaErrorInvalidValue;
  const int64_t grid = p.kv_blocks + p.q_blocks;
  if (grid == 0) return cudaSuccess;
  e = p.d <= 64 ? launch_dim<T, 64>(p, m, grid, st) : launch_dim<T, 128>(p, m, grid, st);
  if (e != cudaSuccess || p.join_blocks == 0) return e;
  return launch_pdl(attention_join_kernel<T>, dim3(static_cast<unsigned>(p.join_blocks)), dim3(kStatThreads), 0,
                    st, p);
}

}  // namespace
}  // namespace gbn
