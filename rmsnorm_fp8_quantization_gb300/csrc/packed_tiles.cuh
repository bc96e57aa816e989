// Which tile of which sequence a CTA takes, where sequences of different lengths are packed.
#pragma once

#include <cstdint>

#include "tensor_core.cuh"

namespace gbn {

// A CTA's tile of a sequence of packed rows (len x mult of them, tiles of `of`).  Sequences
// differ in length, and tiles x sequences CTAs would mostly be empty ones: so there are as
// many as there can be tiles (tile_blocks), and each looks its own up.
struct TilePlace {
  int sequence, tile, tiles;  // tile < 0: none; tiles: of the sequence
};
constexpr int kSortSequences = 256;  // up to so many sequences can be taken by length

inline int64_t tiles(int64_t n, int64_t of) { return (n + of - 1) / of; }
inline int64_t tile_blocks(const int32_t* cu, int64_t rows, int64_t sequences, int64_t most, int64_t of,
                           int64_t mult = 1, bool sort = true) {
  const int64_t all = tiles(most * mult, of) * sequences, some = rows * mult / of + sequences;
  return !cu || (sort && sequences <= kSortSequences && all < some) ? all : some;
}

// By the whole CTA.  SORT and up to kSortSequences sequences: those with the most pairs (rows
// times the other side's) first.  `scratch`: then 2048 bytes of shared memory, used up on return.
template <int THREADS, bool SORT = true>
__device__ __forceinline__ TilePlace find_tile(const int32_t* cu, const int32_t* cu_other, int n, int most,
                                               int most_other, int mult, int of, int index,
                                               uint8_t* scratch) {
  auto tiles_of = [&](int64_t len) {
    return static_cast<int>((min(max(len, int64_t(0)), static_cast<int64_t>(most)) * mult + of - 1) / of);
  };
  if (!cu) {
    const int per = tiles_of(most);
    return {index / per, index % per, per};
  }
  auto length = [&](int i) { return static_cast<int64_t>(cu[i + 1]) - cu[i]; };
  const int tid = threadIdx.x;
  if (n == 1) {
    const int t = tiles_of(length(0));
    return {0, index < t ? index : -1, t};
  }
  if (!SORT || n > kSortSequences) {
    // Sequence b's tiles begin at cu[b] mult / of + b, at least its tiles before the next one's:
    // the last that begins at or before `index`, 32 probes at a time.
    const int lane = tid & 31;
    int lo = 0, hi = n;  // it lies in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5;
      const int at = lo + lane * step;
      const bool before = at < hi && static_cast<int64_t>(cu[at]) * mult / of + at <= index;
      const int c = 31 - __clz(__ballot_sync(0xFFFFFFFFu, before) | 1u);
      lo += c * step;
      hi = min(hi, lo + step);
    }
    const int64_t tile = index - (static_cast<int64_t>(cu[lo]) * mult / of + lo);
    const int t = tiles_of(length(lo));
    return {lo, tile >= 0 && tile < t ? static_cast<int>(tile) : -1, t};
  }
  if (n <= 32) {
    // A sequence by a lane, every warp for itself.
    const int lane = tid & 31, i = min(lane, n - 1);
    const float pairs = static_cast<float>(length(i)) *
                        static_cast<float>(cu_other ? static_cast<int64_t>(cu_other[i + 1]) - cu_other[i] : most_other);
    const int t = lane < n ? tiles_of(length(i)) : 0;
    int before = 0;  // tiles of the sequences taken before this one
    for (int j = 0; j < n; ++j) {
      const float w = __shfl_sync(0xFFFFFFFFu, pairs, j);
      const int tj = __shfl_sync(0xFFFFFFFFu, t, j);
      before += w > pairs || (w == pairs && j < lane) ? tj : 0;
    }
    const uint32_t mine = __ballot_sync(0xFFFFFFFFu, before <= index && index < before + t);
    if (!mine) return {0, -1, 0};
    const int at = __ffs(mine) - 1;
    return {at, index - __shfl_sync(0xFFFFFFFFu, before, at), __shfl_sync(0xFFFFFFFFu, t, at)};
  }
  float* const work = reinterpret_cast<float*>(scratch);
  int* const order = reinterpret_cast<int*>(scratch) + kSortSequences;
  for (int i = tid; i < n; i += THREADS)
    work[i] = static_cast<float>(length(i)) *
              static_cast<float>(cu_other ? static_cast<int64_t>(cu_other[i + 1]) - cu_other[i] : most_other);
  __syncthreads();
  for (int i = tid; i < n; i += THREADS) {
    const float mine = work[i];
    int before = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) before += work[j] > mine || (work[j] == mine && j < i);
    order[before] = i;
  }
  __syncthreads();
  // Every warp adds the tiles up, 32 sequences at a time.
  TilePlace r = {0, -1, 0};
  const int lane = tid & 31;
  int sum = 0;
  for (int from = 0; from < n; from += 32) {
    const int i = from + lane < n ? order[from + lane] : 0;
    const int t = from + lane < n ? tiles_of(length(i)) : 0;
    int upto = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, sum + upto > index);
    if (past) {
      const int at = __ffs(past) - 1;
      r.sequence = __shfl_sync(0xFFFFFFFFu, i, at);
      r.tiles = __shfl_sync(0xFFFFFFFFu, t, at);
      r.tile = index - sum - __shfl_sync(0xFFFFFFFFu, upto - t, at);
      break;
    }
    sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  fence_async_smem();  // (bulk copies may write the scratch next)
  __syncthreads();
  return r;
}

}  // namespace gbn
