// Attention over whole sequences: the C entry points of the forward (its kernel is the prompts' of
// paged_prefill.cu) and of the backward (attention_bwd.cuh).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention_rows.cuh"
#include "packed_tiles.cuh"

namespace gbn {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;

struct AttnSizes {
  int64_t tokens, keys, batches, q_heads, kv_heads, head_dim, max_q, max_k, window;
  bool packed_q, packed_k;  // lengths in cu_seqlens
};

gbn_status check_sizes(const AttnSizes& z, gbn_dtype dtype) {
  if (dtype != GBN_BF16 && dtype != GBN_F16) return GBN_ERR_DTYPE;
  if (z.tokens < 0 || z.keys < 0 || z.batches < 0 || z.batches > GBN_PAGED_MAX_BATCHES ||
      z.q_heads < 1 || z.kv_heads < 1 || z.q_heads % z.kv_heads != 0 || z.q_heads > 65535 ||
      z.head_dim < 8 || z.head_dim > GBN_ATTENTION_MAX_DIM || z.head_dim % 8 != 0 || z.max_q < 0 ||
      z.max_q > kMaxRows || z.max_k < 0 || z.max_k > kMaxRows || z.window < 0 ||
      z.window > INT32_MAX || z.tokens > INT32_MAX || z.keys > INT32_MAX ||
      z.tokens * z.q_heads > INT32_MAX)
    return GBN_ERR_SHAPE;
  if ((!z.packed_q && z.tokens != z.batches * z.max_q) ||
      (!z.packed_k && z.keys != z.batches * z.max_k))
    return GBN_ERR_SHAPE;
  return GBN_OK;
}


// (token, head) strides of a tensor of `rows` tokens: multiples of 16 bytes; `map`: read
// through a tensor map, which takes strides in (0, 2^40) bytes.
gbn_status check_tensor(const void* ptr, const int64_t* st, int64_t rows, int64_t heads, bool map) {
  if ((reinterpret_cast<uintptr_t>(ptr) & 15u) != 0) return GBN_ERR_ALIGNMENT;
  const int64_t extent[2] = {rows, heads};
  for (int i = 0; i < 2; ++i) {
    if (extent[i] <= 1) continue;
    if (st[i] * 2 % 16 != 0) return GBN_ERR_ALIGNMENT;
    if (map && (st[i] <= 0 || st[i] >= (int64_t(1) << 39))) return GBN_ERR_SHAPE;
  }
  return GBN_OK;
}

int64_t align_up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

// Elements of one head's norms of `rows` rows: every sequence's runs behind the last one's.
int64_t norm_elements(int64_t rows, int64_t batches) { return rows / kStatTokens + batches + 1; }
int64_t norm_total(const AttnSizes& z, gbn_dtype dtype) {
  return dtype != GBN_F16 ? 0
                          : align_up(z.q_heads * norm_elements(z.tokens, z.batches) +
                                         z.kv_heads * norm_elements(z.keys, z.batches), 4);
}

// Elements of one head's statistics: every sequence on a multiple of 4, and a whole tile
// behind the last.
int64_t stat_elements(const AttnSizes& z) {
  return align_up(z.tokens + 3 * z.batches + 3 + kBwdTile, 32);
}

// How many CTAs share a tile's steps.  A CTA's steps follow one another (about 1.2 us each for
// dk and dv, 1 us for dq), so a launch takes at least as long as its longest one: where that
// is more than a multiprocessor's share of the whole (152 of them, causal ones half full), it is
// divided, down to 8 steps, below which beginning and end cost as much (one sequence of 4096
// tokens, 8 / 2 heads of 128, causal: 172 us with one CTA a tile, 104 so; 2048 tokens, 5 / 1 of
// 64: 100, 36).
struct BwdPlan {
  int kv_splits, q_splits;  // CTAs that share a tile's steps
  int64_t kv_part, q_part;  // elements
};
BwdPlan plan_bwd(const AttnSizes& z, bool causal) {
  const int64_t q_tiles = tiles(z.max_q, kBwdTile), k_tiles = tiles(z.max_k, kBwdTile);
  const int64_t reach = causal && z.window > 0 ? tiles(z.window, kBwdTile) + 1 : kMaxRows;
  const int64_t kv_steps = z.q_heads / z.kv_heads * std::min(q_tiles, reach), q_steps = std::min(k_tiles, reach);
  const int64_t kv_ctas = std::min(k_tiles * z.batches, z.keys / kBwdTile + z.batches) * z.kv_heads;
  const int64_t q_ctas = std::min(q_tiles * z.batches, z.tokens / kBwdTile + z.batches) * z.q_heads;
  const double all = (causal ? 0.5 : 1.0) * (1.2 * static_cast<double>(kv_ctas) * static_cast<double>(kv_steps) +
                                             static_cast<double>(q_ctas) * static_cast<double>(q_steps));
  const int64_t most = std::max<int64_t>(8, static_cast<int64_t>(all / 152));
  auto share = [&](int64_t steps) {
    return steps * 4 <= most * 5 ? 1 : static_cast<int>(std::min<int64_t>(16, tiles(steps, most)));
  };
  BwdPlan r;
  r.kv_splits = share(kv_steps);
  r.q_splits = share(q_steps);
  r.kv_part = r.kv_splits > 1 ? 2 * r.kv_splits * z.keys * z.kv_heads * z.head_dim : 0;
  r.q_part = r.q_splits > 1 ? r.q_splits * z.tokens * z.q_heads * z.head_dim : 0;
  return r;
}

// Heads of a tile that a CTA takes one after another.  Its beginning and end take as long as four
// steps, and those of a further head in the same CTA as one or two: where tiles have few steps,
// and CTAs enough for three times every multiprocessor are left (five times where lengths
// differ), up to four (8 x 1024 tokens, 32 heads of 64, causal: 254 us with one, 230 with two, 220
// with four; 4 x 2048, 32 / 8 of 128: 385, 373, 364; 9 documents of 17 to 3001, 16 / 4 of 64, window
// 1000: 265, 255, 262).
int heads_each(const AttnSizes& z, bool causal, int64_t x_rows, int64_t x_most, int64_t y_most, int64_t heads,
               int64_t group, int splits, bool ragged) {
  const int64_t x_tiles = tiles(x_most, kBwdTile), y_tiles = tiles(y_most, kBwdTile);
  const int64_t reach = causal && z.window > 0 ? tiles(z.window, kBwdTile) + 1 : kMaxRows;
  const int64_t ctas = std::min(x_tiles * z.batches, x_rows / kBwdTile + z.batches) * heads;
  const double steps = static_cast<double>(group * std::min(y_tiles, reach)) * (causal && reach > y_tiles ? 0.5 : 1.0);
  int each = 1;
  while (splits == 1 && each < 4 && 2 * each <= heads && steps * each < 32 &&
         ctas >= 2 * each * 152 * (ragged ? 5 : 3))
    each *= 2;
  return each;
}

bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale * kAttnLog2e); }

}  // namespace

cudaError_t read_attention_bwd_error(unsigned int* v, bool clear) {
  unsigned int a = 0, b = 0;
  const cudaError_t e = read_attention_bwd_bf16_error(&a, clear), f = read_attention_bwd_f16_error(&b, clear);
  *v = a | b;
  return e != cudaSuccess ? e : f;
}

}  // namespace gbn

using namespace gbn;

extern "C" {

gbn_status gbn_attention_fwd(const gbn_attention_fwd_args* args, cudaStream_t stream) {
  if (!args) return GBN_ERR_NULL;
  const gbn_attention_fwd_args& c = *args;
  const gbn_dtype dtype = static_cast<gbn_dtype>(c.dtype);
  const AttnSizes z{c.tokens, c.keys,  c.batches, c.q_heads, c.kv_heads, c.head_dim,
                    c.max_q,  c.max_k, c.window,  c.cu_q != nullptr, c.cu_k != nullptr};
  gbn_status st = check_sizes(z, dtype);
  if (st != GBN_OK) return st;
  if (!scale_ok(c.scale)) return GBN_ERR_SHAPE;
  // (a bound of 0 leaves no rows, but lengths that do not fit it are flagged)
  if (z.tokens == 0 || z.batches == 0 || (z.max_q == 0 && !z.packed_q)) return GBN_OK;
  if (!c.q || !c.out || (z.keys > 0 && (!c.k || !c.v))) return GBN_ERR_NULL;
  if ((st = check_tensor(c.q, c.q_strides, z.tokens, z.q_heads, false)) != GBN_OK ||
      (st = check_tensor(c.out, c.out_strides, z.tokens, z.q_heads, false)) != GBN_OK ||
      (st = check_tensor(c.k, c.k_strides, z.keys, z.kv_heads, true)) != GBN_OK ||
      (st = check_tensor(c.v, c.v_strides, z.keys, z.kv_heads, true)) != GBN_OK)
    return st;
  AttnParams p = {};
  p.q = c.q;
  // (no keys: nothing is read, but the maps need an address)
  p.k = z.keys > 0 ? c.k : c.q;
  p.v = z.keys > 0 ? c.v : c.q;
  p.out = c.out;
  p.lse = c.lse;
  p.cu = c.cu_q;
  p.cu_k = c.cu_k;
  p.qt = c.q_strides[0];
  p.qh = c.q_strides[1];
  p.ot = c.out_strides[0];
  p.oh = c.out_strides[1];
  p.ks = c.k_strides[0];
  p.kh = c.k_strides[1];
  p.vs = c.v_strides[0];
  p.vh = c.v_strides[1];
  p.tokens = static_cast<int>(z.tokens);
  p.keys = static_cast<int>(z.keys);
  p.batches = static_cast<int>(z.batches);
  p.hq = static_cast<int>(z.q_heads);
  p.hkv = static_cast<int>(z.kv_heads);
  p.group = p.hq / p.hkv;
  p.d = static_cast<int>(z.head_dim);
  p.max_q = static_cast<int>(std::min(z.max_q, z.tokens));
  p.max_kv = static_cast<int>(std::min(z.max_k, z.keys));
  p.causal = c.causal != 0;
  p.window = static_cast<int>(z.window);
  const int64_t blocks = z.max_q > 0 ? tile_blocks(p.cu, z.tokens, z.batches, p.max_q, kPrefillRows, p.group)
                                     : tiles(z.batches, kPrefillRows);
  if (blocks * z.kv_heads > INT32_MAX) return GBN_ERR_SHAPE;
  p.row_tiles = static_cast<int>(blocks);  // of all sequences
  p.splits = 1;
  p.split_len = INT32_MAX;
  p.scale_log2 = c.scale * kAttnLog2e;
  return launch_attention_fwd(p, dtype, stream) == cudaSuccess ? GBN_OK : GBN_ERR_CUDA;
}

gbn_status gbn_attention_bwd_workspace_size(int64_t tokens, int64_t keys, int64_t batches,
                                            int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                            int64_t max_q, int64_t max_k, int64_t window, int causal,
                                            gbn_dtype dtype, size_t* bytes) {
  if (!bytes) return GBN_ERR_NULL;
  const AttnSizes z{tokens, keys, batches, q_heads, kv_heads, head_dim, max_q, max_k, window, true, true};
  const gbn_status st = check_sizes(z, dtype);
  if (st != GBN_OK) return st;
  const BwdPlan a = plan_bwd(z, causal != 0);
  *bytes = static_cast<size_t>(2 * q_heads * stat_elements(z) + norm_total(z, dtype) + a.kv_part + a.q_part) * 4;
  return GBN_OK;
}

gbn_status gbn_attention_bwd(const gbn_attention_bwd_args* args, cudaStream_t stream) {
  if (!args) return GBN_ERR_NULL;
  const gbn_attention_bwd_args& c = *args;
  const gbn_dtype dtype = static_cast<gbn_dtype>(c.dtype);
  const AttnSizes z{c.tokens, c.keys,  c.batches, c.q_heads, c.kv_heads, c.head_dim,
                    c.max_q,  c.max_k, c.window,  c.cu_q != nullptr, c.cu_k != nullptr};
  gbn_status st = check_sizes(z, dtype);
  if (st != GBN_OK) return st;
  if (!scale_ok(c.scale)) return GBN_ERR_SHAPE;
  if (z.batches == 0 || (z.tokens == 0 && z.keys == 0)) return GBN_OK;
  if (z.tokens > 0 && (!c.q || !c.out || !c.dout || !c.lse || !c.dq)) return GBN_ERR_NULL;
  if (z.keys > 0 && (!c.k || !c.v || !c.dk || !c.dv)) return GBN_ERR_NULL;
  if ((st = check_tensor(c.q, c.q_strides, z.tokens, z.q_heads, true)) != GBN_OK ||
      (st = check_tensor(c.dout, c.dout_strides, z.tokens, z.q_heads, true)) != GBN_OK ||
      (st = check_tensor(c.out, c.out_strides, z.tokens, z.q_heads, false)) != GBN_OK ||
      (st = check_tensor(c.dq, c.dq_strides, z.tokens, z.q_heads, false)) != GBN_OK ||
      (st = check_tensor(c.k, c.k_strides, z.keys, z.kv_heads, true)) != GBN_OK ||
      (st = check_tensor(c.v, c.v_strides, z.keys, z.kv_heads, true)) != GBN_OK ||
      (st = check_tensor(c.dk, c.dk_strides, z.keys, z.kv_heads, false)) != GBN_OK ||
      (st = check_tensor(c.dv, c.dv_strides, z.keys, z.kv_heads, false)) != GBN_OK)
    return st;
  size_t need = 0;
  st = gbn_attention_bwd_workspace_size(z.tokens, z.keys, z.batches, z.q_heads, z.kv_heads, z.head_dim, z.max_q,
                                        z.max_k, z.window, c.causal, dtype, &need);
  if (st != GBN_OK) return st;
  if (!c.workspace || c.workspace_bytes < need || (reinterpret_cast<uintptr_t>(c.workspace) & 15u))
    return GBN_ERR_WORKSPACE;

  AttnBwdParams p = {};
  // (no queries or no keys: nothing of them is read, but the maps need an address)
  p.q = z.tokens > 0 ? c.q : c.k;
  p.k = z.keys > 0 ? c.k : c.q;
  p.v = z.keys > 0 ? c.v : c.q;
  p.out = c.out;
  p.dout = z.tokens > 0 ? c.dout : c.k;
  p.lse = c.lse;
  p.cu = c.cu_q;
  p.cu_k = c.cu_k;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.stat_stride = stat_elements(z);
  p.nlse = static_cast<float*>(c.workspace);
  p.ndelta = p.nlse + z.q_heads * p.stat_stride;
  p.q_norm_stride = norm_elements(z.tokens, z.batches);
  p.v_norm_stride = norm_elements(z.keys, z.batches);
  p.q_norms = p.ndelta + z.q_heads * p.stat_stride;  // (f16 only)
  p.v_norms = p.q_norms + z.q_heads * p.q_norm_stride;
  const BwdPlan a = plan_bwd(z, c.causal != 0);
  p.kv_splits = a.kv_splits;
  p.q_splits = a.q_splits;
  p.kv_part = p.q_norms + norm_total(z, dtype);
  p.q_part = p.kv_part + a.kv_part;
  p.qt = c.q_strides[0];
  p.qh = c.q_strides[1];
  p.kt = c.k_strides[0];
  p.kh = c.k_strides[1];
  p.vt = c.v_strides[0];
  p.vh = c.v_strides[1];
  p.ot = c.out_strides[0];
  p.oh = c.out_strides[1];
  p.gt = c.dout_strides[0];
  p.gh = c.dout_strides[1];
  p.dqt = c.dq_strides[0];
  p.dqh = c.dq_strides[1];
  p.dkt = c.dk_strides[0];
  p.dkh = c.dk_strides[1];
  p.dvt = c.dv_strides[0];
  p.dvh = c.dv_strides[1];
  p.tokens = static_cast<int>(z.tokens);
  p.keys = static_cast<int>(z.keys);
  p.batches = static_cast<int>(z.batches);
  p.hq = static_cast<int>(z.q_heads);
  p.hkv = static_cast<int>(z.kv_heads);
  p.group = p.hq / p.hkv;
  p.d = static_cast<int>(z.head_dim);
  p.max_q = static_cast<int>(z.max_q < z.tokens ? z.max_q : z.tokens);
  p.max_k = static_cast<int>(z.max_k < z.keys ? z.max_k : z.keys);
  p.causal = c.causal != 0;
  p.window = static_cast<int>(z.window);
  p.kv_each = heads_each(z, c.causal != 0, z.keys, p.max_k, p.max_q, z.kv_heads, p.group, a.kv_splits, z.packed_k);
  p.q_each = heads_each(z, c.causal != 0, z.tokens, p.max_q, p.max_k, z.q_heads, 1, a.q_splits, z.packed_q);
  const int64_t kv_blocks = tile_blocks(p.cu_k, z.keys, z.batches, p.max_k, kBwdTile) *
                            tiles(z.kv_heads, p.kv_each) * a.kv_splits;
  const int64_t q_blocks = tile_blocks(p.cu, z.tokens, z.batches, p.max_q, kBwdTile) *
                           tiles(z.q_heads, p.q_each) * a.q_splits;
  const int64_t q_stats = tile_blocks(p.cu, z.tokens, z.batches, p.max_q, kStatTokens, 1, false);
  const int64_t v_stats =
      dtype == GBN_F16 ? tile_blocks(p.cu_k, z.keys, z.batches, p.max_k, kStatTokens, 1, false) : 0;
  const int64_t kv_joins =
      a.kv_splits > 1 ? tile_blocks(p.cu_k, z.keys, z.batches, p.max_k, kStatTokens, 1, false) : 0;
  const int64_t q_joins = a.q_splits > 1 ? q_stats : 0;
  if (kv_blocks + q_blocks > INT32_MAX || q_stats + v_stats > INT32_MAX || kv_joins + q_joins > INT32_MAX)
    return GBN_ERR_SHAPE;
  p.kv_join_blocks = static_cast<int>(kv_joins);
  p.join_blocks = static_cast<int>(kv_joins + q_joins);
  p.q_stat_blocks = static_cast<int>(q_stats);
  p.stat_blocks = static_cast<int>(q_stats + v_stats);
  p.kv_blocks = static_cast<int>(kv_blocks);
  p.q_blocks = static_cast<int>(q_blocks);
  p.scale = c.scale;
  p.scale_log2 = c.scale * kAttnLog2e;
  const cudaError_t e = dtype == GBN_BF16 ? launch_attention_bwd_bf16(p, stream)
                                          : launch_attention_bwd_f16(p, stream);
  return e == cudaSuccess ? GBN_OK : GBN_ERR_CUDA;
}

}  // extern "C"
