// Attention over whole sequences, forward (host side; the kernel is the prompts' of
// paged_prefill.cu) and backward.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_rows.cuh"
#include "tensor_core.cuh"

namespace gbn {
namespace {

// ---- row statistics
//
// delta_i = dout_i.out_i for every query and head, and lse beside it in the form and order
// that the kernels of the backward read: by head, then query.  A CTA takes 16 tokens and 32
// heads; a row of 8 elements a lane is C lanes.  Bound by reading out and dout once.
constexpr int kStatTokens = 16, kStatHeads = 32, kStatThreads = 256;

template <typename T, int C>
__global__ void __launch_bounds__(kStatThreads) attention_stats_kernel(const AttnBwdParams p) {
  __shared__ float tile[kStatHeads][kStatTokens + 1];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = (p.max_q + kStatTokens - 1) / kStatTokens;  // of a sequence
  const int b = blockIdx.x / blocks, i0 = blockIdx.x % blocks * kStatTokens, h0 = blockIdx.y * kStatHeads;
  const SeqRange s = bwd_range(p, b, tid == 0 && i0 == 0 && h0 == 0);
  if (i0 >= s.qlen) return;
  constexpr int kRows = 32 / C;  // rows a warp reads at once
  const int c = lane % C;
  for (int r = warp * kRows + lane / C; r < kStatTokens * kStatHeads; r += kStatThreads / 32 * kRows) {
    const int t = r / kStatHeads, hh = r % kStatHeads;
    float sum = 0.f;
    if (i0 + t < s.qlen && h0 + hh < p.hq && c * 8 < p.d) {
      const int64_t at = s.q0 + i0 + t, head = h0 + hh;
      float x[8], y[8];
      eight<T>(p.out, at * p.ot + head * p.oh + c * 8, x);
      eight<T>(p.dout, at * p.gt + head * p.gh + c * 8, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
    }
#pragma unroll
    for (int o = C / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (c == 0) tile[hh][t] = -sum;
  }
  __syncthreads();
  const int64_t base = stat_base(s.q0, b) + i0;
  for (int r = tid; r < kStatTokens * kStatHeads; r += kStatThreads) {
    const int t = r % kStatTokens, hh = r / kStatTokens;
    if (i0 + t >= s.qlen || h0 + hh >= p.hq) continue;
    const int64_t at = (h0 + hh) * p.stat_stride + base + t;
    p.ndelta[at] = tile[hh][t];
    p.nlse[at] = fmaf(p.lse[(s.q0 + static_cast<int64_t>(i0) + t) * p.hq + h0 + hh], -kAttnLog2e,
                      static_cast<float>(kWeightLog2<T>));
  }
}

// ---- the simplest form: a thread computes eight columns of one row

template <typename T, int WHICH>
__global__ void __launch_bounds__(128) attention_bwd_plain_kernel(const AttnBwdParams p) {
  pdl_begin();
  const int b = blockIdx.z, head = blockIdx.y, h = WHICH ? head : head / p.group;
  const SeqRange s = bwd_range(p, b, false);
  const int n = WHICH ? s.kv : s.qlen, chunks = p.d / 8;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  const int row = static_cast<int>(x / chunks), col = static_cast<int>(x % chunks) * 8;
  if (row >= n) return;
  float f[8];
  grad_again<T, WHICH>(p, s, b, head, h, row, col, f);
  T* dst = static_cast<T*>(WHICH == 0 ? p.dq : WHICH == 1 ? p.dk : p.dv);
  const int64_t at = WHICH == 0   ? (s.q0 + static_cast<int64_t>(row)) * p.dqt + head * p.dqh
                     : WHICH == 1 ? (s.k0 + static_cast<int64_t>(row)) * p.dkt + h * p.dkh
                                  : (s.k0 + static_cast<int64_t>(row)) * p.dvt + h * p.dvh;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = narrow2<T>(p2(f[2 * e], f[2 * e + 1]));
  *reinterpret_cast<uint4*>(dst + at + col) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
cudaError_t launch_bwd(const AttnBwdParams& p, cudaStream_t st) {
  const dim3 sg((p.max_q + kStatTokens - 1) / kStatTokens * p.batches, (p.hq + kStatHeads - 1) / kStatHeads);
  cudaError_t e = cudaSuccess;
  if (p.max_q > 0) {
    e = p.d <= 64 ? launch_pdl(attention_stats_kernel<T, 8>, sg, dim3(kStatThreads), 0, st, p)
                  : launch_pdl(attention_stats_kernel<T, 16>, sg, dim3(kStatThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    const unsigned nq = (p.max_q * (p.d / 8) + 127) / 128;
    e = launch_pdl(attention_bwd_plain_kernel<T, 0>, dim3(nq, p.hq, p.batches), dim3(128), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  if (p.max_k == 0) return e;
  const unsigned nk = (p.max_k * (p.d / 8) + 127) / 128;
  e = launch_pdl(attention_bwd_plain_kernel<T, 1>, dim3(nk, p.hkv, p.batches), dim3(128), 0, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attention_bwd_plain_kernel<T, 2>, dim3(nk, p.hkv, p.batches), dim3(128), 0, st, p);
}

// ---- host side

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

int64_t tiles(int64_t n, int64_t of) { return (n + of - 1) / of; }

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

// Elements of one head's statistics: every sequence on a multiple of 4, and a whole tile
// behind the last.
int64_t stat_elements(const AttnSizes& z) {
  return align_up(z.tokens + 3 * z.batches + 3 + kBwdTile, 32);
}

bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale * kAttnLog2e); }

}  // namespace

cudaError_t read_attention_bwd_error(unsigned int* v, bool clear) { return read_paged_error(v, clear); }

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
  if (z.tokens == 0 || z.batches == 0 || z.max_q == 0) return GBN_OK;
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
  p.max_q = static_cast<int>(z.max_q);
  p.max_kv = static_cast<int>(z.max_k);
  p.causal = c.causal != 0;
  p.window = static_cast<int>(z.window);
  const int64_t longest = z.max_q < z.tokens ? z.max_q : z.tokens;
  p.row_tiles = static_cast<int>(tiles(longest * p.group, kPrefillRows));
  p.splits = 1;
  p.split_len = INT32_MAX;
  p.scale_log2 = c.scale * kAttnLog2e;
  if (int64_t(p.row_tiles) * z.batches * z.kv_heads > INT32_MAX) return GBN_ERR_SHAPE;
  return launch_attention_fwd(p, dtype, stream) == cudaSuccess ? GBN_OK : GBN_ERR_CUDA;
}

gbn_status gbn_attention_bwd_workspace_size(int64_t tokens, int64_t batches, int64_t q_heads,
                                            int64_t kv_heads, gbn_dtype dtype, size_t* bytes) {
  if (!bytes) return GBN_ERR_NULL;
  AttnSizes z{tokens, 0, batches, q_heads, kv_heads, 8, 0, 0, 0, true, true};
  const gbn_status st = check_sizes(z, dtype);
  if (st != GBN_OK) return st;
  *bytes = static_cast<size_t>(2 * q_heads * stat_elements(z) * 4 +
                               align_up(dtype == GBN_F16 ? batches * kv_heads * 8 : 0, 256));
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
  st = gbn_attention_bwd_workspace_size(z.tokens, z.batches, z.q_heads, z.kv_heads, dtype, &need);
  if (st != GBN_OK) return st;
  if (!c.workspace || c.workspace_bytes < need || (reinterpret_cast<uintptr_t>(c.workspace) & 15u))
    return GBN_ERR_WORKSPACE;

  AttnBwdParams p = {};
  p.q = c.q;
  p.k = c.k;
  p.v = c.v;
  p.out = c.out;
  p.dout = c.dout;
  p.lse = c.lse;
  p.cu = c.cu_q;
  p.cu_k = c.cu_k;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.stat_stride = stat_elements(z);
  p.nlse = static_cast<float*>(c.workspace);
  p.ndelta = p.nlse + z.q_heads * p.stat_stride;
  p.norms = dtype == GBN_F16 ? reinterpret_cast<uint32_t*>(p.ndelta + z.q_heads * p.stat_stride) : nullptr;
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
  p.scale = c.scale;
  p.scale_log2 = c.scale * kAttnLog2e;
  const cudaError_t e = dtype == GBN_BF16 ? launch_bwd<__nv_bfloat16>(p, stream)
                                          : launch_bwd<__half>(p, stream);
  return e == cudaSuccess ? GBN_OK : GBN_ERR_CUDA;
}

}  // extern "C"
