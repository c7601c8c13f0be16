// Attention of a chunk of new tokens of each sequence over a paged, quantized
// key / value cache that holds them already: causal, with a prefix that every row sees,
// a window, capped scores and a bias by distance.
//
// One warp per row and query head walks the tokens that the row sees, with a
// running maximum and sum; a lane holds D / 32 channels.
#include <algorithm>

#include "kv_common.cuh"
#include "qlin_internal.h"
#include "tree_common.cuh"

namespace qlin {
namespace chunk {
namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr int64_t kMaxLen = 0x7fff0000;

struct Params {
  const uint8_t* q;
  uint8_t* out;
  int64_t qt, qh, ot, oh;
  int32_t hq, hk, dtype, fmt;
  int64_t Tq;
  kv::CacheView cache;
  const int32_t* table;
  int64_t max_pages;
  const int32_t* q_indptr;
  const int32_t* ctx_lens;
  int32_t B, max_new;
  qlin_scores scores;
  float* lse;
  int32_t* err;
};

template <int D>
__device__ __forceinline__ void codes_of(const Params& p, const uint8_t* base, const uint8_t* scales, int64_t page, int64_t row, int lane, float* x) {
  constexpr int kMine = D / 32;
  const uint8_t* sc = scales + page * p.cache.scale_page_stride + row * 4;
  const uint8_t* c = base + page * p.cache.page_stride + row * (p.fmt == QLIN_KV_U4 ? D / 2 : D);
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = lane * kMine + k;
    if (p.fmt == QLIN_KV_U4) {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(sc);
      const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(word & 0xffffu)));
      const float z = tree::odd_zero(word) ? __uint_as_float(0x7fc00000u) : __half2float(__ushort_as_half(static_cast<unsigned short>(word >> 16)));
      x[k] = (static_cast<float>((c[i / 2] >> (4 * (i & 1))) & 15) - z) * s;
    } else if (p.fmt == QLIN_KV_INT8) {
      x[k] = static_cast<float>(reinterpret_cast<const int8_t*>(c)[i]) * *reinterpret_cast<const float*>(sc);
    } else {
      x[k] = kv::unpack2<0>(kv::e4m3x2_to_half2(c[i])).x * *reinterpret_cast<const float*>(sc);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(128) chunk_attention_kernel(const __grid_constant__ Params p) {
  constexpr int kMine = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
  const int64_t row = unit / p.hq;
  const int h = static_cast<int>(unit - row * p.hq);
  if (row >= p.Tq) return;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.q_indptr[mid] <= row) lo = mid; else hi = mid;
  }
  const int64_t q0 = p.q_indptr[lo], q1 = p.q_indptr[lo + 1], ctx = p.ctx_lens[lo];
  if (row < q0 || row >= q1) return;
  const int64_t len = ctx + q1 - q0;
  if (q0 < 0 || q1 > p.Tq || q1 - q0 > p.max_new || ctx < 0 || len > (p.max_pages << p.cache.page_shift) || len > kMaxLen) {
    record_device_error(p.err, kDevErrBadIndex);
    return;
  }
  const int64_t at = ctx + row - q0;
  const int64_t prefix = p.scores.prefix_lens != nullptr ? max(int64_t(0), min(static_cast<int64_t>(p.scores.prefix_lens[lo]), len)) : 0;
  const int64_t low = p.scores.window > 0 ? max(int64_t(0), at - p.scores.window + 1) : 0;
  const int head = h / (p.hq / p.hk);
  float q[kMine], o[kMine] = {};
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const uint16_t u = *reinterpret_cast<const uint16_t*>(p.q + row * p.qt + h * p.qh + (lane * kMine + k) * 2);
    q[k] = p.dtype == QLIN_BF16 ? kv::unpack2<1>(u).x : kv::unpack2<0>(u).x;
  }
  float m = -INFINITY, l = 0.0f;
  const float slope = p.scores.slopes != nullptr ? p.scores.slopes[h] : 0.0f;
  for (int64_t j = prefix > 0 ? 0 : low; j < max(prefix, at + 1); ++j) {
    if (j >= prefix && j < low) j = low;
    const int32_t page = p.table[lo * p.max_pages + (j >> p.cache.page_shift)];
    float x[kMine] = {}, y[kMine] = {};
    if (page >= 0 && page < p.cache.pages) {
      const int64_t r = (static_cast<int64_t>(head) << p.cache.page_shift) + (j & ((1 << p.cache.page_shift) - 1));
      codes_of<D>(p, p.cache.k, p.cache.k_scale, page, r, lane, x);
      codes_of<D>(p, p.cache.v, p.cache.v_scale, page, r, lane, y);
    } else {
      record_device_error(p.err, kDevErrBadIndex);
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kMine; ++k) s += q[k] * x[k];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scores.scale;
    if (p.scores.softcap > 0.0f) s = p.scores.softcap * tanhf(s / p.scores.softcap);
    s -= slope * fabsf(static_cast<float>(at - j));
    const float to = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.0f : __expf(m - to), e = __expf(s - to);
    m = to;
    l = l * keep + e;
#pragma unroll
    for (int k = 0; k < kMine; ++k) o[k] = o[k] * keep + e * y[k];
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const uint32_t u = p.dtype == QLIN_BF16 ? kv::pack2<1>(o[k] / l, 0.0f) : kv::pack2<0>(o[k] / l, 0.0f);
    *reinterpret_cast<uint16_t*>(p.out + row * p.ot + h * p.oh + (lane * kMine + k) * 2) = static_cast<uint16_t>(u);
  }
  if (p.lse != nullptr && lane == 0) p.lse[row * p.hq + h] = m + logf(l);
}

}  // namespace
}  // namespace chunk

int64_t chunk_attention_workspace_bytes(const qlin_kv_cache&, int64_t, int64_t, int64_t) { return 256; }

cudaError_t plan_chunk_attention(const ChunkAttentionArgs& a, Prepared* out) {
  using namespace chunk;
  Params p = {};
  p.q = static_cast<const uint8_t*>(a.q.data);
  p.out = static_cast<uint8_t*>(a.out.data);
  p.qt = 2 * a.q.token_stride;
  p.qh = 2 * a.q.head_stride;
  p.ot = 2 * a.out.token_stride;
  p.oh = 2 * a.out.head_stride;
  p.hq = static_cast<int32_t>(a.q.heads);
  p.hk = static_cast<int32_t>(a.cache.heads);
  p.dtype = a.dtype;
  p.fmt = a.cache.fmt;
  p.Tq = a.Tq;
  p.cache = kv::view_of(a.cache);
  p.table = a.block_table;
  p.max_pages = a.max_pages;
  p.q_indptr = a.q_indptr;
  p.ctx_lens = a.ctx_lens;
  p.B = static_cast<int32_t>(a.B);
  p.max_new = static_cast<int32_t>(a.max_new);
  p.scores = a.scores;
  p.lse = a.lse;
  p.err = device_error_word();
  const void* fn = a.cache.head_dim == 64 ? reinterpret_cast<const void*>(chunk_attention_kernel<64>)
                   : a.cache.head_dim == 128 ? reinterpret_cast<const void*>(chunk_attention_kernel<128>)
                                             : reinterpret_cast<const void*>(chunk_attention_kernel<256>);
  out->count = 1;
  out->launch[0] = {fn, static_cast<uint32_t>((a.Tq * a.q.heads + 3) / 4), 1, 128, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace qlin
