// Attention of the new tokens of each sequence (one, a chain or a tree of
// drafts) over a paged, quantized key / value cache.
//
// The plain kernel: a block per query row and head, four warps that take the
// cached tokens in turn.  Scores, the running maximum, the sum and the output
// are float32.
#include <cmath>

#include "kv_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kWarps = 4;

struct Params {
  const uint8_t* q;
  uint8_t* out;
  int64_t qt, qh, ot, oh;  // strides in bytes
  int32_t hq, group;
  int64_t Tq;
  kv::CacheView cache;
  const int32_t* table;
  int64_t max_pages;
  const int32_t* q_indptr;
  const int32_t* ctx_lens;
  int32_t B;
  const int64_t* mask;
  int32_t mask_words, max_nodes;
  float scale;
  float* lse;
  int32_t* err;
};

template <int FMT, int PER>
__device__ __forceinline__ void load_codes(const uint8_t* row, int lane, uint32_t scale_word, float* x) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = lane * PER + i;
    if constexpr (FMT == QLIN_KV_U4) {
      const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(scale_word & 0xffffu)));
      const float z = __half2float(__ushort_as_half(static_cast<unsigned short>(scale_word >> 16)));
      x[i] = (static_cast<float>((row[c / 2] >> (4 * (c & 1))) & 15) - z) * s;
    } else if constexpr (FMT == QLIN_KV_INT8) {
      x[i] = static_cast<float>(static_cast<int8_t>(row[c])) * __uint_as_float(scale_word);
    } else {
      x[i] = kv::unpack2<0>(kv::e4m3x2_to_half2(row[c])).x * __uint_as_float(scale_word);
    }
  }
}

template <int DT, int D, int FMT>
__global__ void __launch_bounds__(32 * kWarps) tree_attention_plain_kernel(const __grid_constant__ Params p) {
  constexpr int PER = D / 32;
  __shared__ float part[kWarps][D + 2];
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = h / p.group;

  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.q_indptr[mid] <= t) lo = mid; else hi = mid;
  }
  if (t < p.q_indptr[lo] || t >= p.q_indptr[lo + 1]) return;
  const int node = static_cast<int>(t - p.q_indptr[lo]);
  const int nodes = p.q_indptr[lo + 1] - p.q_indptr[lo];
  const int64_t ctx = p.ctx_lens[lo];
  const int64_t len = ctx + nodes;

  float q[PER], o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t u = reinterpret_cast<const uint16_t*>(p.q + t * p.qt + h * p.qh)[lane * PER + i];
    q[i] = kv::unpack2<DT>(u).x * p.scale;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = warp; j < len; j += kWarps) {
    if (j >= ctx) {
      const int b = static_cast<int>(j - ctx);
      const bool seen = p.mask == nullptr ? b <= node : (p.mask[t * p.mask_words + b / 64] >> (b & 63)) & 1;
      if (!seen) continue;
    }
    const int64_t n = j >> p.cache.page_shift;
    const int32_t page = n < p.max_pages ? p.table[lo * p.max_pages + n] : -1;
    if (page < 0 || page >= p.cache.pages) {
      record_device_error(p.err, kDevErrBadIndex);
      continue;
    }
    const int64_t row = (static_cast<int64_t>(hk) << p.cache.page_shift) + (j - (n << p.cache.page_shift));
    const int64_t c = page * p.cache.page_stride + row * kv::row_bytes(FMT, D);
    const int64_t s = page * p.cache.scale_page_stride + row * 4;
    float x[PER];
    load_codes<FMT, PER>(p.cache.k + c, lane, *reinterpret_cast<const uint32_t*>(p.cache.k_scale + s), x);
    float score = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) score = fmaf(q[i], x[i], score);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) score += __shfl_xor_sync(0xffffffffu, score, w);
    load_codes<FMT, PER>(p.cache.v + c, lane, *reinterpret_cast<const uint32_t*>(p.cache.v_scale + s), x);
    const float m_new = fmaxf(m, score);
    const float keep = m == -INFINITY ? 0.0f : __expf(m - m_new);
    const float w = __expf(score - m_new);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * keep + w * x[i];
    m = m_new;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) part[warp][lane * PER + i] = o[i];
  if (lane == 0) {
    part[warp][D] = m;
    part[warp][D + 1] = l;
  }
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY, total = 0.0f, acc[PER] = {};
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][D]);
  for (int w = 0; w < kWarps; ++w) {
    const float keep = part[w][D] == -INFINITY ? 0.0f : __expf(part[w][D] - top);
    total += part[w][D + 1] * keep;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] += part[w][lane * PER + i] * keep;
  }
  const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    reinterpret_cast<uint16_t*>(p.out + t * p.ot + h * p.oh)[lane * PER + i] =
        static_cast<uint16_t>(kv::pack2<DT>(acc[i] * inv, 0.0f));
  if (p.lse != nullptr && lane == 0) p.lse[t * p.hq + h] = top + logf(total);
}

template <int DT, int D>
cudaError_t launch(const Params& p, int fmt, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.Tq), static_cast<unsigned>(p.hq));
  if (fmt == QLIN_KV_INT8) tree_attention_plain_kernel<DT, D, QLIN_KV_INT8><<<grid, 32 * kWarps, 0, stream>>>(p);
  else if (fmt == QLIN_KV_E4M3) tree_attention_plain_kernel<DT, D, QLIN_KV_E4M3><<<grid, 32 * kWarps, 0, stream>>>(p);
  else tree_attention_plain_kernel<DT, D, QLIN_KV_U4><<<grid, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int64_t tree_attention_workspace_bytes(const qlin_kv_cache&, int64_t, int64_t, int64_t) { return 256; }

cudaError_t launch_tree_attention(const TreeAttentionArgs& a, cudaStream_t stream) {
  Params p = {};
  p.q = static_cast<const uint8_t*>(a.q.data);
  p.out = static_cast<uint8_t*>(a.out.data);
  p.qt = 2 * a.q.token_stride;
  p.qh = 2 * a.q.head_stride;
  p.ot = 2 * a.out.token_stride;
  p.oh = 2 * a.out.head_stride;
  p.hq = static_cast<int32_t>(a.q.heads);
  p.group = static_cast<int32_t>(a.q.heads / a.cache.heads);
  p.Tq = a.Tq;
  p.cache = kv::view_of(a.cache);
  p.table = a.block_table;
  p.max_pages = a.max_pages;
  p.q_indptr = a.q_indptr;
  p.ctx_lens = a.ctx_lens;
  p.B = static_cast<int32_t>(a.B);
  p.mask = a.mask;
  p.mask_words = static_cast<int32_t>(a.mask_words);
  p.max_nodes = static_cast<int32_t>(a.max_nodes);
  p.scale = a.scale;
  p.lse = a.lse;
  p.err = device_error_word();
  const int fmt = a.cache.fmt;
  const int64_t d = a.cache.head_dim;
  if (a.dtype == QLIN_F16) {
    if (d == 64) return launch<0, 64>(p, fmt, stream);
    if (d == 128) return launch<0, 128>(p, fmt, stream);
    return launch<0, 256>(p, fmt, stream);
  }
  if (d == 64) return launch<1, 64>(p, fmt, stream);
  if (d == 128) return launch<1, 128>(p, fmt, stream);
  return launch<1, 256>(p, fmt, stream);
}

}  // namespace qlin
