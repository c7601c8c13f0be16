// Reads tokens of a paged, quantized cache back as 16-bit rows: a gather with
// dequantization, bound by HBM (codes and scales in, 16-bit rows out).
//
// A block takes kTokens output rows x the heads that make one pass of its
// threads: groups of D / 8 lanes take a (token, head) each, eight elements per
// lane, so that a lane's code load is 8 bytes (4 for U4) and its store 16, with
// kUnroll rows of keys and values in flight per thread.  A warp per token first
// finds the row's sequence (32 bounds per probe) and its place in the cache.
// Consecutive groups take consecutive tokens of one head: the codes of a page
// are contiguous per head, the outputs are whole 128-byte lines or more either
// way.  Small blocks of one pass fill the GPU from a few hundred rows on.
#include "kv_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;  // one per warp
constexpr int kUnroll = 4;

struct Params {
  kv::CacheView cache;
  const int32_t* table;
  int64_t max_pages;
  const int32_t* starts;
  const int32_t* indptr;
  int32_t B;
  int64_t rows;
  uint8_t* k_out;
  uint8_t* v_out;
  int64_t kt, kh, vt, vh;  // strides in bytes
  int32_t* err;
};

// Eight codes of a row (8 bytes, or 4 for U4) with the row's scale word, as
// the 16-bit values they stand for: one float32 product, rounded once.
template <int DT, int FMT>
__device__ __forceinline__ uint4 dequantize8(uint2 codes, uint32_t scale_word) {
  float x[8];
  if constexpr (FMT == QLIN_KV_U4) {
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(scale_word & 0xffffu)));
    const float z = __half2float(__ushort_as_half(static_cast<unsigned short>(scale_word >> 16)));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (static_cast<float>((codes.x >> (4 * i)) & 15u) - z) * s;
  } else {
    const float s = __uint_as_float(scale_word);
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (FMT == QLIN_KV_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * h + i] = static_cast<float>(static_cast<int8_t>(w[h] >> (8 * i))) * s;
      } else {
        const float2 a = kv::unpack2<0>(kv::e4m3x2_to_half2(static_cast<uint16_t>(w[h])));
        const float2 b = kv::unpack2<0>(kv::e4m3x2_to_half2(static_cast<uint16_t>(w[h] >> 16)));
        x[4 * h] = a.x * s;
        x[4 * h + 1] = a.y * s;
        x[4 * h + 2] = b.x * s;
        x[4 * h + 3] = b.y * s;
      }
    }
  }
  return kv::pack8<DT>(x);
}

template <int DT, int D, int FMT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ Params p) {
  constexpr int LANES = D / 8;
  constexpr int kGroups = kThreads / LANES;
  constexpr int kCode = FMT == QLIN_KV_U4 ? 4 : 8;  // bytes of a lane's eight codes
  __shared__ int64_t place[kTokens];                // page << shift | offset, or -1
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int count = static_cast<int>(min(static_cast<int64_t>(kTokens), p.rows - row0));

  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x / 32;
  if (warp < count) {
    const int l = threadIdx.x % 32;
    const int64_t row = row0 + warp;
    int lo = 0, hi = p.B;  // the last sequence that begins at or before `row` is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int b = lo + l * step;
      const unsigned before = __ballot_sync(0xffffffffu, b < hi && p.indptr[b] <= row);
      const int n = before == 0 ? 0 : 31 - __clz(before);
      lo += n * step;
      hi = min(hi, lo + step);
    }
    if (l == 0) {
      int64_t at = -1;
      if (p.indptr[lo] <= row && row < p.indptr[lo + 1]) {
        const int64_t pos = static_cast<int64_t>(p.starts[lo]) + (row - p.indptr[lo]);
        const int64_t n = pos >> p.cache.page_shift;
        if (pos >= 0 && n < p.max_pages) {
          const int32_t page = p.table[lo * p.max_pages + n];
          if (page >= 0 && page < p.cache.pages)
            at = (static_cast<int64_t>(page) << p.cache.page_shift) | (pos & ((int64_t(1) << p.cache.page_shift) - 1));
        }
      }
      if (at < 0) record_device_error(p.err, kDevErrBadIndex);
      place[warp] = at;
    }
  }
  __syncthreads();

  const int lane = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  constexpr int kHeads = kGroups * kUnroll / kTokens;  // heads of a block
  const int head0 = blockIdx.y * kHeads;
  const int items = count * min(kHeads, p.cache.heads - head0);
  {
    const int i0 = group;
    uint2 kc[kUnroll], vc[kUnroll];
    uint32_t ks[kUnroll], vs[kUnroll];
    int tok[kUnroll], head[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kGroups;
      head[u] = i / count;
      tok[u] = i - head[u] * count;
      head[u] += head0;
      kc[u] = vc[u] = make_uint2(0u, 0u);
      ks[u] = vs[u] = 0u;
      if (i >= items) continue;
      const int64_t at = place[tok[u]];
      if (at < 0) continue;
      const int64_t page = at >> p.cache.page_shift;
      const int64_t row = (static_cast<int64_t>(head[u]) << p.cache.page_shift) + (at - (page << p.cache.page_shift));
      const int64_t c = page * p.cache.page_stride + row * kv::row_bytes(FMT, D) + lane * kCode;
      const int64_t s = page * p.cache.scale_page_stride + row * 4;
      if constexpr (FMT == QLIN_KV_U4) {
        kc[u].x = *reinterpret_cast<const uint32_t*>(p.cache.k + c);
        vc[u].x = *reinterpret_cast<const uint32_t*>(p.cache.v + c);
      } else {
        kc[u] = *reinterpret_cast<const uint2*>(p.cache.k + c);
        vc[u] = *reinterpret_cast<const uint2*>(p.cache.v + c);
      }
      ks[u] = *reinterpret_cast<const uint32_t*>(p.cache.k_scale + s);
      vs[u] = *reinterpret_cast<const uint32_t*>(p.cache.v_scale + s);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (i0 + u * kGroups >= items) continue;
      const int64_t t = row0 + tok[u];
      // a place that is out of range reads as zeros (its scale word is 0)
      *reinterpret_cast<uint4*>(p.k_out + t * p.kt + head[u] * p.kh + lane * 16) = dequantize8<DT, FMT>(kc[u], ks[u]);
      *reinterpret_cast<uint4*>(p.v_out + t * p.vt + head[u] * p.vh + lane * 16) = dequantize8<DT, FMT>(vc[u], vs[u]);
    }
  }
}

template <int DT, int D>
cudaError_t plan(const Params& p, int fmt, Prepared* out) {
  constexpr int kHeads = kThreads / (D / 8) * kUnroll / kTokens;
  const void* fn = fmt == QLIN_KV_INT8   ? reinterpret_cast<const void*>(kv_read_kernel<DT, D, QLIN_KV_INT8>)
                   : fmt == QLIN_KV_E4M3 ? reinterpret_cast<const void*>(kv_read_kernel<DT, D, QLIN_KV_E4M3>)
                                         : reinterpret_cast<const void*>(kv_read_kernel<DT, D, QLIN_KV_U4>);
  out->count = 1;
  out->launch[0] = {fn, static_cast<uint32_t>((p.rows + kTokens - 1) / kTokens),
                    static_cast<uint32_t>((p.cache.heads + kHeads - 1) / kHeads), kThreads, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace

cudaError_t plan_kv_cache_read(const qlin_kv_cache* cache, const int32_t* block_table, int64_t max_pages,
                                 const int32_t* starts, const int32_t* indptr, int64_t B, int64_t rows,
                                 const qlin_heads* k_out, const qlin_heads* v_out, qlin_dtype dtype, Prepared* out) {
  Params p = {};
  p.cache = kv::view_of(*cache);
  p.table = block_table;
  p.max_pages = max_pages;
  p.starts = starts;
  p.indptr = indptr;
  p.B = static_cast<int32_t>(B);
  p.rows = rows;
  p.k_out = static_cast<uint8_t*>(k_out->data);
  p.v_out = static_cast<uint8_t*>(v_out->data);
  p.kt = 2 * k_out->token_stride;
  p.kh = 2 * k_out->head_stride;
  p.vt = 2 * v_out->token_stride;
  p.vh = 2 * v_out->head_stride;
  p.err = device_error_word();
  const int64_t d = cache->head_dim;
  if (dtype == QLIN_F16) {
    if (d == 64) return plan<0, 64>(p, cache->fmt, out);
    if (d == 128) return plan<0, 128>(p, cache->fmt, out);
    return plan<0, 256>(p, cache->fmt, out);
  }
  if (d == 64) return plan<1, 64>(p, cache->fmt, out);
  if (d == 128) return plan<1, 128>(p, cache->fmt, out);
  return plan<1, 256>(p, cache->fmt, out);
}

}  // namespace qlin
