// The accepted path of a sequence's new tokens moved to the places right behind
// its cached ones: token ctx + path[i] becomes token ctx + i, codes and scales of
// every head.
//
// A thread owns 16 bytes (or a scale) of one head's row and moves them for the
// whole path, kBatch tokens at a time: it loads all of a batch before it stores
// any of it.  A path ascends, so path[i] >= i: what a batch stores, at places below
// its end, no later batch reads, and within a thread no other one interferes.
// Bound: latency for few sequences (lengths, path, page, bytes: one conversation's path
// and the read of what it kept take 7.0 us together), memory for many: 192 sequences that
// keep up to 9 of 64 tokens, 32 heads of 128, and that read take 18.3 us for 42 MB
// (6.3 us).
#include <algorithm>

#include "kv_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;

struct Params {
  kv::CacheView cache;
  const int32_t* table;
  int64_t max_pages;
  const int32_t* ctx;
  const int32_t* path;
  const int32_t* count;
  int32_t* lens;
  int32_t max_path;
  int32_t row_bytes, pieces;  // 16-byte pieces of a row of codes, and one for its scale
  int32_t* err;
};

// The row of token `at` of this block's sequence among all (page, place) pairs, or -1.
__device__ __forceinline__ int64_t place_of(const Params& p, const int32_t* table, int64_t at) {
  const int32_t page = table[at >> p.cache.page_shift];
  if (page < 0 || page >= p.cache.pages) return -1;
  return (static_cast<int64_t>(page) << p.cache.page_shift) | (at & ((1 << p.cache.page_shift) - 1));
}

template <class T>
__device__ __forceinline__ void move(const Params& p, uint8_t* base, int64_t page_stride, int64_t row0, int64_t row_bytes, int64_t ctx,
                                     int count, const int32_t* path, const int32_t* table, bool reports) {
  const int64_t in_page = (1 << p.cache.page_shift) - 1;
  for (int i0 = 0; i0 < count; i0 += kBatch) {
    T v[kBatch];
    int64_t to[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      to[k] = -1;
      const int i = i0 + k;
      if (i >= count || path[i] == i) continue;
      const int64_t from = place_of(p, table, ctx + path[i]), dst = place_of(p, table, ctx + i);
      if (from < 0 || dst < 0) {
        if (reports) record_device_error(p.err, kDevErrBadIndex);
        continue;
      }
      to[k] = (dst >> p.cache.page_shift) * page_stride + (row0 + (dst & in_page)) * row_bytes;
      v[k] = *reinterpret_cast<const T*>(base + (from >> p.cache.page_shift) * page_stride + (row0 + (from & in_page)) * row_bytes);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (to[k] >= 0) *reinterpret_cast<T*>(base + to[k]) = v[k];
  }
}

__global__ void __launch_bounds__(kThreads) kv_keep_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = blockIdx.x;
  const int64_t ctx = p.ctx[b];
  const int count = p.count[b];
  const int32_t* path = p.path + b * p.max_path;
  bool bad = count < 0 || count > p.max_path || ctx < 0 || ctx + count > INT32_MAX;  // (lengths are int32)
  if (!bad) {
    for (int i = threadIdx.x; i < count; i += kThreads)
      bad |= path[i] < i || (i > 0 && path[i] <= path[i - 1]) || ((ctx + path[i]) >> p.cache.page_shift) >= p.max_pages;
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    if (bad) record_device_error(p.err, kDevErrBadIndex);
    if (p.lens != nullptr) p.lens[b] = static_cast<int32_t>(bad ? ctx : ctx + count);
  }
  if (bad) return;
  const int32_t* table = p.table + b * p.max_pages;
  const int64_t unit = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
  const int64_t row = unit / p.pieces;  // (head, K or V)
  const int piece = static_cast<int>(unit - row * p.pieces);
  const int64_t head = row >> 1;
  if (head >= p.cache.heads) return;
  const bool v = row & 1;
  const int64_t row0 = head << p.cache.page_shift;
  if (piece < p.pieces - 1)
    move<uint4>(p, (v ? p.cache.v : p.cache.k) + piece * 16, p.cache.page_stride, row0, p.row_bytes, ctx, count, path, table, unit == 0);
  else
    move<uint32_t>(p, v ? p.cache.v_scale : p.cache.k_scale, p.cache.scale_page_stride, row0, 4, ctx, count, path, table, false);
}

}  // namespace

cudaError_t plan_kv_cache_keep(const qlin_kv_cache* cache, const int32_t* block_table, int64_t max_pages, const int32_t* ctx_lens,
                               const int32_t* path, const int32_t* count, int64_t B, int64_t max_path, int32_t* lens, Prepared* out) {
  Params p = {};
  p.cache = kv::view_of(*cache);
  p.table = block_table;
  p.max_pages = max_pages;
  p.ctx = ctx_lens;
  p.path = path;
  p.count = count;
  p.lens = lens;
  p.max_path = static_cast<int32_t>(max_path);
  p.row_bytes = kv::row_bytes(cache->fmt, static_cast<int>(cache->head_dim));
  p.pieces = p.row_bytes / 16 + 1;
  p.err = device_error_word();
  const int64_t units = 2 * cache->heads * p.pieces;
  out->count = 1;
  out->launch[0] = {reinterpret_cast<const void*>(kv_keep_kernel), static_cast<uint32_t>(B),
                    static_cast<uint32_t>((units + kThreads - 1) / kThreads), kThreads, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace qlin
