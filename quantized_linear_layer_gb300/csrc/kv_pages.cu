// Block tables, row bounds, positions and slots of a serving step, from the
// sequences' lengths.
//
// Sequence b needs need = ceil((ctx + new) / page) pages and holds `held`.  It
// gives back give = max(held - need, 0) and asks for take = max(need - held, 0)
// of the stack of free pages.  One block sums along the sequences, 1024 at a time:
// what they give; what they ask for and add, which says who is served; and what of
// that the served ones get.  What moves is then dealt
// out evenly to the threads (a thread finds its sequence in the sums by
// bisection), so one long prompt and a thousand short ones cost alike.  The
// last sequence's last page goes on the stack first, so a step that is taken
// back leaves the stack as it was.
//
// Bound: latency, a chain of dependent reads, scans and barriers of one block: a
// decode step of 64 sequences takes 4.8 us, 600 sequences of 24 tokens each that
// need some 900 pages (0.7 MB written: 0.1 us) 9.8.  Few rows are written by the
// block that works out the sums (one launch); more go to a second kernel over
// the whole GPU.
#include <algorithm>

#include "kv_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kRowThreads = 256;

struct Params {
  int32_t* table;
  int64_t max_pages;
  int32_t* held;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t pages, page_shift;
  const int32_t* ctx;
  const int32_t* add;
  int32_t B;
  int32_t rows_inside;  // the first kernel writes the rows as well
  int64_t T;
  const int32_t* depths;
  int32_t* indptr;
  int64_t* positions;
  int64_t* slots;
  int32_t* err;
};

struct Sums {
  int64_t a, b;
};

// Inclusive sums over the block's threads, and the block's totals; `part` has kWarps + 1 entries.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* part, Sums& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, v.a, o), b = __shfl_up_sync(0xffffffffu, v.b, o);
    if (lane >= o) v.a += a, v.b += b;
  }
  __syncthreads();  // the last use of `part` is over
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    Sums s = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, s.a, o), b = __shfl_up_sync(0xffffffffu, s.b, o);
      if (lane >= o) s.a += a, s.b += b;
    }
    part[lane] = s;
  }
  __syncthreads();
  total = part[kWarps - 1];
  if (warp > 0) v.a += part[warp - 1].a, v.b += part[warp - 1].b;
  return v;
}

struct Request {
  int64_t ctx, add, held, need;
  bool valid;
  __device__ __forceinline__ int64_t give() const { return valid && held > need ? held - need : 0; }
  __device__ __forceinline__ int64_t take() const { return valid && need > held ? need - held : 0; }
};

__device__ __forceinline__ Request request(const Params& p, int64_t b) {
  Request r = {0, 0, 0, 0, false};
  if (b >= p.B) return r;
  r.ctx = p.ctx[b];
  r.add = p.add[b];
  r.held = p.held[b];
  r.need = (r.ctx + r.add + (int64_t(1) << p.page_shift) - 1) >> p.page_shift;
  r.valid = r.ctx >= 0 && r.add >= 0 && r.need <= p.max_pages && r.held >= 0 && r.held <= p.max_pages;
  if (!r.valid) {
    record_device_error(p.err, kDevErrBadIndex);
    r.ctx = r.add = r.need = r.held = 0;
  }
  return r;
}

// The last i in [0, n) with begin[i] <= at (begin does not go down, begin[0] <= at).
template <class T, class V>
__device__ __forceinline__ int last_at(const T* begin, int n, V at) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (begin[mid] <= at) lo = mid; else hi = mid;
  }
  return lo;
}

// Slot and position of row `row`, which is token `i` of the new ones of sequence b (b < 0: of none).
__device__ __forceinline__ void write_row(const Params& p, int64_t row, int b, int64_t i) {
  int64_t slot = -1, position = 0;
  if (b >= 0) {
    const int64_t ctx = p.ctx[b], at = ctx + i;
    const int32_t page = p.table[b * p.max_pages + (at >> p.page_shift)];
    if (page >= 0 && page < p.pages) slot = (static_cast<int64_t>(page) << p.page_shift) + (at & ((1 << p.page_shift) - 1));
    else record_device_error(p.err, kDevErrBadIndex);
    position = ctx + (p.depths != nullptr ? p.depths[row] : i);
  }
  p.slots[row] = slot;
  p.positions[row] = position;
}

__global__ void __launch_bounds__(kThreads) kv_pages_kernel(const __grid_constant__ Params p) {
  __shared__ Sums part[kWarps + 1];
  __shared__ int64_t begin[kThreads + 1];  // what moves before each sequence of the chunk, or its first row
  __shared__ int64_t at_of[kThreads];      // where in the sequence's table row that starts
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x;

  int64_t given = 0;  // by all sequences
  Sums total;
  for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
    block_scan({request(p, b0 + t).give(), 0}, part, total);
    given += total.a;
  }
  int64_t top = *p.free_count;
  if (top < 0 || top + given > p.pages) {  // no stack of this many pages: nothing moves, nobody gets rows
    if (t == 0) record_device_error(p.err, kDevErrBadIndex);
    for (int64_t b = t; b <= p.B; b += kThreads) p.indptr[b] = 0;
    if (p.rows_inside)
      for (int64_t row = t; row < p.T; row += kThreads) write_row(p, row, -1, 0);
    return;
  }

  // back to the stack
  if (given > 0) {
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
      const Request r = request(p, b0 + t);
      const Sums s = block_scan({r.give(), 0}, part, total);
      begin[t] = s.a - r.give();
      at_of[t] = r.need;
      __syncthreads();
      for (int64_t i = t; i < total.a; i += kThreads) {
        const int x = last_at(begin, kThreads, i);
        p.free_pages[top + given - 1 - (before + i)] = p.table[(b0 + x) * p.max_pages + at_of[x] + i - begin[x]];
      }
      before += total.a;
      __syncthreads();
    }
  }
  top += given;
  __syncthreads();  // (and the stack's new pages are there for all threads)

  // from the stack; what the sequences before asked for counts whether they got it or not
  int64_t asked_pages = 0, asked_rows = 0, taken = 0, rows = 0;
  for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
    const int64_t b = b0 + t;
    const Request r = request(p, b);
    const Sums ask = block_scan({r.take(), r.add}, part, total);
    const bool fits = (r.take() == 0 || asked_pages + ask.a <= top) && (r.add == 0 || asked_rows + ask.b <= p.T);
    asked_pages += total.a;
    asked_rows += total.b;
    const int64_t take = fits ? r.take() : 0, add = fits ? r.add : 0;
    const Sums got = block_scan({take, add}, part, total);
    if (b < p.B) {
      if (r.valid) p.held[b] = static_cast<int32_t>(fits ? r.need : min(r.held, r.need));
      p.indptr[b + 1] = static_cast<int32_t>(rows + got.b);
    }
    begin[t] = got.a - take;
    at_of[t] = r.held;
    __syncthreads();
    for (int64_t i = t; i < total.a; i += kThreads) {
      const int x = last_at(begin, kThreads, i);
      p.table[(b0 + x) * p.max_pages + at_of[x] + i - begin[x]] = p.free_pages[top - 1 - (taken + i)];
    }
    __syncthreads();
    begin[t] = got.b - add;  // (used below where there is one chunk)
    taken += total.a;
    rows += total.b;
  }
  if (t == 0) {
    p.indptr[0] = 0;
    *p.free_count = static_cast<int32_t>(top - taken);
  }
  if (!p.rows_inside) return;
  __syncthreads();
  for (int64_t row = t; row < p.T; row += kThreads) {
    const int b = row < rows ? last_at(begin, min(p.B, kThreads), row) : -1;
    write_row(p, row, b, b < 0 ? 0 : row - begin[b]);
  }
}

__global__ void __launch_bounds__(kRowThreads) kv_pages_rows_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (row >= p.T) return;
  const int b = row < p.indptr[p.B] ? last_at(p.indptr, p.B, row) : -1;
  write_row(p, row, b, b < 0 ? 0 : row - p.indptr[b]);
}

}  // namespace

cudaError_t plan_kv_pages_assign(const qlin_kv_pages& c, const int32_t* ctx_lens, const int32_t* new_lens, int64_t B, int64_t T,
                                 const int32_t* depths, int32_t* q_indptr, int64_t* positions, int64_t* slots, Prepared* out) {
  Params p = {};
  p.table = c.block_table;
  p.max_pages = c.max_pages;
  p.held = c.held;
  p.free_pages = c.free_pages;
  p.free_count = c.free_count;
  p.pages = static_cast<int32_t>(c.pages);
  while ((int64_t(1) << p.page_shift) < c.page_size) ++p.page_shift;
  p.ctx = ctx_lens;
  p.add = new_lens;
  p.B = static_cast<int32_t>(B);
  p.T = T;
  p.depths = depths;
  p.indptr = q_indptr;
  p.positions = positions;
  p.slots = slots;
  p.err = device_error_word();
  // one block writes some 1000 rows in the time that a second launch takes
  p.rows_inside = B <= kThreads && T <= 2 * kThreads;
  out->count = p.rows_inside ? 1 : 2;
  out->launch[0] = {reinterpret_cast<const void*>(kv_pages_kernel), 1, 1, kThreads, 0};
  out->launch[1] = {reinterpret_cast<const void*>(kv_pages_rows_kernel),
                    static_cast<uint32_t>(std::max<int64_t>(1, (T + kRowThreads - 1) / kRowThreads)), 1, kRowThreads, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace qlin
