// What the two tree attention kernels share: their parameters, the division of
// the work among blocks, the widening of codes, and the kernel that joins the
// parts of a segment.  The mathematics and the division of the work are
// described in tree_attention.cu.
#pragma once

#include <cmath>

#include "kv_common.cuh"
#include "qlin_internal.h"
#include "tc_common.cuh"

namespace qlin {
namespace tree {

constexpr float kOffset = 13.0f;
constexpr float kSlack = 2.0f;
constexpr float kNoRef = -1e30f;  // before a row has seen anything
constexpr float kHalfExp = -14.0f;
constexpr float kHalfNormal = 6.103515625e-5f;  // 2^-14, the smallest normal fp16
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// What a block leaves for the joining kernel when a segment begins in it and
// ends in a later one.
struct Record {
  int32_t last;  // the block where the segment ends, or -1: nothing to join
  int32_t head, row_tile, nodes;
  int64_t q_row;
};

struct Params {
  const uint8_t* q;
  uint8_t* out;
  int64_t qt, qh, ot, oh;  // strides in bytes
  int32_t hq, hk, group, dtype;
  int64_t Tq;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int64_t page_stride, scale_page_stride;
  int32_t pages, page_shift;
  const int32_t* table;
  int64_t max_pages;
  const int32_t* q_indptr;
  const int32_t* ctx_lens;
  int32_t B;
  const int64_t* mask;
  int32_t mask_words, max_nodes;
  float scale;
  float* lse;
  Record* records;   // [blocks]
  float* part_o;      // [2 blocks][tile_rows][D]
  float2* part_ml;    // [2 blocks][tile_rows]
  int32_t tile_rows;  // rows of a row tile
  int32_t* err;
};

// The longest sequence, nodes included: far enough below 2^31 that the token numbers the kernels form past a sequence's
// end (whole tiles, and the loading warps' 32 boxes of up to 64 tokens) stay in an int32.
constexpr int64_t kMaxLen = 0x7fff0000;

// A sequence's bounds as far as they can be used: nodes = 0 when they cannot.
struct Sequence {
  int64_t q_row;
  int32_t nodes, ctx, len;
  int32_t row_tiles, token_tiles;
};

// In row tiles of ROWS and token tiles of TILE.
template <int ROWS, int TILE>
__device__ __forceinline__ Sequence sequence(const Params& p, int b) {
  Sequence s;
  const int32_t q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
  s.q_row = q0;
  s.nodes = q1 - q0;
  s.ctx = p.ctx_lens[b];
  const int64_t len = static_cast<int64_t>(s.ctx) + s.nodes;
  const bool fits = q0 >= 0 && q1 >= q0 && q1 <= p.Tq && s.nodes <= p.max_nodes && s.ctx >= 0 &&
                    len <= (p.max_pages << p.page_shift) && len <= kMaxLen;
  if (!fits) {
    record_device_error(p.err, kDevErrBadIndex);
    s.nodes = 0;
  }
  s.len = static_cast<int32_t>(len);
  s.row_tiles = (s.nodes * p.group + ROWS - 1) / ROWS;
  s.token_tiles = (s.len + TILE - 1) / TILE;
  if (s.nodes == 0) s.row_tiles = 0;
  return s;
}

__device__ __forceinline__ int64_t units(const Params& p, const Sequence& s) {
  return s.row_tiles == 0 ? 0 : static_cast<int64_t>(p.hk) * s.row_tiles * s.token_tiles;
}

// Walks a block's run of units, one segment at a time.
template <int ROWS, int TILE>
struct Walk {
  int32_t b;
  int64_t at, end;     // next unit, end of the run
  int64_t first;       // first unit of sequence b
  Sequence s;
  // the segment's part that is this block's
  int32_t head, row_tile, tile, tiles;

  __device__ __forceinline__ bool next(const Params& p) {
    if (at >= end) return false;
    int64_t n = units(p, s);
    while (at - first >= n) {
      first += n;
      if (++b >= p.B) return false;  // not reached while the lengths stay as they were counted
      s = sequence<ROWS, TILE>(p, b);
      n = units(p, s);
    }
    const int64_t i = at - first;
    const int32_t seg = static_cast<int32_t>(i / s.token_tiles);
    tile = static_cast<int32_t>(i - static_cast<int64_t>(seg) * s.token_tiles);
    head = seg / s.row_tiles;
    row_tile = seg - head * s.row_tiles;
    tiles = static_cast<int32_t>(min(static_cast<int64_t>(s.token_tiles - tile), end - at));
    at += tiles;
    return true;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The exponent e, in [-126, 113], for which 2^-e puts the largest magnitude of a
// row of 16-bit numbers (`top`, the bits of a float32) into [2^14, 2^15), or
// below it for rows of less than 2^-112; 0 for rows of zeros and rows that hold
// an infinity or a NaN.
__device__ __forceinline__ int row_exponent(uint32_t top) {
  if (top == 0 || top >= 0x7f800000u) return 0;
  return max(static_cast<int>(top >> 23) - 127 - 14, -126);
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

constexpr uint32_t kMagic = 0x64006400u;      // 1024 in both halves: 1024 + n is 0x6400 | n
constexpr uint32_t kInt8Bias = 0x64806480u;   // 1024 + 128

// Four 8-bit codes of one row as two fp16 pairs (codes 0, 1 and 2, 3).
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == QLIN_KV_INT8) {
    w ^= 0x80808080u;  // n + 128, unsigned
    lo = hsub2(__byte_perm(w, kMagic, 0x7170), kInt8Bias);
    hi = hsub2(__byte_perm(w, kMagic, 0x7372), kInt8Bias);
  } else {
    lo = kv::e4m3x2_to_half2(static_cast<uint16_t>(w));
    hi = kv::e4m3x2_to_half2(static_cast<uint16_t>(w >> 16));
  }
}

template <int BYTES>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t* w) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

// The kernels fold log2(sv) of a value scale into the exponent, so they work with scales in [kLeastScale, kMostScale]
// and a factor for each token: sv = usable scale x factor, t and l from the usable scale, P multiplied by the factor
// before it is rounded.  The factor is 1 but for scales that are negative (-1), zero (0), outside the bounds (below: less
// than 1, down to 2^-58 for the smallest subnormal) or not numbers; tiles without such a scale skip it.  A zero (or what
// is not a number) stands at 2^-64, the smallest scale that the cache write gives.  With the lower bound l stays below
// 2^127 for 2^21 tokens of such scales at equal weights, and P of a row of subnormal scales alone keeps its bits.  (A token's
// share of l is lost when its usable scale lies 2^117 or more below that of the token that weighs most.)
constexpr uint32_t kLeastScale = 0x12000000u, kMostScale = 0x7e800000u;  // 2^-91 and 2^126, as bits

template <int FMT>
__device__ __forceinline__ bool odd_scale(uint32_t word) {
  if constexpr (FMT == QLIN_KV_U4) return (word & 0xffffu) - 1u > 0x7bffu - 1u;  // fp16: all positive numbers are usable
  else return word - kLeastScale > kMostScale - kLeastScale;
}

// The scale word with a usable scale in place of an odd one; the factor goes to `factor`.
template <int FMT>
__device__ __forceinline__ uint32_t usable_scale(uint32_t word, float& factor) {
  if constexpr (FMT == QLIN_KV_U4) {
    const uint32_t a = word & 0x7fffu;
    const uint32_t u = a == 0 || a >= 0x7c00u ? 1u : a;  // 2^-24 for what has no logarithm
    factor = __half2float(__ushort_as_half(static_cast<unsigned short>(word))) /
             __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
    return (word & 0xffff0000u) | u;
  } else {
    const uint32_t a = word & 0x7fffffffu;
    const uint32_t u = a == 0 || a >= 0x7f800000u ? 0x1f800000u : min(max(a, kLeastScale), kMostScale);
    factor = __uint_as_float(word) / __uint_as_float(u);
    return u;
  }
}

// Whether the zero-point of a U4 scale word is none: not a whole number from 0 to 15 (1024 + n, n < 16, is 0x6400 | n).
__device__ __forceinline__ bool odd_zero(uint32_t word) {
  const __half z = __ushort_as_half(static_cast<unsigned short>(word >> 16)), big = __float2half_rn(1024.0f);
  const __half b = __hadd(z, big);
  return __half_as_ushort(b) - 0x6400u > 15u || !__heq(__hsub(b, big), z);
}

// One thread's look at 16 bytes of E4M3 codes in shared memory: those that are NaN become 0 there; whether there were any.
// (A product with a probability of 0 keeps a NaN, so what nobody sees must not hold one.)
__device__ __forceinline__ bool clear_nan_codes(uint32_t at) {
  const uint4 u = tc::lds128(at);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t bad[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) bad[i] = __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
  if ((bad[0] | bad[1] | bad[2] | bad[3]) == 0) return false;
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0] & ~bad[0]), "r"(w[1] & ~bad[1]), "r"(w[2] & ~bad[2]),
               "r"(w[3] & ~bad[3])
               : "memory");
  return true;
}

// 16 bytes from global to shared memory, asynchronously, or zeros (bytes = 0: nothing is read); streamed codes leave L2
// first.
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(to), "l"(from), "r"(bytes), "l"(policy)
               : "memory");
}
// Arrives on `bar` (one of its expected arrivals) once this thread's copies so far are there.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A box without a page: behind its sequence's end, where nobody sees its tokens, or with a page number out of range.  Its
// codes and scales are zeros, as the cache read gives them, so that nothing the stage held before reaches a result.
constexpr int32_t kNoPage = -1;

// A page number as the table has it, checked.
__device__ __forceinline__ int32_t checked_page(const Params& p, int32_t page) {
  if (page >= 0 && page < p.pages) return page;
  record_device_error(p.err, kDevErrBadIndex);
  return kNoPage;
}

// One warp's copies of the scales of TOKENS tokens of a key head, from `first` on, into a stage of a ring.  `ahead` is
// the page (or kNoPage) of box `lane` of the 32 boxes of `box` tokens that hold the stage's boxes `at` ...
template <int TOKENS>
__device__ __forceinline__ void copy_scales(const Params& p, int head, int first, int box, int32_t ahead, int at,
                                            uint32_t ks_to, uint32_t vs_to, uint64_t policy) {
  constexpr int kLanes = TOKENS / 4;  // four tokens each: the scales of K, then as many lanes for those of V
  static_assert(2 * kLanes <= 32, "lanes");
  const int lane = threadIdx.x % 32;
  const int token = lane % kLanes * 4;
  const int32_t pg = __shfl_sync(0xffffffffu, ahead, (at + token / box) & 31);
  if (lane >= 2 * kLanes) return;
  const bool k = lane < kLanes;
  const int64_t row = (static_cast<int64_t>(head) << p.page_shift) + ((first + token) & ((1 << p.page_shift) - 1));
  copy16((k ? ks_to : vs_to) + token * 4, (k ? p.k_scale : p.v_scale) + max(pg, 0) * p.scale_page_stride + row * 4,
         pg < 0 ? 0 : 16, policy);
}

// One warp's copies of the codes of TOKENS tokens, page by page, box by box of BOX tokens; the other arguments are those
// of copy_scales, and row_at(r, c) says where 16-byte chunk c of row r lies (its swizzle repeats after eight rows).  The
// rows of a box are contiguous in its page, so a lane's chunks are 512 bytes apart and everything but the page's address
// is known beforehand: the copies of a stage take the warp few instructions (with the box a variable and four copies at
// once, a decode batch took 163 us instead of 149).  A thread's copies arrive in order, which the turns at the ring rest on
// (stage_ring.h); boxes copied through tensor maps, at the same speed, arrive in any.
template <int TOKENS, int BOX, int ROW_BYTES, class RowAt>
__device__ __forceinline__ void copy_codes(const Params& p, int head, int first, int32_t ahead, int at, uint32_t k_to,
                                           uint32_t v_to, uint64_t policy, RowAt row_at) {
  constexpr int kChunks = ROW_BYTES / 16;  // of a row
  constexpr int kRowsAtOnce = 32 / kChunks;
  constexpr int kPeriod = kRowsAtOnce < 8 ? 8 / kRowsAtOnce : 1;
  const int lane = threadIdx.x % 32;
  uint32_t to[kPeriod];
#pragma unroll
  for (int i = 0; i < kPeriod; ++i) to[i] = row_at(i * kRowsAtOnce + lane / kChunks, lane % kChunks);
  const uint32_t step = row_at(kPeriod * kRowsAtOnce, 0);
#pragma unroll
  for (int b = 0; b < TOKENS / BOX; ++b) {
    const int32_t pg = __shfl_sync(0xffffffffu, ahead, (at + b) & 31);
    const uint32_t bytes = pg < 0 ? 0 : 16;
    const int64_t row = (static_cast<int64_t>(head) << p.page_shift) + ((first + b * BOX) & ((1 << p.page_shift) - 1));
    const int64_t codes = max(pg, 0) * p.page_stride + row * ROW_BYTES + lane * 16;
    const uint8_t* k = p.k + codes;
    const uint8_t* v = p.v + codes;
#pragma unroll
    for (int x = 0; x < BOX / kRowsAtOnce; ++x) {
      const int y = b * (BOX / kRowsAtOnce) + x;
      const uint32_t at16 = to[y % kPeriod] + y / kPeriod * step;
      copy16(k_to + at16, k + x * 512, bytes, policy);
      copy16(v_to + at16, v + x * 512, bytes, policy);
    }
  }
}

// The units before each thread's share of the sequences, into scan[THREADS + 1]
// (share b .. b + share - 1 of thread b / share), by all threads of the block.
template <int ROWS, int TILE, int THREADS>
__device__ __forceinline__ void scan_units(const Params& p, int share, int64_t* scan) {
  int64_t sum = 0;
  for (int b = threadIdx.x * share; b < min(p.B, static_cast<int>(threadIdx.x + 1) * share); ++b)
    sum += units(p, sequence<ROWS, TILE>(p, b));
  scan[threadIdx.x + 1] = sum;
  if (threadIdx.x == 0) scan[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t carry = 0;
    for (int i = 0; i < THREADS; i += 32) {
      int64_t v = scan[1 + i + lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      v += carry;
      scan[1 + i + lane] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
}

// The run of units of block `block` of `blocks`.
template <int ROWS, int TILE, int THREADS>
__device__ __forceinline__ Walk<ROWS, TILE> begin_run(const Params& p, int share, const int64_t* scan, int64_t block,
                                                      int64_t blocks) {
  Walk<ROWS, TILE> run;
  const int64_t total = scan[THREADS];
  run.at = total * block / blocks;
  run.end = total * (block + 1) / blocks;
  int lo = 0, hi = THREADS;  // the last share that begins at or before the run
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (scan[mid] <= run.at) lo = mid; else hi = mid;
  }
  run.b = lo * share;
  run.first = scan[lo];
  run.s = sequence<ROWS, TILE>(p, run.b);
  return run;
}

// What the joining kernel needs of the segment that the walk stands at, which
// begins in this block and ends in a later one.
template <int ROWS, int TILE>
__device__ __forceinline__ Record record_of(const Walk<ROWS, TILE>& w, int64_t blocks, int64_t total) {
  const int64_t end = w.at - w.tiles + w.s.token_tiles;  // the segment's end, in units
  Record rec;
  rec.last = static_cast<int32_t>((end * blocks - 1) / total);
  rec.head = w.head;
  rec.row_tile = w.row_tile;
  rec.nodes = w.s.nodes;
  rec.q_row = w.s.q_row;
  return rec;
}

// Joins the parts of a segment that begins in block `blockIdx.x` of the first
// kernel and ends in a later one: one row per block, its parts dealt to the
// warps, D / 4 lanes' worth of float4 each.
template <int D>
static __global__ void __launch_bounds__(128) tree_attention_join_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4 < 32 ? D / 4 : 32;  // lanes that cover a row once
  constexpr int kWide = D / 4 / kLanes;            // float4 a lane
  constexpr int kTeams = 128 / kLanes;
  __shared__ float4 part[kTeams][D / 4];
  __shared__ float2 part_ml[kTeams];
  pdl_wait();
  pdl_launch_dependents();
  const Record rec = p.records[blockIdx.x];
  if (rec.last < 0) return;
  const int row = blockIdx.y;
  const int at = rec.row_tile * p.tile_rows + row;
  const int node = at / p.group;
  if (node >= rec.nodes) return;
  const int team = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int count = rec.last - static_cast<int>(blockIdx.x) + 1;

  float m = -INFINITY, l = 0.0f;
  float4 o[kWide];
#pragma unroll
  for (int i = 0; i < kWide; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = team; i < count; i += kTeams) {
    const int64_t slot = 2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0);
    const float2 e = p.part_ml[slot * p.tile_rows + row];
    const float4* src = reinterpret_cast<const float4*>(p.part_o + (slot * p.tile_rows + row) * D) + lane;
    float4 v[kWide];
#pragma unroll
    for (int x = 0; x < kWide; ++x) v[x] = src[x * kLanes];
    const float to = fmaxf(m, e.x);
    const float fa = m == -INFINITY ? 1.0f : ex2(m - to), fb = e.x == -INFINITY ? 1.0f : ex2(e.x - to);
    m = to;
    l = l * fa + e.y * fb;
#pragma unroll
    for (int x = 0; x < kWide; ++x) {
      o[x].x = o[x].x * fa + v[x].x * fb;
      o[x].y = o[x].y * fa + v[x].y * fb;
      o[x].z = o[x].z * fa + v[x].z * fb;
      o[x].w = o[x].w * fa + v[x].w * fb;
    }
  }
#pragma unroll
  for (int x = 0; x < kWide; ++x) part[team][lane + x * kLanes] = o[x];
  if (lane == 0) part_ml[team] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= D / 4) return;
  float top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kTeams; ++i) top = fmaxf(top, part_ml[i].x);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kTeams; ++i) {
    const float f = part_ml[i].x == -INFINITY ? 1.0f : ex2(part_ml[i].x - top);
    const float4 v = part[i][threadIdx.x];
    sum += f * part_ml[i].y;
    acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
  }
  const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
  const int head = rec.head * p.group + at - node * p.group;
  const int64_t tok = rec.q_row + node;
  const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  const uint2 u = p.dtype == QLIN_BF16 ? make_uint2(kv::pack2<1>(v[0], v[1]), kv::pack2<1>(v[2], v[3]))
                                        : make_uint2(kv::pack2<0>(v[0], v[1]), kv::pack2<0>(v[2], v[3]));
  *reinterpret_cast<uint2*>(p.out + tok * p.ot + head * p.oh + threadIdx.x * 8) = u;
  if (p.lse != nullptr && threadIdx.x == 0) p.lse[tok * p.hq + head] = (lg2(sum) + (top - kOffset)) * kLn2;
}


// Which of the two kernels takes a call (tree_attention.cu).
bool use_wide(int64_t head_dim, int64_t rows);
int wide_blocks();
cudaError_t plan_wide(const Params& p, int fmt, int64_t head_dim, Prepared* out);

}  // namespace tree
}  // namespace qlin
