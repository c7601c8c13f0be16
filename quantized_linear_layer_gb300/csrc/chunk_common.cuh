// What the chunk attention kernel and its joining kernel share: parameters, which
// token tiles a tile of rows sees, and the division of the work among blocks.
#pragma once

#include "tree_common.cuh"

namespace qlin {
namespace chunk {

constexpr int kTile = 128;  // tokens

using Params = tree::ScoredParams;  // (max_nodes: the most new tokens of a sequence)

// A sequence's bounds as far as they can be used: rows = 0 when they cannot.
struct Sequence {
  int64_t q_row;
  int64_t rows;  // new tokens x query heads of a key head
  int32_t n, ctx, len, prefix;
};

__device__ __forceinline__ Sequence sequence(const Params& p, int b) {
  Sequence s;
  const int32_t q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
  s.q_row = q0;
  s.n = q1 - q0;
  s.ctx = p.ctx_lens[b];
  const int64_t len = static_cast<int64_t>(s.ctx) + s.n;
  const bool fits = q0 >= 0 && q1 >= q0 && q1 <= p.Tq && s.n <= p.max_nodes && s.ctx >= 0 &&
                    len <= (p.max_pages << p.page_shift) && len <= tree::kMaxLen;
  if (!fits) {
    record_device_error(p.err, kDevErrBadIndex);
    s.n = 0;
  }
  s.len = static_cast<int32_t>(len);
  s.prefix = p.prefix != nullptr && s.n > 0 ? max(0, min(p.prefix[b], s.len)) : 0;
  s.rows = static_cast<int64_t>(s.n) * p.group;
  return s;
}

// The new token that a row of a key head belongs to (rows lie below 2^32: a row of q has 128 bytes or more).
__device__ __forceinline__ int32_t token_of(const Params& p, int64_t row) {
  return static_cast<int32_t>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.group));
}

// The token tiles that some row of a tile of rows sees: those of the prefix, 0 .. head - 1, and those of the
// window, next .. next + (count - head) - 1.
struct Tiles {
  int32_t head, next, count;
  __device__ __forceinline__ int32_t at(int32_t i) const { return i < head ? i : next + i - head; }
};

// Of rows first .. last (places among the sequence's new tokens) of a sequence.
__device__ __forceinline__ Tiles tiles_of(const Params& p, const Sequence& s, int32_t first, int32_t last) {
  Tiles t;
  t.head = (s.prefix + kTile - 1) / kTile;
  const int32_t low = p.window > 0 ? max(0, s.ctx + first - p.window + 1) : 0;
  t.next = max(low / kTile, t.head);
  t.count = t.head + max((s.ctx + last) / kTile + 1 - t.next, 0);
  return t;
}

template <int ROWS>
__device__ __forceinline__ int32_t row_tiles(const Sequence& s) {
  return static_cast<int32_t>((s.rows + ROWS - 1) / ROWS);
}

template <int ROWS>
__device__ __forceinline__ Tiles tiles_of_row_tile(const Params& p, const Sequence& s, int32_t row_tile) {
  const int64_t first = static_cast<int64_t>(row_tile) * ROWS, last = min(first + ROWS, s.rows) - 1;
  return tiles_of(p, s, token_of(p, first), token_of(p, last));
}

// Token tiles of all row tiles of one key head of a sequence, by a whole warp.
template <int ROWS>
__device__ __forceinline__ int64_t units_of_head(const Params& p, const Sequence& s) {
  const int lane = threadIdx.x % 32, n = row_tiles<ROWS>(s);
  int64_t sum = 0;
  for (int r = lane; r < n; r += 32) sum += tiles_of_row_tile<ROWS>(p, s, r).count;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Units of sequence b (none from `end` on), each lane its own: short ones are counted by their lanes side by side, so that a
// batch of many sequences costs few turns, long ones by the whole warp.
template <int ROWS>
__device__ __forceinline__ int64_t units_of(const Params& p, int b, int end) {
  constexpr int kShort = 4;  // row tiles
  const int lane = threadIdx.x % 32;
  int n = 0;
  int64_t sum = 0;
  if (b < end) {
    const Sequence s = sequence(p, b);
    n = row_tiles<ROWS>(s);
    if (n <= kShort)
      for (int r = 0; r < n; ++r) sum += tiles_of_row_tile<ROWS>(p, s, r).count;
  }
  __syncwarp();
  for (unsigned longer = __ballot_sync(0xffffffffu, n > kShort); longer != 0; longer &= longer - 1) {
    const int of = __ffs(longer) - 1;
    const int64_t v = units_of_head<ROWS>(p, sequence(p, b - lane + of));
    if (lane == of) sum = v;
  }
  return sum * p.hk;
}

// Walks a block's run of units (token tiles of row tiles of key heads of sequences, in this order), one segment (row
// tile) at a time.
template <int ROWS>
struct Walk {
  int64_t at, end;  // next unit, end of the run
  int32_t b, head, row_tile;
  int32_t tile;     // of this segment, the block's first unit
  int32_t tiles;    // and how many
  Tiles seen;
  // Of these tiles' tokens no row sees the `gap` ones from `hidden` on (in whole sixteens), and those from `high` on.
  int32_t hidden, high;
  uint32_t gap;
  Sequence s;
  int32_t next_tile, next_row_tile;  // where the run goes on

  __device__ __forceinline__ bool next(const Params& p) {
    if (at >= end) return false;
    row_tile = next_row_tile;
    tile = next_tile;
    while (row_tile >= row_tiles<ROWS>(s)) {
      row_tile = 0;
      if (++head >= p.hk || s.rows == 0) {
        head = 0;
        if (++b >= p.B) return false;  // not reached while the lengths stay as they were counted
        s = sequence(p, b);
      }
    }
    seen = tiles_of_row_tile<ROWS>(p, s, row_tile);
    const int64_t row0 = static_cast<int64_t>(row_tile) * ROWS;
    hidden = (s.prefix + 15) & ~15;
    const int32_t low = p.window > 0 ? max(0, s.ctx + token_of(p, row0) - p.window + 1) : 0;
    gap = max((low & ~15) - hidden, 0);
    high = max(s.ctx + token_of(p, min(row0 + ROWS, s.rows) - 1) + 1, s.prefix);
    tiles = static_cast<int32_t>(min(static_cast<int64_t>(seen.count - tile), end - at));
    at += tiles;
    next_tile = 0;
    next_row_tile = row_tile + 1;
    return true;
  }
  __device__ __forceinline__ bool begins() const { return tile == 0; }
  __device__ __forceinline__ bool ends() const { return tile + tiles == seen.count; }
};

// The units before each warp's share of the sequences into scan[WARPS + 1], by all threads of the block.
template <int ROWS, int WARPS>
__device__ __forceinline__ void scan_units(const Params& p, int share, int64_t* scan) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int64_t sum = 0;
  const int end = min(p.B, (warp + 1) * share);
  for (int b0 = warp * share; b0 < end; b0 += 32) sum += units_of<ROWS>(p, b0 + lane, end);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) scan[warp + 1] = sum;
  if (threadIdx.x == 0) scan[0] = 0;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 0; i < WARPS; ++i) scan[i + 1] += scan[i];
  __syncthreads();
}

// Sets *run to the beginning of block `block`'s run, by the warp whose share holds it; every thread of the block calls.
template <int ROWS, int WARPS>
__device__ __forceinline__ void begin_run(const Params& p, int share, const int64_t* scan, int64_t block, int64_t blocks, Walk<ROWS>* run) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t total = scan[WARPS], at = total * block / blocks;
  if (scan[warp] <= at && at < scan[warp + 1]) {
    int64_t rest = at - scan[warp];
    const int b_end = min(p.B, (warp + 1) * share);
    for (int b0 = warp * share; b0 < b_end; b0 += 32) {
      const int64_t units = units_of<ROWS>(p, b0 + lane, b_end);
      int64_t sums = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += x;
      }
      const unsigned holds = __ballot_sync(0xffffffffu, sums > rest);
      if (holds == 0) {
        rest -= __shfl_sync(0xffffffffu, sums, 31);
        continue;
      }
      const int of = __ffs(holds) - 1, b = b0 + of;
      rest -= __shfl_sync(0xffffffffu, sums - units, of);
      const int64_t of_head = __shfl_sync(0xffffffffu, units, of) / p.hk;
      const Sequence s = sequence(p, b);
      const int head = static_cast<int>(rest / of_head);
      rest -= head * of_head;
      const int n = row_tiles<ROWS>(s);
      for (int r0 = 0; r0 < n; r0 += 32) {
        const int count = r0 + lane < n ? tiles_of_row_tile<ROWS>(p, s, r0 + lane).count : 0;
        int64_t upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, upto > rest);
        if (past == 0) {
          rest -= __shfl_sync(0xffffffffu, upto, 31);
          continue;
        }
        if (lane == __ffs(past) - 1) {
          run->at = at;
          run->end = total * (block + 1) / blocks;
          run->b = b;
          run->head = head;
          run->s = s;
          run->next_row_tile = r0 + lane;
          run->next_tile = static_cast<int32_t>(rest - (upto - count));
        }
        break;
      }
      break;
    }
  }
  __syncthreads();
}

// What the joining kernel needs of the segment that the walk stands at, which begins in this block and ends in a later one.
template <int ROWS>
__device__ __forceinline__ tree::Record record_of(const Walk<ROWS>& w, int64_t blocks, int64_t total) {
  const int64_t end = w.at + w.seen.count - w.tile - w.tiles;  // the segment's end, in units
  tree::Record rec;
  rec.last = static_cast<int32_t>((end * blocks - 1) / total);
  rec.head = w.head;
  rec.row_tile = w.row_tile;
  rec.nodes = w.s.n;
  rec.q_row = w.s.q_row;
  return rec;
}

}  // namespace chunk
}  // namespace qlin
