// Attention of a chunk of new tokens of each sequence over a paged, quantized
// key / value cache that holds them already, on the tcgen05 tensor cores: causal, with
// a prefix that every row sees, a window, capped scores and a bias by distance.
//
// Mathematics: as in tree_attention.cu, with k_j = sk_j n_j and v_j = sv_j u_j
//   t_ij = log2(e) f(scale sk_j (q_i . n_j)) + log2(sv_j)
//   o_i  = sum_j 2^(t_ij - m_i) u_j / sum_j 2^(t_ij - m_i) / sv_j
// f the cap and the bias.  The codes go to the tensor cores as they are; rows of
// bf16 q that fp16 cannot hold are scaled by a power of two; P = 2^(t - m) is
// rounded to fp16's 11 bits, the one rounding of an operand (below 2^-33 of the row's
// largest it becomes 0).  The reference m_i follows the running maximum lazily: P
// may grow to 2^15 before it moves and the row of O is rescaled.
// The cap is c tanh(s / c) = c (1 - 2 / (1 + 2^(2 log2(e) s / c))); caps above 256, for which that
// loses small scores, have a variant of the kernel with tanh's power series.
//
// Work.  The rows of a key head (token, query head of the group) are cut into
// tiles of 256 (128 for heads of 256), and of the tokens the tiles of 128 that some
// of these rows see are taken.  All (sequence, key head, row tile, token tile) units in
// this order are dealt out evenly to one block per SM, on the device, from the
// lengths; a segment (row tile) cut by a block's border leaves float32 parts
// that a second kernel joins.  So one long prompt, ragged batches and single
// tokens over long contexts load the GPU alike, and a captured call stays right when
// lengths change.
//
// A block has 16 warps, whose registers are dealt out anew by role:
//   0-7    softmax, one thread a row: warps 0-3 the tile's first 128 rows (stream
//          0), 4-7 the others (stream 1); heads of 256 have one stream and two
//          threads a row, 64 tokens each
//   8-11   load codes and scales into registers, a tile ahead, and widen them to fp16
//          in shared memory, in the tensor core's layout: one widening for 256 rows
//   12-13  issue the products of a stream each (one thread)
// Per token tile and stream: S = q n^T into the stream's tensor-memory buffer, which the
// softmax threads turn into P over the same columns; O += P u takes P from there
// and u as it lies (tokens x channels).  A tile's 64 first and 64 last tokens are
// handed over separately: while the softmax has one half, P u of the other and
// then S of the next tile's go through the tensor cores, so that its threads find their
// next scores there (S of 64 tokens costs 54 of the 64 cycles that 128 take, but
// waiting for whole tiles took longer: 3559 -> 3118 us in the case below).  One
// stream: S has two buffers in turn.
// Tensor memory: S/P 2 x 128 columns, O 2 x D (1 x 256).
//
// Bound: the instructions of the softmax and of the widening, and what they wait
// for one another; neither DRAM nor the tensor cores.  8192 tokens behind 16384 (32 query heads on
// 8 of 128, INT8): 2861 us, 961 TFLOP/s, half of what a large product reaches; a
// tile of 256 rows x 128 tokens takes about 5000 cycles, of which the
// products are 2750 (2048 with whole tiles), the exponentials 1024, and issue slots are
// used in 0.53 of the cycles (0.36 tensor, 0.18 exponentials busy).  What has been
// measured: 32 scores at a time instead of 64 3103 us (a step's maximum and vote cost the
// same); 16 softmax warps 3937; one warp for both streams' products 3559; values'
// scales in the exponent 3669.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "chunk_common.cuh"
#include "stage_ring.h"

namespace qlin {
namespace chunk {
namespace {

using namespace tree;  // the widening of codes, scales, pairs of float32
using chunk::Params;
using chunk::Sequence;

constexpr int kSoftmaxWarps = 8;
constexpr int kCols = 4;                            // buffers of the tokens' scales: see the widening warps
constexpr uint32_t kTmemO = 256;

template <int FMT, int D>
struct Geo {
  static constexpr bool kU4 = FMT == QLIN_KV_U4;
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kSubs = 2 / kStreams;  // threads of a row
  static constexpr int kHalves = kStreams;     // a thread takes a tile's scores 64 at a time
  static constexpr int kMine = D / kSubs;      // channels of q and o of each
  static constexpr int kRows = 128 * kStreams;
  static constexpr int kBufs = D == 256 ? 1 : 2;  // of K and of V
  // Warps, whole groups of four, and their registers: what all are launched with is dealt out anew by role.
  static constexpr int kWidenWarps = 4, kMmaWarp = kSoftmaxWarps + kWidenWarps;
  static constexpr int kWarps = kMmaWarp + 4, kThreads = 32 * kWarps, kActive = 32 * (kMmaWarp + kStreams);
  static constexpr int kLaunchRegs = 128;
  // (No role spills at these.  Sixteen bytes of one role's cost 5 % of the time: 72 registers for the products instead of 64 took
  // 4 prompts of 2048 tokens behind 8192 with E4M3 codes from 1140 to 1096 us; INT8 codes and heads of 128 spill at 72, not at 64.)
  static constexpr int kSoftmaxRegs = D == 256 ? 104 : 136, kWidenRegs = D == 256 ? 232 : 168;
  static constexpr int kOtherRegs = FMT == QLIN_KV_INT8 && D == 128 ? 64 : 72;
  static_assert(kSoftmaxWarps * kSoftmaxRegs + kWidenWarps * kWidenRegs + 4 * kOtherRegs <= kWarps * kLaunchRegs, "registers");
  static constexpr int kParts = kTile / 16 / kWidenWarps;  // 16 tokens each, of a widening warp
  static constexpr int kRowBytes = kU4 ? D / 2 : D;
  static constexpr int kBlocks = D / 64;            // 64-channel blocks of 128 rows x 128 bytes
  static constexpr int kOperand = kBlocks * 16384;  // 128 rows of q, K or V in fp16
  static constexpr uint32_t kOCols = D;             // tensor memory columns of a stream's O
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kStreams * kOperand;
  static constexpr int kOffV = kOffK + kBufs * kOperand;
  static constexpr int kOffCol = kOffV + kBufs * kOperand;             // [kCols][scale sk, sv][128]
  static constexpr int kOffPair = kOffCol + kCols * 2 * kTile * 4;     // [32 tokens, in turn][thread of the row][row]
  static constexpr int kOffQmax = kOffPair + 2 * kSubs * 128 * 4;      // [thread of the row][row]
  static constexpr int kOffEnd = kOffQmax + kSubs * 128 * 4;           // [segment parity][thread of the row][row] l
  static constexpr int kOffRow = kOffEnd + 2 * kSubs * 128 * 4;  // [segment parity][softmax thread] RowOf
  static constexpr int kOffBar = kOffRow + 2 * 32 * kSoftmaxWarps * 16;
  static constexpr int kBars = 4 * kBufs + 3 * 4 + kStreams + 1 + kCols;
  static constexpr int kOffMisc = (kOffBar + kBars * 8 + 15) / 16 * 16;  // tensor memory address, flags, exponents
  static constexpr int kOffScan = kOffMisc + 32 + kCols * 16;
  static constexpr int kOffWalk = (kOffScan + (kWarps + 1) * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffWalk + (kMmaWarp + kStreams + 1) * static_cast<int>(sizeof(Walk<kRows>)) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kTmemO + kStreams * kOCols <= 512, "tensor memory");
};

// Tokens that are of the prefix, or from `low` to `high`.
struct Range {
  int32_t prefix, low, high;
};

// The first tokens of the spans of `width` that some row of positions first .. last sees a token of (none if there is no row).
__device__ __forceinline__ Range some_seen(const Params& p, const Sequence& s, int32_t first, int32_t last, int32_t width, bool live) {
  return {live ? s.prefix : 0, p.window > 0 ? first - p.window + 2 - width : INT32_MIN, live ? last : -1};
}
// The first tokens of the spans of `width` that all these rows see all of.
__device__ __forceinline__ Range all_seen(const Params& p, const Sequence& s, int32_t first, int32_t last, int32_t width) {
  return {s.prefix - width + 1, p.window > 0 ? last - p.window + 1 : INT32_MIN, first - width + 1};
}
__device__ __forceinline__ bool within(const Range& r, int32_t j) { return j < r.prefix || (j >= r.low && j <= r.high); }

// That of a stream (its 128 rows of a row tile) for a tile.
template <int ROWS>
__device__ __forceinline__ Range stream_sees(const Params& p, const Walk<ROWS>& w, int x) {
  const int64_t row = static_cast<int64_t>(w.row_tile) * ROWS + x * 128;
  const int32_t first = w.s.ctx + token_of(p, min(row, w.s.rows - 1)), last = w.s.ctx + token_of(p, min(row + 127, w.s.rows - 1));
  return some_seen(p, w.s, first, last, kTile, row < w.s.rows);
}

// What a softmax thread knows of a segment until it writes its row, kept in shared memory: in registers it would take the
// scores'.
struct RowOf {
  int64_t token;  // the row of q and out; -1: none
  int32_t head;   // query head
  int32_t flags;  // 1: the segment begins in this block, 2: it ends in it
};

// Loads that stay where they are written: moved ahead of their use, they would take the registers that the scores need.
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// tc::mbar_wait_quiet in fewer instructions: the loops of all roles have to stay in the instruction cache together.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, int32_t* err, int site) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  uint32_t tries = 0;
#pragma unroll 1
  do {
    if (tc::mbar_try_wait(bar, parity)) return true;
  } while ((++tries & 255) != 0 || clock64() - t0 <= tc::kWaitTimeoutCycles);
  record_device_error(err, kDevErrTimeoutBase + site);
  return false;
}

// Forms of the scores: plain ones (with a window and a prefix or without); a cap or a bias; a cap that large_capped() takes.
enum { kPlainScores, kShaped, kLargeCap };

struct WaitOps {  // for stage_ring.h's wait_or_raise
  volatile uint32_t* flag;
  __device__ __forceinline__ void raise() { *flag = 1; }
};

template <int FMT, int D, int SHAPED>
__global__ void __launch_bounds__(Geo<FMT, D>::kThreads, 1) chunk_attention_kernel(const __grid_constant__ Params p) {
  using G = Geo<FMT, D>;
  constexpr int kRows = G::kRows, kStreams = G::kStreams, kSubs = G::kSubs, kBufs = G::kBufs;
  constexpr int kWidenWarps = G::kWidenWarps, kMmaWarp = G::kMmaWarp, kWarps = G::kWarps;
  using W = Walk<kRows>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - tc::smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const uint32_t bars = base + G::kOffBar;
  const uint32_t k_full = bars, k_free = k_full + 8 * kBufs;                       // [kBufs]
  const uint32_t v_full = k_free + 8 * kBufs, v_free = v_full + 8 * kBufs;         // [kBufs]
  // two streams: S, P and P u of stream x and half h of the tokens at 2 x + h; one stream: of two buffers in turn
  const uint32_t s_full = v_free + 8 * kBufs, p_full = s_full + 32, pv_done = p_full + 32;  // [4] each
  const uint32_t q_full = pv_done + 32;  // [kStreams]
  const uint32_t all_done = q_full + 8 * kStreams;
  const uint32_t col_full = all_done + 8;  // [kCols]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::kOffMisc);
  volatile uint32_t* ran_out = tmem_slot + 1;  // a wait of some role of the block ran out
  volatile uint32_t* odd_tile = tmem_slot + 2;  // [kCols]: 1 + the last tile with a value scale that is not finite
  int32_t* top_exp = reinterpret_cast<int32_t*>(smem + G::kOffMisc + 32);  // [kCols][widening warp]: all its |sv| are below 2^this
  int64_t* scan = reinterpret_cast<int64_t*>(smem + G::kOffScan);
  W* walks = reinterpret_cast<W*>(smem + G::kOffWalk);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBufs; ++i) {
      tc::mbar_init(k_full + 8 * i, kWidenWarps);
      tc::mbar_init(k_free + 8 * i, kStreams);
      tc::mbar_init(v_full + 8 * i, kWidenWarps);
      tc::mbar_init(v_free + 8 * i, kStreams);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(s_full + 8 * i, 1);
      tc::mbar_init(p_full + 8 * i, kSoftmaxWarps / kStreams);
      tc::mbar_init(pv_done + 8 * i, 1);
    }
    for (int i = 0; i < kStreams; ++i) tc::mbar_init(q_full + 8 * i, kSoftmaxWarps / kStreams);
    tc::mbar_init(all_done, kStreams);
    for (int i = 0; i < kCols; ++i) {
      tc::mbar_init(col_full + 8 * i, kWidenWarps);
      odd_tile[i] = 0;
    }
    *ran_out = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int share = (p.B + kWarps - 1) / kWarps;
  scan_units<kRows, kWarps>(p, share, scan);
  const int64_t total = scan[kWarps];
  const int64_t blocks = min(static_cast<int64_t>(gridDim.x), total);  // each of these has a unit or more
  if (threadIdx.x == 0) p.records[blockIdx.x].last = -1;
  if (blockIdx.x >= blocks) return;
  W* origin = walks + kMmaWarp + kStreams;
  begin_run<kRows, kWarps>(p, share, scan, blockIdx.x, blocks, origin);
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // In every role a wait that runs out makes it go on without waiting, so that all loops end and every barrier among
  // threads is met.
  bool dead = false;
  WaitOps ops = {ran_out};
  auto wait = [&](uint32_t bar, uint32_t parity, int site) {
    ring::wait_or_raise(ops, dead, [&]() { return wait_on(bar, parity & 1, p.err, site); });
  };
  // One lane steps a walk in shared memory.
  auto next = [&](W& w) {
    bool more = false;
    __syncwarp();
    if (lane == 0) more = w.next(p);
    __syncwarp();
    return __shfl_sync(0xffffffffu, more, 0) != 0;
  };

  if (warp >= kMmaWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
  if (warp >= kMmaWarp && warp < kMmaWarp + kStreams) {
    // ---------------- products: a warp for each stream ----------------
    // The whole warp runs the loop, so that addresses and descriptors stay in uniform registers; one thread issues.
    const bool leader = elect_one();
    const uint32_t x = warp - kMmaWarp;
    const uint32_t idesc_s = tc::idesc_f16(128, kTile / G::kHalves, 0);
    const uint32_t idesc_o = tc::idesc_f16(128, D, 0) | (1u << 16);  // B with n contiguous
    // a descriptor's address field counts 16 bytes and does not overflow below 256 KB: advancing is an addition
    const uint64_t q_desc = tc::sw128_kmajor_desc(base + G::kOffQ + x * G::kOperand), k_desc = tc::sw128_kmajor_desc(base + G::kOffK);
    const uint64_t v_desc = sw128_nmajor_desc(base + G::kOffV, 16384);
    W& w = walks[warp];
    if (lane == 0) w = *origin;
    asm volatile("bar.sync 15, %0;" ::"n"(G::kActive) : "memory");
    uint32_t t = 0, seg = 0;
    int left = 0, i = 0, prefix_tiles = 0, next_tile = 0;
    Range seen = {};
    bool begun = false;
    bool on = false, first = false;  // whether the tile before has products; whether its P u begins O
    // Two streams: for each half of the tokens, P u of the tile before and S of this one, over P's columns: the softmax threads
    // have the other half meanwhile.  One stream: S of this tile, then P u of the one before, which the softmax threads have
    // turned into P meanwhile.
#pragma unroll 1
    while (true) {
      bool more = left > 0, fresh = false;
      if (!more) {
        more = fresh = next(w);
        if (more) {
          left = w.tiles;
          i = w.tile;
          prefix_tiles = w.seen.head;
          next_tile = w.seen.next - w.seen.head;
          seen = stream_sees(p, w, x);
        }
      }
      const uint32_t kb = t % kBufs, vb = (t - 1) % kBufs;
      const bool here = more && within(seen, (i < prefix_tiles ? i : next_tile + i) * kTile);
#pragma unroll 1
      for (uint32_t h = 0; h < static_cast<uint32_t>(G::kHalves); ++h) {
        auto weighted = [&]() {  // P u of tile t - 1
          const uint32_t bar = kStreams == 2 ? 2 * x + h : (t - 1) & 1;
          wait(p_full + 8 * bar, kStreams == 2 ? t - 1 : (t - 1) >> 1, 0x71);
          if (h == 0) wait(v_full + 8 * vb, (t - 1) / kBufs, 0x72);
          dead = __any_sync(0xffffffffu, dead);
          tc::tc_fence_after();
          if (leader) {
            if (!dead && on) {
              constexpr int kProducts = kTile / 16 / G::kHalves;
              const uint64_t vd = v_desc + vb * (G::kOperand >> 4) + h * (kProducts * 128);
              const uint32_t pt = tmem + (kStreams == 2 ? x : (t - 1) & 1) * 128 + h * 64, ot = tmem + kTmemO + x * G::kOCols;
              const uint32_t keep = h > 0 || !first ? 1u : 0u;
#pragma unroll
              for (int k = 0; k < kProducts; ++k)  // P of 32 tokens lies over the first half of their scores
                tc::mma_f16_ta(ot, pt + 32 * (k >> 1) + 8 * (k & 1), vd + k * 128, idesc_o, k > 0 ? 1u : keep);
            }
            tc::mma_commit(pv_done + 8 * bar);
            if (h == G::kHalves - 1) tc::mma_commit(v_free + 8 * vb);
          }
          __syncwarp();
        };
        if (kStreams == 2 && t > 0) weighted();
        if (more) {
          const uint32_t bar = kStreams == 2 ? 2 * x + h : t & 1;
          if (h == 0) {
            if (fresh) wait(q_full + 8 * x, seg, 0x73);
            wait(k_full + 8 * kb, t / kBufs, 0x74);
          }
          if (t >= (kStreams == 2 ? 1 : 2)) wait(pv_done + 8 * bar, kStreams == 2 ? t - 1 : (t - 2) >> 1, 0x75);
          dead = __any_sync(0xffffffffu, dead);
          tc::tc_fence_after();
          if (leader) {
            if (!dead && here) {
              const uint64_t kd = k_desc + kb * (G::kOperand >> 4) + h * 512;  // 64 rows of 128 bytes
              const uint32_t st = tmem + (kStreams == 2 ? x : t & 1) * 128 + h * 64;
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * 1024 + (k & 3) * 2;
                tc::mma_f16(st, q_desc + off, kd + off, idesc_s, k > 0 ? 1u : 0u);
              }
            }
            tc::mma_commit(s_full + 8 * bar);
            if (h == G::kHalves - 1) tc::mma_commit(k_free + 8 * kb);
          }
          __syncwarp();
        }
        if (kStreams == 1 && t > 0) weighted();
      }
      if (!more) break;
      if (fresh) {
        ++seg;
        begun = false;
      }
      on = here;
      first = !begun;
      begun = begun || here;
      ++t;
      --left;
      ++i;
    }
    // every product is done before the tensor memory is given back, whatever else ran out
    if (leader) tc::mma_commit(all_done);
    __syncwarp();
    tc::mbar_wait_quiet(all_done, 0, p.err, 0x76);
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // (fills up the group)
  } else if (warp >= kSoftmaxWarps) {
    // ---------------- loads and widening ----------------
    if constexpr (G::kWidenRegs > G::kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kWidenRegs));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kWidenRegs));
    constexpr int kParts = G::kParts;
    const int part0 = (warp - kSoftmaxWarps) * kParts;  // this warp's tokens of a tile: 16 each, which lie on one page
    W& w = walks[warp];
    if (lane == 0) w = *origin;
    asm volatile("bar.sync 15, %0;" ::"n"(G::kActive) : "memory");
    // A lane takes 16 bytes of codes of one row at a time and makes kPieces 16-byte chunks of fp16 of them.  Rows and
    // chunks are dealt to lanes such that, for each piece, the eight lanes of a quarter warp write to eight different bank
    // groups, and a lane's row is the same modulo 8 throughout, so that its addresses differ by constants (heads of 256 are
    // two halves of 128 channels, D2):
    //   rows of 128 bytes: rows r, r ^ 5 x four chunks, one row's of one 64-channel block, the other's of the other
    //   rows of 64 bytes, two blocks (U4): rows 0 1 | 6 7 or 2 3 | 4 5 x two chunks of one block | of the other
    //   rows of 64 or 32 bytes, one block: consecutive rows
    constexpr int D2 = D == 256 ? 128 : D, kHalves = D / D2;
    constexpr int kHalfBytes = G::kU4 ? D2 / 2 : D2;  // of a row
    constexpr int kBlocks2 = D2 / 64;
    constexpr int kBlockBytes = kHalfBytes / kBlocks2;  // of a row's codes in one 64-channel block
    constexpr int kPieces = G::kU4 ? 4 : 2;
    constexpr bool kPairs = kHalfBytes == 128, kFours = G::kU4 && kBlocks2 == 2;
    constexpr int kRowsAtOnce = kHalfBytes == 32 || kFours ? 16 : 8;
    constexpr int kLoads = kHalves * 16 / kRowsAtOnce * kBlocks2;  // of 16 bytes, a lane's of K (of V) in a tile
    int row, c, other = 0;  // of the 16 rows; the 16-byte chunk of the row (of the block); the block this lane takes first
    if constexpr (kPairs) {
      row = (lane >> 3) ^ ((lane & 4) ? 5 : 0);
      c = lane & 3;
      other = (lane >> 2) & 1;
    } else if constexpr (kFours) {
      const int i = (lane >> 1) & 3;
      row = 8 * (lane >> 4) + ((lane & 8) ? 2 + i : i + (i & 2) * 2);
      c = lane & 1;
      other = i >> 1;
    } else {
      row = lane / (kHalfBytes / 16);
      c = lane % (kHalfBytes / 16);
    }
    const uint32_t raw_at = static_cast<uint32_t>(row * G::kRowBytes + other * kBlockBytes + c * 16);
    const uint32_t out_at = static_cast<uint32_t>((part0 * 16 + row) * 128 + (((c * kPieces) ^ (row & 7)) << 4)) + other * 16384u;
    const uint32_t second = other ? 0u - 16384u : 16384u;  // from the first block to the second
    const float to_t = SHAPED && p.softcap > 0.0f ? p.scale * (2.0f * kLog2e / p.softcap) : p.scale * kLog2e;

    // Sixteen tokens of a tile: how many of them there are, their row in the page, and the page (not looked at before it is
    // needed).
    struct Part {
      int32_t valid, at, page;
    };
    int i = 0, tiles = 0;
    auto step = [&](Part (&a)[kParts]) {
      if (i == tiles) {
        if (!next(w)) return false;
        i = 0;
        tiles = w.tiles;
      }
      const int j0 = w.seen.at(w.tile + i) * kTile + part0 * 16;
      ++i;
#pragma unroll
      for (int g = 0; g < kParts; ++g) {
        const int j = j0 + g * 16;
        // What no row of the segment sees (a window has left it, and its page may be another's by now) is taken as zeros: its value
        // scale, whatever it is, would count in the bound of the tile's.
        a[g].valid = max(0, static_cast<uint32_t>(j - w.hidden) < w.gap ? 0 : min(w.high - j, 16));
        a[g].at = (w.head << p.page_shift) + (j & ((1 << p.page_shift) - 1));
        a[g].page = a[g].valid > 0 ? p.table[w.b * p.max_pages + (j >> p.page_shift)] : 0;
      }
      return true;
    };
    // a page that is none: zeros
    auto settle = [&](Part (&a)[kParts]) {
#pragma unroll
      for (int g = 0; g < kParts; ++g) {
        if (a[g].page >= 0 && a[g].page < p.pages) continue;
        if (lane == 0) record_device_error(p.err, kDevErrBadIndex);
        a[g].page = 0;
        a[g].valid = 0;
      }
    };
    auto load = [&](const Part (&a)[kParts], const uint8_t* codes, uint4 (&u)[kParts][kLoads]) {
#pragma unroll
      for (int g = 0; g < kParts; ++g) {
        const uint8_t* from = codes + a[g].page * p.page_stride + static_cast<int64_t>(a[g].at) * G::kRowBytes;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int x = 0; x < 16 / kRowsAtOnce; ++x)
#pragma unroll
            for (int b = 0; b < kBlocks2; ++b) {
              uint4& to = u[g][(h * (16 / kRowsAtOnce) + x) * kBlocks2 + b];
              to = make_uint4(0u, 0u, 0u, 0u);
              if (row + x * kRowsAtOnce < a[g].valid)
                to = ldg_v4(from + ((raw_at + x * kRowsAtOnce * G::kRowBytes + h * kHalfBytes) ^ (b * kBlockBytes)));
            }
      }
    };
    auto load_scales = [&](const Part (&a)[kParts], uint32_t (&word)[kParts]) {  // lanes 0-15 those of K, 16-31 those of V
#pragma unroll
      for (int g = 0; g < kParts; ++g) {
        const uint8_t* from = (lane < 16 ? p.k_scale : p.v_scale) + a[g].page * p.scale_page_stride + (static_cast<int64_t>(a[g].at) + (lane & 15)) * 4;
        word[g] = (lane & 15) < a[g].valid ? __ldg(reinterpret_cast<const uint32_t*>(from)) : 0u;
      }
    };
    // `words`: this lane's scale words (of K or of V)
    auto widen = [&](const uint4 (&us)[kParts][kLoads], const uint32_t (&words)[kParts], bool v, uint32_t to) {
#pragma unroll
      for (int gx = 0; gx < kParts * (16 / kRowsAtOnce); ++gx) {
        const int g = gx / (16 / kRowsAtOnce), x = gx % (16 / kRowsAtOnce);
        const uint4* u = us[g];
        const uint32_t word = words[g], out = to + g * 2048 + out_at;
        uint32_t bias = 0;
        if constexpr (G::kU4) {
          // what is no zero-point becomes one: its token counts by its scales, and what is not seen has to stay finite
          const uint32_t sw = __shfl_sync(0xffffffffu, word, (v ? 16 : 0) + row + x * kRowsAtOnce);
          const __half z = __hmin(__hmax(__ushort_as_half(static_cast<unsigned short>(sw >> 16)), __float2half(0.0f)),
                                  __float2half(15.0f));
          const __half2 zz = __half2half2(__hadd(z, __float2half(1024.0f)));
          bias = *reinterpret_cast<const uint32_t*>(&zz);
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int b = 0; b < kBlocks2; ++b) {
            const uint4& r4 = u[(h * (16 / kRowsAtOnce) + x) * kBlocks2 + b];
            const uint32_t wd[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              uint32_t o[4];
              if constexpr (G::kU4) {
#pragma unroll
                for (int m = 0; m < 4; ++m) o[m] = hsub2(((wd[k] >> (4 * m)) & 0x000f000fu) | kMagic, bias);
              } else {
                widen4<FMT>(wd[2 * k], o[0], o[1]);
                widen4<FMT>(wd[2 * k + 1], o[2], o[3]);
              }
              sts128((out ^ (k << 4)) + x * kRowsAtOnce * 128 + h * 32768 + (b ? second : 0u), o[0], o[1], o[2], o[3]);
            }
          }
      }
      tc::fence_proxy_async_smem();
    };

    Part cur[kParts], ahead[kParts];
    uint4 ku[kParts][kLoads], vu[kParts][kLoads];
    uint32_t words[kParts] = {};
    // Per turn: the keys of tile t, then its values; in between and behind, the loads of tile t + 1, whose page numbers came
    // with the turn before, and the page numbers of tile t + 2.
    uint32_t t = 0;
    bool have = false, found = false;  // tile t is loaded; the one behind it is `ahead`
#pragma unroll 1
    while (true) {
      const uint32_t buf = t % kBufs;
      if (have) {
        if (t >= kBufs) wait(k_free + 8 * buf, t / kBufs - 1, 0x77);
        dead = __any_sync(0xffffffffu, dead);
        widen(ku, words, false, base + G::kOffK + buf * G::kOperand);
        // The tokens' scales.  Their buffer was last read for tile t - kCols: S of tile t - kBufs is done, and it was issued
        // after every stream's P of the last but one before it.
        static_assert(kCols >= kBufs + 2, "buffers of scales");
        int32_t top = -64;
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
          const uint32_t word = words[g];
          const int token0 = (part0 + g) * 16;
          float* col = reinterpret_cast<float*>(smem + G::kOffCol) + (t % kCols) * 2 * kTile + token0 + (lane & 15);
          float sc;
          if constexpr (G::kU4)  // without a zero-point a token is not a number
            sc = odd_zero(word) ? __uint_as_float(0x7fc00000u) : __half2float(__ushort_as_half(static_cast<unsigned short>(word & 0xffffu)));
          else
            sc = __uint_as_float(word);
          const uint32_t e = (__float_as_uint(sc) >> 23) & 0xffu;
          if (lane < 16) {
            col[0] = sc * to_t;
          } else {
            col[kTile] = sc;
            if (e == 255) odd_tile[t % kCols] = t + 1;
            else top = max(top, static_cast<int32_t>(e) - 126);
          }
          if constexpr (FMT == QLIN_KV_E4M3) {
            // Value codes that are NaN (which the library never writes) become 0 and their token's scale NaN: a product with
            // a probability of 0 keeps a NaN, and rows that do not see the token must not get one.
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
              bad |= (((vu[g][k].x & 0x7f7f7f7fu) + 0x01010101u) | ((vu[g][k].y & 0x7f7f7f7fu) + 0x01010101u) |
                      ((vu[g][k].z & 0x7f7f7f7fu) + 0x01010101u) | ((vu[g][k].w & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
            if (__any_sync(0xffffffffu, bad != 0)) {
              __syncwarp();
#pragma unroll
              for (int k = 0; k < kLoads; ++k) {
                uint32_t* u = &vu[g][k].x;
                uint32_t any = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t m = __vcmpeq4(u[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  any |= m;
                  u[e] &= ~m;
                }
                const int x = k / kBlocks2 % (16 / kRowsAtOnce);
                if (any != 0) {
                  reinterpret_cast<float*>(smem + G::kOffCol)[((t % kCols) * 2 + 1) * kTile + token0 + row + x * kRowsAtOnce] =
                      __uint_as_float(0x7fc00000u);
                  odd_tile[t % kCols] = t + 1;
                }
              }
            }
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        __syncwarp();  // (what all lanes wrote is there for those who see the arrival)
        if (lane == 0) {
          top_exp[(t % kCols) * 4 + warp - kSoftmaxWarps] = top;
          tc::mbar_arrive(k_full + 8 * buf);
          tc::mbar_arrive(col_full + 8 * (t % kCols));
        }
      }
      uint32_t words_v[kParts];
#pragma unroll
      for (int g = 0; g < kParts; ++g) words_v[g] = words[g];
      const bool go = found;
      if (go) {
        settle(ahead);
        load(ahead, p.k, ku);
        load_scales(ahead, words);
#pragma unroll
        for (int g = 0; g < kParts; ++g) cur[g] = ahead[g];
      }
      found = step(ahead);
      if (have) {
        if (t >= kBufs) wait(v_free + 8 * buf, t / kBufs - 1, 0x78);
        dead = __any_sync(0xffffffffu, dead);
        widen(vu, words_v, true, base + G::kOffV + buf * G::kOperand);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(v_full + 8 * buf);
        ++t;
      }
      if (go) load(cur, p.v, vu);
      have = go;
      if (!go && !found) break;
    }
  } else {
    // ---------------- softmax ----------------
    if constexpr (G::kSoftmaxRegs > G::kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kSoftmaxRegs));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kSoftmaxRegs));
    constexpr int kMine = G::kMine;
    constexpr int kStep = kSubs > 1 ? 32 : 64;  // tokens weighed at a time
    const int quad = warp & 3;
    const int stream = kStreams == 2 ? warp >> 2 : 0, sub = kStreams == 2 ? 0 : warp >> 2;
    const int row = quad * 32 + lane;  // of the stream
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t o_at = lanes + kTmemO + stream * G::kOCols + sub * kMine;
    float* row_max = reinterpret_cast<float*>(smem + G::kOffPair);
    uint32_t* q_max = reinterpret_cast<uint32_t*>(smem + G::kOffQmax);
    float* ends = reinterpret_cast<float*>(smem + G::kOffEnd);
    W& w = walks[warp];
    if (lane == 0) w = *origin;
    asm volatile("bar.sync 15, %0;" ::"n"(G::kActive) : "memory");
    auto sync_rows = [&]() {  // the warps of these rows
      if constexpr (kSubs > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + quad), "n"(32 * kSubs) : "memory");
    };

    RowOf* row_of = reinterpret_cast<RowOf*>(smem + G::kOffRow) + threadIdx.x;  // [2 x 256]
    // The segment that the walk stands at; returns the row's position (of a row that is none: the last one's).
    auto segment = [&](int parity) {
      const int64_t r = static_cast<int64_t>(w.row_tile) * kRows + stream * 128 + row;
      const int64_t at = min(r, w.s.rows - 1);
      const int32_t node = token_of(p, at);
      RowOf o;
      o.token = r < w.s.rows ? w.s.q_row + node : -1;
      o.head = w.head * p.group + static_cast<int32_t>(at - static_cast<int64_t>(node) * p.group);
      o.flags = (w.begins() ? 1 : 0) | (w.ends() ? 2 : 0);
      row_of[parity * 256] = o;
      if (threadIdx.x == 0 && o.flags == 1)
        p.records[blockIdx.x] = record_of(w, min(static_cast<int64_t>(gridDim.x), scan[kWarps]), scan[kWarps]);
      return w.s.ctx + node;
    };

    // q of this thread's part of the row, scaled by a power of two, into shared memory; the factor to undo it
    auto stage_q = [&](int parity, float& row_scale) {
      const RowOf g = row_of[parity * 256];
      uint4 raw[kMine / 8];
      uint32_t top = 0;
      const bool bf16 = p.dtype == QLIN_BF16;
      const uint8_t* src = p.q + g.token * p.qt + g.head * p.qh + sub * kMine * 2;
#pragma unroll
      for (int k = 0; k < kMine / 8; ++k) {
        raw[k] = g.token >= 0 ? ldg_v4(src + k * 16) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        if (bf16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max((u[e] << 16) & 0x7fffffffu, u[e] & 0x7fff0000u));
        }
      }
      if constexpr (kSubs > 1) {
        q_max[sub * 128 + row] = top;
        sync_rows();
        top = max(top, q_max[(sub ^ 1) * 128 + row]);
      }
      // fp16 rows go as they are, and bf16 rows whose largest lies in [2^-4, 2^15): what fp16 drops of those is below
      // 2^-20 of it; others by a power of two that puts the largest into [2^14, 2^15)
      int e = 0;
      if (bf16 && top > 0 && top < 0x7f800000u) {
        const int x = ilogbf(__uint_as_float(top));
        if (x < -4 || x > 14) e = x - 14;
      }
      row_scale = ldexpf(1.0f, e);
      const float s1 = ldexpf(1.0f, -(e / 2)), s2 = ldexpf(1.0f, -(e - e / 2));
#pragma unroll
      for (int k = 0; k < kMine / 8; ++k) {
        uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        if (bf16) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float2 v = kv::unpack2<1>(u[m]);
            u[m] = kv::pack2<0>(v.x * s1 * s2, v.y * s1 * s2);
          }
        }
        const int chunk = sub * (kMine / 8) + k;
        const uint32_t to = base + G::kOffQ + stream * G::kOperand + (chunk >> 3) * 16384 + half_chunk(row, chunk & 7);
        if constexpr (G::kU4)  // the order in which 4-bit codes are widened: 0 4 1 5 2 6 3 7
          sts128(to, __byte_perm(u[0], u[2], 0x5410), __byte_perm(u[0], u[2], 0x7632), __byte_perm(u[1], u[3], 0x5410),
                 __byte_perm(u[1], u[3], 0x7632));
        else
          sts128(to, u[0], u[1], u[2], u[3]);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_full + 8 * stream);
    };

    uint32_t t = 0;
    int parity = 0;  // of the segment
    int32_t at = 0;
    float row_scale = 1.0f, ref = 0.0f, l = 0.0f;
    bool live = false, done_any = false;
    const float cap2 = SHAPED ? p.softcap * kLog2e : 0.0f;
    while (true) {
      // the next segment's q, then the output of the one before it
      const bool more = next(w);
      if (more) {
        at = segment(parity);
        stage_q(parity, row_scale);
      }
      if (done_any) {
        if constexpr (kSubs > 1) {
          sync_rows();
          const float* both = ends + (parity ^ 1) * 256 + row;
          l = both[0] + both[128];  // in one order for both
        }
        wait(pv_done + 8 * (kStreams == 2 ? 2 * stream + 1 : (t - 1) & 1), kStreams == 2 ? t - 1 : (t - 1) >> 1, 0x7c);
        dead = __any_sync(0xffffffffu, dead);
        tc::tc_fence_after();
        const RowOf done = row_of[(parity ^ 1) * 256];
        const bool whole = done.flags == 3;
        // No score above -infinity: l is 0, or NaN where a score is none (maxima drop it), and O holds anything.
        const bool none = ref == kNoRef;
        const float inv = !whole ? 1.0f : __frcp_rn(l);
        const float m = none ? -INFINITY : ref + kOffset;
        const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (done.flags & 1)) * p.tile_rows + stream * 128 + row;
        if (live) {
#pragma unroll 1
          for (int cc = 0; cc < kMine; cc += 16) {
            uint32_t o[16];
            __syncwarp();
            tc::tmem_ld_32x32b_x16(o_at + cc, o);
            tc::tmem_wait_ld(o);
            float f[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              // 4-bit codes: column k of eight is channel k / 2 + 4 (k % 2)
              const int ch = G::kU4 ? (k & 8) + ((k & 7) >> 1) + 4 * (k & 1) : k;
              f[ch] = none ? l : __uint_as_float(o[k]) * inv;
            }
            if (done.token < 0) continue;
            const int ch = sub * kMine + cc;
            if (whole) {
              uint8_t* out = p.out + done.token * p.ot + done.head * p.oh + ch * 2;
#pragma unroll
              for (int k = 0; k < 16; k += 8)
                *reinterpret_cast<uint4*>(out + k * 2) = p.dtype == QLIN_BF16 ? kv::pack8<1>(f + k) : kv::pack8<0>(f + k);
            } else {
              float* out = p.part_o + slot * D + ch;
#pragma unroll
              for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(out + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
            }
          }
        }
        if (done.token >= 0 && sub == 0) {
          if (!whole) p.part_ml[slot] = make_float2(m, l);
          else if (p.lse != nullptr) p.lse[done.token * p.hq + done.head] = (lg2(l) + ref) * kLn2;
        }
        tc::tc_fence_before();
      }
      if (!more) break;
      done_any = true;
      ref = kNoRef;
      uint64_t l2 = pair(0.0f, 0.0f);
      bool begun = false;
      const Range some = stream_sees(p, w, stream);
      const Range all = all_seen(p, w.s, __shfl_sync(0xffffffffu, at, 0), __shfl_sync(0xffffffffu, at, 31), 64);
      const int prefix = w.s.prefix, prefix_tiles = w.seen.head, next_tile = w.seen.next - w.seen.head;
      int i = w.tile;
      const int i_end = w.tile + w.tiles;
      const bool scaled = !__all_sync(0xffffffffu, row_scale == 1.0f);
      float slope2 = 0.0f;
      if constexpr (SHAPED) slope2 = p.slopes != nullptr ? -kLog2e * p.slopes[row_of[parity * 256].head] : 0.0f;
#pragma unroll 1
      for (; i < i_end; ++i, ++t) {
        const int j0 = (i < prefix_tiles ? i : next_tile + i) * kTile;
        const bool here = within(some, j0);  // otherwise nothing is multiplied
        bool odd = false;
        float top = 0.0f;
        if (here) {
          wait(col_full + 8 * (t % kCols), t / kCols, 0x7a);
          odd = odd_tile[t % kCols] == t + 1;
          const int4 te = *reinterpret_cast<const int4*>(top_exp + (t % kCols) * 4);
          top = static_cast<float>(max(max(te.x, te.y), max(te.z, te.w)));
        }
#pragma unroll 1
        for (int h = 0; h < G::kHalves; ++h) {
          const uint32_t bar = kStreams == 2 ? 2 * stream + h : t & 1;
          wait(s_full + 8 * bar, kStreams == 2 ? t : t >> 1, 0x79);
          if (!here) {
            // Not before all lanes have seen this phase: one that still waits would take a phase two later for it and wait for good.
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(p_full + 8 * bar);
            continue;
          }
          dead = __any_sync(0xffffffffu, dead);
          tc::tc_fence_after();
          const int part = kSubs > 1 ? sub : h;  // of the tile's two times 64 tokens
          const uint32_t s_at = lanes + (kStreams == 2 ? stream : t & 1) * 128 + part * 64;
          float keep = 1.0f;
#pragma unroll 1
          for (int c0 = 0; c0 < 64; c0 += kStep) {
            const int jc = j0 + part * 64 + c0;
            const uint32_t col = base + G::kOffCol + ((t % kCols) * 2 * kTile + part * 64 + c0) * 4;

            // t of these tokens from their products
            auto score = [&](uint32_t (&v)[kStep]) {
              if (scaled) {
                const uint64_t rs = pair(row_scale, row_scale);
#pragma unroll
                for (int k = 0; k < kStep; k += 2) {
                  const float2 a = unpair(mul2(pair(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), rs));
                  v[k] = __float_as_uint(a.x);
                  v[k + 1] = __float_as_uint(a.y);
                }
              }
              if (SHAPED && cap2 > 0.0f) {
#pragma unroll
                for (int k = 0; k < kStep; k += 4) {
                  const float4 sk = lds4(col + 4 * k);
                  const float ks[4] = {sk.x, sk.y, sk.z, sk.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float x = __uint_as_float(v[k + e]) * ks[e];
                    v[k + e] = __float_as_uint(SHAPED == kLargeCap ? large_capped(x, cap2) : capped(x, cap2));
                  }
                }
              } else {
#pragma unroll
                for (int k = 0; k < kStep; k += 4) {
                  const float4 sk = lds4(col + 4 * k);
                  const float2 a = unpair(mul2(pair(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), pair(sk.x, sk.y)));
                  const float2 b = unpair(mul2(pair(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), pair(sk.z, sk.w)));
                  v[k] = __float_as_uint(a.x);
                  v[k + 1] = __float_as_uint(a.y);
                  v[k + 2] = __float_as_uint(b.x);
                  v[k + 3] = __float_as_uint(b.y);
                }
              }
              if (SHAPED && p.slopes != nullptr) {
                const float off = static_cast<float>(jc - at);  // exact below 2^24
#pragma unroll
                for (int k = 0; k < kStep; ++k)
                  v[k] = __float_as_uint(fmaf(slope2, fabsf(off + static_cast<float>(k)), __uint_as_float(v[k])));
              }
              if (!within(all, jc)) {
#pragma unroll
                for (int k1 = 0; k1 < kStep; k1 += 32) {
                  const int c = jc + k1;
                  uint32_t bits = low_bits(at + 1 - c);
                  if (p.window > 0) bits &= ~low_bits(max(at + 1 - c, 0) - p.window);  // (without overflow)
                  bits |= low_bits(prefix - c);
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (!((bits >> k) & 1u)) v[k1 + k] = 0xff800000u;
                }
              }
            };
            {
              uint32_t v[kStep];
#pragma unroll
              for (int k = 0; k < kStep; k += 32) tc::tmem_ld_32x32b_x32(s_at + c0 + k, v + k);
              tc::tmem_wait_ld(v);
              score(v);
              float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int k = 0; k < kStep; k += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fmaxf(__uint_as_float(v[k + 2 * e]), __uint_as_float(v[k + 2 * e + 1])));
              float hi = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) + top;  // no product with a value scale is above 2^this
              if constexpr (kSubs > 1) {  // over both threads of the row; and both have their scores: P may go over them
                float* maxima = row_max + (c0 / kStep & 1) * kSubs * 128 + row;
                maxima[sub * 128] = hi;
                sync_rows();
                hi = fmaxf(hi, maxima[(sub ^ 1) * 128]);
              }
              if (__any_sync(0xffffffffu, hi > ref + (kOffset + kSlack))) {  // (the same in all warps of these rows)
                // The reference moves, by a whole number of powers of two, so that the row's probabilities that wait for the products
                // already can be scaled in fp16.  With more to come its largest one goes six bits below the top of fp16, which it may
                // grow by before the row has to be rescaled.
                const float to = hi > ref + (kOffset + kSlack) ? ceilf(hi) - 9.0f : ref;
                const float before = ref, f = ex2(ref - to);
                ref = to;
                keep *= f;
                l2 = mul2(l2, pair(f, f));
                if (c0 > 0) {
                  // in two steps: down to 2^-39 of P may be left, and fp16 ends at 2^-24
                  const float e = fmaxf(before - to, -48.0f), e1 = floorf(0.5f * e);
                  const __half2 f1 = __float2half2_rn(ex2(e1)), f2 = __float2half2_rn(ex2(e - e1));
                  uint32_t o[16];
                  tc::tmem_wait_st();
                  tc::tmem_ld_32x32b_x16(s_at, o);
                  tc::tmem_wait_ld(o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = hmul2(hmul2(o[k], *reinterpret_cast<const uint32_t*>(&f1)), *reinterpret_cast<const uint32_t*>(&f2));
                  tc::tmem_st_32x32b_x16(s_at, o);
                }
              }
              const uint64_t nref = pair(-ref, -ref);
              auto weigh = [&](auto with_odd) {
#pragma unroll
                for (int k = 0; k < kStep; k += 4) {
                  const float4 sv = lds4(col + 4 * (kTile + k));
                  const float ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
                  for (int x = 0; x < 4; x += 2) {
                    const float2 a = unpair(add2(pair(__uint_as_float(v[k + x]), __uint_as_float(v[k + x + 1])), nref));
                    const uint64_t e = pair(ex2(a.x), ex2(a.y));
                    l2 = add2(l2, e);
                    float2 f = unpair(mul2(e, pair(ss[x], ss[x + 1])));
                    if constexpr (decltype(with_odd)::value) {  // (what is hidden has no product with a scale that is not a number)
                      if (v[k + x] == 0xff800000u) f.x = 0.0f;
                      if (v[k + x + 1] == 0xff800000u) f.y = 0.0f;
                    }
                    v[(k + x) / 2] = kv::pack2<0>(f.x, f.y);
                  }
                }
              };
              if (odd) weigh(std::true_type{});
              else weigh(std::false_type{});
#pragma unroll
              for (int k = 0; k < kStep; k += 32) tc::tmem_st_32x32b_x16(s_at + c0 + k, v + k / 2);  // over the first half of their scores
            }
          }
          if (__any_sync(0xffffffffu, keep != 1.0f) && begun) {  // (NaN too)
            // all P u of what came before
            if (kStreams == 1) wait(pv_done + 8 * ((t - 1) & 1), (t - 1) >> 1, 0x7b);
            else wait(pv_done + 8 * (2 * stream + (h ^ 1)), h == 0 ? t - 1 : t, 0x7b);
            dead = __any_sync(0xffffffffu, dead);
            tc::tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < kMine; cc += 16) {
              uint32_t o[16];
              tc::tmem_ld_32x32b_x16(o_at + cc, o);
              tc::tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 f = unpair(mul2(pair(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), pair(keep, keep)));
                o[k] = __float_as_uint(f.x);
                o[k + 1] = __float_as_uint(f.y);
              }
              tc::tmem_st_32x32b_x16(o_at + cc, o);
            }
          }
          begun = true;
          __syncwarp();
          tc::tmem_wait_st();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(p_full + 8 * bar);
        }
      }

      const float2 lp = unpair(l2);
      l = lp.x + lp.y;
      if constexpr (kSubs > 1) ends[parity * 256 + sub * 128 + row] = l;
      live = some.high >= 0;
      parity ^= 1;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a segment that begins in block `blockIdx.x` of the first kernel and ends in a later one, in the order of
// the blocks: a warp a row, D / 4 lanes' worth of float4.
template <int D>
__global__ void __launch_bounds__(128) chunk_attention_join_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4 < 32 ? D / 4 : 32;
  constexpr int kWide = D / 4 / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const tree::Record rec = p.records[blockIdx.x];
  if (rec.last < 0) return;
  const int lane = threadIdx.x % 32;
  const int count = rec.last - static_cast<int>(blockIdx.x) + 1;
  const int64_t rows = static_cast<int64_t>(rec.nodes) * p.group;
  for (int row = blockIdx.y * 4 + threadIdx.x / 32; row < p.tile_rows; row += gridDim.y * 4) {
    const int64_t at = static_cast<int64_t>(rec.row_tile) * (D == 256 ? 128 : 256) + row;
    if (at >= rows) return;
    if (lane >= kLanes) continue;
    float m = -INFINITY, l = 0.0f;
    float4 o[kWide];
#pragma unroll
    for (int i = 0; i < kWide; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const int64_t slot = (2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0)) * p.tile_rows + row;
      const float2 e = p.part_ml[slot];
      const float4* src = reinterpret_cast<const float4*>(p.part_o + slot * D) + lane;
      const float to = fmaxf(m, e.x);
      const float fa = m == -INFINITY ? 1.0f : ex2(m - to), fb = e.x == -INFINITY ? 1.0f : ex2(e.x - to);
      m = to;
      l = l * fa + e.y * fb;
#pragma unroll
      for (int x = 0; x < kWide; ++x) {
        const float4 v = src[x * kLanes];
        o[x].x = o[x].x * fa + v.x * fb;
        o[x].y = o[x].y * fa + v.y * fb;
        o[x].z = o[x].z * fa + v.z * fb;
        o[x].w = o[x].w * fa + v.w * fb;
      }
    }
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
    const int64_t node = at / p.group;
    const int head = rec.head * p.group + static_cast<int>(at - node * p.group);
    const int64_t tok = rec.q_row + node;
#pragma unroll
    for (int x = 0; x < kWide; ++x) {
      const float v[4] = {o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv};
      const uint2 u = p.dtype == QLIN_BF16 ? make_uint2(kv::pack2<1>(v[0], v[1]), kv::pack2<1>(v[2], v[3]))
                                           : make_uint2(kv::pack2<0>(v[0], v[1]), kv::pack2<0>(v[2], v[3]));
      *reinterpret_cast<uint2*>(p.out + tok * p.ot + head * p.oh + (lane + x * kLanes) * 8) = u;
    }
    if (p.lse != nullptr && lane == 0) p.lse[tok * p.hq + head] = (lg2(l) + (m - kOffset)) * kLn2;
  }
}

template <int FMT, int D, int SHAPED>
cudaError_t plan(const Params& p, Prepared* out) {
  const void* fn = reinterpret_cast<const void*>(chunk_attention_kernel<FMT, D, SHAPED>);
  const cudaError_t e = ensure_max_dynamic_smem(fn);
  if (e != cudaSuccess) return e;
  const uint32_t blocks = static_cast<uint32_t>(sm_count());
  out->count = 2;
  out->launch[0] = {fn, blocks, 1, Geo<FMT, D>::kThreads, Geo<FMT, D>::kSmem};
  out->launch[1] = {reinterpret_cast<const void*>(chunk_attention_join_kernel<D>), blocks,
                    static_cast<uint32_t>((p.tile_rows + 7) / 8), 128, 0};
  out->set(p);
  return cudaSuccess;
}

template <int FMT, int D>
cudaError_t plan(const Params& p, Prepared* out) {
  if (p.softcap > kPlainCap) return plan<FMT, D, kLargeCap>(p, out);
  return p.softcap > 0.0f || p.slopes != nullptr ? plan<FMT, D, kShaped>(p, out) : plan<FMT, D, kPlainScores>(p, out);
}

template <int FMT>
cudaError_t plan(const Params& p, int64_t d, Prepared* out) {
  return d == 64 ? plan<FMT, 64>(p, out) : d == 128 ? plan<FMT, 128>(p, out) : plan<FMT, 256>(p, out);
}

// Rows of a part in the workspace.
int64_t part_rows(const qlin_kv_cache& c, int64_t hq, int64_t max_new) {
  const int64_t group = hq / c.heads;
  return std::min<int64_t>(c.head_dim == 256 ? 128 : 256, max_new > 256 ? 256 : max_new * group);
}

// Calls of few rows per key head go to tree attention's kernels, which have no tile of 256 rows to fill: up to 16 in any form,
// plain ones up to 64 (heads of 256 have no such kernel there).  INT8, 32 heads on 8 of 128, there / here: 64 single tokens
// behind 1000 51 / 122 us (61 with a cap), 4 x 4 tokens behind 16000 49 / 91; of 32 rows 95 / 123 and 77 / 91, of 64 101 / 124
// and 84 / 92, of 128 125 / 140 and 97 / 97.
constexpr int64_t kFewRows = 16, kFewPlainRows = 64;
int64_t rows_of(const qlin_kv_cache& c, int64_t hq, int64_t max_new) { return max_new * (hq / c.heads); }
bool few_rows(const qlin_kv_cache& c, int64_t rows, bool plain) {
  return rows <= kFewRows || (plain && c.head_dim <= 128 && rows <= kFewPlainRows);
}

}  // namespace
}  // namespace chunk

int64_t chunk_attention_workspace_bytes(const qlin_kv_cache& cache, int64_t hq, int64_t max_new, int64_t B) {
  const int64_t blocks = sm_count();
  const int64_t own = blocks * static_cast<int64_t>(sizeof(tree::Record)) + 256 +
                      2 * blocks * chunk::part_rows(cache, hq, max_new) * (cache.head_dim * 4 + static_cast<int64_t>(sizeof(float2)));
  const bool other = chunk::few_rows(cache, chunk::rows_of(cache, hq, max_new), true);
  return other ? std::max(own, tree_attention_workspace_bytes(cache, hq, max_new, B)) : own;
}

cudaError_t plan_chunk_attention(const ChunkAttentionArgs& a, Prepared* out) {
  chunk::Params p = {};
  const qlin_kv_cache& c = a.cache;
  const bool plain = a.scores.softcap == 0.0f && a.scores.slopes == nullptr && a.scores.window == 0 && a.scores.prefix_lens == nullptr;
  if (chunk::few_rows(c, chunk::rows_of(c, a.q.heads, a.max_new), plain)) {
    TreeAttentionArgs t = {};
    t.q = a.q;
    t.out = a.out;
    t.dtype = a.dtype;
    t.Tq = a.Tq;
    t.cache = c;
    t.block_table = a.block_table;
    t.max_pages = a.max_pages;
    t.q_indptr = a.q_indptr;
    t.ctx_lens = a.ctx_lens;
    t.B = a.B;
    t.max_nodes = a.max_new;
    t.scale = a.scores.scale;
    t.lse = a.lse;
    t.workspace = a.workspace;
    return plain ? plan_tree_attention(t, out) : plan_chain_attention(t, a.scores, out);
  }
  p.q = static_cast<const uint8_t*>(a.q.data);
  p.out = static_cast<uint8_t*>(a.out.data);
  p.qt = 2 * a.q.token_stride;
  p.qh = 2 * a.q.head_stride;
  p.ot = 2 * a.out.token_stride;
  p.oh = 2 * a.out.head_stride;
  p.hq = static_cast<int32_t>(a.q.heads);
  p.hk = static_cast<int32_t>(c.heads);
  p.group = p.hq / p.hk;
  p.dtype = a.dtype;
  p.Tq = a.Tq;
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.page_stride = c.page_stride;
  p.k_scale = static_cast<const uint8_t*>(c.k_scale);
  p.v_scale = static_cast<const uint8_t*>(c.v_scale);
  p.scale_page_stride = c.scale_page_stride;
  const kv::CacheView view = kv::view_of(c);
  p.pages = view.pages;
  p.page_shift = view.page_shift;
  p.table = a.block_table;
  p.max_pages = a.max_pages;
  p.q_indptr = a.q_indptr;
  p.ctx_lens = a.ctx_lens;
  p.B = static_cast<int32_t>(a.B);
  p.max_nodes = static_cast<int32_t>(a.max_new);
  p.scale = a.scores.scale;
  p.softcap = a.scores.softcap;
  p.slopes = a.scores.slopes;
  p.window = a.scores.window >= tree::kMaxLen ? 0 : static_cast<int32_t>(a.scores.window);  // no sequence is longer
  p.prefix = a.scores.prefix_lens;
  p.lse = a.lse;
  p.tile_rows = static_cast<int32_t>(chunk::part_rows(c, a.q.heads, a.max_new));
  const int64_t blocks = sm_count(), rows = 2 * blocks * p.tile_rows;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  ws += rows * c.head_dim * 4;
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += rows * static_cast<int64_t>(sizeof(float2));
  p.records = reinterpret_cast<tree::Record*>(ws);
  p.err = device_error_word();
  if (c.fmt == QLIN_KV_INT8) return chunk::plan<QLIN_KV_INT8>(p, c.head_dim, out);
  if (c.fmt == QLIN_KV_E4M3) return chunk::plan<QLIN_KV_E4M3>(p, c.head_dim, out);
  return chunk::plan<QLIN_KV_U4>(p, c.head_dim, out);
}

}  // namespace qlin
