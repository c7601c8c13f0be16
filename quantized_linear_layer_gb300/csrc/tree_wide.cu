// Tree attention for many rows per key head (nodes x query heads of a group),
// on the tcgen05 tensor cores.  The mathematics, the division of the work and
// the joining kernel are those of tree_attention.cu; here a row tile has 128
// rows and a token tile 128 tokens, so that one widening of the codes serves
// 128 rows and the products run at the full tensor rate.
//
// A block (one per SM) has 28 warps, whose registers are dealt out anew by role:
//   0-15   softmax: four threads per row, 32 of a tile's tokens each
//   16-23  widen codes to fp16 in shared memory, in the tensor core's layout
//   24     copies codes and scales into a ring of half tiles
//   25     issues the products (one thread)
// Per token tile: S = q n^T (128 x 128, operands from shared memory) into one of
// two tensor-memory buffers; the softmax threads read their 32 columns of it,
// turn them into probabilities and write these as fp16 over the same buffer;
// O += P u takes P from tensor memory and the codes of v from shared memory as
// they lie (tokens x channels, the operand's other major order), so neither K
// nor V is transposed.  S of the next tile is issued before P u of this one,
// so the tensor cores work while the softmax of a tile runs.
//
// The four threads of a row agree on the reference through shared memory; when
// it moves, each rescales a quarter of the row of O in tensor memory, after its
// probabilities are written, when P u of the tile before is done.
// Probabilities below fp16's normal range are written apart, times 2^29, into
// the buffer's other half, and go to a second accumulator O2 (o = O + 2^-29 O2)
// in the tiles that hold any.
//
// Tensor memory, all 512 columns: S/P 2 x 128, O 128, O2 128.
//
// Bound: a tile takes about 3900 cycles whatever its rows.  Shared memory is busy
// for about 2900 of them: 768 to 1024 for the products' operands, 1000 for the
// codes in and out of their widening, 900 for the tokens' scales, which every
// warp of rows reads; issue slots take 2600 of each scheduler's, products 1024 to
// 1536, exponentials 1024.  One tree of 26 nodes (104 rows a key head) over 131001
// tokens, U4: 139 us; 16 sequences of 33 to 64 nodes (782 in all) x 64 query heads
// over up to 8192 tokens, INT8: 344 us, 407 TFLOP/s; 32 sequences of 8 to 16 nodes
// (407) over up to 32768, E4M3: 500 us, 2310 GB/s.  Prompt chunks, 8 sequences of 256
// nodes x 32 query heads, INT8: 71 us behind no token, 302 behind 4096 (483
// TFLOP/s), 958 behind 16384 (582).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "stage_ring.h"
#include "tree_common.cuh"

namespace qlin {
namespace tree {
namespace {

constexpr int kRows = 128;
constexpr int kTile = 128;
constexpr int kHalf = 64;  // tokens of a stage of the ring
constexpr int kSoftmaxWarps = 16;
constexpr int kSubs = kSoftmaxWarps / 4;  // threads of a row
constexpr int kSpan = kTile / kSubs;      // tokens of each
constexpr int kWidenWarps = 8;
constexpr int kLoadWarp = kSoftmaxWarps + kWidenWarps;
constexpr int kMmaWarp = kLoadWarp + 1;
constexpr int kThreads = 32 * 28;  // whole groups of four warps
// Registers: 896 threads are launched with 72 each, 64512 in all; 512 x 88 + 256 x 48 + 128 x 56 = 64512.
constexpr int kSoftmaxRegs = 88, kWidenRegs = 48, kOtherRegs = 56;
constexpr int kStages = 4;
constexpr int kCols = 4;  // buffers of the tokens' scales: see the widening warps
constexpr float kShiftUp = 536870912.0f;              // 2^29: the small probabilities lie below 2^15
constexpr float kShiftDown = 1.862645149230957e-9f;  // 2^-29
using W = Walk<kRows, kTile>;

// tensor memory columns
constexpr uint32_t kTmemO = 256, kTmemO2 = 384;

template <int FMT, int D>
struct Geo {
  static constexpr bool kU4 = FMT == QLIN_KV_U4;
  static constexpr int kRowBytes = kU4 ? D / 2 : D;
  static constexpr int kBlocks = D / 64;                // 64-channel blocks of 128 rows x 128 bytes
  static constexpr int kOperand = kBlocks * 16384;      // q, K or V of a tile in fp16
  static constexpr int kRawCode = kHalf * kRowBytes;    // K or V codes of a stage
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kOperand;
  static constexpr int kOffV = kOffK + kOperand;        // two buffers
  static constexpr int kOffRaw = kOffV + 2 * kOperand;
  static constexpr int kOffScale = kOffRaw + kStages * 2 * kRawCode;
  static constexpr int kOffCol = kOffScale + kStages * 2 * kHalf * 4;  // [kCols][scale log2(e) sk, log2 sv, 1 / sv, factor][128]
  static constexpr int kOffPair = kOffCol + kCols * 4 * kTile * 4;     // [tile parity][thread of the row][row]
  static constexpr int kOffQmax = kOffPair + 2 * kSubs * kRows * 4;    // [thread of the row][row]
  static constexpr int kOffEnd = kOffQmax + kSubs * kRows * 4;         // [thread of the row][row] (l, small)
  static constexpr int kOffBar = kOffEnd + kSubs * kRows * 8;
  static constexpr int kBars = 2 * kStages + 1 + 1 + 2 + 2 + 2 + 2 + 1 + 1 + kCols;
  static constexpr int kOffMisc = kOffBar + kBars * 8;  // tensor memory address, flags
  static constexpr int kOffScan = kOffMisc + 32;
  static constexpr int kOffWalk = (kOffScan + (kThreads + 1) * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffWalk + (kSoftmaxWarps + kWidenWarps) * static_cast<int>(sizeof(W)) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");

};

// Halves below fp16's normal range become 0.
__device__ __forceinline__ __half2 flush(uint32_t v) {
  uint32_t r;
  asm("mul.rn.ftz.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x3c003c00u));
  return *reinterpret_cast<const __half2*>(&r);
}

// Two probabilities as fp16: what fp16 cannot hold as a normal number is 0 in `large` and, times `up` (2^29), in `small`.
__device__ __forceinline__ void split(uint64_t e, uint64_t up, uint32_t& large, uint32_t& small) {
  const float2 f = unpair(e), s = unpair(mul2(e, up));
  const __half2 p16 = flush(kv::pack2<0>(f.x, f.y));
  large = *reinterpret_cast<const uint32_t*>(&p16);
  small = kv::pack2<0>(s.x, s.y) & __heq2_mask(p16, __float2half2_rn(0.0f));
}

// Which of the 64 tokens from node `first` on (negative: cached tokens) node
// `node` sees, one bit each.
__device__ __forceinline__ uint64_t seen_bits(const Params& p, const Sequence& s, int node, int first) {
  if (first <= -64) return ~0ull;
  uint64_t v = 0;
  const int from = max(first, 0), n = min(s.nodes - from, 64);  // nodes from .. from + n - 1
  if (node >= 0 && node < s.nodes && n > 0) {
    if (p.mask == nullptr) {
      const int m = node + 1 - from;
      v = m <= 0 ? 0 : m >= 64 ? ~0ull : (1ull << m) - 1;
    } else {
      const int64_t* words = p.mask + (s.q_row + node) * p.mask_words;
      const int w = from >> 6, sh = from & 63;
      v = static_cast<uint64_t>(words[w]) >> sh;
      if (sh != 0 && w + 1 < p.mask_words) v |= static_cast<uint64_t>(words[w + 1]) << (64 - sh);
    }
    if (n < 64) v &= (1ull << n) - 1;
  }
  if (first < 0) v = (v << -first) | ((1ull << -first) - 1);
  return v;
}

// The ring of half tiles, for stage_ring.h.
struct RingOps {
  uint32_t full, free;  // barriers, [kStages]
  volatile uint32_t* flag;
  int32_t* err;
  __device__ __forceinline__ bool wait_full(uint32_t stage, uint32_t parity) {
    return tc::mbar_wait_quiet(full + 8 * stage, parity, err, 0x6f);
  }
  __device__ __forceinline__ bool wait_free(uint32_t stage, uint32_t parity) {
    return tc::mbar_wait_quiet(free + 8 * stage, parity, err, 0x60);
  }
  __device__ __forceinline__ bool raised() { return *flag != 0; }
  __device__ __forceinline__ void raise() {
    *flag = 1;
    __threadfence_block();
  }
  __device__ __forceinline__ bool any(bool b) { return __any_sync(0xffffffffu, b); }
};

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_attention_wide_kernel(const __grid_constant__ Params p) {
  using G = Geo<FMT, D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - tc::smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const uint32_t bars = base + G::kOffBar;
  const uint32_t raw_full = bars, raw_free = raw_full + 8 * kStages;  // [kStages]
  const uint32_t k_full = raw_free + 8 * kStages, k_free = k_full + 8;
  const uint32_t v_full = k_free + 8;       // [2]
  const uint32_t s_full = v_full + 16;      // [2]
  const uint32_t p_full = s_full + 16;      // [2]
  const uint32_t pv_done = p_full + 16;     // [2]
  const uint32_t q_full = pv_done + 16;
  const uint32_t all_done = q_full + 8;
  const uint32_t col_full = all_done + 8;   // [kCols]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::kOffMisc);
  volatile uint32_t* ran_out = tmem_slot + 1;  // a wait of some role of the block ran out
  volatile uint32_t* small_tile = reinterpret_cast<volatile uint32_t*>(smem + G::kOffMisc + 8);  // [2]: 1 + the last tile with any
  volatile uint32_t* odd_tile = small_tile + 2;  // [kCols]: 1 + the last tile with a factor (usable_scale) that is not 1
  int64_t* scan = reinterpret_cast<int64_t*>(smem + G::kOffScan);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(raw_full + 8 * i, 33);
      tc::mbar_init(raw_free + 8 * i, kWidenWarps / 2);
    }
    tc::mbar_init(k_full, kWidenWarps);
    tc::mbar_init(k_free, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(v_full + 8 * i, kWidenWarps);
      tc::mbar_init(s_full + 8 * i, 1);
      tc::mbar_init(p_full + 8 * i, kSoftmaxWarps);
      tc::mbar_init(pv_done + 8 * i, 1);
      small_tile[i] = 0;
    }
    tc::mbar_init(q_full, kSoftmaxWarps);
    tc::mbar_init(all_done, 1);
    for (int i = 0; i < kCols; ++i) {
      tc::mbar_init(col_full + 8 * i, kWidenWarps);
      odd_tile[i] = 0;
    }
    *ran_out = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int share = (p.B + kThreads - 1) / kThreads;
  scan_units<kRows, kTile, kThreads>(p, share, scan);
  const int64_t total = scan[kThreads];
  const int64_t blocks = min(static_cast<int64_t>(gridDim.x), total);  // each of these has a unit or more
  if (threadIdx.x == 0) p.records[blockIdx.x].last = -1;
  if (blockIdx.x >= blocks) return;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  W run = begin_run<kRows, kTile, kThreads>(p, share, scan, blockIdx.x, blocks);

  // In every role a wait that runs out makes it go on without waiting, so that
  // all loops end and every barrier among threads is met; the block's flag tells
  // the loading warp (stage_ring.h).
  bool dead = false;
  RingOps ops = {raw_full, raw_free, ran_out, p.err};
  auto wait = [&](uint32_t bar, uint32_t parity, int site) {
    ring::wait_or_raise(ops, dead, [&]() { return tc::mbar_wait_quiet(bar, parity & 1, p.err, site); });
  };

  if (warp >= kLoadWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kLoadWarp) {
    // ---------------- loads ----------------
    ring::Filler<kStages> fill;
    bool zeroed = false;
    const int page = 1 << p.page_shift;
    const int box = min(page, kHalf);
    const int boxes = kHalf / box;
    const uint64_t policy = tc::l2_policy_evict_first();
    while (run.next(p)) {
      const int32_t* table = p.table + run.b * p.max_pages;
      const int end = min(run.s.len, (run.tile + run.tiles) * kTile);
      int32_t ahead = kNoPage;  // the page of box `lane` of the 32 boxes from half tile `from` on
      unsigned bad = 0;  // of them, those whose page is out of range
      int from = 0;
      for (int t = 2 * run.tile; t < 2 * (run.tile + run.tiles); ++t) {
        if (t == 2 * run.tile || (t - from) * boxes == 32) {
          from = t;
          const int j = t * kHalf + lane * box;
          ahead = kNoPage;
          if (j < end) ahead = checked_page(p, table[j >> p.page_shift]);
          bad = __ballot_sync(0xffffffffu, j < end && ahead < 0);
        }
        if (!fill.wait(ops)) continue;
        const uint32_t stage = fill.stage();
        // a box's codes are contiguous in its page: one bulk copy each of K and V; its scales go by small copies
        const uint32_t bar = raw_full + 8 * stage;
        const int32_t pg = __shfl_sync(0xffffffffu, ahead, ((t - from) * boxes + lane) & 31);
        const bool load = lane < boxes && pg >= 0;
        const int good = __popc(__ballot_sync(0xffffffffu, load));
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, good * box * 2 * G::kRowBytes);
        __syncwarp();
        const uint32_t raw = base + G::kOffRaw + stage * 2 * G::kRawCode;
        if (load) {
          const int64_t row = static_cast<int64_t>(run.head) * page + ((t * kHalf + lane * box) & (page - 1));
          const int64_t codes = pg * p.page_stride + row * G::kRowBytes;
          const uint32_t to = raw + lane * box * G::kRowBytes;
          if (zeroed) tc::fence_proxy_async_smem();  // the stage may hold zeros from below: written by another proxy
          tc::bulk_load_policy(to, p.k + codes, box * G::kRowBytes, bar, policy);
          tc::bulk_load_policy(to + G::kRawCode, p.v + codes, box * G::kRowBytes, bar, policy);
        }
        const uint32_t scales = base + G::kOffScale + stage * 2 * kHalf * 4;
        copy_scales<kHalf>(p, run.head, t * kHalf, box, ahead, (t - from) * boxes, scales, scales + kHalf * 4, policy);
        if (bad != 0) {
          for (int b = 0; b < boxes; ++b)
            if ((bad >> ((t - from) * boxes + b)) & 1) {
              const uint32_t to = raw + b * box * G::kRowBytes;
              for (int x = lane * 16; x < box * G::kRowBytes; x += 512) {
                copy16(to + x, p.k, 0, policy);
                copy16(to + G::kRawCode + x, p.v, 0, policy);
              }
              zeroed = true;
            }
        }
        copies_arrive(bar);
        ++fill.filled;
      }
    }
    copies_wait();
    fill.drain(ops);
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    // The whole warp runs the loop, so that addresses and descriptors stay in uniform registers; one thread issues.
    const bool leader = elect_one();
    const uint32_t idesc_s = tc::idesc_f16(kRows, kTile, 0);
    const uint32_t idesc_o = tc::idesc_f16(kRows, D, 0) | (1u << 16);  // B with n contiguous
    // a descriptor's address field counts 16 bytes and does not overflow below 256 KB: advancing is an addition
    const uint64_t q_desc = tc::sw128_kmajor_desc(base + G::kOffQ), k_desc = tc::sw128_kmajor_desc(base + G::kOffK);
    const uint64_t v_desc = sw128_nmajor_desc(base + G::kOffV, 16384);
    uint32_t t = 0, seg = 0;
    bool o2_begun = false;
    auto second = [&](uint32_t x, bool first) {  // O += P u of tile x, the first of its segment or not
      const uint32_t buf = x & 1;
      wait(p_full + 8 * buf, x >> 1, 0x61);
      wait(v_full + 8 * buf, x >> 1, 0x62);
      dead = __any_sync(0xffffffffu, dead);
      tc::tc_fence_after();
      if (first) o2_begun = false;
      const uint64_t vd = v_desc + buf * (G::kOperand >> 4);
      const uint32_t pt = tmem + buf * 128;
      const bool small = __any_sync(0xffffffffu, small_tile[buf] == x + 1);
      if (!dead) {
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            tc::mma_f16_ta(tmem + kTmemO, pt + 8 * k, vd + k * 128, idesc_o, !first || k > 0 ? 1u : 0u);
          if (small) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              tc::mma_f16_ta(tmem + kTmemO2, pt + 64 + 8 * k, vd + k * 128, idesc_o, o2_begun || k > 0 ? 1u : 0u);
          }
        }
        o2_begun = o2_begun || small;
      }
      if (leader) tc::mma_commit(pv_done + 8 * buf);
      __syncwarp();
    };
    bool pending_first = false;
    while (run.next(p)) {
      for (int i = 0; i < run.tiles; ++i, ++t) {
        const uint32_t buf = t & 1;
        if (i == 0) wait(q_full, seg, 0x63);
        wait(k_full, t, 0x64);
        if (t >= 2) wait(pv_done + 8 * buf, (t - 2) >> 1, 0x65);
        dead = __any_sync(0xffffffffu, dead);
        tc::tc_fence_after();
        if (leader) {
          if (!dead) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * 1024 + (k & 3) * 2;
              tc::mma_f16(tmem + buf * 128, q_desc + off, k_desc + off, idesc_s, k > 0 ? 1u : 0u);
            }
          }
          tc::mma_commit(s_full + 8 * buf);
          tc::mma_commit(k_free);
        }
        __syncwarp();
        if (t > 0) second(t - 1, pending_first);
        pending_first = i == 0;
      }
      ++seg;
    }
    second(t - 1, pending_first);
    // every product is done before the tensor memory is given back, whatever else ran out
    if (leader) tc::mma_commit(all_done);
    __syncwarp();
    tc::mbar_wait_quiet(all_done, 0, p.err, 0x66);
    __syncwarp();
  } else if (warp > kMmaWarp) {
    // (fills up the group)
  } else if (warp >= kSoftmaxWarps) {
    // ---------------- widening ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWidenRegs));
    const int part = warp - kSoftmaxWarps;  // this warp's 16 tokens of a tile
    const int h = part / 4;                 // the half tile they lie in
    W& w = reinterpret_cast<W*>(smem + G::kOffWalk)[warp];
    if (lane == 0) w = run;
    uint32_t t = 0;
    // A lane takes 16 bytes of codes of one row at a time and makes kPieces 16-byte chunks of fp16 of them.  The codes lie
    // as they do in their pages; rows and chunks are dealt to lanes such that the eight lanes of a quarter warp read from,
    // and for each piece write to, eight different bank groups, and a lane's row is the same modulo 8 throughout, so that
    // its addresses differ by constants:
    //   rows of 128 bytes: rows r, r ^ 5 x four chunks, one row's of one 64-channel block, the other's of the other
    //   rows of 64 bytes, two blocks (U4): rows 0 1 | 6 7 or 2 3 | 4 5 x two chunks of one block | of the other
    //   rows of 64 or 32 bytes, one block: consecutive rows
    constexpr int kPieces = G::kU4 ? 4 : 2;
    constexpr bool kPairs = G::kRowBytes == 128, kFours = G::kU4 && G::kBlocks == 2;
    constexpr int kRowsAtOnce = G::kRowBytes == 32 || kFours ? 16 : 8;
    int row, c;     // of the 16 rows, and the 16-byte chunk of the row (of the block)
    int other = 0;  // the block this lane takes first
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
      row = lane / (G::kRowBytes / 16);
      c = lane % (G::kRowBytes / 16);
    }
    constexpr int kBlockBytes = G::kRowBytes / G::kBlocks;  // of a row's codes in one 64-channel block
    const uint32_t raw_at = static_cast<uint32_t>(row * G::kRowBytes + other * kBlockBytes + c * 16);
    const uint32_t out_at = static_cast<uint32_t>(row * 128 + (((c * kPieces) ^ (row & 7)) << 4)) + other * 16384u;
    const uint32_t second = other ? 0u - 16384u : 16384u;  // from the first block to the second
    while (true) {
      bool more = false;
      __syncwarp();
      if (lane == 0) more = w.next(p);
      __syncwarp();
      if (!__shfl_sync(0xffffffffu, more, 0)) break;
      const int len = w.s.len;
      for (int i = 0; i < w.tiles; ++i, ++t) {
        const int j0 = (w.tile + i) * kTile;
        const uint32_t stage = (2 * t + h) % kStages;
        const uint32_t raw = base + G::kOffRaw + stage * 2 * G::kRawCode;
        const uint8_t* scales = smem + G::kOffScale + stage * 2 * kHalf * 4;
        // K or V (v) of this warp's tokens into `to`
        auto widen = [&](bool v, uint32_t to) {
          const uint32_t from = raw + (v ? G::kRawCode : 0) + (part & 3) * 16 * G::kRowBytes + raw_at;
          const uint8_t* sc = scales + (v ? kHalf * 4 : 0) + ((part & 3) * 16 + row) * 4;
          const uint32_t out = to + part * 16 * 128 + out_at;
          uint4 u[G::kBlocks * 16 / kRowsAtOnce];
#pragma unroll
          for (int x = 0; x < 16 / kRowsAtOnce; ++x)
#pragma unroll
            for (int b = 0; b < G::kBlocks; ++b)
              u[x * G::kBlocks + b] = tc::lds128((from + x * kRowsAtOnce * G::kRowBytes) ^ (b * kBlockBytes));
#pragma unroll
          for (int x = 0; x < 16 / kRowsAtOnce; ++x) {
            uint32_t bias = 0;
            if constexpr (G::kU4) {
              const uint32_t word = *reinterpret_cast<const uint32_t*>(sc + x * kRowsAtOnce * 4);
              // what is no zero-point becomes one: its token counts by its score and its factor, and what is not seen has
              // to stay finite
              const __half z = __hmin(__hmax(__ushort_as_half(static_cast<unsigned short>(word >> 16)), __float2half(0.0f)),
                                      __float2half(15.0f));
              const __half2 zz = __half2half2(__hadd(z, __float2half(1024.0f)));
              bias = *reinterpret_cast<const uint32_t*>(&zz);
            }
#pragma unroll
            for (int b = 0; b < G::kBlocks; ++b) {
              const uint4& r4 = u[x * G::kBlocks + b];
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
                sts128((out ^ (k << 4)) + x * kRowsAtOnce * 128 + (b ? second : 0u), o[0], o[1], o[2], o[3]);
              }
            }
          }
          tc::fence_proxy_async_smem();
        };

        // K, once S of the tile before is done
        wait(raw_full + 8 * stage, (2 * t + h) / kStages, 0x67);
        if (t >= 1) wait(k_free, t - 1, 0x68);
        dead = __any_sync(0xffffffffu, dead);
        widen(false, base + G::kOffK);
        // The tokens' scales.  Their buffer was last read for tile t - kCols; K of this tile could be written
        // only after S of tile t - 1, which needed p of tile t - 3.
        if (lane < 16) {
          const int token = (part & 3) * 16 + lane;  // of the half tile
          const uint32_t kw = *reinterpret_cast<const uint32_t*>(scales + token * 4);
          uint32_t vw = *reinterpret_cast<const uint32_t*>(scales + (kHalf + token) * 4);
          float factor = 1.0f;
          bool odd = odd_scale<FMT>(vw);
          if (odd) vw = usable_scale<FMT>(vw, factor);
          if constexpr (G::kU4) {  // without a zero-point a token is not a number: its factor here, its score below
            if (odd_zero(vw)) odd = true, factor = __uint_as_float(0x7fc00000u);
          }
          if constexpr (FMT == QLIN_KV_E4M3) {  // among the values of nodes, or behind the end
            if (j0 + part * 16 + lane >= w.s.ctx) {
              bool nan_codes = false;
#pragma unroll 1
              for (int x = 0; x < G::kRowBytes; x += 16) nan_codes |= clear_nan_codes(raw + G::kRawCode + token * G::kRowBytes + x);
              if (nan_codes) odd = true, factor = __uint_as_float(0x7fc00000u);
            }
          }
          if (odd && j0 + part * 16 + lane < len) odd_tile[t % kCols] = t + 1;
          float sk, sv;
          if constexpr (G::kU4) {
            sk = odd_zero(kw) ? __uint_as_float(0x7fc00000u) : __half2float(__ushort_as_half(static_cast<unsigned short>(kw & 0xffffu)));
            sv = __half2float(__ushort_as_half(static_cast<unsigned short>(vw & 0xffffu)));
          } else {
            sk = __uint_as_float(kw);
            sv = __uint_as_float(vw);
          }
          float* col = reinterpret_cast<float*>(smem + G::kOffCol) + (t % kCols) * 4 * kTile + part * 16 + lane;
          col[0] = sk * (p.scale * kLog2e);
          col[kTile] = lg2(sv);
          col[2 * kTile] = rcp(sv);
          col[3 * kTile] = factor;
        }
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(k_full);
          tc::mbar_arrive(col_full + 8 * (t % kCols));
        }
        // V, once P u of the tile before the last is done
        if (t >= 2) wait(pv_done + 8 * (t & 1), (t - 2) >> 1, 0x69);
        dead = __any_sync(0xffffffffu, dead);
        widen(true, base + G::kOffV + (t & 1) * G::kOperand);
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(v_full + 8 * (t & 1));
          tc::mbar_arrive(raw_free + 8 * stage);
        }
      }
    }
  } else {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int quad = warp & 3, sub = warp >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    constexpr int kMine = D / kSubs;  // channels of q and o that this thread takes
    float* row_max = reinterpret_cast<float*>(smem + G::kOffPair);
    uint32_t* q_max = reinterpret_cast<uint32_t*>(smem + G::kOffQmax);
    float2* ends = reinterpret_cast<float2*>(smem + G::kOffEnd);
    W& w = reinterpret_cast<W*>(smem + G::kOffWalk)[warp];
    auto sync_rows = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + quad), "n"(32 * kSubs) : "memory"); };  // the warps of these rows

    // What is left to do for a segment once its last product is issued, and what its rows are.
    struct Segment {
      Sequence s;
      int32_t head, row_tile, node;
      bool begins, ends;
    };

    // q of this thread's part of the row, scaled by a power of two, into shared memory; the factor to undo it
    auto stage_q = [&](const Segment& g, float& row_scale) {
      const int at = g.row_tile * kRows + row;
      const bool live = g.node < g.s.nodes;
      uint4 raw[kMine / 8];
      uint32_t top = 0;
      const bool bf16 = p.dtype == QLIN_BF16;
      const uint8_t* src = p.q + (g.s.q_row + g.node) * p.qt + (g.head * p.group + at - g.node * p.group) * p.qh + sub * kMine * 2;
#pragma unroll
      for (int i = 0; i < kMine / 8; ++i) {
        raw[i] = live ? ldg_v4(src + i * 16) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = bf16 ? kv::unpack2<1>(u[k]) : kv::unpack2<0>(u[k]);
          top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
        }
      }
      q_max[sub * kRows + row] = top;
      sync_rows();
#pragma unroll
      for (int x = 1; x < kSubs; ++x) top = max(top, q_max[(sub ^ x) * kRows + row]);
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
      for (int i = 0; i < kMine / 8; ++i) {
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = bf16 ? kv::unpack2<1>(u[k]) : kv::unpack2<0>(u[k]);
          f[2 * k] = v.x * s1 * s2;
          f[2 * k + 1] = v.y * s1 * s2;
        }
        const int chunk = sub * (kMine / 8) + i;
        const uint32_t to = base + G::kOffQ + (chunk >> 3) * 16384 + half_chunk(row, chunk & 7);
        if constexpr (G::kU4)  // the order in which 4-bit codes are widened
          sts128(to, kv::pack2<0>(f[0], f[4]), kv::pack2<0>(f[1], f[5]), kv::pack2<0>(f[2], f[6]), kv::pack2<0>(f[3], f[7]));
        else
          sts128(to, kv::pack2<0>(f[0], f[1]), kv::pack2<0>(f[2], f[3]), kv::pack2<0>(f[4], f[5]), kv::pack2<0>(f[6], f[7]));
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_full);
    };

    auto segment = [&]() {
      Segment g;
      g.s = w.s;
      g.head = w.head;
      g.row_tile = w.row_tile;
      g.node = (w.row_tile * kRows + row) / p.group;
      g.begins = w.tile == 0;
      g.ends = w.tile + w.tiles == w.s.token_tiles;
      if (threadIdx.x == 0 && g.begins && !g.ends) p.records[blockIdx.x] = record_of(w, blocks, total);
      return g;
    };
    auto next = [&]() {
      bool more = false;
      __syncwarp();
      if (lane == 0) more = w.next(p);
      __syncwarp();
      return __shfl_sync(0xffffffffu, more, 0) != 0;
    };

    if (lane == 0) w = run;
    uint32_t t = 0;
    bool more = next();
    Segment g = segment();
    float row_scale;
    stage_q(g, row_scale);
    while (more) {
      float ref = kNoRef;
      uint64_t l2 = pair(0.0f, 0.0f);
      bool had_small = false;
      const int tiles = w.tiles, tile0 = w.tile;
      // where a moved reference puts the row's largest probability: with more tiles to come, six bits below the
      // top of fp16, which it may grow by before the row has to be rescaled
      const float put = tiles > 1 ? 9.0f : kOffset;
      for (int i = 0; i < tiles; ++i, ++t) {
        const uint32_t buf = t & 1;
        wait(s_full + 8 * buf, t >> 1, 0x6a);
        wait(col_full + 8 * (t % kCols), t / kCols, 0x6b);
        dead = __any_sync(0xffffffffu, dead);
        tc::tc_fence_after();
        const bool odd = odd_tile[t % kCols] == t + 1;  // read before it is needed: 40 cycles of a tile's 3900
        const uint32_t s_at = lanes + buf * 128;
        uint32_t v[kSpan];
        tc::tmem_ld_32x32b_x32(s_at + sub * kSpan, v);
        tc::tmem_wait_ld(v);
        const float* col = reinterpret_cast<const float*>(smem + G::kOffCol) + (t % kCols) * 4 * kTile + sub * kSpan;
        if (!__all_sync(0xffffffffu, row_scale == 1.0f)) {
          const uint64_t rs = pair(row_scale, row_scale);
#pragma unroll
          for (int k = 0; k < kSpan; k += 2) {
            const float2 a = unpair(mul2(pair(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), rs));
            v[k] = __float_as_uint(a.x);
            v[k + 1] = __float_as_uint(a.y);
          }
        }
        float hi = -INFINITY;
#pragma unroll
        for (int k = 0; k < kSpan; k += 4) {
          const float4 sk = *reinterpret_cast<const float4*>(col + k);
          const float4 ls = *reinterpret_cast<const float4*>(col + kTile + k);
          const float2 a = unpair(fma2(pair(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), pair(sk.x, sk.y), pair(ls.x, ls.y)));
          const float2 b =
              unpair(fma2(pair(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), pair(sk.z, sk.w), pair(ls.z, ls.w)));
          v[k] = __float_as_uint(a.x);
          v[k + 1] = __float_as_uint(a.y);
          v[k + 2] = __float_as_uint(b.x);
          v[k + 3] = __float_as_uint(b.y);
        }
        const int first = (tile0 + i) * kTile + sub * kSpan - g.s.ctx;  // the node that column 0 is
        if (first > -kSpan) {
          const uint32_t seen = static_cast<uint32_t>(seen_bits(p, g.s, g.node, first));
#pragma unroll
          for (int k = 0; k < kSpan; ++k)
            if (!((seen >> k) & 1u)) v[k] = 0xff800000u;
        }
#pragma unroll
        for (int k = 0; k < kSpan; ++k) hi = fmaxf(hi, __uint_as_float(v[k]));
        float* maxima = row_max + buf * kSubs * kRows + row;
        maxima[sub * kRows] = hi;
        sync_rows();
#pragma unroll
        for (int x = 1; x < kSubs; ++x) hi = fmaxf(hi, maxima[(sub ^ x) * kRows]);
        const bool move = hi > ref + (kOffset + kSlack);
        const float to = move ? hi - put : ref;
        const float keep = ex2(ref - to);
        ref = to;
        l2 = mul2(l2, pair(keep, keep));

        const uint64_t nref = pair(-ref, -ref), up = pair(kShiftUp, kShiftUp);
        uint32_t any_small = 0;
        auto weigh = [&](auto with_factors) {
          uint32_t pk[16], ps[16];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 rv = *reinterpret_cast<const float4*>(col + 2 * kTile + k);
            const float rr[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              const int i0 = k + x;
              const float2 a = unpair(add2(pair(__uint_as_float(v[i0]), __uint_as_float(v[i0 + 1])), nref));
              uint64_t e = pair(ex2(a.x), ex2(a.y));
              l2 = fma2(e, pair(rr[x], rr[x + 1]), l2);
              if constexpr (decltype(with_factors)::value) {  // (what is hidden has no product with a factor that is not a number)
                const float2 f = unpair(e);
                e = pair(v[i0] == 0xff800000u ? 0.0f : f.x * col[3 * kTile + i0],
                         v[i0 + 1] == 0xff800000u ? 0.0f : f.y * col[3 * kTile + i0 + 1]);
              }
              split(e, up, pk[i0 / 2], ps[i0 / 2]);
            }
            any_small |= ps[k / 2] | ps[k / 2 + 1];
          }
          tc::tmem_st_32x32b_x16(s_at + sub * kSpan / 2, pk);
          tc::tmem_st_32x32b_x16(s_at + 64 + sub * kSpan / 2, ps);
        };
        if (odd) weigh(std::true_type{});
        else weigh(std::false_type{});
        had_small = had_small || any_small != 0;
        if (__any_sync(0xffffffffu, any_small != 0) && lane == 0) small_tile[buf] = t + 1;
        if (__any_sync(0xffffffffu, move) && i > 0) {  // the same in all warps of these rows
          wait(pv_done + 8 * ((t - 1) & 1), (t - 1) >> 1, 0x6c);
          dead = __any_sync(0xffffffffu, dead);
          tc::tc_fence_after();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int cc = 0; cc < kMine; cc += 16) {
              const uint32_t at = lanes + (x == 0 ? kTmemO : kTmemO2) + sub * kMine + cc;
              uint32_t o[16];
              tc::tmem_ld_32x32b_x16(at, o);
              tc::tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 f = unpair(mul2(pair(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), pair(keep, keep)));
                o[k] = __float_as_uint(f.x);
                o[k + 1] = __float_as_uint(f.y);
              }
              tc::tmem_st_32x32b_x16(at, o);
            }
          }
        }
        __syncwarp();
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + 8 * buf);
      }

      // the next segment's q, then this one's output
      const Segment done = g;
      const float2 lp = unpair(l2);
      float l = lp.x + lp.y;
      ends[sub * kRows + row] = make_float2(l, had_small ? 1.0f : 0.0f);
      more = next();
      if (more) {
        g = segment();
        stage_q(g, row_scale);
      }
      sync_rows();
      l = 0.0f;  // in one order for all four
#pragma unroll
      for (int x = 0; x < kSubs; ++x) {
        const float2 e = ends[x * kRows + row];
        l += e.x;
        had_small = had_small || e.y != 0.0f;
      }
      wait(pv_done + 8 * ((t - 1) & 1), (t - 1) >> 1, 0x6d);
      dead = __any_sync(0xffffffffu, dead);
      tc::tc_fence_after();
      const bool live = done.node < done.s.nodes;
      const bool whole = done.begins && done.ends;
      const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : __frcp_rn(l);
      const float m = ref == kNoRef ? -INFINITY : ref + kOffset;
      const int head = done.head * p.group + done.row_tile * kRows + row - done.node * p.group;
      const int64_t tok = done.s.q_row + done.node;
      const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (done.begins ? 1 : 0)) * kRows + row;
#pragma unroll 1
      for (int cc = 0; cc < kMine; cc += 16) {
        uint32_t o[16], s[16];
        __syncwarp();
        tc::tmem_ld_32x32b_x16(lanes + kTmemO + sub * kMine + cc, o);
        tc::tmem_ld_32x32b_x16(lanes + kTmemO2 + sub * kMine + cc, s);
        tc::tmem_wait_ld(o);
        tc::tmem_wait_ld(s);
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          // 4-bit codes: column k of eight is channel k / 2 + 4 (k % 2)
          const int to = G::kU4 ? (k & 8) + ((k & 7) >> 1) + 4 * (k & 1) : k;
          // O2 holds anything until a tile with small ones
          f[to] = (__uint_as_float(o[k]) + (had_small ? __uint_as_float(s[k]) * kShiftDown : 0.0f)) * inv;
        }
        if (!live) continue;
        const int ch = sub * kMine + cc;
        if (whole) {
          uint8_t* to = p.out + tok * p.ot + head * p.oh + ch * 2;
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(to + k * 2) = p.dtype == QLIN_BF16 ? kv::pack8<1>(f + k) : kv::pack8<0>(f + k);
        } else {
          float* to = p.part_o + slot * D + ch;
#pragma unroll
          for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(to + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
      }
      if (live && sub == 0) {
        if (!whole) p.part_ml[slot] = make_float2(m, l);
        else if (p.lse != nullptr) p.lse[tok * p.hq + head] = (lg2(l) + (m - kOffset)) * kLn2;
      }
      tc::tc_fence_before();
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int D>
cudaError_t plan(const Params& p, Prepared* out) {
  const void* fn = reinterpret_cast<const void*>(tree_attention_wide_kernel<FMT, D>);
  const cudaError_t e = ensure_max_dynamic_smem(fn);
  if (e != cudaSuccess) return e;
  const uint32_t blocks = static_cast<uint32_t>(wide_blocks());
  const uint32_t rows = static_cast<uint32_t>(std::min<int64_t>(kRows, static_cast<int64_t>(p.max_nodes) * p.group));
  out->count = 2;
  out->launch[0] = {fn, blocks, 1, kThreads, Geo<FMT, D>::kSmem};
  out->launch[1] = {reinterpret_cast<const void*>(tree_attention_join_kernel<D>), blocks, rows, 128, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace

int wide_blocks() { return sm_count(); }

cudaError_t plan_wide(const Params& p, int fmt, int64_t head_dim, Prepared* out) {
  if (head_dim == 64) {
    if (fmt == QLIN_KV_INT8) return plan<QLIN_KV_INT8, 64>(p, out);
    if (fmt == QLIN_KV_E4M3) return plan<QLIN_KV_E4M3, 64>(p, out);
    return plan<QLIN_KV_U4, 64>(p, out);
  }
  if (fmt == QLIN_KV_INT8) return plan<QLIN_KV_INT8, 128>(p, out);
  if (fmt == QLIN_KV_E4M3) return plan<QLIN_KV_E4M3, 128>(p, out);
  return plan<QLIN_KV_U4, 128>(p, out);
}

}  // namespace tree
}  // namespace qlin
