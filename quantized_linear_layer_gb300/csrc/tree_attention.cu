// Attention of the new tokens of each sequence (one, a chain or a tree of
// drafts) over a paged, quantized key / value cache, on the warp-level tensor
// cores, split over the cached tokens.
//
// Mathematics.  With k_j = sk_j n_j and v_j = sv_j u_j (n, u the codes, small
// integers or E4M3 numbers, exact in fp16):
//   t_ij = log2(e) scale sk_j (q_i . n_j) + log2(sv_j)
//   o_i  = sum_j 2^(t_ij - m_i) u_j / sum_j 2^(t_ij - m_i) / sv_j
// for any reference m_i (scales that are zero, negative or out of range: usable_scale
// in tree_common.cuh), so the codes go to the tensor cores as they are and
// neither product rounds an operand except the probabilities 2^(t - m) (to
// fp16).  q rows are scaled by a power of two to below 2^15 before they become
// fp16: exact for fp16, and for bf16 down to 2^-31 of the row's largest (smaller
// elements in steps of 2^-39 of it).  The
// reference m_i follows the running maximum of t lazily: it moves when t
// exceeds it by more than 2, and the exponent carries an offset of 13, so that
// the probabilities lie below 2^15 and those down to 2^-27 of the reference are
// normal fp16 numbers.  Smaller ones matter where the large ones meet codes of
// 0: when a unit of 16 x 32 holds any, these go through a second product, times
// 2^24 against codes times 2^-24 (2^15 for E4M3), both exact in fp16, so that
// every probability keeps 11 bits down to 2^-51 (2^-42) of the largest.
//
// Work.  The rows of one key head (node, query head of the group) are cut
// into tiles of kRows = 16, the tokens into tiles of kTile = 32.  All (sequence,
// key head, row tile, token tile) units in this order are dealt out evenly to
// a grid that just fills the GPU: a block takes a run of units, which touches
// as many segments (sequence, head, row tile) as it happens to.  The division
// is worked out on the device from the lengths, so ragged batches and one long
// sequence load the GPU alike, and a captured call stays right when lengths
// change.  A segment cut by a block's border leaves float32 partial results
// (o, m, l), which a second kernel joins in the order of the blocks; a
// sequence's result depends on the lengths, not on timing.
//
// A block has five compute warps (six or seven where registers allow) and one that
// loads.  The loading warp keeps a ring of stages filled by asynchronous
// copies: one unit's codes of K and V (rows of 128, 64 or 32 bytes, their
// 16-byte chunks swizzled) and their scales.  Units go to the compute warps in
// turn; a warp takes all rows of its unit, with its own running maximum, sums
// and output, so that nothing but the ring lies between warps until a segment
// ends.  Codes are widened to fp16 in registers, straight into the operand
// layout of mma.m16n8k16: the order of channels in q . n and of output channels
// is permuted such that a lane's operands are contiguous bytes of a row, read
// without bank conflicts through the swizzle.
//
// Bound: up to eight rows per key head no unit is full (issue slots 38 %, HBM 5.1
// TB/s over equal lengths): a unit is one chain of about 700 instructions, ten
// compute and two loading warps share an SM at 168 registers, and shorter code in
// either has given a few percent each time.  64 ragged sequences of
// up to 8191 tokens, 8 key heads of 128, E4M3, one node of 32 query heads each:
// 141 us, 4540 GB/s (one copy would take 96 us); INT8 152, U4 189 (twice the
// widening for half the bytes); heads of 256, as many bytes, 163.  Twelve of the 16
// operand rows are padding there.  At 16 rows the widening takes as long as the loads.
// One sequence of 500 tokens, 32 heads: 11 us, two launches' latency.
//
// Chains whose scores have another form (ScoredParams: a cap, a bias by distance, a window, a
// prefix) are a variant of their own: a cap's exponential and reciprocal and the bias
// are a few instructions for each score, and of the tokens only the tiles that some
// row sees are units.  64 single tokens behind 1000, INT8, 32 heads on 8 of 128:
// 51 us plain, 61 capped, 50 with a window of 512; 4 x 4 behind 16000 with that
// window 22 (49 without).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "stage_ring.h"
#include "tree_common.cuh"

namespace qlin {
namespace {

constexpr int kTile = 32;
constexpr int kRows = 16;

using namespace tree;

// The geometry of one (format, head size).
template <int FMT, int D>
struct Geo {
  static constexpr bool kU4 = FMT == QLIN_KV_U4;
  static constexpr int kRowBytes = kU4 ? D / 2 : D;
  static constexpr int kSub = kRowBytes > 128 ? 2 : 1;      // 128-byte column blocks of a row
  static constexpr int kW = kRowBytes / kSub;               // bytes of a row in one of them
  static constexpr int kSubBytes = kTile * kW;
  static constexpr int kCodeBytes = kTile * kRowBytes;      // K or V of a stage
  static constexpr int kScaleBytes = kTile * 4;
  static constexpr int kStage = 2 * kCodeBytes;
  static constexpr int kPerSub = kU4 ? 2 * kW : kW;         // channels of a column block
  static constexpr int kKLane = kW / 4;                     // bytes of a row a lane takes for q . k
  static constexpr int kVLane = kW / 8;                     // and for p . v
  static constexpr int kNPerSub = kPerSub / 8;              // output tiles of a column block
  // 168 registers a thread (D = 128) let 12 warps live on an SM (ten compute), 128 (D = 64) 16 (14), 255 (D = 256) 8 (6 or 7)
  static constexpr int kBlocksPerSm = D == 256 ? 1 : 2;
  // (six stages of rows of 256 bytes fit beside the merge area: no more than six warps may take turns at them)
  static constexpr int kStages = kRowBytes >= 256 ? 6 : kRowBytes == 128 ? 8 : kRowBytes == 64 ? 12 : 16;
  static constexpr int kWarps = D == 128 ? 5 : kStages < 7 ? kStages : 7;
  static_assert(ring::turns_are_safe(kStages, kWarps), "a warp's wait could be a whole round of the ring ahead");
  static constexpr int kThreads = 32 * (kWarps + 1);
  // 2^24 (2^15 for E4M3): codes times 2^-kShift are fp16 numbers, exactly
  static constexpr float kShiftUp = FMT == QLIN_KV_E4M3 ? 32768.0f : 16777216.0f;
  static constexpr uint32_t kShiftDown = FMT == QLIN_KV_E4M3 ? 0x02000200u : 0x00010001u;
  // shared memory: stages, scales, merge area, q_max etc.
  static constexpr int kOffScale = kStages * kStage;
  static constexpr int kOffMerge = kOffScale + kStages * 2 * kScaleBytes;
  static constexpr int kMergeRow = D + 4;  // floats
  static constexpr int kOffMl = kOffMerge + kWarps * kRows * kMergeRow * 4;
  static constexpr int kOffFactor = kOffMl + kWarps * kRows * 8;  // [warp][token]: see usable_scale
  static constexpr int kOffBar = kOffFactor + kWarps * kTile * 4;
  static constexpr int kOffScan = kOffBar + 2 * kStages * 8;
  static constexpr int kOffWalk = (kOffScan + (kThreads + 1) * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffWalk + kWarps * static_cast<int>(sizeof(Walk<kRows, kTile>)) + 1024;  // + alignment of the base
  static_assert(kBlocksPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");

  // where 16-byte chunk c of row r of a column block lies
  static __device__ __forceinline__ uint32_t chunk(int r, int c) {
    const int s = kW == 128 ? (r & 7) : kW == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
    return static_cast<uint32_t>(r * kW + ((c ^ s) << 4));
  }
};

// P: Params, or ScoredParams or LargeCapParams (chains whose scores have another form).
template <int FMT, int D, class P>
__global__ void __launch_bounds__(Geo<FMT, D>::kThreads, Geo<FMT, D>::kBlocksPerSm)
    tree_attention_kernel(const __grid_constant__ P p) {
  constexpr bool kScored = kIsScored<P>;
  using G = Geo<FMT, D>;
  constexpr int kWarps = G::kWarps, kThreads = G::kThreads;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - tc::smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t bar_full = base + G::kOffBar, bar_free = bar_full + G::kStages * 8;
  int64_t* scan = reinterpret_cast<int64_t*>(smem + G::kOffScan);  // [kThreads + 1]

  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      tc::mbar_init(bar_full + 8 * i, 32);
      tc::mbar_init(bar_free + 8 * i, 1);
    }
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

  auto run = begin_run<kRows, kTile, kThreads>(p, share, scan, blockIdx.x, blocks);

  if (warp == kWarps) {  // ---- the loading warp
    auto& w = run;
    int stage = 0;
    uint32_t phase = 1;  // the first round finds every stage free
    bool dead = false;
    const int page = 1 << p.page_shift;
    const int box = min(page, kTile);
    const int boxes = kTile / box;  // of a unit
    const uint64_t policy = tc::l2_policy_evict_first();
    while (!dead && w.next(p)) {
      const int32_t* table = p.table + w.b * p.max_pages;
      int32_t ahead = kNoPage;  // the page of box `lane` of the 32 boxes from unit `from` on
      int from = 0;
      for (int t = w.tile; t < w.tile + w.tiles; ++t) {
        if (t == w.tile || (t - from) * boxes == 32 || (kScored && t == w.s.prefix_tiles)) {
          from = t;
          const int first = w.s.template token_tile<P>(t);
          // (up to where the tiles are those of consecutive tokens)
          const int past = kScored && t < w.s.prefix_tiles ? min(w.tile + w.tiles, w.s.prefix_tiles) : w.tile + w.tiles;
          const int j = first * kTile + lane * box;
          ahead = kNoPage;
          bool seen = j < min(w.s.len, (first + past - t) * kTile);
          if constexpr (kScored)  // a box that every window has left has no page: its number may be none by now
            seen = seen && (j < w.s.prefix || p.window == 0 || j + box > w.s.ctx - p.window + 1);
          if (seen) ahead = checked_page(p, table[j >> p.page_shift]);
        }
        if (!tc::mbar_wait_quiet(bar_free + 8 * stage, phase, p.err, 0x50)) dead = true;
        if (__any_sync(0xffffffffu, dead)) {
          dead = true;
          break;
        }
        const uint32_t codes = base + stage * G::kStage, scales = base + G::kOffScale + stage * 2 * G::kScaleBytes;
        auto row_at = [](int r, int c) { return c / (G::kW / 16) * G::kSubBytes + G::chunk(r, c % (G::kW / 16)); };
        const int at = (t - from) * boxes;
        const int j0 = w.s.template token_tile<P>(t) * kTile;
        copy_scales<kTile>(p, w.head, j0, box, ahead, at, scales, scales + G::kScaleBytes, policy);
        if (box == kTile)
          copy_codes<kTile, kTile, G::kRowBytes>(p, w.head, j0, ahead, at, codes, codes + G::kCodeBytes, policy, row_at);
        else
          copy_codes<kTile, 16, G::kRowBytes>(p, w.head, j0, ahead, at, codes, codes + G::kCodeBytes, policy, row_at);
        copies_arrive(bar_full + 8 * stage);
        if (++stage == G::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    copies_wait();  // none outlives the block, also where a wait ran out
    return;
  }

  // ---- the compute warps
  const int g = lane >> 2, r = lane & 3;
  uint32_t unit0 = 0;  // units of the run before this segment
  bool dead = false;  // a wait ran out: go on without waiting, so that every barrier is met
  // the walk stays in shared memory, out of the registers of the loop below
  Walk<kRows, kTile>& w = reinterpret_cast<Walk<kRows, kTile>*>(smem + G::kOffWalk)[warp];
  if (lane == 0) w = run;
  while (true) {
    bool more = false;
    __syncwarp();
    if (lane == 0) more = w.next(p);
    __syncwarp();
    if (!__shfl_sync(0xffffffffu, more, 0)) break;
    // q of this lane's rows g and g + 8, as fp16 operands scaled by a power of two
    uint32_t qa[D / 16][4];
    float row_scale[2], slope2[2] = {0.0f, 0.0f};
    int32_t row_node[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = w.row_tile * kRows + g + 8 * i;
      const int node = row / p.group;
      const bool live = node < w.s.nodes;
      row_node[i] = live ? node : -1;
      if constexpr (kScored) {
        if (p.slopes != nullptr && live) slope2[i] = -kLog2e * p.slopes[w.head * p.group + row - node * p.group];
      }
      const uint8_t* src = p.q + (w.s.q_row + node) * p.qt + (w.head * p.group + row - node * p.group) * p.qh;
      uint32_t raw[D / 8];  // this lane's D / 4 channels: kPerSub / 4 contiguous ones of each column block
      uint32_t top = 0;
#pragma unroll
      for (int h = 0; h < G::kSub; ++h) {
#pragma unroll
        for (int c = 0; c < G::kPerSub / 32; ++c) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live) v = ldg_v4(src + 2 * (h * G::kPerSub + r * (G::kPerSub / 4) + 8 * c));
          uint32_t* to = raw + h * (G::kPerSub / 8) + 4 * c;
          to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
        }
      }
      const bool bf16 = p.dtype == QLIN_BF16;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const float2 f = bf16 ? kv::unpack2<1>(raw[c]) : kv::unpack2<0>(raw[c]);
        top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = row_exponent(top);
      row_scale[i] = p.scale * kLog2e * power_of_two(e);
      const float down = power_of_two(-e);
      uint16_t q16[D / 4];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const float2 f = bf16 ? kv::unpack2<1>(raw[c]) : kv::unpack2<0>(raw[c]);
        const uint32_t u = kv::pack2<0>(f.x * down, f.y * down);
        q16[2 * c] = static_cast<uint16_t>(u);
        q16[2 * c + 1] = static_cast<uint16_t>(u >> 16);
      }
      // the order in which the widened codes of a lane's bytes meet the k index
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int x = G::kU4 ? 8 * (ks / 2) + 2 * (ks % 2) + h : 4 * ks + 2 * h;
          const int y = G::kU4 ? x + 4 : x + 1;
          qa[ks][i + 2 * h] = static_cast<uint32_t>(q16[x]) | (static_cast<uint32_t>(q16[y]) << 16);
        }
      }
    }

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float ref[2] = {kNoRef, kNoRef}, l[2] = {0.0f, 0.0f};

    // this warp's units of the segment
    uint32_t u = unit0 + (warp + kWarps - unit0 % kWarps) % kWarps;
    const bool took = u < unit0 + w.tiles;
    for (; u < unit0 + w.tiles; u += kWarps) {
      const uint32_t stage = u % G::kStages;
      if (!dead) dead = !tc::mbar_wait_quiet(bar_full + 8 * stage, (u / G::kStages) & 1, p.err, 0x51);
      dead = __any_sync(0xffffffffu, dead);
      const int j0 = w.s.template token_tile<P>(w.tile + static_cast<int>(u - unit0)) * kTile;  // the unit's first token
      const uint32_t ks_at = base + stage * G::kStage;
      const uint32_t vs_at = ks_at + G::kCodeBytes;
      const uint8_t* sc = smem + G::kOffScale + stage * 2 * G::kScaleBytes;
      bool masked = j0 + kTile > w.s.ctx;
      if constexpr (kScored)
        masked = j0 + kTile > w.s.prefix && (masked || (p.window > 0 && w.s.ctx + w.s.nodes - 1 - j0 >= p.window));

      // odd value scales of the unit (it is this warp's alone until it is given free), those behind the end among them
      float* factors = reinterpret_cast<float*>(smem + G::kOffFactor) + warp * kTile;
      bool odd = false;  // a token of the sequence has one
      {
        uint32_t* of_k = reinterpret_cast<uint32_t*>(smem + G::kOffScale + stage * 2 * G::kScaleBytes) + lane;
        uint32_t* word = of_k + kTile;
        bool mine = odd_scale<FMT>(*word);
        if constexpr (G::kU4) mine = mine || odd_zero(*of_k) || odd_zero(*word);
        bool nan_codes = false;  // among the values of tokens that some row does not see, or behind the end
        if constexpr (FMT == QLIN_KV_E4M3) {
          if (masked && (kScored || j0 + lane >= w.s.ctx)) {
#pragma unroll 1
            for (int c = 0; c < G::kRowBytes / 16; ++c)
              nan_codes |= clear_nan_codes(vs_at + c / (G::kW / 16) * G::kSubBytes + G::chunk(lane, c % (G::kW / 16)));
          }
          mine = mine || nan_codes;
        }
        if (__any_sync(0xffffffffu, mine)) {
          odd = __any_sync(0xffffffffu, mine && j0 + lane < w.s.len);
          float factor = 1.0f;
          if (mine) {
            uint32_t v = *word;
            if (odd_scale<FMT>(v)) v = usable_scale<FMT>(v, factor);
            if constexpr (G::kU4) {  // without a zero-point a token is not a number: its score, or its factor
              if (odd_zero(*of_k)) *of_k = 0x7fffu;
              if (odd_zero(v)) v &= 0xffffu, factor = __uint_as_float(0x7fc00000u);
            }
            if (nan_codes) factor = __uint_as_float(0x7fc00000u);
            *word = v;
          }
          factors[lane] = factor;
          __syncwarp();
        }
      }

      // scores of 16 rows x 32 tokens; this lane's: rows g, g + 8, tokens 8 n + 2 r + {0, 1}
      float s[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
        const int tok = 8 * n + g;
        uint32_t kz = 0;
        if constexpr (G::kU4) {
          const uint32_t kw = *reinterpret_cast<const uint32_t*>(sc + tok * 4);
          const __half2 b = __hadd2(__half2half2(__ushort_as_half(static_cast<unsigned short>(kw >> 16))),
                                    __float2half2_rn(1024.0f));
          kz = *reinterpret_cast<const uint32_t*>(&b);
        }
#pragma unroll
        for (int h = 0; h < G::kSub; ++h) {
          constexpr int kLoad = G::kKLane < 16 ? G::kKLane : 16;
#pragma unroll
          for (int c = 0; c < G::kKLane / kLoad; ++c) {
            uint32_t wd[4];
            const int byte = r * G::kKLane + c * 16;
            lds<kLoad>(ks_at + h * G::kSubBytes + G::chunk(tok, byte / 16) + byte % 16, wd);
#pragma unroll
            for (int i = 0; i < kLoad / 4; ++i) {
              if constexpr (G::kU4) {
                const int ks = h * (G::kPerSub / 16) + (c * (kLoad / 4) + i) * 2;
                const uint32_t x0 = hsub2((wd[i] & 0x000f000fu) | kMagic, kz);
                const uint32_t x1 = hsub2(((wd[i] >> 4) & 0x000f000fu) | kMagic, kz);
                const uint32_t x2 = hsub2(((wd[i] >> 8) & 0x000f000fu) | kMagic, kz);
                const uint32_t x3 = hsub2(((wd[i] >> 12) & 0x000f000fu) | kMagic, kz);
                mma16816(s[n], qa[ks], x0, x1);
                mma16816(s[n], qa[ks + 1], x2, x3);
              } else {
                const int ks = h * (G::kPerSub / 16) + c * (kLoad / 4) + i;
                uint32_t lo, hi;
                widen4<FMT>(wd[i], lo, hi);
                mma16816(s[n], qa[ks], lo, hi);
              }
            }
          }
        }
      }

      // t, hiding what a row does not see
      float rsv[8];
      uint32_t vz[4];  // U4: 1024 + the zero-points of the tokens, per pair
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int tok = 8 * n + 2 * r;
        const uint2 kw = *reinterpret_cast<const uint2*>(sc + tok * 4);
        const uint2 vw = *reinterpret_cast<const uint2*>(sc + G::kScaleBytes + tok * 4);
        const uint32_t kws[2] = {kw.x, kw.y}, vws[2] = {vw.x, vw.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float sk, sv;
          if constexpr (G::kU4) {
            sk = __half2float(__ushort_as_half(static_cast<unsigned short>(kws[i] & 0xffffu)));
            sv = __half2float(__ushort_as_half(static_cast<unsigned short>(vws[i] & 0xffffu)));
          } else {
            sk = __uint_as_float(kws[i]);
            sv = __uint_as_float(vws[i]);
          }
          const float lsv = lg2(sv);
          rsv[2 * n + i] = rcp(sv);
          if constexpr (kScored) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float t = s[n][2 * x + i] * row_scale[x] * sk;
              if (p.softcap > 0.0f) {
                const float cap2 = p.softcap * kLog2e, at = t * __fdividef(2.0f, p.softcap);
                t = std::is_same<P, LargeCapParams>::value ? large_capped(at, cap2) : capped(at, cap2);
              }
              if (p.slopes != nullptr) t = fmaf(slope2[x], fabsf(static_cast<float>(w.s.ctx + row_node[x] - j0 - tok - i)), t);
              s[n][2 * x + i] = t + lsv;
            }
          } else {
            s[n][i] = fmaf(s[n][i] * row_scale[0], sk, lsv);
            s[n][2 + i] = fmaf(s[n][2 + i] * row_scale[1], sk, lsv);
          }
        }
        if constexpr (G::kU4) {
          const uint32_t z = __byte_perm(vw.x, vw.y, 0x7632);
          const __half2 b = __hadd2(*reinterpret_cast<const __half2*>(&z), __float2half2_rn(1024.0f));
          vz[n] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      if (masked) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + 8 * n + 2 * r + (i & 1) - w.s.ctx;  // the node that the token is
            const int node = row_node[i >> 1];
            bool seen = j < 0;
            if constexpr (kScored) {
              seen = node >= 0 && j < w.s.nodes && (j + w.s.ctx < w.s.prefix || (j <= node && (p.window == 0 || node - j < p.window)));
            } else if (!seen && j < w.s.nodes && node >= 0) {
              seen = p.mask == nullptr
                         ? j <= node
                         : ((p.mask[(w.s.q_row + node) * p.mask_words + (j >> 6)] >> (j & 63)) & 1) != 0;
            }
            if (!seen) s[n][i] = -INFINITY;
          }
        }
      }

      // move the reference where t leaves it behind
      float hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        hi[i] = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
        lo[i] = fminf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
        for (int n = 1; n < 4; ++n) {
          hi[i] = fmaxf(hi[i], fmaxf(s[n][2 * i], s[n][2 * i + 1]));
          lo[i] = fminf(lo[i], fminf(s[n][2 * i], s[n][2 * i + 1]));
        }
      }
      if (__any_sync(0xffffffffu, fmaxf(hi[0] - ref[0], hi[1] - ref[1]) > kOffset + kSlack)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = hi[i];
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float to = fmaxf(ref[i], top - kOffset);
          const float keep = ex2(ref[i] - to);
          ref[i] = to;
          l[i] *= keep;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            o[c][2 * i] *= keep;
            o[c][2 * i + 1] *= keep;
          }
        }
      }
      const bool small = odd || __any_sync(0xffffffffu, fminf(lo[0] - ref[0], lo[1] - ref[1]) < kHalfExp);
      uint32_t pa[4][2];
      auto weigh = [&](auto with_factors) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float t = s[n][i];
            s[n][i] = ex2(t - ref[i >> 1]);
            l[i >> 1] = fmaf(s[n][i], rsv[2 * n + (i & 1)], l[i >> 1]);
            if constexpr (decltype(with_factors)::value)  // (what is hidden has no product with a factor that is not a number)
              s[n][i] = t == -INFINITY ? 0.0f : s[n][i] * factors[8 * n + 2 * r + (i & 1)];
          }
          pa[n][0] = kv::pack2<0>(s[n][0], s[n][1]);
          pa[n][1] = kv::pack2<0>(s[n][2], s[n][3]);
        }
      };
      if (odd) weigh(std::true_type{});
      else weigh(std::false_type{});

      // p . v: the lane's tokens 16 k + 2 r + {0, 1, 8, 9}, contiguous channels of each
      auto accumulate = [&](auto shifted) {
        constexpr bool kShifted = decltype(shifted)::value;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t pr[4] = {pa[2 * k][0], pa[2 * k][1], pa[2 * k + 1][0], pa[2 * k + 1][1]};
          auto product = [&](float* acc, uint32_t b0, uint32_t b1) {
            if constexpr (kShifted) {
              b0 = hmul2(b0, G::kShiftDown);
              b1 = hmul2(b1, G::kShiftDown);
            }
            mma16816(acc, pr, b0, b1);
          };
#pragma unroll
          for (int h = 0; h < G::kSub; ++h) {
            constexpr int kLoad = G::kVLane;  // 16, 8 or 4 bytes
            uint32_t wd[4][kLoad / 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = 16 * k + 2 * r + (i & 1) + 8 * (i >> 1);
              const int byte = g * kLoad;
              lds<kLoad>(vs_at + h * G::kSubBytes + G::chunk(tok, byte / 16) + byte % 16, wd[i]);
            }
#pragma unroll
            for (int c = 0; c < kLoad / 4; ++c) {
              if constexpr (G::kU4) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint32_t sel = half ? 0x7632u : 0x5410u;
                  const uint32_t a = __byte_perm(wd[0][c], wd[1][c], sel), b = __byte_perm(wd[2][c], wd[3][c], sel);
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    product(o[h * G::kNPerSub + 8 * c + 4 * half + i],
                            hsub2(((a >> (4 * i)) & 0x000f000fu) | kMagic, vz[2 * k]),
                            hsub2(((b >> (4 * i)) & 0x000f000fu) | kMagic, vz[2 * k + 1]));
                }
              } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint32_t sel = half ? 0x7362u : 0x5140u;
                  uint32_t a0, a1, b0, b1;
                  widen4<FMT>(__byte_perm(wd[0][c], wd[1][c], sel), a0, a1);
                  widen4<FMT>(__byte_perm(wd[2][c], wd[3][c], sel), b0, b1);
                  const int n = h * G::kNPerSub + 4 * c + 2 * half;
                  product(o[n], a0, b0);
                  product(o[n + 1], a1, b1);
                }
              }
            }
          }
        }
      };
      if (small) {
        // some lie below fp16's normal range: these times 2^kShift first, then the others
        uint32_t rest[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = s[n][2 * h], b = s[n][2 * h + 1];
            const bool sa = fabsf(a) < kHalfNormal, sb = fabsf(b) < kHalfNormal;
            rest[n][h] = kv::pack2<0>(sa ? 0.0f : a, sb ? 0.0f : b);
            pa[n][h] = kv::pack2<0>(sa ? a * G::kShiftUp : 0.0f, sb ? b * G::kShiftUp : 0.0f);
          }
        accumulate(std::true_type{});
#pragma unroll
        for (int n = 0; n < 4; ++n) pa[n][0] = rest[n][0], pa[n][1] = rest[n][1];
      }
      accumulate(std::false_type{});
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_free + 8 * stage);
    }
    unit0 += w.tiles;

    // join the warps: each scaled to the common reference
    float* area = reinterpret_cast<float*>(smem + G::kOffMerge);
    float2* ml = reinterpret_cast<float2*>(smem + G::kOffMl);  // [warp][row]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (r == 0) ml[warp * kRows + g + 8 * i] = make_float2(ref[i] == kNoRef ? -INFINITY : ref[i] + kOffset, l[i]);
      if (!took) continue;
      float* to = area + (warp * kRows + g + 8 * i) * G::kMergeRow;
#pragma unroll
      for (int h = 0; h < G::kSub; ++h)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int c = 0; c < G::kNPerSub; c += 4) {
            const int n = h * G::kNPerSub + c;
            *reinterpret_cast<float4*>(to + h * G::kPerSub + (2 * r + y) * G::kNPerSub + c) =
                make_float4(o[n][2 * i + y], o[n + 1][2 * i + y], o[n + 2][2 * i + y], o[n + 3][2 * i + y]);
          }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    const bool begins = w.tile == 0, ends = w.tile + w.tiles == w.s.token_tiles;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (begins ? 1 : 0);
    constexpr int kPer = D / 4;  // threads a row
    for (int row = threadIdx.x / kPer; row < kRows; row += 32 * kWarps / kPer) {
      const int c = threadIdx.x % kPer * 4;
      const int at = w.row_tile * kRows + row;
      const int node = at / p.group;
      if (node >= w.s.nodes) break;
      float2 e[kWarps];
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        e[i] = ml[i * kRows + row];
        top = fmaxf(top, e[i].x);
      }
      float sum = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        // a warp that saw nothing has o = l = 0 (and may not have written o), or NaN where the query is NaN
        if (e[i].x == -INFINITY && e[i].y == 0.0f) continue;
        const float f = e[i].x == -INFINITY ? 1.0f : ex2(e[i].x - top);
        const float4 v = *reinterpret_cast<const float4*>(area + (i * kRows + row) * G::kMergeRow + c);
        sum += f * e[i].y;
        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
      }
      if (begins && ends) {
        const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        const int head = w.head * p.group + at - node * p.group;
        const int64_t tok = w.s.q_row + node;
        const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
        const uint2 u = p.dtype == QLIN_BF16 ? make_uint2(kv::pack2<1>(v[0], v[1]), kv::pack2<1>(v[2], v[3]))
                                              : make_uint2(kv::pack2<0>(v[0], v[1]), kv::pack2<0>(v[2], v[3]));
        *reinterpret_cast<uint2*>(p.out + tok * p.ot + head * p.oh + c * 2) = u;
        if (p.lse != nullptr && c == 0) p.lse[tok * p.hq + head] = (lg2(sum) + (top - kOffset)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * kRows + row) * D + c) = acc;
        if (c == 0) p.part_ml[slot * kRows + row] = make_float2(top, sum);
      }
    }
    if (begins && !ends && threadIdx.x == 0) p.records[blockIdx.x] = record_of(w, blocks, total);
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");  // the merge area is free again
  }
}

int grid_blocks(int64_t head_dim) { return sm_count() * (head_dim == 256 ? 1 : 2); }

template <int FMT, int D, class P>
cudaError_t plan(const P& p, Prepared* out) {
  using G = Geo<FMT, D>;
  const void* fn = reinterpret_cast<const void*>(tree_attention_kernel<FMT, D, P>);
  const cudaError_t e = ensure_max_dynamic_smem(fn);
  if (e != cudaSuccess) return e;
  const uint32_t blocks = static_cast<uint32_t>(grid_blocks(D));
  const uint32_t rows = static_cast<uint32_t>(std::min<int64_t>(kRows, static_cast<int64_t>(p.max_nodes) * p.group));
  out->count = 2;
  out->launch[0] = {fn, blocks, 1, G::kThreads, G::kSmem};
  out->launch[1] = {reinterpret_cast<const void*>(tree_attention_join_kernel<D>), blocks, rows, 128, 0};
  out->set(p);
  return cudaSuccess;
}

template <int FMT, class P>
cudaError_t plan(const P& p, int64_t d, Prepared* out) {
  if (d == 64) return plan<FMT, 64>(p, out);
  if (d == 128) return plan<FMT, 128>(p, out);
  return plan<FMT, 256>(p, out);
}

}  // namespace

namespace tree {

// Rows of one key head above which a tile of 128 rows on tcgen05 beats tiles of 16 on the warp-level tensor cores: a
// second tile of 16 doubles the time here, while the wide kernel's hardly depends on the rows.  16 sequences of 16384
// tokens, 8 key heads of 128, INT8, this kernel / the wide one: 16 rows 131 / 225 us, 20 rows 242 / 223, 64 rows 472 /
// 233; 4 sequences of 600 tokens: 19.7 / 17.9, 19.2 / 18.9, 22.9 / 26.6.  A head of 256 channels does not fit the wide
// kernel's tensor memory.
bool use_wide(int64_t head_dim, int64_t rows) { return head_dim <= 128 && rows > 16; }

}  // namespace tree

namespace {

struct Shape {
  bool wide;
  int64_t blocks, rows;  // of the grid, and of a row tile
};

Shape shape_of(const qlin_kv_cache& cache, int64_t hq, int64_t max_nodes) {
  Shape s;
  s.wide = use_wide(cache.head_dim, max_nodes * (hq / cache.heads));
  s.blocks = s.wide ? wide_blocks() : grid_blocks(cache.head_dim);
  s.rows = s.wide ? 128 : kRows;
  return s;
}

}  // namespace

int64_t tree_attention_workspace_bytes(const qlin_kv_cache& cache, int64_t hq, int64_t max_nodes, int64_t) {
  const Shape s = shape_of(cache, hq, max_nodes);
  return s.blocks * static_cast<int64_t>(sizeof(Record)) + 256 +
         2 * s.blocks * s.rows * (cache.head_dim * 4 + static_cast<int64_t>(sizeof(float2)));
}

namespace {

void fill(Params& p, const TreeAttentionArgs& a, const Shape& shape) {
  const qlin_kv_cache& c = a.cache;
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
  p.mask = a.mask;
  p.mask_words = static_cast<int32_t>(a.mask_words);
  p.max_nodes = static_cast<int32_t>(a.max_nodes);
  p.scale = a.scale;
  p.lse = a.lse;
  p.tile_rows = static_cast<int32_t>(shape.rows);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  ws += 2 * shape.blocks * shape.rows * c.head_dim * 4;
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += 2 * shape.blocks * shape.rows * static_cast<int64_t>(sizeof(float2));
  p.records = reinterpret_cast<Record*>(ws);
  p.err = device_error_word();
}

template <class P>
cudaError_t plan(const P& p, const qlin_kv_cache& c, Prepared* out) {
  if (c.fmt == QLIN_KV_INT8) return plan<QLIN_KV_INT8>(p, c.head_dim, out);
  if (c.fmt == QLIN_KV_E4M3) return plan<QLIN_KV_E4M3>(p, c.head_dim, out);
  return plan<QLIN_KV_U4>(p, c.head_dim, out);
}

}  // namespace

cudaError_t plan_tree_attention(const TreeAttentionArgs& a, Prepared* out) {
  const qlin_kv_cache& c = a.cache;
  const Shape shape = shape_of(c, a.q.heads, a.max_nodes);
  Params p = {};
  fill(p, a, shape);
  return shape.wide ? plan_wide(p, c.fmt, c.head_dim, out) : plan(p, c, out);
}

cudaError_t plan_chain_attention(const TreeAttentionArgs& a, const qlin_scores& scores, Prepared* out) {
  LargeCapParams p = {};
  fill(p, a, shape_of(a.cache, a.q.heads, a.max_nodes));
  p.softcap = scores.softcap;
  p.slopes = scores.slopes;
  p.window = scores.window >= kMaxLen ? 0 : static_cast<int32_t>(scores.window);  // no sequence is longer
  p.prefix = scores.prefix_lens;
  return p.softcap > kPlainCap ? plan(p, a.cache, out) : plan(static_cast<const ScoredParams&>(p), a.cache, out);
}

}  // namespace qlin
