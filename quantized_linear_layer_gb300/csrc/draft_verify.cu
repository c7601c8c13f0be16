// Drafted tokens verified against the target's probabilities, and the next
// token drawn, from given random numbers.
//
// Mathematics.  At the node reached so far, with target row p and draft row q,
// the children are tried in order.  After k rejections there the target is
// left with
//   r_k = max(p - c_k q, 0),  W_k = sum r_k,  c_0 = 0, W_0 = 1, c_{k+1} = c_k + W_k
// (taking the draft's share away k times, max(r_{k-1} - W_{k-1} q, 0), in closed
// form), and a child with token x is accepted when u W_k q(x) < r_k(x).  Where no
// child is, the next token is drawn from r_k.  Without draft probabilities a
// rejected token leaves p: r_k is p without the rejected tokens, W_{k+1} =
// W_k - p(x), accepted when u W_k < p(x).
//
// Sums are of integers, in steps of 2^-52, so they are exact and do not depend on
// any order: the threads may take a row apart in any way and the token found is
// the one of the definition.  (A float32 sum over a row of 128256 would miss it once in
// some dozens of draws.)
//
// A cluster of two to eight blocks takes a sequence.  What the decisions read,
// one number of p and of q for each node, is loaded for all nodes at once; a row
// is read only where a sum is needed, so a sequence costs one row of the target
// and, after a rejection, one of the draft.  Each of the cluster's warps sums a
// contiguous part of the row, the loads of a turn under way while the turn
// before is summed; after the blocks have exchanged the sums, the block whose
// part holds the drawn place looks it up there (its part comes from L2), a piece
// to a warp.
//
// Bound: memory while rows are summed (64 sequences of 128256 tokens with a rejection
// each: 66 MB in some 11 us; repeated, 51 MB of it come from DRAM and the rest from L2),
// a chain of dependent reads before and behind: lengths, nodes, their
// probabilities, the walk, the sums' exchange, the look-up, 8 us together.
// 64 chains of 128256 tokens take 25.6 us (66 MB at most: 9.9 us at the copy rate),
// one of 32000 8.6 us, 32 trees of 50257 12.6 us.
#include <algorithm>

#include "kv_common.cuh"
#include "qlin_internal.h"
#include "tc_common.cuh"

namespace qlin {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNodes = 256;
constexpr uint64_t kOne = uint64_t(1) << 52;
constexpr uint64_t kFull = ~uint64_t(0);  // a sum that does not fit: no row of probabilities

struct Params {
  const float* target;
  const float* draft;
  int64_t target_stride, draft_stride, V;
  const int32_t* parents;
  const int64_t* tokens;
  const int32_t* q_indptr;
  const float* accept;
  const float* sample;
  int32_t* path;
  int32_t* count;
  int64_t* next;
  int64_t Tq;
  int32_t max_nodes;
  int32_t wide;  // rows of both arrays begin on 16 bytes
  int32_t* err;
};

// A probability (what is not in [0, 1] counts as the end it is nearest to, what is no number as 0) in steps of 2^-52.
__device__ __forceinline__ uint64_t steps(float x) {
  const uint32_t b = __float_as_uint(__saturatef(x));
  const uint64_t m = static_cast<uint64_t>((b & 0x7fffffu) | 0x800000u) << 29;  // 1.f at 2^52
  uint64_t w;
  asm("shr.b64 %0, %1, %2;" : "=l"(w) : "l"(m), "r"(127u - (b >> 23)));  // (0 from 64 on)
  return w;
}

// c q, both in steps (c below 2^61, q at most one).
__device__ __forceinline__ uint64_t times(uint64_t c, uint64_t q) { return __umul64hi(c << 2, q << 10); }

__device__ __forceinline__ uint64_t add_full(uint64_t a, uint64_t b) {
  const uint64_t s = a + b;
  return s < a ? kFull : s;
}

// A number of [0, 1) in steps of 2^-64 (what lies outside counts as the nearest inside).
__device__ __forceinline__ uint64_t fraction(float u) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(u, 0.0f), 0.99999994f));
  const uint64_t m = static_cast<uint64_t>((b & 0x7fffffu) | 0x800000u) << 40;  // 0.1f at 2^64
  return m >> min(126u - (b >> 23), 63u);
}

__device__ __forceinline__ float unit(float x) { return fminf(fmaxf(x, 0.0f), 1.0f); }

struct Shared {
  int32_t parent[kMaxNodes];
  int64_t token[kMaxNodes];
  double p[kMaxNodes], q[kMaxNodes], u[kMaxNodes];
  double share[kMaxNodes];  // p in whole steps
  int32_t path[kMaxNodes];
  int64_t gone[kMaxNodes];  // tokens rejected at this node (no draft probabilities)
  uint64_t own[2][kWarps];  // this block's sums, of this pass and of the one before
  uint64_t part[kMaxCluster * kWarps];  // all of the cluster's
  uint64_t total;
  uint64_t c;               // the pass asked for
  int32_t at, rejected, done;
  int32_t plain;            // nothing was left of the row at `at`: it is taken as it is
  int32_t holder;           // the warp whose part holds the drawn place, and what lies before it
  uint64_t base;
  uint64_t piece[kWarps];   // sums of the pieces of that part
};

// What is left of a number.  After one rejection c is one.
enum class Gone { kNothing, kOnce, kMore };
template <Gone GONE>
__device__ __forceinline__ uint64_t weight(float p, float q, uint64_t c) {
  const uint64_t w = steps(p);
  if (GONE == Gone::kNothing) return w;
  const uint64_t gone = GONE == Gone::kOnce ? steps(q) : times(c, steps(q));
  return w > gone ? w - gone : 0;
}
__device__ __forceinline__ uint64_t weight(float p, float q, uint64_t c) {
  return c == 0 ? weight<Gone::kNothing>(p, q, c) : weight<Gone::kMore>(p, q, c);
}

// Four numbers of a row from element i on; those from `end` on are 0.
template <bool WIDE>
__device__ __forceinline__ float4 load4(const float* row, int64_t i, int64_t end) {
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (WIDE) {
    if (i + 3 < end) x = __ldcg(reinterpret_cast<const float4*>(row + i));
  } else {
    if (i < end) x.x = __ldcg(row + i);
    if (i + 1 < end) x.y = __ldcg(row + i + 1);
    if (i + 2 < end) x.z = __ldcg(row + i + 2);
    if (i + 3 < end) x.w = __ldcg(row + i + 3);
  }
  return x;
}

// What is left of the numbers begin .. begin + 3, begin + 128 .. begin + 131 and so on before `end`, of a lane.  While the numbers
// of one turn are summed those of the next are on their way.
template <bool WIDE, Gone GONE>
__device__ __forceinline__ uint64_t sum_left(const float* prow, const float* qrow, uint64_t c, int64_t begin, int64_t end) {
  constexpr bool kBoth = GONE != Gone::kNothing;
  constexpr int kAtOnce = kBoth ? 2 : 4, kTurn = kAtOnce * 128;
  float4 x[kAtOnce], y[kAtOnce];
  auto load = [&](int64_t i) {
#pragma unroll
    for (int g = 0; g < kAtOnce; ++g) {
      x[g] = load4<WIDE>(prow, i + g * 128, end);
      if (kBoth) y[g] = load4<WIDE>(qrow, i + g * 128, end);
    }
  };
  load(begin);
  uint64_t sum = 0;
#pragma unroll 1
  for (int64_t i = begin; i < end; i += kTurn) {
    float4 a[kAtOnce], b[kAtOnce];
#pragma unroll
    for (int g = 0; g < kAtOnce; ++g) {
      a[g] = x[g];
      if (kBoth) b[g] = y[g];
    }
    load(i + kTurn);
#pragma unroll
    for (int g = 0; g < kAtOnce; ++g)
      sum += (weight<GONE>(a[g].x, b[g].x, c) + weight<GONE>(a[g].y, b[g].y, c)) +
             (weight<GONE>(a[g].z, b[g].z, c) + weight<GONE>(a[g].w, b[g].w, c));
  }
  if (WIDE) {  // a row's last numbers that are not four
    const int64_t tail = end & ~int64_t(3);
    if (tail < end && tail >= begin && (tail - begin) % 128 == 0)
      for (int64_t i = tail; i < end; ++i) sum += weight<GONE>(__ldcg(prow + i), kBoth ? __ldcg(qrow + i) : 0.0f, c);
  }
  return sum;
}
template <bool WIDE>
__device__ __forceinline__ uint64_t sum_left(const float* prow, const float* qrow, uint64_t c, int64_t begin, int64_t end) {
  return c == 0      ? sum_left<WIDE, Gone::kNothing>(prow, qrow, c, begin, end)
         : c == kOne ? sum_left<WIDE, Gone::kOnce>(prow, qrow, c, begin, end)
                     : sum_left<WIDE, Gone::kMore>(prow, qrow, c, begin, end);
}
// (one piece of code for both of its uses: a launch begins with no instructions in the caches)
__device__ __noinline__ uint64_t sum_left(bool wide, const float* prow, const float* qrow, uint64_t c, int64_t begin,
                                          int64_t end) {
  return wide ? sum_left<true>(prow, qrow, c, begin, end) : sum_left<false>(prow, qrow, c, begin, end);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint64_t load_remote(uint32_t addr, int rank) {
  uint64_t v;
  asm volatile("{ .reg .u32 a; mapa.shared::cluster.u32 a, %1, %2; ld.shared::cluster.u64 %0, [a]; }" : "=l"(v) : "r"(addr), "r"(rank) : "memory");
  return v;
}

template <int CLUSTER>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(kThreads, 2) draft_verify_kernel(const __grid_constant__ Params p) {
  constexpr int kParts = CLUSTER * kWarps;  // (a multiple of 32)
  __shared__ Shared s;
  const int rank = blockIdx.x % CLUSTER, t = threadIdx.x, lane = t % 32, warp = t / 32;
  const int64_t b = blockIdx.x / CLUSTER;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t q0 = p.q_indptr[b];
  int64_t n = static_cast<int64_t>(p.q_indptr[b + 1]) - q0;
  if (q0 < 0 || n < 0 || q0 + n > p.Tq || n > p.max_nodes) {
    if (t == 0) record_device_error(p.err, kDevErrBadIndex);
    n = 0;
  }
  if (n == 0) {  // all blocks of the cluster alike
    if (rank == 0) {
      for (int i = t; i < p.max_nodes; i += kThreads) p.path[b * p.max_nodes + i] = -1;
      if (t == 0) p.count[b] = 0, p.next[b] = -1;
    }
    return;
  }
  if (t < n) {
    const int64_t row = q0 + t;
    int32_t parent = t == 0 ? -1 : p.parents != nullptr ? p.parents[row] : t - 1;
    const int64_t token = t == 0 ? 0 : p.tokens[row];
    float pp = 0.0f, qq = 0.0f;
    if (t > 0) {
      if (parent < 0 || parent >= t || token < 0 || token >= p.V) {
        record_device_error(p.err, kDevErrBadIndex);
        parent = -1;  // nobody's child
      } else {
        pp = unit(__ldcg(p.target + (q0 + parent) * p.target_stride + token));
        if (p.draft != nullptr) qq = unit(__ldcg(p.draft + (q0 + parent) * p.draft_stride + token));
      }
    }
    s.parent[t] = parent;
    s.token[t] = token;
    s.p[t] = pp;
    s.q[t] = qq;
    s.u[t] = t == 0 ? 0.0f : fminf(unit(p.accept[row]), 0.99999994f);
    s.share[t] = static_cast<double>(steps(pp)) * 0x1p-52;
  }
  if (t == 0) {
    s.path[0] = 0;
    s.holder = -1;
  }
  __syncthreads();

  // The walk is thread 0's, the same in every block of the cluster; sums are everybody's.
  int at = 0, length = 1, child = 1, rejected = 0, pass = 0;
  uint64_t c = 0, w = kOne;
  double left = 1.0;  // W: that of w, or without draft probabilities what the rejected tokens leave
  const int64_t span = (p.V + kParts * 128 - 1) / (kParts * 128) * 128;  // of a warp
  const int64_t begin = (static_cast<int64_t>(rank) * kWarps + warp) * span, end = min(begin + span, p.V);
  bool have = false;   // the sums at hand are those of (at, c)
  bool plain = false;  // s.plain
  while (true) {
    if (t == 0) {
      bool ask = false;
      for (; child < n && !ask; ++child) {
        if (s.parent[child] != at) continue;
        bool seen = false;
        for (int i = 0; i < rejected && !seen; ++i) seen = s.gone[i] == s.token[child];
        double rest = seen ? 0.0 : s.p[child], need = s.u[child] * left;
        if (p.draft != nullptr) {
          if (c != 0) rest = fmax(rest - static_cast<double>(c) * 0x1p-52 * s.q[child], 0.0);
          need *= s.q[child];
        }
        if (need < rest) {
          at = child;
          s.path[length++] = child;
          c = 0, w = kOne, left = 1.0, rejected = 0, have = false;
        } else if (p.draft == nullptr) {
          if (!seen) {
            left = fmax(left - s.share[child], 0.0);  // (exact: whole steps)
            s.gone[rejected++] = s.token[child];
          }
        } else if (w != 0) {
          c += w;
          ask = true;
        }
      }
      // Nothing left where the walk ends (not before: a child behind the rejected one may be tried still, and most nodes behind it
      // are no children of this one): one more sum, of the row as it is.
      const bool again = !ask && have && w == 0 && !plain && (c != 0 || rejected > 0);
      s.plain = plain || again;
      s.done = !ask && have && !again;
      s.at = at;
      s.c = c;
      s.rejected = rejected;
      have = true;
    }
    __syncthreads();
    if (s.done) break;
    plain = s.plain != 0;
    // sums of what is left of the row
    const float* prow = p.target + (q0 + s.at) * p.target_stride;
    const uint64_t cc = plain ? 0 : s.c;
    const float* qrow = cc != 0 ? p.draft + (q0 + s.at) * p.draft_stride : prow;
    uint64_t sum = sum_left(p.wide != 0, prow, qrow, cc, begin + lane * 4, end);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = add_full(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    if (!plain && s.rejected > 0) {
      uint64_t out = 0;
      for (int i = lane; i < s.rejected; i += 32)
        if (s.gone[i] >= begin && s.gone[i] < end) out += steps(__ldcg(prow + s.gone[i]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
      if (sum != kFull) sum -= out;
    }
    if (lane == 0) s.own[pass & 1][warp] = sum;
    cluster_sync();
    if (warp < kParts / 32) {
      const int i = warp * 32 + lane;
      s.part[i] = load_remote(tc::smem_u32(&s.own[pass & 1][i % kWarps]), i / kWarps);
    }
    __syncthreads();
    if (warp == 0) {
      uint64_t all = 0;
#pragma unroll
      for (int i = 0; i < kParts; i += 32) all = add_full(all, s.part[i + lane]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all = add_full(all, __shfl_xor_sync(0xffffffffu, all, o));
      if (lane == 0) s.total = all;
    }
    __syncthreads();
    w = s.total;
    left = static_cast<double>(w) * 0x1p-52;
    ++pass;
  }

  // the drawn place
  const uint64_t total = s.total;
  const uint64_t place = __umul64hi(fraction(p.sample[b]), total);
  uint64_t before = 0;
  const int mine = rank * kWarps + warp;
  for (int i = lane; i < mine; i += 32) before += s.part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const bool drawn = total != 0 && total != kFull;
  if (lane == 0 && drawn && place >= before && place - before < s.part[mine]) {
    s.holder = warp;
    s.base = before;
  }
  __syncthreads();
  if (s.holder >= 0) {
    // the block's warps sum a piece each of the part that holds it, and one of them looks through its own
    const float* prow = p.target + (q0 + s.at) * p.target_stride;
    const uint64_t cc = plain ? 0 : s.c;
    const float* qrow = cc != 0 ? p.draft + (q0 + s.at) * p.draft_stride : prow;
    const int rej = plain ? 0 : s.rejected;
    const int64_t piece = span / kWarps;  // a multiple of 8
    const int64_t from = (static_cast<int64_t>(rank) * kWarps + s.holder) * span + warp * piece, to = min(from + piece, p.V);
    uint64_t sum = sum_left(p.wide != 0, prow, qrow, cc, from + lane * 4, to);
    for (int g = lane; g < rej; g += 32)
      if (s.gone[g] >= from && s.gone[g] < to) sum -= steps(__ldcg(prow + s.gone[g]));  // (may pass below 0 until all are added)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s.piece[warp] = sum;
    __syncthreads();
    before = s.base;
    for (int i = 0; i < warp; ++i) before += s.piece[i];
    if (place >= before && place - before < sum) {
      for (int64_t i0 = from; i0 < to; i0 += 128) {
        const int64_t i = i0 + lane * 4;
        const float4 x = load4<false>(prow, i, to);
        const float4 y = cc != 0 ? load4<false>(qrow, i, to) : x;
        uint64_t v[4] = {weight(x.x, y.x, cc), weight(x.y, y.y, cc), weight(x.z, y.z, cc), weight(x.w, y.w, cc)};
        for (int g = 0; g < rej; ++g) {
          const int64_t k = s.gone[g] - i;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k == e) v[e] = 0;
        }
        const uint64_t four = (v[0] + v[1]) + (v[2] + v[3]);
        uint64_t upto = four;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t x2 = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x2;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > place);
        if (past != 0) {
          if (lane == __ffs(past) - 1) {
            uint64_t at = before + upto - four;
            int e = 0;
            while (e < 3 && at + v[e] <= place) at += v[e++];
            p.next[b] = i + e;
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  if (rank == 0) {
    if (t == 0) {
      p.count[b] = length;
      if (!drawn) p.next[b] = -1;
      if (total == kFull) record_device_error(p.err, kDevErrBadIndex);
      s.done = length;
    }
    __syncthreads();
    for (int i = t; i < p.max_nodes; i += kThreads) p.path[b * p.max_nodes + i] = i < s.done ? s.path[i] : -1;
  }
  cluster_sync();  // no block ends while another one reads its sums
}

}  // namespace

cudaError_t plan_verify_drafts(const VerifyDraftsArgs& a, Prepared* out) {
  Params p = {};
  p.target = a.target;
  p.draft = a.draft;
  p.target_stride = a.target_stride;
  p.draft_stride = a.draft_stride;
  p.V = a.V;
  p.parents = a.parents;
  p.tokens = a.tokens;
  p.q_indptr = a.q_indptr;
  p.accept = a.accept_u;
  p.sample = a.sample_u;
  p.path = a.path;
  p.count = a.count;
  p.next = a.next_token;
  p.Tq = a.Tq;
  p.max_nodes = static_cast<int32_t>(a.max_nodes);
  p.wide = ((reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) & 15) == 0 && a.target_stride % 4 == 0 &&
           a.draft_stride % 4 == 0;
  p.err = device_error_word();
  // Two blocks fit an SM, and all sequences should be under way at the same time.  Of 8 | 4 | 2 blocks a sequence, 64 of 128256
  // tokens take 32.0 | 26.2 | 27.7 us, 32 of 50257 14.3 | 12.8 | 14.3, one of 32000 8.9 | 9.3 | 9.2.
  const int64_t sms = sm_count();
  const int cluster = a.B * 8 <= sms ? 8 : a.B * 4 <= 2 * sms ? 4 : 2;
  const void* fn = cluster == 8   ? reinterpret_cast<const void*>(draft_verify_kernel<8>)
                   : cluster == 4 ? reinterpret_cast<const void*>(draft_verify_kernel<4>)
                                  : reinterpret_cast<const void*>(draft_verify_kernel<2>);
  out->count = 1;
  out->launch[0] = {fn, static_cast<uint32_t>(a.B * cluster), 1, kThreads, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace qlin
