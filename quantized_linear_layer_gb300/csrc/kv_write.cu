// Head norms and the position rotation of q and k in one pass, with k and v
// quantized into the paged cache in the same pass when there is one.
//
// A row is one head of one token, D 16-bit elements, held by a group of D / 8
// lanes, eight elements each, as two pieces of four: a lane's pieces are the two
// sides of four rotated pairs (halves: channels 4 l .. and rot / 2 + 4 l ..;
// interleaved: eight consecutive channels), so that the rotation exchanges
// nothing between lanes, and a lane needs four angles whatever the head.  A
// group takes one token's heads `parts` apart (all of them, or a share where
// there are few tokens): it works out its lanes' four sines and cosines once per
// token and keeps them and the gammas in registers over the heads, the next rows
// loaded ahead.
//
// Angles: a position times inv_freq, modulo a full turn.  The frequency in
// turns is kept as a 64-bit fraction (worked out once per block in float64);
// position x fraction modulo 2^64 is then one integer product that drops the
// whole turns exactly, and what is left converts to a float in [-1/2, 1/2)
// for sincospif.  The product is exact, the fraction within 2^-52 of its
// frequency, so an angle of any position below 2^31 is off by less than 2^-21
// radians for |inv_freq| <= 1 (and by |inv_freq| times that above), without a
// float64 operation per angle (float64 runs at a small fraction of the float32
// rate here).
//
// The mean of squares, the norm, the rotation and the scales are float32; a
// row is rounded once, to its 16-bit output or to its codes.  Integer codes
// are rounded by adding 1.5 x 2^23 (nearest even, the code in the low bits),
// which is the float-to-integer conversion at the rate of an addition.
// Bound: below about a thousand tokens a launch's latency (64 tokens x 48 heads
// into the cache: 4.3 us).  Above, the latency of the rows' loads: neither HBM (half
// to two thirds of the copy rate) nor the issue slots (56 % rotating, 64 to 70 %
// quantizing) are full, but the loads ahead begin anew with q, k and v and with
// every token, whose first row and place are waited for.  8192 tokens x 40 heads of
// 128 rotated: 40.3 us (4170 GB/s); 5028 x 96, 64 channels of each turned, into the
// cache: 67 us INT8 (3080 GB/s), 68 E4M3, 78 U4 (2400); k and v of 8192 tokens x 16
// heads as they are: 16.3 us INT8, 17.6 E4M3, 20.7 U4, part of it in L2.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 256;
// Rows a group takes at once, and blocks that share an SM.  Rotation alone does little per row, so two rows at once and
// 80 registers; quantizing fills a warp's issue slots by itself, and the shorter code and a fourth block count for
// more.  Rotation of 8192 tokens x 40 heads of 128: 39.3 us at two rows and three blocks, 45.5 at one and four.
// Appending 5028 tokens x 96 heads, the read of them behind it: 92.5 and 90.4 us; 64 tokens x 48 heads: 8.5 and 7.1 us
// (a sweep before the quantizer's last step, graph replays).
__host__ __device__ constexpr int unroll_of(int fmt) { return fmt < 0 ? 2 : 1; }
__host__ __device__ constexpr int blocks_of(int fmt) { return fmt < 0 ? 3 : 4; }
constexpr int kFlat = 2;  // rows a group of the plain write takes at once
constexpr float kRoundMagic = 12582912.0f;  // 1.5 x 2^23
constexpr float kScaleFloor = 5.42101086e-20f;  // 2^-64

struct Params {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* q_out;
  uint8_t* k_out;
  int64_t qt, qh, kt, kh, vt, vh, qot, qoh, kot, koh;  // strides in bytes
  int32_t hq, hk, hv;  // heads of q, k and v (0: absent)
  int32_t heads;       // their sum
  int32_t parts;       // groups that share a token's heads
  int64_t T;
  const int64_t* positions;
  const double* inv_freq;
  const void* q_gamma;
  const void* k_gamma;
  int32_t half_rot, interleaved;
  float eps;
  const int64_t* slots;
  kv::CacheView cache;
  int32_t* err;
};

// The largest and smallest of three, NaN if one is NaN (fmaxf and fminf drop it).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// x / d rounded to nearest even from r = 1 / d rounded to nearest, as div_by_rcp,
// but for the sign of a quotient of zero.
__device__ __forceinline__ float divide(float x, float d, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

// Quantizes the row held by this group of lanes (four values from channel ca
// on, four from cb on each; JOINED: cb = ca + 4) and writes its codes and scale.  All lanes of the
// warp call it (shuffles); `write` says whether this group's row is stored.
template <int FMT, int LANES, bool JOINED>
__device__ __forceinline__ void quantize_row(const float* y, int lane, int ca, int cb, bool write, uint8_t* codes,
                                             uint8_t* scale_at) {
  if constexpr (FMT == QLIN_KV_U4) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      lo = min3(lo, y[i], y[i + 1]);
      hi = max3(hi, y[i], y[i + 1]);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      const float l = __shfl_xor_sync(0xffffffffu, lo, o), h = __shfl_xor_sync(0xffffffffu, hi, o);
      lo = min3(lo, l, l);
      hi = max3(hi, h, h);
    }
    const bool finite = hi < INFINITY && lo > -INFINITY;
    const float span = fmaxf(__fsub_rn(hi, lo), 1e-5f);
    // (a span that overflowed to infinity stays one)
    const __half s16 = __float2half_rn(span < INFINITY ? fminf(divide(span, 15.0f, 1.0f / 15.0f), 65504.0f) : 65504.0f);
    const float s = __half2float(s16);  // at least the fp16 nearest 1e-5 / 15, a normal float32
    const float r = __frcp_rn(s);
    const float z = fminf(fmaxf(rintf(divide(-lo, s, r)), 0.0f), 15.0f);
    // rint(y / s) + z in [0, 15]: the clamp first (z is an integer), the rounding and + z in the magic sum
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = fminf(fmaxf(divide(y[i], s, r), -z), 15.0f - z);
      packed |= (__float_as_uint((n + kRoundMagic) + z) & 15u) << (4 * i);
    }
    if (write) {
      if (!finite) packed = 0;
      if constexpr (JOINED) {
        *reinterpret_cast<uint32_t*>(codes + ca / 2) = packed;
      } else {
        *reinterpret_cast<uint16_t*>(codes + ca / 2) = static_cast<uint16_t>(packed);
        *reinterpret_cast<uint16_t*>(codes + cb / 2) = static_cast<uint16_t>(packed >> 16);
      }
      if (lane == 0) {
        const uint32_t word = static_cast<uint32_t>(__half_as_ushort(s16)) |
                              (static_cast<uint32_t>(__half_as_ushort(__float2half_rn(z))) << 16);
        *reinterpret_cast<uint32_t*>(scale_at) = finite ? word : 0x00007fffu;
      }
    }
  } else {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) amax = max3(amax, fabsf(y[i]), fabsf(y[i + 1]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, amax, o);
      amax = max3(amax, a, a);
    }
    const bool finite = amax < INFINITY;
    constexpr float kTop = FMT == QLIN_KV_INT8 ? 127.0f : 448.0f;
    float s = fmaxf(divide(amax, kTop, 1.0f / kTop), kScaleFloor);  // exact where it is above the floor
    if (amax == 0.0f) s = 1.0f;
    const float r = __frcp_rn(s);  // s lies in [2^-64, 2^122]: normal, as is its reciprocal
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = divide(y[4 * h + i], s, r);
      if constexpr (FMT == QLIN_KV_INT8) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(n[i] + kRoundMagic);
        w[h] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // a quotient that is zero keeps the sign of y
          n[i] = __uint_as_float((__float_as_uint(n[i]) & 0x7fffffffu) | (__float_as_uint(y[4 * h + i]) & 0x80000000u));
        w[h] = kv::floats_to_e4m3x2(n[0], n[1]) | (kv::floats_to_e4m3x2(n[2], n[3]) << 16);
      }
    }
    if (write) {
      if (!finite) w[0] = w[1] = 0;
      if constexpr (JOINED) {
        *reinterpret_cast<uint2*>(codes + ca) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t*>(codes + ca) = w[0];
        *reinterpret_cast<uint32_t*>(codes + cb) = w[1];
      }
      if (lane == 0) *reinterpret_cast<float*>(scale_at) = finite ? s : __uint_as_float(0x7fc00000u);
    }
  }
}

// DT: 0 fp16, 1 bf16.  FMT: the cache's format, or -1 without a cache.
template <int DT, int D, int FMT>
__global__ void __launch_bounds__(kThreads, blocks_of(FMT)) norm_rope_write_kernel(const __grid_constant__ Params p) {
  constexpr int LANES = D / 8;
  constexpr int kGroups = kThreads / LANES;
  constexpr int kUnroll = unroll_of(FMT);
  __shared__ __align__(16) uint64_t freq[D / 2];  // fractions of a turn
  const int lane = threadIdx.x % LANES;
  const int hqk = p.hq + p.hk;

  // this lane's channels: ca .. ca + 3 and cb .. cb + 3
  const bool turns = 4 * lane < p.half_rot;
  int ca = 8 * lane, cb = ca + 4;
  if (turns && !p.interleaved) {
    ca = 4 * lane;
    cb = p.half_rot + 4 * lane;
  }

  pdl_wait();
  pdl_launch_dependents();
  const int64_t tasks = p.T * p.parts;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t task = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LANES;
  int64_t t;
  int part;
  auto locate = [&]() {  // the task's token and share of its heads
    t = tasks <= 0xffffffffll ? static_cast<uint32_t>(task) / static_cast<uint32_t>(p.parts) : task / p.parts;
    part = static_cast<int>(task - t * p.parts);
  };
  locate();
  int64_t pos = 0;
  if (p.half_rot > 0 && t < p.T) pos = p.positions[t];

  // the gammas of this lane's channels
  float gq[8], gk[8];
  {
    const int c[2] = {ca, cb};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gq[i] = p.q_gamma != nullptr ? load_elem<DT>(p.q_gamma, c[i / 4] + i % 4) : 1.0f;
      gk[i] = p.k_gamma != nullptr ? load_elem<DT>(p.k_gamma, c[i / 4] + i % 4) : 1.0f;
    }
  }
  if (p.half_rot > 0) {
    for (int i = threadIdx.x; i < p.half_rot; i += kThreads) {
      const double x = p.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
      freq[i] = static_cast<uint64_t>((x - floor(x)) * 18446744073709551616.0);
    }
    __syncthreads();
  }

  // The rows of one kind, from head `h` of the task on, kUnroll at once and as many loaded ahead; `finish(row, head,
  // live)` takes each.  All groups of the warp go round together (the shuffles need every lane).
  auto rows = [&](int& h, int count, bool live, const uint8_t* base, int64_t pitch, auto finish) {
    uint4 next[kUnroll];
    auto load = [&](int at) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int head = at + u * p.parts;
        uint2 a = make_uint2(0u, 0u), b = a;
        if (live && head < count) {
          const uint8_t* src = base + head * pitch;
          a = *reinterpret_cast<const uint2*>(src + 2 * ca);
          b = *reinterpret_cast<const uint2*>(src + 2 * cb);
        }
        next[u] = make_uint4(a.x, a.y, b.x, b.y);
      }
    };
    load(h);
    while (__any_sync(0xffffffffu, live && h < count)) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) raw[u] = next[u];
      load(h + kUnroll * p.parts);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float y[8];
        kv::unpack8<DT>(raw[u], y);
        const int head = h + u * p.parts;
        finish(y, head, live && head < count);
      }
      h += kUnroll * p.parts;
    }
    // the first of this task's heads past the kind's last
    if (h >= count) h -= (h - count) / p.parts * p.parts;
    h -= count;
  };
  // Norm and rotation of a row, with the factors of the token: (a, b) -> (a fac[0..3] - b fac[4..7],
  // b fac[8..11] + a fac[12..15]) for a lane that turns, channel by channel times fac[0..3] and fac[8..11] else.
  auto norm_turn = [&](float* y, bool norm, const float* fac) {
    if (norm) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= inv;
    }
    if (!turns) {  // not a turn by zero: its b x 0 would make NaN of an infinity, and lose a zero's sign
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] *= p.interleaved ? (i & 1 ? fac[8 + i / 2] : fac[i / 2]) : fac[i];
        y[4 + i] *= p.interleaved ? (i & 1 ? fac[10 + i / 2] : fac[2 + i / 2]) : fac[8 + i];
      }
    } else if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = fmaf(a, fac[i], -(b * fac[4 + i]));
        y[2 * i + 1] = fmaf(b, fac[8 + i], a * fac[12 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[i], b = y[4 + i];
        y[i] = fmaf(a, fac[i], -(b * fac[4 + i]));
        y[4 + i] = fmaf(b, fac[8 + i], a * fac[12 + i]);
      }
    }
  };

  while (__any_sync(0xffffffffu, task < tasks)) {
    const bool live = task < tasks;
    int64_t slot = -1;
    if constexpr (FMT >= 0) {
      if (live) slot = p.slots[t];
    }
    float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {};
    if (turns && live && part < hqk) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t turn = static_cast<uint64_t>(pos) * freq[4 * lane + i];
        // the fraction of a turn, as a signed number of half turns
        sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 1.08420217e-19f, &sn[i], &cs[i]);  // 2^-63
      }
    }
    auto factors = [&](const float* g, float* fac) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ga = p.interleaved ? g[2 * i] : g[i], gb = p.interleaved ? g[2 * i + 1] : g[4 + i];
        fac[i] = ga * cs[i];
        fac[4 + i] = gb * sn[i];
        fac[8 + i] = gb * cs[i];
        fac[12 + i] = ga * sn[i];
      }
    };
    auto store_row = [&](uint8_t* to, const float* y) {
      const uint4 o = kv::pack8<DT>(y);
      *reinterpret_cast<uint2*>(to + 2 * ca) = make_uint2(o.x, o.y);
      *reinterpret_cast<uint2*>(to + 2 * cb) = make_uint2(o.z, o.w);
    };
    // this token's place in the cache
    const int64_t page = slot >> p.cache.page_shift;
    const bool stored = slot >= 0 && page < p.cache.pages;
    if (FMT >= 0 && slot >= 0 && !stored) record_device_error(p.err, kDevErrBadIndex);
    auto quantize = [&](const float* y, int head, bool there, uint8_t* codes, uint8_t* scale) {
      if constexpr (FMT >= 0) {
        const int64_t row = (static_cast<int64_t>(head) << p.cache.page_shift) +
                            (slot & ((int64_t(1) << p.cache.page_shift) - 1));
        quantize_row<FMT, LANES, false>(y, lane, ca, cb, there && stored,
                                 codes + page * p.cache.page_stride + row * kv::row_bytes(FMT, D),
                                 scale + page * p.cache.scale_page_stride + row * 4);
      }
    };

    int h = part;
    float fac[16];
    factors(gq, fac);
    rows(h, p.hq, live, p.q + t * p.qt, p.qh, [&](float* y, int head, bool there) {
      norm_turn(y, p.q_gamma != nullptr, fac);
      if (there && p.q_out != nullptr) store_row(p.q_out + t * p.qot + head * p.qoh, y);
    });
    factors(gk, fac);
    rows(h, p.hk, live, p.k + t * p.kt, p.kh, [&](float* y, int head, bool there) {
      norm_turn(y, p.k_gamma != nullptr, fac);
      if (there && p.k_out != nullptr) store_row(p.k_out + t * p.kot + head * p.koh, y);
      quantize(y, head, there, p.cache.k, p.cache.k_scale);
    });
    if constexpr (FMT >= 0) {
      rows(h, p.hv, live, p.v + t * p.vt, p.vh,
           [&](float* y, int head, bool there) { quantize(y, head, there, p.cache.v, p.cache.v_scale); });
    }
    task += stride;
    locate();
    if (p.half_rot > 0 && task < tasks) pos = p.positions[t];
  }
}

// k and v as they are: the rows of all tokens in one flat (token, head) order, kFlat rows a group at once.
template <int DT, int D, int FMT>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ Params p) {
  constexpr int LANES = D / 8;
  constexpr int kGroups = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t count = p.T * p.heads;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups * kFlat;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kGroups * kFlat; row0 < count; row0 += stride) {
    uint4 raw[kFlat];
    int64_t slot[kFlat];
    int head[kFlat];
#pragma unroll
    for (int u = 0; u < kFlat; ++u) {
      const int64_t at = row0 + u * kGroups + threadIdx.x / LANES;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      slot[u] = -1;
      head[u] = 0;
      if (at < count) {
        const int64_t t = count <= 0xffffffffll ? static_cast<uint32_t>(at) / static_cast<uint32_t>(p.heads) : at / p.heads;
        head[u] = static_cast<int>(at - t * p.heads);
        const uint8_t* src = head[u] < p.hk ? p.k + t * p.kt + head[u] * p.kh : p.v + t * p.vt + (head[u] - p.hk) * p.vh;
        raw[u] = *reinterpret_cast<const uint4*>(src + lane * 16);
        slot[u] = p.slots[t];
      }
    }
#pragma unroll
    for (int u = 0; u < kFlat; ++u) {
      const int64_t page = slot[u] >> p.cache.page_shift;
      const bool stored = slot[u] >= 0 && page < p.cache.pages;
      if (slot[u] >= 0 && !stored) record_device_error(p.err, kDevErrBadIndex);
      float y[8];
      kv::unpack8<DT>(raw[u], y);
      const bool is_k = head[u] < p.hk;
      const int64_t row = (static_cast<int64_t>(is_k ? head[u] : head[u] - p.hk) << p.cache.page_shift) +
                          (slot[u] & ((int64_t(1) << p.cache.page_shift) - 1));
      quantize_row<FMT, LANES, true>(y, lane, 8 * lane, 8 * lane + 4, stored,
                                     (is_k ? p.cache.k : p.cache.v) + page * p.cache.page_stride + row * kv::row_bytes(FMT, D),
                                     (is_k ? p.cache.k_scale : p.cache.v_scale) + page * p.cache.scale_page_stride + row * 4);
    }
  }
}

template <int DT, int D>
cudaError_t plan(Params p, int fmt, Prepared* out) {
  constexpr int kGroups = kThreads / (D / 8);
  p.heads = p.hq + p.hk + p.hv;
  out->count = 1;
  if (p.hq == 0 && p.half_rot == 0 && p.k_gamma == nullptr && p.k_out == nullptr && fmt >= 0) {
    const void* fn = fmt == QLIN_KV_INT8   ? reinterpret_cast<const void*>(write_kernel<DT, D, QLIN_KV_INT8>)
                     : fmt == QLIN_KV_E4M3 ? reinterpret_cast<const void*>(write_kernel<DT, D, QLIN_KV_E4M3>)
                                           : reinterpret_cast<const void*>(write_kernel<DT, D, QLIN_KV_U4>);
    const int64_t blocks = (p.T * p.heads + kGroups * kFlat - 1) / (kGroups * kFlat);
    out->launch[0] = {fn, static_cast<uint32_t>(std::min<int64_t>(blocks, sm_count() * 8)), 1, kThreads, 0};
    out->set(p);
    return cudaSuccess;
  }
  // four tasks for every group that fits on the GPU at once, as far as there are heads to share: the angles cost
  // about one row's work per task
  const int64_t resident = static_cast<int64_t>(sm_count()) * blocks_of(fmt);
  p.parts = static_cast<int32_t>(std::min<int64_t>(p.heads, (4 * resident * kGroups + p.T - 1) / p.T));
  const int64_t blocks = (p.T * p.parts + kGroups - 1) / kGroups;
  const int64_t grid = std::min<int64_t>(blocks, resident);
  const void* fn = fmt < 0                ? reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, -1>)
                   : fmt == QLIN_KV_INT8 ? reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, QLIN_KV_INT8>)
                   : fmt == QLIN_KV_E4M3 ? reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, QLIN_KV_E4M3>)
                                         : reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, QLIN_KV_U4>);
  out->launch[0] = {fn, static_cast<uint32_t>(grid), 1, kThreads, 0};
  out->set(p);
  return cudaSuccess;
}

}  // namespace

cudaError_t plan_qk_norm_rope(const qlin_heads* q, const qlin_heads* k, const qlin_heads* v, const qlin_heads* q_out,
                                const qlin_heads* k_out, qlin_dtype dtype, int64_t T, int64_t D, const qlin_rope* rope,
                                const int64_t* slots, const qlin_kv_cache* cache, Prepared* out) {
  Params p = {};
  p.T = T;
  if (q != nullptr) {
    p.q = static_cast<const uint8_t*>(q->data);
    p.qt = 2 * q->token_stride;
    p.qh = 2 * q->head_stride;
    p.hq = static_cast<int32_t>(q->heads);
    p.q_out = static_cast<uint8_t*>(q_out->data);
    p.qot = 2 * q_out->token_stride;
    p.qoh = 2 * q_out->head_stride;
  }
  if (k != nullptr) {
    p.k = static_cast<const uint8_t*>(k->data);
    p.kt = 2 * k->token_stride;
    p.kh = 2 * k->head_stride;
    p.hk = static_cast<int32_t>(k->heads);
  }
  if (k_out != nullptr) {
    p.k_out = static_cast<uint8_t*>(k_out->data);
    p.kot = 2 * k_out->token_stride;
    p.koh = 2 * k_out->head_stride;
  }
  if (v != nullptr) {
    p.v = static_cast<const uint8_t*>(v->data);
    p.vt = 2 * v->token_stride;
    p.vh = 2 * v->head_stride;
    p.hv = static_cast<int32_t>(v->heads);
  }
  p.positions = rope->positions;
  p.inv_freq = rope->inv_freq;
  p.half_rot = static_cast<int32_t>(rope->rot / 2);
  p.interleaved = rope->interleaved;
  p.q_gamma = rope->q_gamma;
  p.k_gamma = rope->k_gamma;
  p.eps = rope->eps;
  int fmt = -1;
  if (cache != nullptr) {
    p.slots = slots;
    p.cache = kv::view_of(*cache);
    fmt = cache->fmt;
  }
  p.err = device_error_word();
  if (dtype == QLIN_F16) {
    if (D == 64) return plan<0, 64>(p, fmt, out);
    if (D == 128) return plan<0, 128>(p, fmt, out);
    return plan<0, 256>(p, fmt, out);
  }
  if (D == 64) return plan<1, 64>(p, fmt, out);
  if (D == 128) return plan<1, 128>(p, fmt, out);
  return plan<1, 256>(p, fmt, out);
}

}  // namespace qlin
