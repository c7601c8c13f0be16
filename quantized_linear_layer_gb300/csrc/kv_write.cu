// Head norms and the position rotation of q and k in one pass, with k and v
// quantized into the paged cache in the same pass when there is one.
//
// A row is one head of one token, D 16-bit elements, held by D / 8 lanes of
// eight elements (one 16-byte load each).  A block takes kRows consecutive
// rows of the flat (token, head) order per step: D / 8 lanes x kUnroll rows
// per lane group.  While a step's loads are under way the block works out the
// angles of the next step's tokens into the other of two buffers; then it
// finishes the step's rows and issues the next loads; one barrier a step.
//
// Angles: a position times inv_freq, modulo a full turn.  The frequency in
// turns is kept as a 64-bit fraction (worked out once per block in float64);
// position x fraction modulo 2^64 is then one integer product that drops the
// whole turns exactly, and what is left converts to a float in [-1/2, 1/2)
// for sincospif.  An angle of any position below 2^31 is off by less than
// 2^-21 radians, without a float64 operation per angle (float64 runs at a
// small fraction of the float32 rate here).
//
// The mean of squares, the norm, the rotation and the scales are float32; a
// row is rounded once, to its 16-bit output or to its codes.  Integer codes
// are rounded by adding 1.5 x 2^23 (nearest even, the code in the low bits),
// which is the float-to-integer conversion at the rate of an addition.  The
// kernel is bound by HBM from about a thousand tokens on, by launch latency
// below.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows per lane group and step: 64 bytes in flight per thread
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
  uint32_t magic;      // ceil(2^32 / heads) where at x magic / 2^32 is exact for every `at` of a step, or 0
  int64_t T;
  const int64_t* positions;
  const double* inv_freq;
  const void* q_gamma;
  const void* k_gamma;
  int32_t half_rot, interleaved;
  int32_t step_tokens;  // tokens that one step of a block can touch
  float eps;
  const int64_t* slots;
  kv::CacheView cache;
  int32_t* err;
};

// The largest of the lanes' values in groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// x / d rounded to nearest even from r = __frcp_rn(d), as div_by_rcp, but for
// the sign of a quotient of zero.
__device__ __forceinline__ float divide(float x, float d, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

// Quantizes the row held by this group of lanes (eight values each) and
// writes its codes and scale.  All lanes of the warp call it (shuffles);
// `write` says whether this group's row is stored.
template <int FMT, int LANES>
__device__ __forceinline__ void quantize_row(const float* y, int lane, bool write, uint8_t* codes, uint8_t* scale_at) {
  uint32_t amax_bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax_bits = max(amax_bits, __float_as_uint(y[i]) & 0x7fffffffu);
  amax_bits = group_max_u32<LANES>(amax_bits);  // as integers a NaN or an infinity is above every finite value
  const bool finite = amax_bits < 0x7f800000u;
  if constexpr (FMT == QLIN_KV_U4) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, y[i]);
      hi = fmaxf(hi, y[i]);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const float span = fmaxf(__fsub_rn(hi, lo), 1e-5f);
    const __half s16 = __float2half_rn(fminf(__fdiv_rn(span, 15.0f), 65504.0f));
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
      *reinterpret_cast<uint32_t*>(codes + 4 * lane) = finite ? packed : 0u;
      if (lane == 0) {
        const uint32_t word = static_cast<uint32_t>(__half_as_ushort(s16)) |
                              (static_cast<uint32_t>(__half_as_ushort(__float2half_rn(z))) << 16);
        *reinterpret_cast<uint32_t*>(scale_at) = finite ? word : 0x00007fffu;
      }
    }
  } else {
    const float amax = __uint_as_float(amax_bits);
    float s = fmaxf(__fdiv_rn(amax, FMT == QLIN_KV_INT8 ? 127.0f : 448.0f), kScaleFloor);
    if (amax_bits == 0) s = 1.0f;
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
      *reinterpret_cast<uint2*>(codes + 8 * lane) = finite ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
      if (lane == 0) *reinterpret_cast<float*>(scale_at) = finite ? s : __uint_as_float(0x7fc00000u);
    }
  }
}

// DT: 0 fp16, 1 bf16.  FMT: the cache's format, or -1 without a cache.
template <int DT, int D, int FMT>
__global__ void __launch_bounds__(kThreads) norm_rope_write_kernel(const __grid_constant__ Params p) {
  constexpr int LANES = D / 8;
  constexpr int kGroups = kThreads / LANES;
  constexpr int kRows = kGroups * kUnroll;
  // [D / 2 fractions of a turn][gammas of q and k as float, D each][two buffers of angles]
  extern __shared__ __align__(16) uint8_t smem[];
  uint64_t* freq = reinterpret_cast<uint64_t*>(smem);
  float* gammas = reinterpret_cast<float*>(freq + D / 2);
  float* trig = gammas + 2 * D;
  const int per_token = 2 * p.half_rot;  // cosines, then sines; see trig_at
  const int per_buffer = per_token * p.step_tokens;

  const int lane = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  const int64_t rows = p.T * p.heads;
  const bool normed = p.q_gamma != nullptr || p.k_gamma != nullptr;

  pdl_launch_dependents();
  pdl_wait();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  int64_t t0 = 0;                        // the first row's token
  int32_t tok[kUnroll], head[kUnroll];   // token after t0; head in the order q, k, v (-1: no row)
  uint4 raw[kUnroll];
  int64_t slot[kUnroll];
  auto load_rows = [&]() {
    t0 = row0 / p.heads;
    const int32_t h0 = static_cast<int32_t>(row0 - t0 * p.heads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t at = h0 + group + u * kGroups;
      tok[u] = p.magic == 0 ? at / p.heads : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(at), p.magic));
      head[u] = at - tok[u] * p.heads;
      slot[u] = -1;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      const int64_t t = t0 + tok[u];
      if (t >= p.T) {
        head[u] = -1;
      } else {
        const uint8_t* src;
        if (head[u] < p.hq) {
          src = p.q + t * p.qt + head[u] * p.qh;
        } else {
          const int32_t h = head[u] - p.hq;
          src = h < p.hk ? p.k + t * p.kt + h * p.kh : p.v + t * p.vt + (h - p.hk) * p.vh;
          if constexpr (FMT >= 0) slot[u] = p.slots[t];
        }
        raw[u] = *reinterpret_cast<const uint4*>(src + lane * 16);
      }
    }
  };
  load_rows();

  for (int i = threadIdx.x; i < p.half_rot; i += kThreads) {
    const double turns = p.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    freq[i] = static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);
  }
  if (normed) {
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      const void* from = i < D ? p.q_gamma : p.k_gamma;
      if (from != nullptr) gammas[i] = load_elem<DT>(from, i < D ? i : i - D);
    }
  }
  // Where the cosine of frequency i lies in a token's block (its sine half_rot behind).  Halves: the four
  // that a lane reads at once are together, lanes 16 bytes apart, free of bank conflicts.
  auto trig_at = [&](int i) {
    return p.interleaved ? i : ((i >> 2) & 1) * (p.half_rot / 2) + (i >> 3) * 4 + (i & 3);
  };
  auto angles = [&](int64_t row0, float* to) {
    const int64_t t0 = row0 / p.heads;
    const int64_t last = min(rows - 1, row0 + kRows - 1) / p.heads;
    const int count = static_cast<int>(last - t0 + 1) * p.half_rot;
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const int j = i / p.half_rot, f = i - j * p.half_rot;
      const uint64_t turn = static_cast<uint64_t>(p.positions[t0 + j]) * freq[f];
      float s, c;  // the fraction of a turn, as a signed number of half turns
      sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 1.08420217e-19f, &s, &c);  // 2^-63
      float* at = to + j * per_token + trig_at(f);
      at[0] = c;
      at[p.half_rot] = s;
    }
  };

  if (p.half_rot > 0 || normed) __syncthreads();  // freq and gammas are there
  if (p.half_rot > 0) {
    angles(row0, trig);
    __syncthreads();
  }
  for (int buffer = 0;; buffer ^= 1) {
    if (p.half_rot > 0 && row0 + stride < rows) angles(row0 + stride, trig + (buffer ^ 1) * per_buffer);

#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t t = t0 + tok[u];
      const bool is_q = head[u] >= 0 && head[u] < p.hq;
      const bool is_k = head[u] >= p.hq && head[u] < p.hq + p.hk;
      float y[8];
      kv::unpack8<DT>(raw[u], y);

      if (normed) {  // uniform: the shuffles below need every lane
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((is_q && p.q_gamma != nullptr) || (is_k && p.k_gamma != nullptr)) {
          const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
          const float4* g4 = reinterpret_cast<const float4*>(gammas + (is_q ? 0 : D) + lane * 8);
          const float4 ga = g4[0], gb = g4[1];
          const float g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * g[i];
        }
      }

      if (p.half_rot > 0) {
        const float* cs = trig + buffer * per_buffer + tok[u] * per_token;
        if (p.interleaved) {
          const int c0 = lane * 4;  // this lane's first frequency
          if ((is_q || is_k) && c0 < p.half_rot) {
            const float4 c = *reinterpret_cast<const float4*>(cs + c0);
            const float4 s = *reinterpret_cast<const float4*>(cs + p.half_rot + c0);
            const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = y[2 * i], b = y[2 * i + 1];
              y[2 * i] = a * cc[i] - b * sn[i];
              y[2 * i + 1] = b * cc[i] + a * sn[i];
            }
          }
        } else {
          const int step = p.half_rot / 8;  // lanes between the two of a pair
          const bool first = lane < step, second = lane >= step && lane < 2 * step;
          const int from = (threadIdx.x & 31) + (first ? step : second ? -step : 0);
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], from);
          if ((is_q || is_k) && (first || second)) {
            const float* at = cs + 4 * (first ? lane : lane - step);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 c = *reinterpret_cast<const float4*>(at + h * (p.half_rot / 2));
              const float4 s = *reinterpret_cast<const float4*>(at + h * (p.half_rot / 2) + p.half_rot);
              const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[4 * h + i] = y[4 * h + i] * cc[i] + (first ? -o[4 * h + i] : o[4 * h + i]) * sn[i];
            }
          }
        }
      }

      if (is_q && p.q_out != nullptr)
        *reinterpret_cast<uint4*>(p.q_out + t * p.qot + head[u] * p.qoh + lane * 16) = kv::pack8<DT>(y);
      if (is_k && p.k_out != nullptr)
        *reinterpret_cast<uint4*>(p.k_out + t * p.kot + (head[u] - p.hq) * p.koh + lane * 16) = kv::pack8<DT>(y);

      if constexpr (FMT >= 0) {
        bool write = head[u] >= p.hq && slot[u] >= 0;
        const int64_t page = slot[u] >> p.cache.page_shift;
        if (write && page >= p.cache.pages) {
          record_device_error(p.err, kDevErrBadIndex);
          write = false;
        }
        if (__any_sync(0xffffffffu, write)) {
          const int32_t h = is_k ? head[u] - p.hq : head[u] - p.hq - p.hk;
          const int64_t row = (static_cast<int64_t>(h) << p.cache.page_shift) +
                              (slot[u] & ((int64_t(1) << p.cache.page_shift) - 1));
          uint8_t* codes = (is_k ? p.cache.k : p.cache.v) + page * p.cache.page_stride + row * kv::row_bytes(FMT, D);
          uint8_t* scale = (is_k ? p.cache.k_scale : p.cache.v_scale) + page * p.cache.scale_page_stride + row * 4;
          quantize_row<FMT, LANES>(y, lane, write, codes, scale);
        }
      }
    }
    row0 += stride;
    if (row0 >= rows) break;
    load_rows();
    if (p.half_rot > 0) __syncthreads();
  }
}

template <int DT, int D>
cudaError_t plan(Params p, int fmt, Prepared* out) {
  constexpr int kRows = kThreads / (D / 8) * kUnroll;
  p.heads = p.hq + p.hk + p.hv;
  p.magic = p.heads > 1 && p.heads <= 16384 ? static_cast<uint32_t>(((uint64_t(1) << 32) + p.heads - 1) / p.heads) : 0;
  const int64_t steps = (p.T * p.heads + kRows - 1) / kRows;
  // tokens that one step can touch
  p.step_tokens = p.heads >= kRows ? 2 : (kRows + p.heads - 2) / p.heads + 1;
  const int64_t grid = std::min<int64_t>(steps, sm_count() * 6);
  const int buffers = steps > grid ? 2 : 1;
  const size_t smem = D / 2 * 8 + 2 * D * 4 + 8 * static_cast<size_t>(p.half_rot) * p.step_tokens * buffers;
  const void* fn = fmt < 0                ? reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, -1>)
                   : fmt == QLIN_KV_INT8 ? reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, QLIN_KV_INT8>)
                   : fmt == QLIN_KV_E4M3 ? reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, QLIN_KV_E4M3>)
                                         : reinterpret_cast<const void*>(norm_rope_write_kernel<DT, D, QLIN_KV_U4>);
  if (smem > 48 * 1024) {
    const cudaError_t e = ensure_max_dynamic_smem(fn);
    if (e != cudaSuccess) return e;
  }
  out->count = 1;
  out->launch[0] = {fn, static_cast<uint32_t>(grid), 1, kThreads, static_cast<uint32_t>(smem)};
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
