// What the kernels over a quantized key / value cache share: 16-bit element
// conversions and the cache's addresses.
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"
#include "qlin.h"

namespace qlin {
namespace kv {

// The cache as a kernel sees it; offsets are 64-bit throughout (a cache may
// hold more than 2^32 bytes).
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t page_stride, scale_page_stride;
  int32_t pages, heads, page_shift;  // page_size = 1 << page_shift
};

inline CacheView view_of(const qlin_kv_cache& c) {
  CacheView v;
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.k_scale = static_cast<uint8_t*>(c.k_scale);
  v.v_scale = static_cast<uint8_t*>(c.v_scale);
  v.page_stride = c.page_stride;
  v.scale_page_stride = c.scale_page_stride;
  v.pages = static_cast<int32_t>(c.pages);
  v.heads = static_cast<int32_t>(c.heads);
  v.page_shift = 0;
  while ((int64_t(1) << v.page_shift) < c.page_size) ++v.page_shift;
  return v;
}

// Bytes of one row of D codes.
__host__ __device__ constexpr int row_bytes(int fmt, int d) { return fmt == QLIN_KV_U4 ? d / 2 : d; }

// Two elements of a 16-bit dtype (0: fp16, 1: bf16) as float32, and back
// (rounded to nearest even).
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (DT == 0) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  else return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == 0) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<DT>(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
}

// Two E4M3 codes (low byte first) as fp16: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t u) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(u));
  return h;
}

// Two float32 as E4M3 codes, a in the low byte, saturating.
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float a, float b) {
  uint16_t u;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(b), "f"(a));
  return u;
}

}  // namespace kv
}  // namespace qlin
