// Eight-element vectors of a row: streaming loads kept in their storage type,
// unpacking to float32, and stores that round once to the storage type.
#pragma once
#include "common.cuh"

namespace svg {

constexpr int kVec = 8;  // elements per vector

template <typename T>
struct Raw;
template <>
struct Raw<bf16> {
  uint4 u;
};
template <>
struct Raw<float> {
  float4 a, b;
};

__device__ __forceinline__ void load_raw(Raw<bf16>& v, const bf16* p) { v.u = __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void load_raw(Raw<float>& v, const float* p) {
  v.a = __ldcs(reinterpret_cast<const float4*>(p));
  v.b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void zero_raw(Raw<bf16>& v) { v.u = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero_raw(Raw<float>& v) { v.a = v.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void unpack(const Raw<bf16>& v, float (&f)[kVec]) {
  const uint32_t w[4] = {v.u.x, v.u.y, v.u.z, v.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float>& v, float (&f)[kVec]) {
  f[0] = v.a.x; f[1] = v.a.y; f[2] = v.a.z; f[3] = v.a.w;
  f[4] = v.b.x; f[5] = v.b.y; f[6] = v.b.z; f[7] = v.b.w;
}
__device__ __forceinline__ void store_raw(bf16* p, const Raw<bf16>& v) { *reinterpret_cast<uint4*>(p) = v.u; }
__device__ __forceinline__ void store_raw(float* p, const Raw<float>& v) {
  reinterpret_cast<float4*>(p)[0] = v.a;
  reinterpret_cast<float4*>(p)[1] = v.b;
}
__device__ __forceinline__ void store_vec(bf16* p, const float (&f)[kVec]) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store_vec(float* p, const float (&f)[kVec]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void load_f8(float (&f)[kVec], const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Sums over the `width` lanes of a worker: 4, 8, 16 or 32 lanes of a warp, or a
// whole block of up to 32 warps.  Every thread of the block calls it the same
// number of times; `scratch` ([2][32]) alternates between two halves, so one
// barrier per sum suffices: a half is written again only behind the next
// sum's barrier, which every reader of it has reached.
struct RowSum {
  float2* scratch;
  int width, phase;
  __device__ __forceinline__ float2 operator()(float2 v) {
    for (int o = (width < 32 ? width : 32) >> 1; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (width > 32) {
      float2* s = scratch + phase * 32;
      phase ^= 1;
      if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
      __syncthreads();
      const int nw = width >> 5, lane = threadIdx.x & 31;
      v = lane < nw ? s[lane] : make_float2(0.f, 0.f);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
    }
    return v;
  }
  __device__ __forceinline__ float operator()(float v) { return (*this)(make_float2(v, 0.f)).x; }
};

}  // namespace svg
