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
// Two floats in one register pair: the packed float32 instructions of sm_100
// do twice the work per issue slot.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ f2 pair(float x) { return pair(x, x); }
__device__ __forceinline__ float2 halves(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// A vector as four pairs.
struct Vec {
  f2 v[4];
};
__device__ __forceinline__ void unpack(const Raw<bf16>& r, Vec& f) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Raw<float>& r, Vec& f) {
  f.v[0] = pair(r.a.x, r.a.y);
  f.v[1] = pair(r.a.z, r.a.w);
  f.v[2] = pair(r.b.x, r.b.y);
  f.v[3] = pair(r.b.z, r.b.w);
}
__device__ __forceinline__ void store_vec(bf16* p, const Vec& f) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = halves(f.v[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(h.x, h.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store_vec(float* p, const Vec& f) {
  const float2 a = halves(f.v[0]), b = halves(f.v[1]), c = halves(f.v[2]), d = halves(f.v[3]);
  reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
}
__device__ __forceinline__ void load_vec(Vec& f, const float* p) {
  Raw<float> r;
  r.a = reinterpret_cast<const float4*>(p)[0];
  r.b = reinterpret_cast<const float4*>(p)[1];
  unpack(r, f);
}
__device__ __forceinline__ void fill(Vec& f, float x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = pair(x);
}

// Sums over the lanes of a worker.  STEPS < 0: `width` = 4, 8, 16 or 32 lanes of
// a warp.  Otherwise a whole block of `width` / 32 <= 2^STEPS warps; every
// thread of the block calls it the same number of times.  `scratch` ([2][32], for
// two pairs at once [4][32]) alternates between two halves, so one barrier per sum
// suffices: a half is written again only behind the next sum's barrier, which
// every reader of it has reached.
template <int STEPS>
struct RowSum {
  static constexpr bool kBlock = STEPS >= 0;
  static constexpr int kMask = kBlock ? (1 << STEPS) - 1 : 0;
  float2* scratch;
  int width, phase;
  __device__ __forceinline__ RowSum(float2* s, int w) : scratch(s), width(w), phase(0) {}
  __device__ __forceinline__ float lanes(float v) const {
    if (kBlock) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
      for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  }
  __device__ __forceinline__ float2 lanes(float2 v) const { return make_float2(lanes(v.x), lanes(v.y)); }
  __device__ __forceinline__ float2 other(const float2* s) const {
    const int i = threadIdx.x & kMask;
    return i < width >> 5 ? s[i] : make_float2(0.f, 0.f);
  }
  // Trades the warps' values: lane i gets warp (i & kMask)'s, zeros behind the last warp.
  __device__ __forceinline__ float2 trade(float2 v) {
    float2* s = scratch + phase * 32;
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    return other(s);
  }
  __device__ __forceinline__ float warps(float v) const {
#pragma unroll
    for (int o = (kMask + 1) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ float2 operator()(float2 v) {
    v = lanes(v);
    if (kBlock) {
      v = trade(v);
      v = make_float2(warps(v.x), warps(v.y));
    }
    return v;
  }
  // Trades two pairs behind one barrier.
  __device__ __forceinline__ void trade(float2& a, float2& b) {
    float2* s = scratch + 64 + phase * 32;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = b;
    a = trade(a);
    b = other(s);
  }
  // Sums of two pairs behind one barrier.
  __device__ __forceinline__ void both(float2& a, float2& b) {
    a = lanes(a);
    b = lanes(b);
    if (kBlock) {
      trade(a, b);
      a = make_float2(warps(a.x), warps(a.y));
      b = make_float2(warps(b.x), warps(b.y));
    }
  }
  __device__ __forceinline__ float operator()(float v) {
    v = lanes(v);
    return kBlock ? warps(trade(make_float2(v, 0.f)).x) : v;
  }
};

}  // namespace svg
