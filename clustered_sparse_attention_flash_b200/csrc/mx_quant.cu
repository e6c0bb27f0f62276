// Microscaled 4-bit floats (OCP Microscaling Formats v1.0, MXFP4): blocks of 32
// consecutive elements of a row, E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// sign) under one E8M0 scale 2^(byte - 127).
//
// Quantisation as in section 6.3 of the specification: the scale's exponent is
// floor(log2 amax) - 2, clamped to the format's range; elements are x / scale
// rounded to nearest even, magnitudes above 6 saturate.  A block that holds a
// NaN or an infinity gets the NaN scale (255) and zero codes, so the fault
// shows in everything computed from it.
//
// HBM-bound: x in, half a byte plus 1/32 byte per element out.  Measured on a
// B200 (share of a plain copy's 6,544 GB/s; above 1 where part of the output
// is still in the L2 at the end): 75,600 x 5,120, quantisation of rows bf16 148 us
// (1.01), float32 259 us (1.03), head-major bf16 168 us (0.89), float32 274 us
// (0.98); dequantisation to bf16 147 us (1.02), to float32 356 us (0.75), whose
// stores are 16 bytes of every 32 at a time.  32,768 x 2,048 bf16: rows 26.1 us,
// head-major 27.0 us, dequantisation 27.8 us.  With the maximum taken element by
// element in float32 the issue slots bound it: 31.5 and 30.5 us.
#include <cuda_fp16.h>

#include "chain.cuh"
#include "common.cuh"
#include "internal.h"
#include "rowvec.cuh"

namespace svg {

namespace {

// Eight floats to eight E2M1 codes, element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&f)[kVec]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight E2M1 codes to floats (by way of fp16, which holds each exactly).
__device__ __forceinline__ void unpack_e2m1(uint32_t c, float (&f)[kVec]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ float e8m0(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // vectors of a thread in flight

// The largest magnitude of a vector, as the bits of a float (a NaN is above all).
__device__ __forceinline__ uint32_t top_bits(const Raw<float>& r) {
  const uint32_t m = 0x7fffffffu;
  const uint32_t a = max(__float_as_uint(r.a.x) & m, __float_as_uint(r.a.y) & m), b = max(__float_as_uint(r.a.z) & m, __float_as_uint(r.a.w) & m);
  const uint32_t c = max(__float_as_uint(r.b.x) & m, __float_as_uint(r.b.y) & m), d = max(__float_as_uint(r.b.z) & m, __float_as_uint(r.b.w) & m);
  return max(max(a, b), max(c, d));
}
__device__ __forceinline__ uint32_t top_bits(const Raw<bf16>& r) {
  auto mag = [](uint32_t w) {
    w &= 0x7fff7fffu;
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  };
  const __nv_bfloat162 t = __hmax2_nan(__hmax2_nan(mag(r.u.x), mag(r.u.y)), __hmax2_nan(mag(r.u.z), mag(r.u.w)));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&t);
  return max(w << 16, w & 0xffff0000u);
}

// One vector of a block of 32: its codes and the scale byte, which the block's
// four lanes agree on.
template <typename T>
__device__ __forceinline__ uint32_t quantise(const Raw<T>& r, uint32_t& byte) {
  uint32_t top = top_bits(r);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t e = top >> 23;  // biased exponent of the largest magnitude
  const bool bad = e == 255u;
  byte = bad ? 255u : e > 2u ? e - 2u : 0u;
  // 1 / scale = 2^(127 - byte): a normal float for every byte up to 252
  const f2 inv = pair(__uint_as_float((254u - byte) << 23));
  Vec v;
  unpack(r, v);
  float f[kVec];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = halves(mul2(v.v[i], inv));
    f[2 * i] = h.x;
    f[2 * i + 1] = h.y;
  }
  const uint32_t c = pack_e2m1(f);
  return bad ? 0u : c;
}

// X is [M][K] (head_d = 0) or head-major [K/head_d][M][head_d]; four threads
// share a block of 32 elements.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_quantize(const T* __restrict__ X, long long vecs, int M, int vpr, int head_d,
                                                          uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  launch_next();
  const long long base = (long long)blockIdx.x * (kThreads * kBatch);
  const long long row0 = base / vpr;  // one 64-bit division per block
  const uint32_t in0 = (uint32_t)(base - row0 * vpr) + threadIdx.x;
  const uint32_t left = (uint32_t)min(vecs - base, (long long)(kThreads * kBatch));
  Raw<T> r[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    zero_raw(r[u]);
    const uint32_t i = u * kThreads + threadIdx.x;
    if (i >= left) continue;
    long long at = (base + i) * kVec;
    if (head_d) {
      const uint32_t in = in0 + u * kThreads, dr = in / (uint32_t)vpr, col = (in - dr * vpr) * kVec, h = col / (uint32_t)head_d;
      at = ((long long)h * M + row0 + dr) * head_d + (col - h * head_d);
    }
    load_raw(r[u], X + at);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    uint32_t byte;
    const uint32_t c = quantise(r[u], byte), i = u * kThreads + threadIdx.x;
    if (i < left) {
      codes[base + i] = c;
      if ((threadIdx.x & 3) == 0) scales[(base + i) >> 2] = (uint8_t)byte;
    }
  }
}

// Head-major X whose heads are 2^n vectors wide: a block takes kThreads / 2^n
// tokens of kBatch neighbouring heads, so that it reads whole kilobytes (32,768
// tokens of 16 heads of 128, before the packed maximum: 43.9 us in the order of
// the rows, 30.4 us in this; now 29.2 us with the head groups of a run of tokens
// in neighbouring blocks, 27.0 us in this order).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_quantize_heads(const T* __restrict__ X, int M, int H, int log_vph,
                                                                uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  launch_next();
  const int vph = 1 << log_vph, vec = threadIdx.x & (vph - 1);
  const long long row = (long long)blockIdx.x * (kThreads >> log_vph) + (threadIdx.x >> log_vph);
  const int h0 = blockIdx.y * kBatch;
  Raw<T> r[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    zero_raw(r[u]);
    if (row < M && h0 + u < H) load_raw(r[u], X + (((long long)(h0 + u) * M + row) * vph + vec) * kVec);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    uint32_t byte;
    const uint32_t c = quantise(r[u], byte);
    if (row < M && h0 + u < H) {
      const long long i = (row * H + h0 + u) * vph + vec;
      codes[i] = c;
      if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(const uint32_t* codes, const uint8_t* scales, long long vecs, T* Y) {
  wait_previous(codes, scales, Y);
  const long long base = (long long)blockIdx.x * (kThreads * kBatch) + threadIdx.x;
  uint32_t c[kBatch], e[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const long long i = base + u * kThreads;
    c[u] = i < vecs ? __ldcs(codes + i) : 0u;
    e[u] = i < vecs ? scales[i >> 2] : 0u;
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const long long i = base + u * kThreads;
    if (i >= vecs) return;
    float f[kVec];
    unpack_e2m1(c[u], f);
    const float s = e8m0(e[u]);
#pragma unroll
    for (int k = 0; k < kVec; ++k) f[k] *= s;
    store_vec(Y + i * kVec, f);
  }
}

}  // namespace

template <typename T>
static void quantize(const void* X, int M, int K, int head_d, uint32_t* codes, uint8_t* scales, cudaStream_t st) {
  const T* x = static_cast<const T*>(X);
  int log_vph = 0;
  while ((kVec << log_vph) < head_d) ++log_vph;
  const int H = head_d ? K / head_d : 0;
  // whole blocks of 32 in a head, a head within a thread block, heads within the grid's second axis
  if (head_d >= 32 && (kVec << log_vph) == head_d && (1 << log_vph) <= kThreads && H <= 65535 * kBatch) {
    const int rows = kThreads >> log_vph;
    k_mx_quantize_heads<T><<<dim3((M + rows - 1) / rows, (H + kBatch - 1) / kBatch), kThreads, 0, st>>>(x, M, H, log_vph, codes, scales);
  } else {
    const long long vecs = (long long)M * (K / kVec);
    const int grid = (int)((vecs + kThreads * kBatch - 1) / (kThreads * kBatch));
    k_mx_quantize<T><<<grid, kThreads, 0, st>>>(x, vecs, M, K / kVec, head_d, codes, scales);
  }
  note_launch();
}

cudaError_t mx_quantize_run(const void* X, int dtype, int M, int K, int head_d, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st) {
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (dtype == DT_F32) quantize<float>(X, M, K, head_d, c, scales, st);
  else quantize<bf16>(X, M, K, head_d, c, scales, st);
  return cudaGetLastError();
}

cudaError_t mx_dequantize_run(const uint8_t* codes, const uint8_t* scales, int M, int K, void* Y, int dtype,
                              cudaStream_t st) {
  const long long vecs = (long long)M * (K / kVec);
  const int grid = (int)((vecs + kThreads * kBatch - 1) / (kThreads * kBatch));
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  note_launch();
  if (dtype == DT_F32) return launch_chained(k_mx_dequantize<float>, grid, kThreads, 0, 0, st, c, scales, vecs, static_cast<float*>(Y));
  return launch_chained(k_mx_dequantize<bf16>, grid, kThreads, 0, 0, st, c, scales, vecs, static_cast<bf16*>(Y));
}

}  // namespace svg
