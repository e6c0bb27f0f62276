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
// HBM-bound: x in, half a byte plus 1/32 byte per element out.
#include <algorithm>

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

// Eight E2M1 codes to floats.
__device__ __forceinline__ void unpack_e2m1(uint32_t c, float (&f)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const uint32_t n = c >> (4 * i) & 15u, e = n >> 1 & 3u, m = n & 1u;
    // exponent 0: m * 0.5; else (1 + m/2) 2^(e-1)
    const float v = e ? __uint_as_float((126u + e) << 23 | m << 22) : 0.5f * (float)m;
    f[i] = n & 8u ? -v : v;
  }
}

__device__ __forceinline__ float e8m0(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

// X is [M][K] (head_d = 0) or head-major [K/head_d][M][head_d]; four threads
// share a block of 32 elements.
template <typename T>
__global__ void __launch_bounds__(256) k_mx_quantize(const T* __restrict__ X, long long vecs, int M, int vpr, int head_d,
                                                     uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const long long base = (long long)blockIdx.x * blockDim.x;
  const long long row0 = base / vpr;  // one 64-bit division per block
  const uint32_t in = (uint32_t)(base - row0 * vpr) + threadIdx.x;
  const uint32_t dr = in / (uint32_t)vpr;
  const long long row = row0 + dr;
  const int vec = (int)(in - dr * vpr);
  const bool on = base + threadIdx.x < vecs;
  float f[kVec];
  Raw<T> r;
  zero_raw(r);
  if (on) {
    long long at = row * vpr * kVec + vec * kVec;
    if (head_d) {
      const int h = vec * kVec / head_d;
      at = ((long long)h * M + row) * head_d + (vec * kVec - h * head_d);
    }
    load_raw(r, X + at);
  }
  unpack(r, f);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t e = top >> 23;  // biased exponent of the largest magnitude
  const bool bad = e == 255u;
  const uint32_t byte = bad ? 255u : e > 2u ? e - 2u : 0u;
  // 1 / scale = 2^(127 - byte): a normal float for every byte up to 252
  const float inv = bad ? 0.f : __uint_as_float((254u - byte) << 23);
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = bad ? 0.f : f[i] * inv;
  if (on) {
    codes[base + threadIdx.x] = pack_e2m1(f);
    if ((threadIdx.x & 3) == 0) scales[(base + threadIdx.x) >> 2] = (uint8_t)byte;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_mx_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                       long long vecs, T* __restrict__ Y) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= vecs) return;
  float f[kVec];
  unpack_e2m1(codes[i], f);
  const float s = e8m0(scales[i >> 2]);
#pragma unroll
  for (int k = 0; k < kVec; ++k) f[k] *= s;
  store_vec(Y + i * kVec, f);
}

}  // namespace

cudaError_t mx_quantize_run(const void* X, int dtype, int M, int K, int head_d, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st) {
  const long long vecs = (long long)M * (K / kVec);
  const int grid = (int)((vecs + 255) / 256);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (dtype == DT_F32)
    k_mx_quantize<float><<<grid, 256, 0, st>>>(static_cast<const float*>(X), vecs, M, K / kVec, head_d, c, scales);
  else
    k_mx_quantize<bf16><<<grid, 256, 0, st>>>(static_cast<const bf16*>(X), vecs, M, K / kVec, head_d, c, scales);
  note_launch();
  return cudaGetLastError();
}

cudaError_t mx_dequantize_run(const uint8_t* codes, const uint8_t* scales, int M, int K, void* Y, int dtype,
                              cudaStream_t st) {
  const long long vecs = (long long)M * (K / kVec);
  const int grid = (int)((vecs + 255) / 256);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (dtype == DT_F32) k_mx_dequantize<float><<<grid, 256, 0, st>>>(c, scales, vecs, static_cast<float*>(Y));
  else k_mx_dequantize<bf16><<<grid, 256, 0, st>>>(c, scales, vecs, static_cast<bf16*>(Y));
  note_launch();
  return cudaGetLastError();
}

}  // namespace svg
