// From the rows of a Q/K/V projection to the attention's operands: optional RMS
// norm of Q and K (per head or over the whole token), rotary positions on
// three axes, and the move from token-major [B,N,H,d] to head-major
// [B*H,N,d].  HBM-bound: every element is read once and written once.
//
// A pair (a, b) of a head turns by the angle pos_axis theta^(-2i/d_axis):
//   (a cos - b sin, a sin + b cos).
// An angle in float32 loses its low bits at far positions, so it is reduced in
// float64, in turns: t = pos f, t - rint(t); the remainder, at most half a
// turn, goes to float32 sincospi.  One table of cos/sin per token serves every
// head of Q and K.
//
// A worker (4, 8, 16 or 32 lanes of a warp, or a block) owns a token at a
// time; a thread owns 16 elements of one head, columns [8j, 8j+8) and
// [d/2 + 8j, d/2 + 8j + 8), so that both pairings find their partners in one
// thread: adjacent pairs inside each vector, half-split pairs across the two.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "rowvec.cuh"

namespace svg {

namespace {

constexpr int kMaxPairs = 64;

struct RopeArgs {
  const void* in[3];    // q, k, v rows (backward: q, k)
  const void* grad[3];  // backward: dQ, dK, dV, head-major
  void* out[3];         // Q, K, V head-major; backward: dq, dk, dv rows
  long long ld[3], batch[3], out_ld, out_batch;
  const float* w[2];
  const int32_t* pos;
  long long pos_batch;  // int32 per batch entry (0: shared)
  float* part;          // backward: [workers][2][C] partial weight gradients
  int B, N, H, d, out_tokens, norm, tpt, chunk;
  int pairs0, pairs01, pairs;  // pairs of axis 0, of axes 0-1, of all axes
  int g1, g2, vol;             // grid extents of axes 1 and 2, grid tokens
  int origin[3];
  float eps;
  double freq[kMaxPairs];  // turns per position
};

// cos/sin of one token's pairs; identity where nothing turns.
__device__ __forceinline__ void token_table(const RopeArgs& p, int b, int n, float2* cs, int lane, int width) {
  for (int i = lane; i < p.d / 2; i += width) {
    float2 v = make_float2(1.f, 0.f);
    if (i < p.pairs) {
      const int ax = i < p.pairs0 ? 0 : i < p.pairs01 ? 1 : 2;
      int x = 0;
      bool turn = true;
      if (p.pos) {
        x = p.pos[(long long)b * p.pos_batch + (long long)n * 3 + ax];
      } else if (n < p.vol) {
        x = ax == 2 ? n % p.g2 : ax == 1 ? n / p.g2 % p.g1 : n / p.g2 / p.g1;
      } else {
        turn = false;
      }
      if (turn) {
        double t = ((double)x + p.origin[ax]) * p.freq[i];
        t -= rint(t);
        sincospif(2.f * (float)t, &v.y, &v.x);
      }
    }
    cs[i] = v;
  }
}

// Turns the 16 elements of a thread by its 8 angles (sign -1: back).
template <bool HALF>
__device__ __forceinline__ void turn16(float (&lo)[kVec], float (&hi)[kVec], const float2 (&cs)[kVec], float sign) {
  if (HALF) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float a = lo[i], b = hi[i], s = sign * cs[i].y;
      lo[i] = a * cs[i].x - b * s;
      hi[i] = a * s + b * cs[i].x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = lo[2 * i], b = lo[2 * i + 1], s = sign * cs[i].y;
      lo[2 * i] = a * cs[i].x - b * s;
      lo[2 * i + 1] = a * s + b * cs[i].x;
      a = hi[2 * i], b = hi[2 * i + 1], s = sign * cs[4 + i].y;
      hi[2 * i] = a * cs[4 + i].x - b * s;
      hi[2 * i + 1] = a * s + b * cs[4 + i].x;
    }
  }
}

__device__ __forceinline__ float dot16(const float (&a)[kVec], const float (&b)[kVec], const float (&c)[kVec],
                                       const float (&d)[kVec]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) s = fmaf(a[i], b[i], fmaf(c[i], d[i], s));
  return s;
}

// Sum over the threads of a head (d/16 lanes) or of the token.
__device__ __forceinline__ float norm_sum(float v, int norm, int lanes, RowSum& sum) {
  if (norm == SVGEAR_QKNORM_TOKEN) return sum(v);
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What both kernels know about a thread: its worker, its place in a token.
struct Place {
  int slot, lane, lanes, j, off;  // off: element offset of the low vector in a token
  bool on;
  long long t, end;               // tokens [t, end) of this worker, b*N + n
};

__device__ __forceinline__ Place place(const RopeArgs& p) {
  Place q;
  q.slot = threadIdx.x / p.tpt;
  q.lane = threadIdx.x - q.slot * p.tpt;
  q.lanes = p.d / 16;
  const int head = q.lane / q.lanes;
  q.j = q.lane - head * q.lanes;
  q.on = head < p.H;
  q.off = head * p.d + q.j * kVec;
  const long long total = (long long)p.B * p.N;
  q.t = ((long long)blockIdx.x * (blockDim.x / p.tpt) + q.slot) * p.chunk;
  q.end = q.t + p.chunk < total ? q.t + p.chunk : total;
  return q;
}

template <bool HALF>
__device__ __forceinline__ void read_angles(const float2* cs, int j, int d, float2 (&c)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) c[i] = HALF ? cs[j * 8 + i] : i < 4 ? cs[j * 4 + i] : cs[d / 4 + j * 4 + i - 4];
}

// Block classes: most threads of a block, and the blocks an SM is to hold (the
// launch bounds set the registers, the grid counts on them).
template <int MAXT, bool BACK>
struct Class {
  static constexpr int kThreads = MAXT == 128 ? (BACK ? 384 : 512) : MAXT == 384 ? (BACK ? 384 : 768) : 1024;  // per SM
  static constexpr int kBlocks = kThreads / MAXT;
};

template <typename T, bool HALF, int MAXT>
__global__ void __launch_bounds__(MAXT, (Class<MAXT, false>::kBlocks)) k_qkv_rope(const __grid_constant__ RopeArgs p) {
  __shared__ float2 scratch[64];
  __shared__ float2 table[2][MAXT == 128 ? 32 : 1][kMaxPairs];
  constexpr bool kAhead = sizeof(T) == 2 && MAXT < 1024;  // the next token is loaded while this one is computed
  RowSum sum(scratch, p.tpt);
  const Place pl = place(p);
  const int half = p.d / 2, head = pl.off / p.d;
  const float inv_c = 1.f / (float)(p.norm == SVGEAR_QKNORM_TOKEN ? p.H * p.d : p.d);
  Raw<T> next[3][2];
  auto fetch = [&](long long t, Raw<T>(&raw)[3][2]) {
    const int b = (int)(t / p.N), n = (int)(t - (long long)b * p.N);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      zero_raw(raw[k][0]);
      zero_raw(raw[k][1]);
      if (p.in[k] && t < pl.end && pl.on) {
        const T* x = static_cast<const T*>(p.in[k]) + b * p.batch[k] + n * p.ld[k] + pl.off;
        load_raw(raw[k][0], x);
        load_raw(raw[k][1], x + half);
      }
    }
  };
  if (kAhead) fetch(pl.t, next);
  for (int it = 0; it < p.chunk; ++it) {
    const long long t = pl.t + it;
    const bool live = t < pl.end;
    if (p.tpt >= 32 && !live) break;  // uniform over the worker
    const int b = live ? (int)(t / p.N) : 0, n = live ? (int)(t - (long long)b * p.N) : 0;
    float2* cs = table[it & 1][pl.slot];
    const long long o = ((long long)(b * p.H + head) * p.out_tokens + n) * p.d + pl.j * kVec;
    Raw<T> raw[3][2];
    if (kAhead) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        raw[k][0] = next[k][0];
        raw[k][1] = next[k][1];
      }
    } else {
      fetch(t, raw);
    }
    if (p.in[2] && live && pl.on) {
      T* out = static_cast<T*>(p.out[2]) + o;
      store_raw(out, raw[2][0]);
      store_raw(out + half, raw[2][1]);
    }
    if (kAhead) fetch(t + 1, next);
    token_table(p, b, n, cs, pl.lane, p.tpt);
    if (p.tpt > 32) __syncthreads(); else __syncwarp();
    float2 c[kVec];
    read_angles<HALF>(cs, pl.j, p.d, c);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!p.in[k]) continue;
      float lo[kVec], hi[kVec];
      unpack(raw[k][0], lo);
      unpack(raw[k][1], hi);
      if (p.norm != SVGEAR_QKNORM_NONE) {
        const float inv = rsqrtf(norm_sum(dot16(lo, lo, hi, hi), p.norm, pl.lanes, sum) * inv_c + p.eps);
        float wl[kVec], wh[kVec];
        const int wo = p.norm == SVGEAR_QKNORM_TOKEN ? pl.off : pl.j * kVec;
        if (pl.on && p.w[k]) {
          load_f8(wl, p.w[k] + wo);
          load_f8(wh, p.w[k] + wo + half);
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) wl[i] = wh[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          lo[i] *= inv * wl[i];
          hi[i] *= inv * wh[i];
        }
      }
      turn16<HALF>(lo, hi, c, 1.f);
      if (live && pl.on) {
        T* out = static_cast<T*>(p.out[k]) + o;
        store_vec(out, lo);
        store_vec(out + half, hi);
      }
    }
  }
}

template <typename T, bool HALF, int MAXT>
__global__ void __launch_bounds__(MAXT, (Class<MAXT, true>::kBlocks)) k_qkv_rope_back(const __grid_constant__ RopeArgs p) {
  __shared__ float2 scratch[64];
  constexpr int kTable = 2 * (MAXT == 128 ? 32 : 1) * kMaxPairs;
  constexpr int kRed = MAXT / 32 * kMaxPairs;  // [warps][2 * kMaxPairs] floats, in the table's place at the end
  __shared__ float2 store[kTable > kRed ? kTable : kRed];
  constexpr bool kAhead = sizeof(T) == 2 && MAXT < 1024;
  RowSum sum(scratch, p.tpt);
  const Place pl = place(p);
  const int half = p.d / 2, head = pl.off / p.d;
  const float inv_c = 1.f / (float)(p.norm == SVGEAR_QKNORM_TOKEN ? p.H * p.d : p.d);
  float dw[2][2][kVec];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < kVec; ++i) dw[k][0][i] = dw[k][1][i] = 0.f;
  Raw<T> next[5][2];  // dQ, dK, dV, q, k
  auto fetch = [&](long long t, Raw<T>(&raw)[5][2]) {
    const int b = (int)(t / p.N), n = (int)(t - (long long)b * p.N);
    const bool ok = t < pl.end && pl.on;
    const long long o = ((long long)(b * p.H + head) * p.out_tokens + n) * p.d + pl.j * kVec;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      zero_raw(raw[k][0]);
      zero_raw(raw[k][1]);
      const T* x;
      if (k < 3) {
        if (!ok || !p.grad[k]) continue;
        x = static_cast<const T*>(p.grad[k]) + o;
      } else {
        if (!ok || p.norm == SVGEAR_QKNORM_NONE || !p.grad[k - 3]) continue;
        x = static_cast<const T*>(p.in[k - 3]) + b * p.batch[k - 3] + n * p.ld[k - 3] + pl.off;
      }
      load_raw(raw[k][0], x);
      load_raw(raw[k][1], x + half);
    }
  };
  if (kAhead) fetch(pl.t, next);
  for (int it = 0; it < p.chunk; ++it) {
    const long long t = pl.t + it;
    const bool live = t < pl.end;
    if (p.tpt >= 32 && !live) break;
    const int b = live ? (int)(t / p.N) : 0, n = live ? (int)(t - (long long)b * p.N) : 0;
    const long long go = b * p.out_batch + n * p.out_ld + pl.off;
    float2* cs = store + ((it & 1) * (MAXT == 128 ? 32 : 1) + pl.slot) * kMaxPairs;
    Raw<T> raw[5][2];
    if (kAhead) {
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        raw[k][0] = next[k][0];
        raw[k][1] = next[k][1];
      }
    } else {
      fetch(t, raw);
    }
    if (p.grad[2] && live && pl.on) {
      T* out = static_cast<T*>(p.out[2]) + go;
      store_raw(out, raw[2][0]);
      store_raw(out + half, raw[2][1]);
    }
    if (kAhead) fetch(t + 1, next);
    token_table(p, b, n, cs, pl.lane, p.tpt);
    if (p.tpt > 32) __syncthreads(); else __syncwarp();
    float2 c[kVec];
    read_angles<HALF>(cs, pl.j, p.d, c);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!p.grad[k]) continue;
      float lo[kVec], hi[kVec];
      unpack(raw[k][0], lo);
      unpack(raw[k][1], hi);
      turn16<HALF>(lo, hi, c, -1.f);
      if (p.norm != SVGEAR_QKNORM_NONE) {
        float nl[kVec], nh[kVec];
        unpack(raw[3 + k][0], nl);
        unpack(raw[3 + k][1], nh);
        const float inv = rsqrtf(norm_sum(dot16(nl, nl, nh, nh), p.norm, pl.lanes, sum) * inv_c + p.eps);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          nl[i] *= inv;
          nh[i] *= inv;
          dw[k][0][i] = fmaf(lo[i], nl[i], dw[k][0][i]);
          dw[k][1][i] = fmaf(hi[i], nh[i], dw[k][1][i]);
        }
        if (pl.on && p.w[k]) {
          const int wo = p.norm == SVGEAR_QKNORM_TOKEN ? pl.off : pl.j * kVec;
          float wl[kVec], wh[kVec];
          load_f8(wl, p.w[k] + wo);
          load_f8(wh, p.w[k] + wo + half);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            lo[i] *= wl[i];
            hi[i] *= wh[i];
          }
        }
        const float mean = norm_sum(dot16(lo, nl, hi, nh), p.norm, pl.lanes, sum) * inv_c;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          lo[i] = inv * (lo[i] - nl[i] * mean);
          hi[i] = inv * (hi[i] - nh[i] * mean);
        }
      }
      if (live && pl.on) {
        T* out = static_cast<T*>(p.out[k]) + go;
        store_vec(out, lo);
        store_vec(out + half, hi);
      }
    }
  }
  if (!p.part) return;
  const long long worker = (long long)blockIdx.x * (blockDim.x / p.tpt) + pl.slot;
  const bool mine = pl.t < (long long)p.B * p.N;  // workers without a token have no slot
  if (p.norm == SVGEAR_QKNORM_TOKEN) {
    if (mine && pl.on)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* part = p.part + ((size_t)worker * 2 + k) * p.H * p.d + pl.off;
        store_vec(part, dw[k][0]);
        store_vec(part + half, dw[k][1]);
      }
    return;
  }
  // Per-head weights: add the heads of this worker, in a warp, then over its warps.
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        for (int s = pl.lanes; s < (p.tpt < 32 ? p.tpt : 32); s <<= 1)
          dw[k][h][i] += __shfl_xor_sync(0xffffffffu, dw[k][h][i], s);
  if (p.tpt <= 32) {
    if (mine && pl.lane < pl.lanes)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* part = p.part + ((size_t)worker * 2 + k) * p.d + pl.j * kVec;
        store_vec(part, dw[k][0]);
        store_vec(part + half, dw[k][1]);
      }
    return;
  }
  float(*wred)[2 * kMaxPairs] = reinterpret_cast<float(*)[2 * kMaxPairs]>(store);
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
    if ((threadIdx.x & 31) < pl.lanes)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        wred[threadIdx.x >> 5][pl.j * kVec + i] = dw[k][0][i];
        wred[threadIdx.x >> 5][half + pl.j * kVec + i] = dw[k][1][i];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += blockDim.x) {
      float s = 0.f;
      for (int w = 0; w < p.tpt / 32; ++w) s += wred[w][i];
      if (mine) p.part[((size_t)worker * 2 + k) * p.d + i] = s;
    }
  }
}

constexpr int kSumLanes = 16;

// Adds the workers' partial weight gradients in a fixed order.
__global__ void __launch_bounds__(32 * kSumLanes) k_rope_weight_sums(const float* part, long long workers, int C, float* dwq,
                                                                     float* dwk) {
  __shared__ float red[kSumLanes][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dwk : dwq;
  if (!out) return;
  float s = 0.f;
  if (col < C)
    for (long long i = w; i < workers; i += kSumLanes) s += part[((size_t)i * 2 + blockIdx.y) * C + col];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < C) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumLanes; ++i) s += red[i][lane];
    out[col] = s;
  }
}

struct Shape {
  int tpt, block, cls, chunk, grid;
  long long workers;
};

Shape rope_shape(const svgear_rope_params* p, bool back) {
  Shape s;
  const int items = p->H * p->d / 16;
  if (items <= 32) {
    s.tpt = items <= 4 ? 4 : items <= 8 ? 8 : items <= 16 ? 16 : 32;
    s.block = 128;
  } else {
    s.tpt = s.block = (items + 31) / 32 * 32;
  }
  s.cls = s.block <= 128 ? 128 : s.block <= 384 ? 384 : 1024;
  const int per = s.block / s.tpt;
  const long long tokens = (long long)p->B * p->N;
  // As many blocks as the SMs hold at once, each with a run of tokens.
  const int threads = s.cls == 1024 ? 1024
                      : s.cls == 384 ? (back ? Class<384, true>::kThreads : Class<384, false>::kThreads)
                                     : (back ? Class<128, true>::kThreads : Class<128, false>::kThreads);
  long long want = std::min(tokens, 148LL * (threads / s.block) * per);
  if (back) want = std::min(want, 4096LL);
  s.chunk = (int)((tokens + want - 1) / want);
  s.workers = (tokens + s.chunk - 1) / s.chunk;
  s.grid = (int)((s.workers + per - 1) / per);
  return s;
}

RopeArgs rope_args(const svgear_rope_params* p, const float* wq, const float* wk, const int32_t* pos, const Shape& s) {
  RopeArgs a{};
  for (int k = 0; k < 3; ++k) {
    a.ld[k] = p->ld[k];
    a.batch[k] = p->batch[k];
    a.origin[k] = p->origin[k];
  }
  a.out_ld = p->grad_ld;
  a.out_batch = p->grad_batch;
  a.w[0] = wq;
  a.w[1] = wk;
  a.pos = pos;
  a.pos_batch = p->pos_per_batch ? (long long)p->N * 3 : 0;
  a.B = p->B; a.N = p->N; a.H = p->H; a.d = p->d;
  a.out_tokens = p->out_tokens > 0 ? p->out_tokens : p->N;
  a.norm = p->norm;
  a.tpt = s.tpt;
  a.chunk = s.chunk;
  a.pairs0 = p->axes[0] / 2;
  a.pairs01 = a.pairs0 + p->axes[1] / 2;
  a.pairs = a.pairs01 + p->axes[2] / 2;
  a.g1 = std::max(p->grid[1], 1);
  a.g2 = std::max(p->grid[2], 1);
  a.vol = pos ? 0 : p->grid[0] * p->grid[1] * p->grid[2];
  a.eps = p->eps;
  const double turn = 6.283185307179586476925286766559;
  for (int ax = 0, at = 0; ax < 3; ++ax) {
    // f_i = scale theta^(-2i/d_ax) / 2 pi, by repeated products: one pow per axis
    const double ratio = p->axes[ax] ? std::pow((double)p->theta[ax], -2.0 / p->axes[ax]) : 1.0;
    double f = (double)p->pos_scale[ax] / turn;
    for (int i = 0; i < p->axes[ax] / 2; ++i, f *= ratio) a.freq[at++] = f;
  }
  return a;
}

template <typename T, bool HALF, int MAXT>
void launch_class(const RopeArgs& a, const Shape& s, bool back, cudaStream_t st) {
  if (back) k_qkv_rope_back<T, HALF, MAXT><<<s.grid, s.block, 0, st>>>(a);
  else k_qkv_rope<T, HALF, MAXT><<<s.grid, s.block, 0, st>>>(a);
  note_launch();
}

template <typename T, bool HALF>
void launch_half(const RopeArgs& a, const Shape& s, bool back, cudaStream_t st) {
  if (s.cls == 128) launch_class<T, HALF, 128>(a, s, back, st);
  else if (s.cls == 384) launch_class<T, HALF, 384>(a, s, back, st);
  else launch_class<T, HALF, 1024>(a, s, back, st);
}

template <typename T>
void launch_rope(const RopeArgs& a, const Shape& s, bool half, bool back, cudaStream_t st) {
  if (half) launch_half<T, true>(a, s, back, st);
  else launch_half<T, false>(a, s, back, st);
}

}  // namespace

cudaError_t qkv_rope_run(const void* const in[3], const float* wq, const float* wk, const int32_t* pos,
                         const svgear_rope_params* p, void* const out[3], cudaStream_t st) {
  const Shape s = rope_shape(p, false);
  RopeArgs a = rope_args(p, wq, wk, pos, s);
  for (int k = 0; k < 3; ++k) {
    a.in[k] = in[k];
    a.out[k] = out[k];
  }
  const bool half = p->pairing == SVGEAR_PAIR_HALF;
  if (p->dtype == DT_F32) launch_rope<float>(a, s, half, false, st);
  else launch_rope<bf16>(a, s, half, false, st);
  return cudaGetLastError();
}

size_t qkv_rope_back_ws_bytes(const svgear_rope_params* p) {
  if (p->norm == SVGEAR_QKNORM_NONE) return 0;
  const Shape s = rope_shape(p, true);
  return align_up((size_t)s.workers * 2 * (p->norm == SVGEAR_QKNORM_TOKEN ? p->H * p->d : p->d) * sizeof(float), 256);
}

cudaError_t qkv_rope_back_run(const void* const grad[3], const void* const in[2], const float* wq, const float* wk,
                              const int32_t* pos, const svgear_rope_params* p, void* const out[3], float* dwq, float* dwk,
                              void* ws, cudaStream_t st) {
  const Shape s = rope_shape(p, true);
  RopeArgs a = rope_args(p, wq, wk, pos, s);
  for (int k = 0; k < 3; ++k) {
    a.grad[k] = grad[k];
    a.out[k] = out[k];
    if (k < 2) a.in[k] = in[k];
  }
  const bool sums = p->norm != SVGEAR_QKNORM_NONE && (dwq || dwk);
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  const bool half = p->pairing == SVGEAR_PAIR_HALF;
  if (p->dtype == DT_F32) launch_rope<float>(a, s, half, true, st);
  else launch_rope<bf16>(a, s, half, true, st);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && sums) {
    const int C = p->norm == SVGEAR_QKNORM_TOKEN ? p->H * p->d : p->d;
    k_rope_weight_sums<<<dim3((C + 31) / 32, 2), 32 * kSumLanes, 0, st>>>(a.part, s.workers, C, dwq, dwk);
    note_launch();
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace svg
