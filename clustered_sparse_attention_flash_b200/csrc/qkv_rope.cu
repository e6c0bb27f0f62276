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
//
// Measured on a B200 behind other work (share of a plain copy's 6,544 GB/s), norm
// over the token: 75,600 tokens of 40 heads of 128, bf16 747 us (0.95; 769 us each
// in a hundred calls in a row), float32 1,521 us (0.93); backward of 32,768 tokens
// of 16 heads bf16 184 us (0.89), float32 355 us (0.93), of 40 heads bf16 505 us
// (0.81).  262,144 tokens of one head of 64 without a norm 55 us (0.56): the sines
// of a token cost as much as its one head, and those of the axes that did not move
// are computed again.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "rowvec.cuh"
#include "tc_common.cuh"

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
  int B, N, H, out_tokens, norm, tpt, chunk, stages, ring_bytes, weight_bytes, table_tokens, grads_at;
  int pairs0, pairs01, pairs;  // pairs of axis 0, of axes 0-1, of all axes
  int g1, g2, vol;             // grid extents of axes 1 and 2, grid tokens
  int origin[3];
  float eps;
  int* status;
  double freq[kMaxPairs];  // turns per position
};

// Where a token sits on the three axes; `on`: it turns at all.
struct Spot {
  int x[3];
  bool on;
};
__device__ __forceinline__ Spot spot(const RopeArgs& p, int b, int n) {
  Spot s;
  s.on = p.pos || n < p.vol;
  if (p.pos) {
    const int32_t* at = p.pos + (long long)b * p.pos_batch + (long long)n * 3;
    s.x[0] = at[0]; s.x[1] = at[1]; s.x[2] = at[2];
  } else {
    const int q = (int)((unsigned)n / (unsigned)p.g2), t = (int)((unsigned)q / (unsigned)p.g1);
    s.x[0] = t;
    s.x[1] = q - t * p.g1;
    s.x[2] = n - q * p.g2;
  }
  return s;
}

// cos and sin of pair i of a token; the identity where nothing turns.
__device__ __forceinline__ float2 cos_sin(const RopeArgs& p, const Spot& s, int i) {
  float2 v = make_float2(1.f, 0.f);
  if (s.on && i < p.pairs) {
    const bool a0 = i < p.pairs0, a1 = i < p.pairs01;
    double t = ((double)(a0 ? s.x[0] : a1 ? s.x[1] : s.x[2]) + (a0 ? p.origin[0] : a1 ? p.origin[1] : p.origin[2])) * p.freq[i];
    t -= rint(t);
    sincospif(2.f * (float)t, &v.y, &v.x);
  }
  return v;
}

// A thread's 16 elements of a head as two sets of packed floats: A the first
// and B the second members of its eight pairs, in the order of its angles.
struct Sixteen {
  f2 A[4], B[4];
};

__device__ __forceinline__ f2 low_bf16(uint32_t a, uint32_t b) { return pair(__uint_as_float(a << 16), __uint_as_float(b << 16)); }
__device__ __forceinline__ f2 high_bf16(uint32_t a, uint32_t b) {
  return pair(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u));
}
template <bool HALF>
__device__ __forceinline__ void spread(const Raw<bf16>& lo, const Raw<bf16>& hi, Sixteen& z) {
  if (HALF) {
    Vec a, b;
    unpack(lo, a);
    unpack(hi, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) { z.A[i] = a.v[i]; z.B[i] = b.v[i]; }
  } else {
    z.A[0] = low_bf16(lo.u.x, lo.u.y); z.B[0] = high_bf16(lo.u.x, lo.u.y);
    z.A[1] = low_bf16(lo.u.z, lo.u.w); z.B[1] = high_bf16(lo.u.z, lo.u.w);
    z.A[2] = low_bf16(hi.u.x, hi.u.y); z.B[2] = high_bf16(hi.u.x, hi.u.y);
    z.A[3] = low_bf16(hi.u.z, hi.u.w); z.B[3] = high_bf16(hi.u.z, hi.u.w);
  }
}
template <bool HALF>
__device__ __forceinline__ void spread(const Raw<float>& lo, const Raw<float>& hi, Sixteen& z) {
  if (HALF) {
    Vec a, b;
    unpack(lo, a);
    unpack(hi, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) { z.A[i] = a.v[i]; z.B[i] = b.v[i]; }
  } else {
    z.A[0] = pair(lo.a.x, lo.a.z); z.B[0] = pair(lo.a.y, lo.a.w);
    z.A[1] = pair(lo.b.x, lo.b.z); z.B[1] = pair(lo.b.y, lo.b.w);
    z.A[2] = pair(hi.a.x, hi.a.z); z.B[2] = pair(hi.a.y, hi.a.w);
    z.A[3] = pair(hi.b.x, hi.b.z); z.B[3] = pair(hi.b.y, hi.b.w);
  }
}
// The two vectors in memory order.
template <bool HALF>
__device__ __forceinline__ void gather(const Sixteen& z, Vec& lo, Vec& hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (HALF) {
      lo.v[i] = z.A[i];
      hi.v[i] = z.B[i];
    } else {
      const float2 a = halves(z.A[i]), b = halves(z.B[i]);
      Vec& o = i < 2 ? lo : hi;
      o.v[2 * (i & 1)] = pair(a.x, b.x);
      o.v[2 * (i & 1) + 1] = pair(a.y, b.y);
    }
  }
}
template <typename T, bool HALF>
__device__ __forceinline__ void put(T* at, int half, const Sixteen& z) {
  Vec lo, hi;
  gather<HALF>(z, lo, hi);
  store_vec(at, lo);
  store_vec(at + half, hi);
}

// z turned by its angles; `sign` -1 turns back.
__device__ __forceinline__ void turn(Sixteen& z, const f2 (&c)[4], const f2 (&s)[4], float sign) {
  const f2 k = pair(sign), nk = pair(-sign);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 a = z.A[i];
    z.A[i] = fma2(mul2(s[i], nk), z.B[i], mul2(a, c[i]));
    z.B[i] = fma2(mul2(s[i], k), a, mul2(z.B[i], c[i]));
  }
}
__device__ __forceinline__ float dot(const Sixteen& x, const Sixteen& y) {
  f2 q = mul2(x.A[0], y.A[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i) q = fma2(x.A[i], y.A[i], q);
    q = fma2(x.B[i], y.B[i], q);
  }
  const float2 h = halves(q);
  return h.x + h.y;
}

// Where a thread works: its worker, its place in a token, its run of tokens.
template <int D>
struct Place {
  static constexpr int lanes = D / 16;
  int slot, lane, j, head, off;  // off: element offset of the low vector in a token
  bool on;
  int t, end;                           // tokens [t, end), counted b * N + n
};
template <int D>
__device__ __forceinline__ Place<D> place(const RopeArgs& p) {
  Place<D> q;
  q.slot = threadIdx.x / p.tpt;
  q.lane = threadIdx.x - q.slot * p.tpt;
  q.head = q.lane / q.lanes;
  q.j = q.lane - q.head * q.lanes;
  q.on = q.head < p.H;
  q.off = q.head * D + q.j * kVec;
  const long long total = (long long)p.B * p.N, first = ((long long)blockIdx.x * (blockDim.x / p.tpt) + q.slot) * p.chunk;
  q.t = (int)min(first, total);
  q.end = (int)min(first + p.chunk, total);
  return q;
}

// Batch entry and token, stepped without divisions.
struct Token {
  int b, n;
  __device__ __forceinline__ Token(const RopeArgs& p, int t) : b(t / p.N), n(t - t / p.N * p.N) {}
  __device__ __forceinline__ void step(int N) {
    if (++n == N) { n = 0; ++b; }
  }
};

// Shared memory: ring stages, then per thread the weights of its elements
// ([2][4][threads] of 16 bytes), then cos and sin of the tokens in work.
__device__ __forceinline__ uint8_t* shared_base() {
  extern __shared__ __align__(128) uint8_t dyn[];
  return dyn;
}

// SHARED: in shared memory, each thread its own elements; otherwise (tokens too
// wide for that) read from global memory, where they stay in the L1.
template <bool HALF, bool SHARED, int D>
struct Weights {
  const RopeArgs& p;
  const Place<D>& pl;
  ulonglong2* at;
  __device__ __forceinline__ void load(int k, Sixteen& z) const {
    const int o = p.norm == SVGEAR_QKNORM_TOKEN ? pl.off : pl.j * kVec;
    Raw<float> lo, hi;
    lo.a = lo.b = hi.a = hi.b = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.w[k] && pl.on) {
      const float4* w = reinterpret_cast<const float4*>(p.w[k] + o);
      const float4* v = reinterpret_cast<const float4*>(p.w[k] + o + D / 2);
      lo.a = w[0]; lo.b = w[1]; hi.a = v[0]; hi.b = v[1];
    }
    spread<HALF>(lo, hi, z);
  }
  __device__ __forceinline__ Weights(const RopeArgs& args, const Place<D>& place)
      : p(args), pl(place), at(reinterpret_cast<ulonglong2*>(shared_base() + args.ring_bytes) + threadIdx.x) {
    if (!SHARED || p.norm == SVGEAR_QKNORM_NONE) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Sixteen z;
      load(k, z);
      const f2 v[8] = {z.A[0], z.A[1], z.A[2], z.A[3], z.B[0], z.B[1], z.B[2], z.B[3]};
#pragma unroll
      for (int i = 0; i < 4; ++i) at[(k * 4 + i) * blockDim.x] = make_ulonglong2(v[2 * i], v[2 * i + 1]);
    }
  }
  // z *= weight
  __device__ __forceinline__ void apply(int k, Sixteen& z) const {
    Sixteen w;
    if (SHARED) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const ulonglong2 a = at[(k * 4 + i) * blockDim.x], b = at[(k * 4 + 2 + i) * blockDim.x];
        w.A[2 * i] = a.x; w.A[2 * i + 1] = a.y;
        w.B[2 * i] = b.x; w.B[2 * i + 1] = b.y;
      }
    } else {
      load(k, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z.A[i] = mul2(z.A[i], w.A[i]);
      z.B[i] = mul2(z.B[i], w.B[i]);
    }
  }
};

// cos and sin, per token cos[d/2] then sin[d/2].  A block fills the tables of
// `table_tokens` tokens at once, so that every thread has a pair to compute; a
// worker inside a warp fills its own token's.  Two buffers: one is filled again
// only behind the barrier that follows the filling of the other.
template <int D>
struct Tables {
  static constexpr int half = D / 2;
  float* base;
  int left, buf, tok;
  __device__ __forceinline__ Tables(const RopeArgs& p, int slot)
      : base(reinterpret_cast<float*>(shared_base() + p.ring_bytes + p.weight_bytes)),
        left(0), buf(1), tok(0) {
    if (p.tpt <= 32) base += slot * 2 * D;
  }
  __device__ __forceinline__ void next(const RopeArgs& p, const Token& t, int lane) {
    if (p.tpt <= 32) {
      buf ^= 1;
      float* at = base + buf * D;
      const Spot s = spot(p, t.b, t.n);
      for (int i = lane; i < half; i += p.tpt) {
        const float2 v = cos_sin(p, s, i);
        at[i] = v.x;
        at[half + i] = v.y;
      }
      __syncwarp();
      return;
    }
    ++tok;
    if (left-- == 0) {
      left = p.table_tokens - 1;
      tok = 0;
      buf ^= 1;
      const int mine = threadIdx.x / half, i = threadIdx.x - mine * half;
      if (mine < p.table_tokens) {
        int b = t.b, n = t.n + mine;
        while (n >= p.N) { n -= p.N; ++b; }
        if (b < p.B) {
          const float2 v = cos_sin(p, spot(p, b, n), i);
          float* at = base + (buf * p.table_tokens + mine) * D;
          at[i] = v.x;
          at[half + i] = v.y;
        }
      }
      __syncthreads();
    }
  }
  template <bool HALF>
  __device__ __forceinline__ void read(const RopeArgs& p, int j, f2 (&c)[4], f2 (&s)[4]) const {
    const float* at = base + (p.tpt <= 32 ? buf : buf * p.table_tokens + tok) * D;
    const int o0 = HALF ? j * 8 : j * 4, o1 = HALF ? j * 8 + 4 : half / 2 + j * 4;
    const ulonglong2 c0 = *reinterpret_cast<const ulonglong2*>(at + o0), c1 = *reinterpret_cast<const ulonglong2*>(at + o1);
    const ulonglong2 s0 = *reinterpret_cast<const ulonglong2*>(at + half + o0), s1 = *reinterpret_cast<const ulonglong2*>(at + half + o1);
    c[0] = c0.x; c[1] = c0.y; c[2] = c1.x; c[3] = c1.y;
    s[0] = s0.x; s[1] = s0.y; s[2] = s1.x; s[3] = s1.y;
  }
};

// Token-major rows of up to OPS operands: workers inside a warp load them
// straight into registers, one token ahead; blocks take them from a ring of
// bulk copies in shared memory.
template <typename T, int OPS, int D>
struct Direct {
  const RopeArgs& p;
  const Place<D>& pl;
  Token ahead;
  int t;
  Raw<T> nx[OPS][2];
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int k = 0; k < OPS; ++k) {
      zero_raw(nx[k][0]);
      zero_raw(nx[k][1]);
      if (p.in[k] && t < pl.end && pl.on) {
        const T* x = static_cast<const T*>(p.in[k]) + ahead.b * p.batch[k] + ahead.n * p.ld[k] + pl.off;
        load_raw(nx[k][0], x);
        load_raw(nx[k][1], x + D / 2);
      }
    }
  }
  __device__ __forceinline__ Direct(const RopeArgs& args, const Place<D>& place)
      : p(args), pl(place), ahead(args, place.t), t(place.t) {
    load();
  }
  __device__ __forceinline__ void take(Raw<T> (&r)[OPS][2]) {
#pragma unroll
    for (int k = 0; k < OPS; ++k) {
      r[k][0] = nx[k][0];
      r[k][1] = nx[k][1];
    }
    ++t;
    ahead.step(p.N);
    load();
  }
  __device__ __forceinline__ void release() {}
};

constexpr int kMaxStages = 8;

template <typename T, int OPS, int D>
struct Ring {
  const RopeArgs& p;
  const Place<D>& pl;
  Token ahead;       // the next token to be copied
  int t;
  uint32_t row;      // bytes of a token's row
  uint64_t* full;
  volatile int* abort_flag;
  int slot;
  uint32_t parity;
  int stop;          // a wait has given up
  // One thread: the copies of token `ahead` into stage s.
  __device__ __forceinline__ void issue(int s) {
    if (t >= pl.end || stop) return;
    uint32_t bytes = 0;
#pragma unroll
    for (int k = 0; k < OPS; ++k) bytes += p.in[k] ? row : 0u;
    if (bytes) {
      tc::mbar_arrive_expect_tx(full + s, bytes);
      const uint32_t dst = tc::smem_u32(shared_base()) + s * OPS * row;
#pragma unroll
      for (int k = 0; k < OPS; ++k)
        if (p.in[k]) tc::bulk_g2s(dst + k * row, static_cast<const T*>(p.in[k]) + ahead.b * p.batch[k] + ahead.n * p.ld[k], row, full + s);
    }
    ++t;
    ahead.step(p.N);
  }
  __device__ __forceinline__ Ring(const RopeArgs& args, const Place<D>& place)
      : p(args), pl(place), ahead(args, place.t), t(place.t), row(args.H * D * sizeof(T)), slot(0), parity(0), stop(0) {
    __shared__ uint64_t bars[kMaxStages];
    __shared__ int flag;
    full = bars;
    abort_flag = &flag;
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.stages; ++i) tc::mbar_init(full + i, 1);
      flag = 0;
      tc::mbar_fence_init();
      for (int i = 0; i < p.stages; ++i) issue(i);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void take(Raw<T> (&r)[OPS][2]) {
    bool any = false;
#pragma unroll
    for (int k = 0; k < OPS; ++k) any |= p.in[k] != nullptr;
    // A wait that gives up records it; the block goes on with what is there, so every thread still meets every
    // barrier, and copies no more: the stage's last copy may not have ended.  Those in flight were issued before the
    // wait began and have had its limit to end.
    if (any) tc::mbar_wait(full + slot, parity, abort_flag, p.status);
    // threads without a head read the first one's elements: their sums are replaced by zeros, and they store nothing
    const uint8_t* at = shared_base() + slot * OPS * row + (pl.on ? pl.off : 0) * sizeof(T);
#pragma unroll
    for (int k = 0; k < OPS; ++k) {
      if (p.in[k]) {
        r[k][0] = *reinterpret_cast<const Raw<T>*>(at + k * row);
        r[k][1] = *reinterpret_cast<const Raw<T>*>(at + k * row + D / 2 * sizeof(T));
      } else {
        zero_raw(r[k][0]);
        zero_raw(r[k][1]);
      }
    }
    stop = *abort_flag;  // read here, it costs nothing; in release() 2 to 11 %
  }
  // Behind a barrier that follows take(): the stage is free for a later token.
  __device__ __forceinline__ void release() {
    if (threadIdx.x == 0) issue(slot);
    if (++slot == p.stages) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// Block classes: most threads of a block and the threads an SM is to hold (the
// launch bounds set the registers, the grid and the ring count on them).
// 0: tokens of up to 512 columns; 1, 2, 3: up to 2,048, 6,144 and 16,384.
template <int CLS, bool BACK>
struct Class {
  static constexpr int kMax = CLS <= 1 ? 128 : CLS == 2 ? 384 : 1024;
  static constexpr int kThreads = CLS == 0 ? (BACK ? 256 : 512) : CLS == 1 ? (BACK ? 384 : 512) : CLS == 2 ? 384 : 1024;
};

// Gradients of Q, K and V of a token, head-major: each thread copies its own
// vectors into its own slots of shared memory, two tokens ahead (as registers
// they would spill), so no barrier is needed before it reads them back.
// Without slots (float32 rows, wide blocks) they are loaded where they are used.
constexpr int kAheadStages = 2;
template <typename T>
constexpr bool ahead_of(int cls) {
  return sizeof(T) == 2 && cls < 3;
}

template <typename T, bool AHEAD, int D>
struct Gradients {
  static constexpr int kParts = sizeof(Raw<T>) / 16;
  const RopeArgs& p;
  const Place<D>& pl;
  Token ahead;
  int t;
  uint32_t at;
  int slot;
  uint8_t* mem;
  __device__ __forceinline__ const T* source(int k, const Token& tk) const {
    return static_cast<const T*>(p.grad[k]) + ((long long)(tk.b * p.H + pl.head) * p.out_tokens + tk.n) * D + pl.j * kVec;
  }
  __device__ __forceinline__ void issue(int s) {
    if (t < pl.end && pl.on) {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (p.grad[k]) {
          const T* x = source(k, ahead);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kParts; ++i)
              tc::cp_async16(at + (((s * 3 + k) * 2 + h) * kParts + i) * blockDim.x * 16,
                             reinterpret_cast<const uint8_t*>(x + h * (D / 2)) + i * 16, 16);
        }
    }
    tc::cp_async_commit();
    ++t;
    ahead.step(p.N);
  }
  __device__ __forceinline__ Gradients(const RopeArgs& args, const Place<D>& place, uint8_t* slots)
      : p(args), pl(place), ahead(args, place.t), t(place.t), slot(0), mem(slots + threadIdx.x * 16) {
    at = tc::smem_u32(mem);
    if (AHEAD)
      for (int i = 0; i < kAheadStages - 1; ++i) issue(i);
  }
  __device__ __forceinline__ void take(const Token& tk, bool mine, Raw<T> (&g)[3][2]) {
    if (AHEAD) {
      issue(slot == 0 ? kAheadStages - 1 : slot - 1);  // the slot read last
      tc::cp_async_wait_group<kAheadStages - 1>();
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        zero_raw(g[k][h]);
        if (!p.grad[k] || !mine) continue;
        if (AHEAD) {
          uint4* r = reinterpret_cast<uint4*>(&g[k][h]);
#pragma unroll
          for (int i = 0; i < kParts; ++i)
            r[i] = *reinterpret_cast<const uint4*>(mem + (((slot * 3 + k) * 2 + h) * kParts + i) * blockDim.x * 16);
        } else {
          load_raw(g[k][h], source(k, tk) + h * (D / 2));
        }
      }
    if (AHEAD && ++slot == kAheadStages) slot = 0;
  }
};

template <typename T, bool HALF, int CLS, int D>
__global__ void __launch_bounds__(Class<CLS, false>::kMax, (Class<CLS, false>::kThreads / Class<CLS, false>::kMax))
    k_qkv_rope(const __grid_constant__ RopeArgs p) {
  __shared__ float2 scratch[64];
  RowSum<CLS == 0 ? -1 : CLS == 1 ? 2 : CLS == 2 ? 4 : 5> sum(scratch, p.tpt);
  const Place<D> pl = place<D>(p);
  constexpr int half = D / 2;
  const float inv_c = 1.f / (float)(p.norm == SVGEAR_QKNORM_TOKEN ? p.H * D : D);
  const Weights<HALF, CLS != 3, D> w(p, pl);
  Tables<D> tables(p, pl.slot);
  typename std::conditional<CLS == 0, Direct<T, 3, D>, Ring<T, 3, D>>::type rows(p, pl);
  Token tk(p, pl.t);
  for (int it = 0; it < p.chunk; ++it, tk.step(p.N)) {
    const bool live = pl.t + it < pl.end;
    if (p.tpt >= 32 && !live) break;  // uniform over the worker
    if (!live) tk.b = tk.n = 0;       // lanes of a warp whose other workers still run
    tables.next(p, tk, pl.lane);
    Raw<T> raw[3][2];
    rows.take(raw);
    const bool mine = live && pl.on;
    const long long o = ((long long)(tk.b * p.H + pl.head) * p.out_tokens + tk.n) * D + pl.j * kVec;
    if (p.in[2] && mine) {
      T* out = static_cast<T*>(p.out[2]) + o;
      store_raw(out, raw[2][0]);
      store_raw(out + half, raw[2][1]);
    }
    Sixteen z[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) spread<HALF>(raw[k][0], raw[k][1], z[k]);
    if (p.norm != SVGEAR_QKNORM_NONE) {
      float2 s = make_float2(dot(z[0], z[0]), dot(z[1], z[1]));
      if (!pl.on) s = make_float2(0.f, 0.f);
      if (p.norm == SVGEAR_QKNORM_TOKEN) {
        s = sum(s);
      } else {
        for (int i = pl.lanes >> 1; i > 0; i >>= 1) {
          s.x += __shfl_xor_sync(0xffffffffu, s.x, i);
          s.y += __shfl_xor_sync(0xffffffffu, s.y, i);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f2 inv = pair(rsqrtf(fmaf(k ? s.y : s.x, inv_c, p.eps)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[k].A[i] = mul2(z[k].A[i], inv);
          z[k].B[i] = mul2(z[k].B[i], inv);
        }
        w.apply(k, z[k]);
      }
    }
    f2 c[4], sn[4];
    tables.read<HALF>(p, pl.j, c, sn);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (p.in[k] && mine) {
        turn(z[k], c, sn, 1.f);
        put<T, HALF>(static_cast<T*>(p.out[k]) + o, half, z[k]);
      }
    if (CLS != 0 && p.norm != SVGEAR_QKNORM_TOKEN) __syncthreads();  // else the sum's barrier frees the stage
    rows.release();
  }
}

// Backward: g = the gradient turned back; with a norm, n = x inv, u = g w:
//   dx = inv (u - n mean(u n)) = inv u - x inv^3 sum(u x) / C,  dw += g n,
// so that sum(x^2) and sum(u x) of Q and of K share one barrier.
template <typename T, bool HALF, int CLS, int D>
__global__ void __launch_bounds__(Class<CLS, true>::kMax, (Class<CLS, true>::kThreads / Class<CLS, true>::kMax))
    k_qkv_rope_back(const __grid_constant__ RopeArgs p) {
  __shared__ float2 scratch[128];
  constexpr bool kAhead = ahead_of<T>(CLS);
  RowSum<CLS == 0 ? -1 : CLS == 1 ? 2 : CLS == 2 ? 4 : 5> sum(scratch, p.tpt);
  const Place<D> pl = place<D>(p);
  constexpr int half = D / 2;
  const float inv_c = 1.f / (float)(p.norm == SVGEAR_QKNORM_TOKEN ? p.H * D : D);
  const Weights<HALF, CLS != 3, D> w(p, pl);
  Tables<D> tables(p, pl.slot);
  typename std::conditional<CLS == 0, Direct<T, 2, D>, Ring<T, 2, D>>::type rows(p, pl);
  Gradients<T, kAhead, D> grads(p, pl, shared_base() + p.grads_at);
  Token tk(p, pl.t);
  Sixteen dw[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[k].A[i] = dw[k].B[i] = pair(0.f);
  for (int it = 0; it < p.chunk; ++it, tk.step(p.N)) {
    const bool live = pl.t + it < pl.end;
    if (p.tpt >= 32 && !live) break;
    if (!live) tk.b = tk.n = 0;
    const bool mine = live && pl.on;
    const long long go = tk.b * p.out_batch + tk.n * p.out_ld + pl.off;
    Raw<T> g[3][2];
    grads.take(tk, mine, g);
    if (p.grad[2] && mine) {
      T* out = static_cast<T*>(p.out[2]) + go;
      store_raw(out, g[2][0]);
      store_raw(out + half, g[2][1]);
    }
    tables.next(p, tk, pl.lane);
    Raw<T> raw[2][2];
    rows.take(raw);
    Sixteen z[2];
    {
      f2 c[4], sn[4];
      tables.read<HALF>(p, pl.j, c, sn);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        spread<HALF>(g[k][0], g[k][1], z[k]);
        turn(z[k], c, sn, -1.f);
      }
    }
    if (p.norm != SVGEAR_QKNORM_NONE) {
      Sixteen x[2];
      float2 s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        spread<HALF>(raw[k][0], raw[k][1], x[k]);
        Sixteen u = z[k];
        w.apply(k, u);
        s[k] = make_float2(dot(x[k], x[k]), dot(u, x[k]));
        if (!pl.on) s[k] = make_float2(0.f, 0.f);
      }
      if (p.norm == SVGEAR_QKNORM_TOKEN) {
        sum.both(s[0], s[1]);
      } else {
        for (int i = pl.lanes >> 1; i > 0; i >>= 1)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            s[k].x += __shfl_xor_sync(0xffffffffu, s[k].x, i);
            s[k].y += __shfl_xor_sync(0xffffffffu, s[k].y, i);
          }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float r = rsqrtf(fmaf(s[k].x, inv_c, p.eps));
        const f2 inv = pair(r), m = pair(-(s[k].y * inv_c) * r * r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k].A[i] = mul2(x[k].A[i], inv);
          x[k].B[i] = mul2(x[k].B[i], inv);
          dw[k].A[i] = fma2(z[k].A[i], x[k].A[i], dw[k].A[i]);
          dw[k].B[i] = fma2(z[k].B[i], x[k].B[i], dw[k].B[i]);
        }
        w.apply(k, z[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[k].A[i] = fma2(x[k].A[i], m, mul2(z[k].A[i], inv));
          z[k].B[i] = fma2(x[k].B[i], m, mul2(z[k].B[i], inv));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (p.grad[k] && mine) put<T, HALF>(static_cast<T*>(p.out[k]) + go, half, z[k]);
    if (CLS != 0 && p.norm != SVGEAR_QKNORM_TOKEN) __syncthreads();
    rows.release();
  }
  if (!p.part) return;
  const long long worker = (long long)blockIdx.x * (blockDim.x / p.tpt) + pl.slot;
  const bool has = pl.t < pl.end;  // workers without a token have no slot
  if (p.norm == SVGEAR_QKNORM_TOKEN) {
    if (has && pl.on)
#pragma unroll
      for (int k = 0; k < 2; ++k) put<float, HALF>(p.part + ((size_t)worker * 2 + k) * p.H * D + pl.off, half, dw[k]);
    return;
  }
  // Per-head weights: add the heads of this worker, in a warp, then over its warps.
  // A thread without a head has multiplied zero gradients by another's elements, which gave NaN where those are
  // infinite.  (pl.on, kept over the loop for this, would spill; threads inside a warp loaded zeros.)
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 a = halves(dw[k].A[i]), b = halves(dw[k].B[i]);
      if (CLS != 0 && (int)threadIdx.x / pl.lanes >= p.H) a = b = make_float2(0.f, 0.f);
      for (int s = pl.lanes; s < (p.tpt < 32 ? p.tpt : 32); s <<= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, s);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, s);
        b.x += __shfl_xor_sync(0xffffffffu, b.x, s);
        b.y += __shfl_xor_sync(0xffffffffu, b.y, s);
      }
      dw[k].A[i] = pair(a.x, a.y);
      dw[k].B[i] = pair(b.x, b.y);
    }
  if (p.tpt <= 32) {
    if (has && pl.lane < pl.lanes)
#pragma unroll
      for (int k = 0; k < 2; ++k) put<float, HALF>(p.part + ((size_t)worker * 2 + k) * D + pl.j * kVec, half, dw[k]);
    return;
  }
  float* red = reinterpret_cast<float*>(shared_base());  // [warps][d], over the ring, whose copies have all been taken
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
    if ((threadIdx.x & 31) < pl.lanes) put<float, HALF>(red + (threadIdx.x >> 5) * D + pl.j * kVec, half, dw[k]);
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
      float s = 0.f;
      for (int v = 0; v < p.tpt / 32; ++v) s += red[v * D + i];
      if (has) p.part[((size_t)worker * 2 + k) * D + i] = s;
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
  if (col < C) {
#pragma unroll 4
    for (long long i = w; i < workers; i += kSumLanes) s += part[((size_t)i * 2 + blockIdx.y) * C + col];
  }
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
  int cls, tpt, block, chunk, grid, stages, ring_bytes, weight_bytes, table_tokens, grads_at, smem;
  long long workers;
};

constexpr int kSmemPerSm = 228 * 1024, kSmemPerBlock = 3 * 1024;  // 1 KB per block is the system's, the rest static arrays
// What the rings of an SM's blocks hold together at most.  More than about 80 KB
// in flight only queues reads before the writes and takes the L1 away
// (float32, 40 heads, 32,768 tokens: 748 us with 180 KB, 685 us).
constexpr int kRingPerSm = 92 * 1024;
// The forward pass takes no more blocks than hold two stages each in this (16
// heads of 128, share of the copy rate with 3 / 4 blocks: 0.91 / 0.79; 12 heads
// with 4 / 5: 0.86 / 0.79; 8 heads with 7 / 8: 0.85 / 0.77).
constexpr int kBlocksRing = 85 * 1024;

Shape rope_shape(const svgear_rope_params* p, bool back) {
  Shape s;
  const int items = p->H * p->d / 16;
  const bool normed = p->norm != SVGEAR_QKNORM_NONE;
  int threads;
  if (items <= 32) {
    s.cls = 0;
    s.tpt = items <= 4 ? 4 : items <= 8 ? 8 : items <= 16 ? 16 : 32;
    s.block = 128;
    threads = back ? Class<0, true>::kThreads : Class<0, false>::kThreads;
  } else {
    s.tpt = s.block = (items + 31) / 32 * 32;
    s.cls = s.block <= 128 ? 1 : s.block <= 384 ? 2 : 3;
    threads = s.cls == 1   ? (back ? Class<1, true>::kThreads : Class<1, false>::kThreads)
              : s.cls == 2 ? (back ? Class<2, true>::kThreads : Class<2, false>::kThreads)
                           : Class<3, true>::kThreads;
  }
  const int per = s.block / s.tpt;
  const long long tokens = (long long)p->B * p->N;
  s.table_tokens = s.cls == 0 ? per : std::max(1, s.block / (p->d / 2));
  s.weight_bytes = normed && s.cls != 3 ? 128 * s.block : 0;
  const int front = s.weight_bytes + 2 * s.table_tokens * p->d * (int)sizeof(float);
  const int fixed = front + (back && p->dtype == DT_BF16 && ahead_of<bf16>(s.cls) ? kAheadStages * 6 * 16 * s.block : 0);
  // The forward pass brings q, k and v through the ring, the backward pass q and k where a norm needs them.
  const int stage = s.cls == 0 ? 0 : (back ? (normed ? 2 : 0) : 3) * p->H * p->d * (p->dtype == DT_F32 ? 4 : 2);
  int blocks = std::max(1, std::min(threads / s.block, 8));
  if (stage && !back) blocks = std::min(blocks, std::max(2, kBlocksRing / (2 * stage)));
  auto stages = [&]() { return stage ? (kSmemPerSm / blocks - kSmemPerBlock - fixed) / stage : 1; };
  while (stage && blocks > 1 && stages() < 2) --blocks;
  // As many workers as the SMs hold at once, each with a run of tokens.
  long long want = std::min(tokens, 148LL * blocks * per);
  if (back) want = std::min(want, 4096LL);
  s.chunk = (int)((tokens + want - 1) / want);
  s.workers = (tokens + s.chunk - 1) / s.chunk;
  s.grid = (int)((s.workers + per - 1) / per);
  s.stages = std::max(1, std::min({stages(), kMaxStages, s.chunk, std::max(2, kRingPerSm / blocks / std::max(stage, 1))}));
  s.ring_bytes = s.stages * stage;
  s.grads_at = s.ring_bytes + front;
  s.smem = s.ring_bytes + fixed;
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
  a.B = p->B; a.N = p->N; a.H = p->H;
  a.out_tokens = p->out_tokens > 0 ? p->out_tokens : p->N;
  a.norm = p->norm;
  a.tpt = s.tpt;
  a.chunk = s.chunk;
  a.stages = s.stages;
  a.ring_bytes = s.ring_bytes;
  a.table_tokens = s.table_tokens;
  a.weight_bytes = s.weight_bytes;
  a.grads_at = s.grads_at;
  a.status = status_word();
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

template <typename T, bool HALF, int CLS, int D>
cudaError_t launch_class(const RopeArgs& a, const Shape& s, bool back, cudaStream_t st) {
  const auto kernel = back ? k_qkv_rope_back<T, HALF, CLS, D> : k_qkv_rope<T, HALF, CLS, D>;
  if (s.smem > 32 * 1024) {
    const cudaError_t e = allow_dynamic_smem(kernel, kSmemPerSm - kSmemPerBlock);
    if (e != cudaSuccess) return e;
  }
  kernel<<<s.grid, s.block, s.smem, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

template <typename T, bool HALF, int D>
cudaError_t launch_half(const RopeArgs& a, const Shape& s, bool back, cudaStream_t st) {
  if (s.cls == 0) return launch_class<T, HALF, 0, D>(a, s, back, st);
  if (s.cls == 1) return launch_class<T, HALF, 1, D>(a, s, back, st);
  if (s.cls == 2) return launch_class<T, HALF, 2, D>(a, s, back, st);
  return launch_class<T, HALF, 3, D>(a, s, back, st);
}

cudaError_t launch_rope(const RopeArgs& a, const Shape& s, const svgear_rope_params* p, bool back, cudaStream_t st) {
  if (!a.status) return cudaErrorInvalidValue;
  const bool half = p->pairing == SVGEAR_PAIR_HALF;
  if (p->d == 128) {
    if (p->dtype == DT_F32) return half ? launch_half<float, true, 128>(a, s, back, st) : launch_half<float, false, 128>(a, s, back, st);
    return half ? launch_half<bf16, true, 128>(a, s, back, st) : launch_half<bf16, false, 128>(a, s, back, st);
  }
  if (p->dtype == DT_F32) return half ? launch_half<float, true, 64>(a, s, back, st) : launch_half<float, false, 64>(a, s, back, st);
  return half ? launch_half<bf16, true, 64>(a, s, back, st) : launch_half<bf16, false, 64>(a, s, back, st);
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
  return launch_rope(a, s, p, false, st);
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
    if (k < 2 && grad[k]) a.in[k] = in[k];  // null without a norm
  }
  const bool sums = p->norm != SVGEAR_QKNORM_NONE && (dwq || dwk);
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  cudaError_t e = launch_rope(a, s, p, true, st);
  if (e == cudaSuccess && sums) {
    const int C = p->norm == SVGEAR_QKNORM_TOKEN ? p->H * p->d : p->d;
    k_rope_weight_sums<<<dim3((C + 31) / 32, 2), 32 * kSumLanes, 0, st>>>(a.part, s.workers, C, dwq, dwk);
    note_launch();
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace svg
