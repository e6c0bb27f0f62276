// Gated residual and norms around an attention block (row-wise, HBM-bound).
//
//   m = P(y)              P, Q: none, RMS norm or layer norm of a row
//   r = a x + g m w2      (r = x without y)
//   n = Q(r),  h = (n w + b)(1 + s) + t
//
// One pass: a row is loaded once, its statistics are taken in registers, and r
// and h leave from there; h is formed from the unrounded r.  The per-column
// coefficients (1+s) w, b (1+s) + t and g w2 are formed once per group of a run.
//
// Rows are taken by workers: a warp takes one to four rows of up to 256 columns
// side by side, a whole block one wider row (two 8-element vectors per thread).
// A worker walks a contiguous run of rows, so column sums of the backward pass
// stay in registers until the group or the run ends; partial sums then go to
// slot (worker + group), which no other pair maps to because both only grow
// along the rows, and are added in slot order: no atomics, the same bits every
// time.
//
// What bounds it is HBM, once three things are out of the way: instructions
// (packed float32, two vectors per thread, statistics behind one barrier: 458
// to about 220 per warp and row), spills (with the ring's shared memory there
// is no L1 left to catch them) and reads so far ahead that the writes wait (see
// kBlocksRing).  Measured on a B200 (share of a plain copy's 6,544 GB/s), gated
// residual and layer norm, stream / branch types:
//   forward   75,600 x 5,120 bf16 525 us (0.90), float32 / bf16 770 us (0.92);
//             40,000 x 2,048 float32 215 us (0.93), float32 / bf16 157 us (0.96)
//   backward  32,768 x 2,048 bf16 148 us (0.83), of which 13 us are the column
//             sums, float32 / bf16 199 us (0.93), float32 258 us (0.95);
//             32,768 x 5,120 bf16 480 us (0.64), float32 / bf16 556 us (0.83),
//             float32 631 us (0.98)
// The backward pass of wide bf16 rows is the one far from its bytes: float32 rows,
// twice as long, take a third more.  An SM holds one block of ten warps there,
// which issue 700 instructions a row each and all stop at the same barriers.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "rowvec.cuh"
#include "tc_common.cuh"

namespace svg {

namespace {

struct NormArgs {
  const void *x, *y, *dr, *dh;
  const float *gate, *scale, *shift, *weight, *bias, *post_weight;
  const int32_t* offsets;
  int N, D, G, pre, post, clear, tpr, chunk, stages, ring_bytes;
  float eps, a;
  void *r, *h, *dx, *dy;
  float* part;  // backward: [slots][3][D] partial column sums
  int* status;
};

// First row behind group g (offsets are clamped, so bad ones stay in range).
__device__ __forceinline__ int group_end(const NormArgs& p, int g) {
  if (!p.offsets) return (int)((long long)(g + 1) * (p.N / p.G));
  const int e = p.offsets[g + 1];
  return e < 0 ? 0 : (e > p.N ? p.N : e);
}
// The first group whose end lies behind `row` (G: the row is in no group).
__device__ __forceinline__ int group_of(const NormArgs& p, int row) {
  int lo = 0, hi = p.G;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (group_end(p, mid) > row) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// What a thread knows of its row: which of its V vectors exist, and the number
// of columns of its warp and of the warp whose totals RowSum::trade hands it.
template <int V>
struct Columns {
  int col[V];
  bool on[V];
  float inv_d, d, inv_own, n, inv_n;
  template <typename SUM>
  __device__ __forceinline__ void init(int D, int tpr, int lane, const SUM&) {
    d = (float)D;
    inv_d = 1.f / d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      col[v] = (v * tpr + lane) * kVec;
      on[v] = col[v] < D;
    }
    auto columns_of = [&](int w) {
      int c = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) c += max(0, min(D - (v * tpr + 32 * w) * kVec, 32 * kVec));
      return (float)c;
    };
    const float own = tpr > 32 ? columns_of(lane >> 5) : d;
    inv_own = own > 0.f ? 1.f / own : 0.f;
    const int other = threadIdx.x & SUM::kMask;
    n = tpr > 32 && other < tpr >> 5 ? columns_of(other) : 0.f;
    inv_n = n > 0.f ? 1.f / n : 0.f;
  }
};

template <int V>
__device__ __forceinline__ float total(const Vec (&f)[V], const Columns<V>& c) {
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float2 h = halves(add2(add2(f[v].v[0], f[v].v[1]), add2(f[v].v[2], f[v].v[3])));
    s += c.on[v] ? h.x + h.y : 0.f;
  }
  return s;
}

// Sum of (f - mean)^2 over this thread's columns.
template <int V>
__device__ __forceinline__ float squares(const Vec (&f)[V], const Columns<V>& c, float mean) {
  float s = 0.f;
  const f2 m = pair(-mean);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f2 q = pair(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 e = add2(f[v].v[i], m);
      q = fma2(e, e, q);
    }
    const float2 h = halves(q);
    s += c.on[v] ? h.x + h.y : 0.f;
  }
  return s;
}

// s / d rounded like a division, so that a constant row's mean is its value.
__device__ __forceinline__ float over(float s, float d, float inv_d) {
  const float q = s * inv_d;
  return fmaf(fmaf(-q, d, s), inv_d, q);
}

// Mean and 1/deviation of a row with one barrier: a warp takes the mean and the
// squared deviations of its own columns, and the warps' pairs (sum, squares)
// are joined by
//   squares = sum_w squares_w + n_w (mean_w - mean)^2,
// every term of which is a square: nothing cancels, whatever the mean.
template <int V, typename SUM>
__device__ __forceinline__ float2 statistics(const Vec (&f)[V], const Columns<V>& c, int kind, float eps, SUM& sum) {
  if (kind == SVGEAR_NORM_RMS) return make_float2(0.f, rsqrtf(fmaf(sum(squares(f, c, 0.f)), c.inv_d, eps)));
  const float s = sum.lanes(total(f, c));
  if (!SUM::kBlock) {
    const float mean = over(s, c.d, c.inv_d);
    return make_float2(mean, rsqrtf(fmaf(sum.lanes(squares(f, c, mean)), c.inv_d, eps)));
  }
  const float q = sum.lanes(squares(f, c, s * c.inv_own));
  const float2 v = sum.trade(make_float2(s, q));
  const float mean = over(sum.warps(v.x), c.d, c.inv_d), e = v.x * c.inv_n - mean;
  return make_float2(mean, rsqrtf(fmaf(sum.warps(fmaf(c.n * e, e, v.y)), c.inv_d, eps)));
}

// f = (f - mean) inv
template <int V>
__device__ __forceinline__ void apply(Vec (&f)[V], float2 st) {
  const f2 m = pair(-st.x), inv = pair(st.y);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) f[v].v[i] = mul2(add2(f[v].v[i], m), inv);
}

// f becomes the normalised row; returns 1 / deviation.
template <int V, typename SUM>
__device__ __forceinline__ float normalise(Vec (&f)[V], const Columns<V>& c, int kind, float eps, SUM& sum) {
  if (kind == SVGEAR_NORM_NONE) return 1.f;
  const float2 st = statistics(f, c, kind, eps, sum);
  apply<V>(f, st);
  return st.y;
}

// Rows of a worker, one at a time, behind one interface: narrow rows straight
// from global memory (the next row is loaded while this one is computed), wide
// rows through a ring of bulk copies in shared memory, so that the bytes in
// flight do not depend on how many threads are resident.  Rows come in order;
// operand k of the current row is read when it is needed.  Threads without a
// column read the last ones: they add to no sum and store nothing.
enum Operand { kX = 0, kY = 1, kDr = 2, kDh = 3 };

template <typename TX, typename TY, int OPS, int V>
struct Direct {
  const NormArgs& p;
  const Columns<V>& c;
  int end;
  Raw<TX> x[V], dr[V], nx[V], ndr[V];
  Raw<TY> y[V], dh[V], ny[V], ndh[V];
  template <typename T>
  __device__ __forceinline__ void one(Raw<T>& r, const void* base, long long at, bool ok) {
    zero_raw(r);
    if (ok && base) load_raw(r, static_cast<const T*>(base) + at);
  }
  __device__ __forceinline__ void load(int row) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const long long at = (long long)row * p.D + c.col[v];
      const bool ok = c.on[v] && row < end;
      one(nx[v], p.x, at, ok);
      one(ny[v], p.y, at, ok);
      if (OPS == 4) {
        one(ndr[v], p.dr, at, ok);
        one(ndh[v], p.dh, at, ok);
      }
    }
  }
  __device__ __forceinline__ Direct(const NormArgs& args, const Columns<V>& cols, int first, int last)
      : p(args), c(cols), end(last) {
    load(first);
  }
  // The row loaded last becomes the current one, `next` is loaded.
  __device__ __forceinline__ void take(int next) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = nx[v];
      y[v] = ny[v];
      if (OPS == 4) {
        dr[v] = ndr[v];
        dh[v] = ndh[v];
      }
    }
    load(next);
  }
  template <int K>
  __device__ __forceinline__ void read(Vec (&f)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (K == kX) unpack(x[v], f[v]);
      if (K == kY) unpack(y[v], f[v]);
      if (K == kDr) unpack(dr[v], f[v]);
      if (K == kDh) unpack(dh[v], f[v]);
    }
  }
  __device__ __forceinline__ void release(int) {}
  __device__ __forceinline__ void release_previous(int) {}
};

constexpr int kMaxStages = 16;

template <typename TX, typename TY, int OPS, int V>
struct Ring {
  const NormArgs& p;
  int first, end;
  uint32_t bx, by, stage;  // bytes of a row of either type, of a stage
  uint32_t col[V];
  uint8_t* buf;
  uint64_t* full;
  volatile int* abort_flag;
  int slot;         // the stage of the current row,
  uint32_t parity;  // and the parity of its phase
  int stop;         // a wait has given up
  // One thread: the copies of `row` into stage s.
  __device__ __forceinline__ void issue(int row, int s) {
    if (row >= end || stop) return;
    tc::mbar_arrive_expect_tx(full + s, bx + (p.y ? by : 0u) + (OPS == 4 ? (p.dr ? bx : 0u) + (p.dh ? by : 0u) : 0u));
    const uint32_t dst = tc::smem_u32(buf) + s * stage;
    tc::bulk_g2s(dst, static_cast<const char*>(p.x) + (long long)row * bx, bx, full + s);
    if (p.y) tc::bulk_g2s(dst + bx, static_cast<const char*>(p.y) + (long long)row * by, by, full + s);
    if (OPS == 4) {
      if (p.dr) tc::bulk_g2s(dst + bx + by, static_cast<const char*>(p.dr) + (long long)row * bx, bx, full + s);
      if (p.dh) tc::bulk_g2s(dst + 2 * bx + by, static_cast<const char*>(p.dh) + (long long)row * by, by, full + s);
    }
  }
  __device__ __forceinline__ Ring(const NormArgs& args, const Columns<V>& cols, int row, int last)
      : p(args), first(row), end(last), slot(-1), parity(1), stop(0) {
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ uint64_t bars[kMaxStages];
    __shared__ int flag;
    bx = p.D * sizeof(TX);
    by = p.D * sizeof(TY);
    stage = (OPS / 2) * (bx + by);
#pragma unroll
    for (int v = 0; v < V; ++v) col[v] = min(cols.col[v], p.D - kVec);
    buf = dyn;
    full = bars;
    abort_flag = &flag;
    slot = p.stages - 1;
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.stages; ++i) tc::mbar_init(full + i, 1);
      flag = 0;
      tc::mbar_fence_init();
      for (int i = 0; i < p.stages; ++i) issue(first + i, i);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void take(int) {
    if (++slot == p.stages) {
      slot = 0;
      parity ^= 1;
    }
    // A wait that gives up records it; the block goes on with what is there, so every thread still meets every
    // barrier, and copies no more: the stage's last copy may not have ended.  Those in flight were issued before the
    // wait began and have had its limit to end.
    tc::mbar_wait(full + slot, parity, abort_flag, p.status);
    stop = *abort_flag;
  }
  template <int K>
  __device__ __forceinline__ void read(Vec (&f)[V]) const {
    const uint8_t* at = buf + slot * stage + (K == kX ? 0u : K == kY ? bx : K == kDr ? bx + by : 2 * bx + by);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (K == kX || K == kDr) unpack(*reinterpret_cast<const Raw<TX>*>(at + col[v] * sizeof(TX)), f[v]);
      else unpack(*reinterpret_cast<const Raw<TY>*>(at + col[v] * sizeof(TY)), f[v]);
    }
  }
  // Behind a barrier that every thread reached after its last read of `row`.
  __device__ __forceinline__ void release(int row) {
    if (threadIdx.x == 0) issue(row + p.stages, slot);
  }
  // Behind a barrier in `row`: the row before it has been read by every thread.
  __device__ __forceinline__ void release_previous(int row) {
    if (threadIdx.x == 0 && row != first) issue(row - 1 + p.stages, slot == 0 ? p.stages - 1 : slot - 1);
  }
};

// The worker of a thread and its run of rows, up to the last group's end.  A
// worker takes `step` rows at a time, this thread's being `sub` behind the
// first; no step reaches over a group's end.
struct Place {
  int worker, row, end, lane, sub, step;
};
template <bool NARROW>
__device__ __forceinline__ Place place(const NormArgs& p) {
  Place q;
  if (NARROW) {
    q.worker = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    q.step = 32 / p.tpr;
    q.sub = (threadIdx.x & 31) / p.tpr;
    q.lane = threadIdx.x & (p.tpr - 1);
  } else {
    q.worker = blockIdx.x;
    q.step = 1;
    q.sub = 0;
    q.lane = threadIdx.x;
  }
  const long long first = (long long)q.worker * p.chunk;
  q.end = (int)min(first + p.chunk, (long long)group_end(p, p.G - 1));
  q.row = (int)min(first, (long long)p.N);
  return q;
}

// The rows of a worker's run behind the last group, which belong to none: zeros,
// or those of `from`.  A run's rows lie side by side.
template <bool NARROW, typename T>
__device__ __forceinline__ void clear_rest(const NormArgs& p, const Place& q, void* to, const void* from = nullptr) {
  if (!to) return;
  const int threads = NARROW ? 32 : blockDim.x, t = NARROW ? threadIdx.x & 31 : threadIdx.x;
  const long long till = min((long long)q.row + p.chunk, (long long)p.N) * p.D;
  for (long long i = (long long)max(q.row, q.end) * p.D + t * kVec; i < till; i += threads * kVec) {
    Raw<T> v;
    zero_raw(v);
    if (from) load_raw(v, static_cast<const T*>(from) + i);
    store_raw(static_cast<T*>(to) + i, v);
  }
}

// Steps through a run: `base` the first row of this step, `next` of the one
// behind it, `g` the rows' group, which ends (for this run) at `stop`.
struct Walk {
  int base, next, stop, end, g, step;
  __device__ __forceinline__ Walk(const NormArgs& p, const Place& pl)
      : base(pl.row), next(pl.row), stop(pl.row), end(pl.end), g(pl.row < pl.end ? group_of(p, pl.row) : 0), step(pl.step) {}
  __device__ __forceinline__ bool more() const { return base < end; }
  // True when this step opens a group.
  __device__ __forceinline__ bool open(const NormArgs& p) {
    const bool fresh = base >= stop;
    if (fresh) {
      int e;
      while ((e = group_end(p, g)) <= base && g + 1 < p.G) ++g;
      stop = min(e, end);
    }
    next = min(base + step, stop);
    return fresh;
  }
  __device__ __forceinline__ void advance() { base = next; }
};

// The coefficients of this thread's columns in group g: (1 + scale) weight,
// bias (1 + scale) + shift (forward), gate post_weight.  Narrow rows keep them in
// registers; wide rows keep two of them in shared memory, each thread its own
// columns: in registers they would cost a block per SM, or spill to local
// memory (75,600 x 5,120: 632 us and 879 us, against 538 us).
template <int V, bool SHARED>
struct Coefficients;
template <int V>
struct Coefficients<V, false> {
  Vec a[V], b[V], g[V];
  __device__ __forceinline__ Coefficients(const NormArgs&, const Columns<V>&, uint8_t*) {}
  __device__ __forceinline__ void put(int which, int v, const Vec& t) { (which == 0 ? b : g)[v] = t; }
  __device__ __forceinline__ Vec get_a(int v) const { return a[v]; }
  __device__ __forceinline__ Vec get_b(int v) const { return b[v]; }
  __device__ __forceinline__ Vec get_g(int v) const { return g[v]; }
};
template <int V>
struct Coefficients<V, true> {
  Vec a[V];
  float* at[V];
  int D;
  __device__ __forceinline__ Coefficients(const NormArgs& p, const Columns<V>& c, uint8_t* mem) : D(p.D) {
#pragma unroll
    for (int v = 0; v < V; ++v) at[v] = reinterpret_cast<float*>(mem) + (c.on[v] ? c.col[v] : 0);
  }
  __device__ __forceinline__ void put(int which, int v, const Vec& t) { store_vec(at[v] + which * D, t); }
  __device__ __forceinline__ Vec get_a(int v) const { return get_b(v); }  // backward: in b's place
  __device__ __forceinline__ Vec get_b(int v) const { Vec t; load_vec(t, at[v]); return t; }
  __device__ __forceinline__ Vec get_g(int v) const { Vec t; load_vec(t, at[v] + D); return t; }
};

template <int V, bool SHARED>
__device__ __forceinline__ void load_coefficients(const NormArgs& p, int g, const Columns<V>& c, Coefficients<V, SHARED>& k,
                                                  bool want_b) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!c.on[v]) continue;
    const size_t at = (size_t)g * p.D + c.col[v];
    Vec a, o, t;
    fill(a, 1.f);
    if (p.scale) {
      load_vec(t, p.scale + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) a.v[i] = add2(a.v[i], t.v[i]);
    }
    if (want_b) {
      fill(o, 0.f);
      if (p.bias) {
        load_vec(t, p.bias + c.col[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = mul2(t.v[i], a.v[i]);
      }
      if (p.shift) {
        load_vec(t, p.shift + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = add2(o.v[i], t.v[i]);
      }
      k.put(0, v, o);
    }
    if (p.weight) {
      load_vec(t, p.weight + c.col[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) a.v[i] = mul2(a.v[i], t.v[i]);
    }
    k.a[v] = a;
    if (SHARED && !want_b) k.put(0, v, a);
    fill(o, 1.f);
    if (p.gate) load_vec(o, p.gate + at);
    if (p.post_weight) {
      load_vec(t, p.post_weight + c.col[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) o.v[i] = mul2(o.v[i], t.v[i]);
    }
    k.put(1, v, o);
  }
}

// Block classes: vectors per thread, most threads of a block, and the threads
// an SM is to hold (the launch bounds set the registers, the grid and the ring
// count on them).  0: rows of up to 256 columns; 1, 2, 3: up to 2,048, 5,120
// and 8,192 columns, two vectors per thread.
template <int CLS, bool BACK>
struct Class {
  static constexpr int kV = CLS == 0 ? 1 : 2;
  static constexpr int kMax = CLS == 0 ? 128 : CLS == 1 ? 128 : CLS == 2 ? 320 : 512;
  static constexpr int kThreads = CLS == 0 ? (BACK ? 512 : 768) : CLS == 1 ? 512 : CLS == 2 ? (BACK ? 320 : 640) : 512;
};

// Shared memory of the wide rows: the ring's stages, then two coefficients per column.
__device__ __forceinline__ uint8_t* coefficient_memory(const NormArgs& p) {
  extern __shared__ __align__(128) uint8_t dyn[];
  return dyn + p.ring_bytes;
}

template <int CLS>
using Sum = RowSum<CLS == 0 ? -1 : CLS == 1 ? 2 : 4>;  // up to 4, 10 and 16 warps

template <typename TX, typename TY, int CLS>
__global__ void __launch_bounds__(Class<CLS, false>::kMax, (Class<CLS, false>::kThreads / Class<CLS, false>::kMax))
    k_block_norm(const __grid_constant__ NormArgs p) {
  constexpr int V = Class<CLS, false>::kV;
  __shared__ float2 scratch[64];
  Sum<CLS> sum(scratch, p.tpr);
  const Place pl = place<CLS == 0>(p);
  Columns<V> c;
  c.init(p.D, p.tpr, pl.lane, sum);
  typename std::conditional<CLS == 0, Direct<TX, TY, 2, V>, Ring<TX, TY, 2, V>>::type rows(p, c, pl.row + pl.sub, pl.end);
  if (p.clear && pl.end < pl.row + p.chunk) {
    clear_rest<CLS == 0, TX>(p, pl, p.r);
    clear_rest<CLS == 0, TY>(p, pl, p.h);
  }
  Walk at(p, pl);
  // a sum over the block is the barrier behind which a stage is free
  const bool barrier = (p.y && p.post != SVGEAR_NORM_NONE) || (p.h && p.pre != SVGEAR_NORM_NONE);
  Coefficients<V, CLS != 0> k(p, c, coefficient_memory(p));
  for (; at.more(); at.advance()) {
    if (at.open(p)) load_coefficients(p, at.g, c, k, true);
    const int row = at.base + pl.sub;
    const bool live = CLS != 0 || row < at.stop;
    rows.take(at.next + pl.sub);
    const long long out = (long long)row * p.D;
    Vec f[V], m[V];
    rows.template read<kX>(f);
    if (p.y) {
      rows.template read<kY>(m);
      normalise<V>(m, c, p.post, p.eps, sum);
      const f2 a = pair(p.a);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Vec cg = k.get_g(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[v].v[i] = fma2(a, f[v].v[i], mul2(cg.v[i], m[v].v[i]));
        if (live && c.on[v]) store_vec(static_cast<TX*>(p.r) + out + c.col[v], f[v]);
      }
    }
    if (p.h) {
      const float2 st = p.pre == SVGEAR_NORM_NONE ? make_float2(0.f, 1.f) : statistics<V>(f, c, p.pre, p.eps, sum);
      const f2 mean = pair(-st.x), inv = pair(st.y);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Vec cb = k.get_b(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[v].v[i] = fma2(mul2(add2(f[v].v[i], mean), inv), k.a[v].v[i], cb.v[i]);
        if (live && c.on[v]) store_vec(static_cast<TY*>(p.h) + out + c.col[v], f[v]);
      }
    }
    if (CLS != 0 && !barrier) __syncthreads();
    rows.release(row);
  }
}

// What the gradient of a norm's input needs of its row r and of u, the gradient
// of the normalised row n: R = inv (u - mu - n mun), mu = mean(u) (layer norm
// only), mun = mean(u n).  One barrier for all of it: with the squares go
// sum u and sum u (r - mean_w) of every warp, joined by
//   sum u (r - mean) = sum_w c_w + (mean_w - mean) sum_w u.
struct BackStats {
  float mean, inv, mu, mun;
};
template <int V, typename SUM>
__device__ __forceinline__ BackStats back_statistics(const Vec (&r)[V], const Vec (&u)[V], const Columns<V>& c, int kind,
                                                     float eps, SUM& sum) {
  if (kind == SVGEAR_NORM_NONE) return {0.f, 1.f, 0.f, 0.f};
  auto dot = [&](float mean) {
    float s = 0.f;
    const f2 m = pair(-mean);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f2 q = pair(0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(u[v].v[i], add2(r[v].v[i], m), q);
      const float2 h = halves(q);
      s += c.on[v] ? h.x + h.y : 0.f;
    }
    return s;
  };
  if (kind == SVGEAR_NORM_RMS) {
    const float2 q = sum(make_float2(squares(r, c, 0.f), dot(0.f)));
    const float inv = rsqrtf(fmaf(q.x, c.inv_d, eps));
    return {0.f, inv, 0.f, q.y * c.inv_d * inv};
  }
  const float s = sum.lanes(total(r, c));
  const float pivot = SUM::kBlock ? s * c.inv_own : over(s, c.d, c.inv_d);
  float q = sum.lanes(squares(r, c, pivot));
  float2 w = sum.lanes(make_float2(total(u, c), dot(pivot)));
  float mean = pivot;
  if (SUM::kBlock) {
    float2 v = make_float2(s, q);
    sum.trade(v, w);
    mean = over(sum.warps(v.x), c.d, c.inv_d);
    const float e = v.x * c.inv_n - mean;
    q = sum.warps(fmaf(c.n * e, e, v.y));
    w = make_float2(sum.warps(w.x), sum.warps(fmaf(e, w.x, w.y)));
  }
  const float inv = rsqrtf(fmaf(q, c.inv_d, eps));
  return {mean, inv, w.x * c.inv_d, w.y * c.inv_d * inv};
}

// du -> the gradient of the norm's input: inv (du - n mean(du n) - mean(du)),
// the last term for a layer norm only.  n is the normalised row.
template <int V, typename SUM>
__device__ __forceinline__ void norm_back(Vec (&du)[V], const Vec (&n)[V], const Columns<V>& c, float inv, int kind, SUM& sum) {
  if (kind == SVGEAR_NORM_NONE) return;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f2 q = pair(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) q = fma2(du[v].v[i], n[v].v[i], q);
    const float2 h = halves(q);
    s.x += c.on[v] ? h.x + h.y : 0.f;
  }
  if (kind == SVGEAR_NORM_LAYER) {
    s.y = total(du, c);
    s = sum(s);
  } else {
    s.x = sum(s.x);
  }
  const f2 c1 = pair(-s.x * c.inv_d), c0 = pair(-s.y * c.inv_d), k = pair(inv);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) du[v].v[i] = mul2(k, add2(fma2(n[v].v[i], c1, c0), du[v].v[i]));
}

template <typename TX, typename TY, int CLS>
__global__ void __launch_bounds__(Class<CLS, true>::kMax, (Class<CLS, true>::kThreads / Class<CLS, true>::kMax))
    k_block_norm_back(const __grid_constant__ NormArgs p) {
  constexpr int V = Class<CLS, true>::kV;
  __shared__ float2 scratch[128];
  Sum<CLS> sum(scratch, p.tpr);
  const Place pl = place<CLS == 0>(p);
  Columns<V> c;
  c.init(p.D, p.tpr, pl.lane, sum);
  typename std::conditional<CLS == 0, Direct<TX, TY, 4, V>, Ring<TX, TY, 4, V>>::type rows(p, c, pl.row + pl.sub, pl.end);
  if (p.clear && pl.end < pl.row + p.chunk) {
    clear_rest<CLS == 0, TX>(p, pl, p.dx, p.y ? nullptr : p.dr);  // without y, r is x there too
    clear_rest<CLS == 0, TY>(p, pl, p.dy);
  }
  Walk at(p, pl);
  // Rows are read to the end of their iteration.  With four stages or more the
  // barrier in the next row's sum frees them; otherwise one at the end does.
  const bool late = p.dh && p.pre != SVGEAR_NORM_NONE && p.stages > 3;
  const f2 a = pair(p.y ? p.a : 1.f);
  Coefficients<V, CLS != 0> k(p, c, coefficient_memory(p));
  Vec s1[V], s2[V], su[V];
  auto flush = [&](int g) {
    float* part = p.part + (size_t)(pl.worker + g) * 3 * p.D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (CLS == 0) {  // the sums of the rows taken side by side
        const auto across = [&](Vec& s) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 h = halves(s.v[i]);
            for (int o = p.tpr; o < 32; o <<= 1) {
              h.x += __shfl_xor_sync(0xffffffffu, h.x, o);
              h.y += __shfl_xor_sync(0xffffffffu, h.y, o);
            }
            s.v[i] = pair(h.x, h.y);
          }
        };
        across(s1[v]);
        across(s2[v]);
        across(su[v]);
      }
      if (c.on[v] && pl.sub == 0) {
        store_vec(part + c.col[v], s1[v]);
        store_vec(part + p.D + c.col[v], s2[v]);
        store_vec(part + 2 * p.D + c.col[v], su[v]);
      }
    }
  };
  int open = -1;  // the group whose sums are being taken
  for (; at.more(); at.advance()) {
    if (at.open(p)) {
      if (open >= 0) flush(open);
      open = at.g;
      load_coefficients(p, at.g, c, k, false);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        fill(s1[v], 0.f);
        fill(s2[v], 0.f);
        fill(su[v], 0.f);
      }
    }
    const int row = at.base + pl.sub;
    const bool live = CLS != 0 || row < at.stop;
    rows.take(at.next + pl.sub);
    const long long out = (long long)row * p.D;
    Vec n[V], R[V];
    float2 st_m = make_float2(0.f, 1.f);  // mean and 1/deviation of y
    rows.template read<kX>(n);
    if (p.y) {
      rows.template read<kY>(R);
      if (p.post != SVGEAR_NORM_NONE) {
        st_m = statistics<V>(R, c, p.post, p.eps, sum);
        apply<V>(R, st_m);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Vec cg = k.get_g(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) n[v].v[i] = fma2(a, n[v].v[i], mul2(cg.v[i], R[v].v[i]));
      }
    }
    if (p.dh) {
      rows.template read<kDh>(R);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Vec ca = k.get_a(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (CLS != 0 || live) s1[v].v[i] = add2(s1[v].v[i], R[v].v[i]);
          R[v].v[i] = mul2(R[v].v[i], ca.v[i]);
        }
      }
      const BackStats st = back_statistics<V>(n, R, c, p.pre, p.eps, sum);
      if (late) rows.release_previous(row);
      const f2 mean = pair(-st.mean), inv = pair(st.inv), mu = pair(-st.mu), mun = pair(-st.mun);
      Vec dh[V];
      rows.template read<kDh>(dh);  // again: kept in registers it would cost the fourth block per SM
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 x = mul2(add2(n[v].v[i], mean), inv);
          if (CLS != 0 || live) s2[v].v[i] = fma2(dh[v].v[i], x, s2[v].v[i]);
          R[v].v[i] = mul2(inv, add2(fma2(x, mun, mu), R[v].v[i]));
        }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) fill(R[v], 0.f);
    }
    if (p.dr) {
      rows.template read<kDr>(n);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) R[v].v[i] = add2(R[v].v[i], n[v].v[i]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) n[v].v[i] = mul2(a, R[v].v[i]);
      if (live && c.on[v]) store_vec(static_cast<TX*>(p.dx) + out + c.col[v], n[v]);
    }
    if (p.y) {
      rows.template read<kY>(n);  // again, like dh
      if (p.post != SVGEAR_NORM_NONE) apply<V>(n, st_m);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Vec cg = k.get_g(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (CLS != 0 || live) su[v].v[i] = fma2(R[v].v[i], n[v].v[i], su[v].v[i]);
          R[v].v[i] = mul2(R[v].v[i], cg.v[i]);
        }
      }
      norm_back<V>(R, n, c, st_m.y, p.post, sum);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (live && c.on[v]) store_vec(static_cast<TY*>(p.dy) + out + c.col[v], R[v]);
    }
    if (CLS != 0 && !late) {
      __syncthreads();  // the row has been read
      rows.release(row);
    }
  }
  if (open >= 0) flush(open);
}

struct SumArgs {
  const float* part;
  const float *gate, *scale, *weight, *bias, *post_weight;
  float *dgate, *dscale, *dshift, *dweight, *dbias, *dpost_weight;
  float* sums;  // [G][3][D] group sums, kept when a weight's gradient is wanted
};

constexpr int kSumLanes = 16;
constexpr int kSumCols = 128;

// Column sums of one group: 128 columns per block, the group's slots dealt to
// 16 warps, their results added in warp order.
__global__ void __launch_bounds__(32 * kSumLanes) k_group_sums(const __grid_constant__ NormArgs p, const __grid_constant__ SumArgs q) {
  __shared__ float4 red[3][kSumLanes][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * kSumCols + lane * 4;
  const size_t plane = (size_t)p.D;
  for (int g = blockIdx.y; g < p.G; g += gridDim.y) {
    const int beg = g ? group_end(p, g - 1) : 0, end = group_end(p, g);
    float4 s[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (end > beg && col < p.D) {
      const int c1 = (end - 1) / p.chunk + g;
#pragma unroll 2
      for (int c = beg / p.chunk + g + w; c <= c1; c += kSumLanes) {
        const float* part = q.part + (size_t)c * 3 * plane + col;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(part + k * plane);
          s[k].x += v.x; s[k].y += v.y; s[k].z += v.z; s[k].w += v.w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) red[k][w][lane] = s[k];
    __syncthreads();
    // one column per thread from here
    const int at = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.x < kSumCols && at < p.D) {
      float t[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < kSumLanes; ++i) t[k] += reinterpret_cast<const float*>(red[k][i])[threadIdx.x];
      const size_t o = (size_t)g * plane + at;
      const float wt = p.weight ? p.weight[at] : 1.f, b = p.bias ? p.bias[at] : 0.f;
      if (q.dshift) q.dshift[o] = t[0];
      if (q.dscale) q.dscale[o] = fmaf(wt, t[1], b * t[0]);
      if (q.dgate) q.dgate[o] = p.post_weight ? p.post_weight[at] * t[2] : t[2];
      if (q.sums)
#pragma unroll
        for (int k = 0; k < 3; ++k) q.sums[((size_t)g * 3 + k) * plane + at] = t[k];
    }
    __syncthreads();
  }
}

// Gradients of the affine weights: the groups' sums weighted by 1 + s or g.
__global__ void __launch_bounds__(32 * kSumLanes) k_weight_sums(const __grid_constant__ NormArgs p, const __grid_constant__ SumArgs q) {
  __shared__ float red[3][kSumLanes][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s[3] = {0.f, 0.f, 0.f};
  if (col < p.D)
    for (int g = w; g < p.G; g += kSumLanes) {
      const float* v = q.sums + (size_t)g * 3 * p.D + col;
      const size_t at = (size_t)g * p.D + col;
      const float sc = p.scale ? 1.f + p.scale[at] : 1.f, gt = p.gate ? p.gate[at] : 1.f;
      s[0] = fmaf(sc, v[0], s[0]);
      s[1] = fmaf(sc, v[p.D], s[1]);
      s[2] = fmaf(gt, v[2 * (size_t)p.D], s[2]);
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) red[k][w][lane] = s[k];
  __syncthreads();
  if (w == 0 && col < p.D) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      s[k] = 0.f;
#pragma unroll
      for (int i = 0; i < kSumLanes; ++i) s[k] += red[k][i][lane];
    }
    if (q.dbias) q.dbias[col] = s[0];
    if (q.dweight) q.dweight[col] = s[1];
    if (q.dpost_weight) q.dpost_weight[col] = s[2];
  }
}

// Launch shape: block class, threads per row, rows per worker, ring stages.
struct Shape {
  int cls, tpr, block, chunk, grid, stages, ring_bytes, smem;
  long long workers;
};

// Per block 1 KB is the system's, 1.25 KB are static arrays.
constexpr int kSmemPerSm = 228 * 1024, kSmemPerBlock = 2304;
// What the rings of an SM's blocks hold together.  Beyond about 80 KB more reads
// in flight only delay the writes (share of the copy rate: bf16 65,536 x 2,048
// with 64 / 96 / 195 KB 0.94 / 0.84 / 0.80; float32 40,000 x 2,048 with 64 / 96
// KB 0.93 / 0.85; 80,000 x 1,024 with 64 / 80 KB 0.97 / 0.86).  So the blocks per
// SM are those whose two stages stay within kBlocksRing, or as many as give
// kThreadBytes / (bytes of an x and a y element) threads where those are
// more (bf16 75,600 x 5,120 with one / two blocks 0.76 / 0.91), and deeper rings
// stay within kRingPerSm.  The backward pass computes more for each byte.
constexpr int kBlocksRing = 76 * 1024, kBlocksRingBack = 132 * 1024, kThreadBytes = 2048;
constexpr int kRingPerSm = 88 * 1024;

Shape norm_shape(const svgear_norm_params* p, bool back) {
  Shape s;
  const int nvec = p->D / kVec, N = p->N;
  int threads;  // resident per SM
  if (nvec <= 32) {
    s.cls = 0;
    s.tpr = nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
    s.block = 128;
    threads = back ? Class<0, true>::kThreads : Class<0, false>::kThreads;
  } else {
    s.tpr = s.block = std::max(64, (nvec + 63) / 64 * 32);
    s.cls = s.block <= 128 ? 1 : s.block <= 320 ? 2 : 3;
    threads = s.cls == 1   ? (back ? Class<1, true>::kThreads : Class<1, false>::kThreads)
              : s.cls == 2 ? (back ? Class<2, true>::kThreads : Class<2, false>::kThreads)
                           : Class<3, true>::kThreads;
  }
  const int per = s.cls == 0 ? s.block / 32 : 1, step = s.cls == 0 ? 32 / s.tpr : 1;  // workers of a block, rows of a step
  const int stage = p->D * ((p->res_dtype == DT_F32 ? 4 : 2) + (p->dtype == DT_F32 ? 4 : 2)) * (back ? 2 : 1);
  const int coefs = 2 * p->D * (int)sizeof(float);
  // Blocks per SM: what the registers allow, as long as each has two stages, and
  // no more than kBlocksRing says unless the threads were too few to keep up.
  int blocks = std::max(1, std::min(threads / s.block, 8));
  auto stages = [&]() { return (kSmemPerSm / blocks - kSmemPerBlock - coefs) / stage; };
  if (s.cls != 0) {
    const int pair_bytes = (p->res_dtype == DT_F32 ? 4 : 2) + (p->dtype == DT_F32 ? 4 : 2);
    const int enough = (kThreadBytes / pair_bytes + s.block - 1) / s.block;
    blocks = std::min(blocks, std::max(enough, (back ? kBlocksRingBack : kBlocksRing) / (2 * stage)));
    while (blocks > 1 && stages() < 2) --blocks;
  }
  // As many workers as the SMs hold at once, each with whole steps; more would
  // only add partial sums.
  const long long want = std::min<long long>((N + step - 1) / step, 148LL * blocks * per);
  s.chunk = (int)(((N + want - 1) / want + step - 1) / step * step);
  s.workers = (N + s.chunk - 1) / s.chunk;
  s.grid = (int)((s.workers + per - 1) / per);
  const int deep = std::max(blocks == 1 ? 3 : 2, kRingPerSm / blocks / stage);
  s.stages = s.cls == 0 ? 0 : std::max(1, std::min({stages(), kMaxStages, s.chunk, deep}));
  s.ring_bytes = s.stages * stage;
  s.smem = s.cls == 0 ? 0 : s.ring_bytes + coefs;
  return s;
}

NormArgs norm_args(const BlockNorm& b, const Shape& s) {
  NormArgs p{};
  p.x = b.x; p.y = b.y; p.dr = b.dr; p.dh = b.dh;
  p.gate = b.gate; p.scale = b.scale; p.shift = b.shift; p.weight = b.weight; p.bias = b.bias;
  p.post_weight = b.post_weight;
  p.offsets = b.offsets;
  p.N = b.p->N; p.D = b.p->D; p.G = b.p->G; p.pre = b.p->pre & ~SVGEAR_NORM_CLEAR_REST; p.post = b.p->post;
  p.clear = b.offsets && (b.p->pre & SVGEAR_NORM_CLEAR_REST);
  p.tpr = s.tpr; p.chunk = s.chunk; p.stages = s.stages; p.ring_bytes = s.ring_bytes;
  p.eps = b.p->eps; p.a = b.p->res_scale;
  p.r = b.r; p.h = b.h; p.dx = b.dx; p.dy = b.dy;
  p.status = status_word();
  return p;
}

template <typename TX, typename TY, int CLS>
cudaError_t launch_class(const NormArgs& p, const Shape& s, bool back, cudaStream_t st) {
  const auto kernel = back ? k_block_norm_back<TX, TY, CLS> : k_block_norm<TX, TY, CLS>;
  if (s.smem > 32 * 1024) {
    const cudaError_t e = allow_dynamic_smem(kernel, kSmemPerSm - kSmemPerBlock);
    if (e != cudaSuccess) return e;
  }
  kernel<<<s.grid, s.block, s.smem, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t launch_norm(const NormArgs& p, const Shape& s, bool back, cudaStream_t st) {
  if (s.cls == 0) return launch_class<TX, TY, 0>(p, s, back, st);
  if (s.cls == 1) return launch_class<TX, TY, 1>(p, s, back, st);
  if (s.cls == 2) return launch_class<TX, TY, 2>(p, s, back, st);
  return launch_class<TX, TY, 3>(p, s, back, st);
}

cudaError_t launch_typed(const BlockNorm& b, const NormArgs& p, const Shape& s, bool back, cudaStream_t st) {
  if (!p.status) return cudaErrorInvalidValue;
  if (b.p->dtype == DT_F32) return launch_norm<float, float>(p, s, back, st);
  if (b.p->res_dtype == DT_F32) return launch_norm<float, bf16>(p, s, back, st);
  return launch_norm<bf16, bf16>(p, s, back, st);
}

}  // namespace

size_t block_norm_back_ws_bytes(const svgear_norm_params* p) {
  const Shape s = norm_shape(p, true);
  Carve cv(nullptr);
  cv.take<float>((size_t)(s.workers + p->G) * 3 * p->D);
  cv.take<float>((size_t)p->G * 3 * p->D);
  return cv.used();
}

cudaError_t block_norm_run(const BlockNorm& b, cudaStream_t st) {
  const Shape s = norm_shape(b.p, false);
  return launch_typed(b, norm_args(b, s), s, false, st);
}

cudaError_t block_norm_back_run(const BlockNorm& b, void* ws, cudaStream_t st) {
  const Shape s = norm_shape(b.p, true);
  NormArgs p = norm_args(b, s);
  Carve cv(ws);
  p.part = cv.take<float>((size_t)(s.workers + p.G) * 3 * p.D);
  SumArgs q{};
  q.part = p.part;
  q.dgate = b.dgate; q.dscale = b.dscale; q.dshift = b.dshift;
  q.dweight = b.dweight; q.dbias = b.dbias; q.dpost_weight = b.dpost_weight;
  if (q.dweight || q.dbias || q.dpost_weight) q.sums = cv.take<float>((size_t)p.G * 3 * p.D);
  cudaError_t e = launch_typed(b, p, s, true, st);
  if (e == cudaSuccess && (q.dgate || q.dscale || q.dshift || q.sums)) {
    k_group_sums<<<dim3((p.D + kSumCols - 1) / kSumCols, std::min(p.G, 32768)), 32 * kSumLanes, 0, st>>>(p, q);
    note_launch();
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && q.sums) {
    k_weight_sums<<<(p.D + 31) / 32, 32 * kSumLanes, 0, st>>>(p, q);
    note_launch();
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace svg
