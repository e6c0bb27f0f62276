// Gated residual and norms around an attention block (row-wise, HBM-bound).
//
//   m = P(y)              P, Q: none, RMS norm or layer norm of a row
//   r = a x + g m w2      (r = x without y)
//   n = Q(r),  h = (n w + b)(1 + s) + t
//
// One pass: a row is loaded once into registers, its statistics are taken
// there (mean first, then the squared deviations, so nothing cancels), and r
// and h leave from the same registers.  h is formed from the unrounded r.
// The per-column coefficients (1+s) w, b (1+s) + t and g w2 stay in registers
// while consecutive rows belong to one group.
//
// A row is owned by a worker: 8, 16 or 32 lanes of a warp for D <= 256,
// otherwise a whole block (one 8-element vector per thread, two above 5,120
// columns).  A worker walks a contiguous run of rows, so column sums of the
// backward pass stay in registers until the group or the run ends; partial
// sums then go to slot (worker + group), which no other pair maps to because
// both only grow along the rows, and are added in slot order: no atomics, the
// same bits every time.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "rowvec.cuh"

namespace svg {

namespace {

struct NormArgs {
  const void *x, *y, *dr, *dh;
  const float *gate, *scale, *shift, *weight, *bias, *post_weight;
  const int32_t* offsets;
  int N, D, G, pre, post, tpr, chunk;
  float eps, a;
  void *r, *h, *dx, *dy;
  float* part;  // backward: [slots][3][D] partial column sums
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

// Row statistics of f (inactive vectors hold zeros): f becomes the normalised
// row, the return value is 1 / deviation.  The deviations from the rounded
// mean sum to D times what the mean is off, which the second sum carries along
// with the squares: mean and variance are both corrected by it.  A constant
// row of a large value would otherwise show its mean's last bit, magnified by
// 1/sqrt(eps).
template <int V>
__device__ __forceinline__ float normalise(float (&f)[V][kVec], const bool (&on)[V], int kind, float d, float eps,
                                           RowSum& sum) {
  if (kind == SVGEAR_NORM_NONE) return 1.f;
  float2 q = make_float2(0.f, 0.f);
  if (kind == SVGEAR_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < kVec; ++i) s += f[v][i];
    const float mean = sum(s) / d;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        f[v][i] = on[v] ? f[v][i] - mean : 0.f;
        q.y += f[v][i];
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < kVec; ++i) q.x = fmaf(f[v][i], f[v][i], q.x);
  q = sum(q);
  const float off = q.y / d;  // 0 for an RMS norm
  const float inv = rsqrtf(fmaxf(fmaf(-off, off, q.x / d), 0.f) + eps);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[v][i] = on[v] ? (f[v][i] - off) * inv : 0.f;
  return inv;
}

template <typename TX, typename TY, int V>
__global__ void __launch_bounds__(V == 1 ? 640 : 512) k_block_norm(const NormArgs p) {
  __shared__ float2 scratch[64];
  RowSum sum{scratch, p.tpr, 0};
  const int slot = threadIdx.x / p.tpr, lane = threadIdx.x - slot * p.tpr;
  const long long worker = (long long)blockIdx.x * (blockDim.x / p.tpr) + slot;
  const float d = (float)p.D;
  long long row = worker * p.chunk;
  const long long end = row + p.chunk < p.N ? row + p.chunk : p.N;
  const TX* x = static_cast<const TX*>(p.x);
  const TY* y = static_cast<const TY*>(p.y);
  int col[V];
  bool on[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = (v * p.tpr + lane) * kVec;
    on[v] = col[v] < p.D;
  }
  int g = row < end ? group_of(p, (int)row) : p.G;
  long long gend = row;  // forces the first coefficient load
  bool first = true;
  float ca[V][kVec], cb[V][kVec], cg[V][kVec];
  Raw<TX> xr[V];
  Raw<TY> yr[V];
  auto fetch = [&](long long rw) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool ok = on[v] && rw < end;
      zero_raw(xr[v]);
      if (ok) load_raw(xr[v], x + rw * p.D + col[v]);
      if (y) {
        zero_raw(yr[v]);
        if (ok) load_raw(yr[v], y + rw * p.D + col[v]);
      }
    }
  };
  fetch(row);
  for (int it = 0; it < p.chunk; ++it, ++row) {
    // rows of this worker are done, or lie behind the last group; whole blocks leave together
    if (g < p.G && row < end && (first || row >= gend)) {
      while (g < p.G && (gend = group_end(p, g)) <= row) ++g;
      first = false;
      if (g < p.G) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float w[kVec], t[kVec];
#pragma unroll
          for (int i = 0; i < kVec; ++i) { ca[v][i] = 1.f; cb[v][i] = 0.f; cg[v][i] = 1.f; }
          if (!on[v]) continue;
          const size_t at = (size_t)g * p.D + col[v];
          if (p.scale) {
            load_f8(t, p.scale + at);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ca[v][i] += t[i];
          }
          if (p.bias) {
            load_f8(w, p.bias + col[v]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) cb[v][i] = w[i] * ca[v][i];
          }
          if (p.shift) {
            load_f8(t, p.shift + at);
#pragma unroll
            for (int i = 0; i < kVec; ++i) cb[v][i] += t[i];
          }
          if (p.weight) {
            load_f8(w, p.weight + col[v]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ca[v][i] *= w[i];
          }
          if (p.gate) load_f8(cg[v], p.gate + at);
          if (p.post_weight) {
            load_f8(w, p.post_weight + col[v]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) cg[v][i] *= w[i];
          }
        }
      }
    }
    const bool live = g < p.G && row < end;
    if (p.tpr >= 32 && !live) break;  // uniform over the worker, which is whole warps
    float f[V][kVec], m[V][kVec];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack(xr[v], f[v]);
      if (y) unpack(yr[v], m[v]);
    }
    fetch(row + 1);
    if (y) {
      normalise<V>(m, on, p.post, d, p.eps, sum);
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[v][i] = on[v] ? fmaf(p.a, f[v][i], cg[v][i] * m[v][i]) : 0.f;
        if (live && on[v]) store_vec(static_cast<TX*>(p.r) + row * p.D + col[v], f[v]);
      }
    }
    if (p.h) {
      normalise<V>(f, on, p.pre, d, p.eps, sum);
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[v][i] = fmaf(f[v][i], ca[v][i], cb[v][i]);
        if (live && on[v]) store_vec(static_cast<TY*>(p.h) + row * p.D + col[v], f[v]);
      }
    }
  }
}

// du -> the gradient of the norm's input: inv (du - n mean(du n) - mean(du)),
// the last term for a layer norm only.  n is the normalised row.
template <int V>
__device__ __forceinline__ void norm_back(float (&du)[V][kVec], const float (&n)[V][kVec], const bool (&on)[V], float inv,
                                          int kind, float inv_d, RowSum& sum) {
  if (kind == SVGEAR_NORM_NONE) return;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      s.x = fmaf(du[v][i], n[v][i], s.x);
      s.y += du[v][i];
    }
  s = sum(s);
  const float c1 = s.x * inv_d, c0 = kind == SVGEAR_NORM_LAYER ? s.y * inv_d : 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < kVec; ++i) du[v][i] = on[v] ? inv * (du[v][i] - c0 - n[v][i] * c1) : 0.f;
}

template <typename TX, typename TY, int V>
__global__ void __launch_bounds__(V == 1 ? 640 : 512) k_block_norm_back(const NormArgs p) {
  __shared__ float2 scratch[64];
  RowSum sum{scratch, p.tpr, 0};
  const int slot = threadIdx.x / p.tpr, lane = threadIdx.x - slot * p.tpr;
  const long long worker = (long long)blockIdx.x * (blockDim.x / p.tpr) + slot;
  const float d = (float)p.D;
  long long row = worker * p.chunk;
  const long long end = row + p.chunk < p.N ? row + p.chunk : p.N;
  const TX *x = static_cast<const TX*>(p.x), *dr = static_cast<const TX*>(p.dr);
  const TY *y = static_cast<const TY*>(p.y), *dh = static_cast<const TY*>(p.dh);
  int col[V];
  bool on[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = (v * p.tpr + lane) * kVec;
    on[v] = col[v] < p.D;
  }
  int g = row < end ? group_of(p, (int)row) : p.G;
  long long gend = row;
  bool first = true;
  float ca[V][kVec], cg[V][kVec];
  float s1[V][kVec], s2[V][kVec], su[V][kVec];
  Raw<TX> xr[V], rr[V];
  Raw<TY> yr[V], hr[V];
  auto fetch = [&](long long rw) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool ok = on[v] && rw < end;
      const long long at = rw * p.D + col[v];
      zero_raw(xr[v]); zero_raw(yr[v]); zero_raw(rr[v]); zero_raw(hr[v]);
      if (ok) load_raw(xr[v], x + at);
      if (ok && y) load_raw(yr[v], y + at);
      if (ok && dr) load_raw(rr[v], dr + at);
      if (ok && dh) load_raw(hr[v], dh + at);
    }
  };
  auto flush = [&]() {
    float* part = p.part + (size_t)(worker + g) * 3 * p.D;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (on[v]) {
        store_vec(part + col[v], s1[v]);
        store_vec(part + p.D + col[v], s2[v]);
        store_vec(part + 2 * (size_t)p.D + col[v], su[v]);
      }
  };
  fetch(row);
  for (int it = 0; it < p.chunk; ++it, ++row) {
    if (g < p.G && row < end && (first || row >= gend)) {
      if (!first) flush();
      while (g < p.G && (gend = group_end(p, g)) <= row) ++g;
      first = false;
      if (g < p.G) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float w[kVec];
#pragma unroll
          for (int i = 0; i < kVec; ++i) { ca[v][i] = cg[v][i] = 1.f; s1[v][i] = s2[v][i] = su[v][i] = 0.f; }
          if (!on[v]) continue;
          const size_t at = (size_t)g * p.D + col[v];
          if (p.scale) {
            load_f8(w, p.scale + at);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ca[v][i] += w[i];
          }
          if (p.weight) {
            load_f8(w, p.weight + col[v]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ca[v][i] *= w[i];
          }
          if (p.gate) load_f8(cg[v], p.gate + at);
          if (p.post_weight) {
            load_f8(w, p.post_weight + col[v]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) cg[v][i] *= w[i];
          }
        }
      }
    }
    const bool live = g < p.G && row < end;
    if (p.tpr >= 32 && !live) break;
    float n[V][kVec], m[V][kVec], R[V][kVec];
    float inv_m = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack(xr[v], n[v]);
      unpack(yr[v], m[v]);
      unpack(hr[v], R[v]);
    }
    Raw<TX> rc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rc[v] = rr[v];
    fetch(row + 1);
    if (y) {
      inv_m = normalise<V>(m, on, p.post, d, p.eps, sum);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) n[v][i] = on[v] ? fmaf(p.a, n[v][i], cg[v][i] * m[v][i]) : 0.f;
    }
    if (dh) {
      const float inv_n = normalise<V>(n, on, p.pre, d, p.eps, sum);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if (live) {
            s1[v][i] += R[v][i];
            s2[v][i] = fmaf(R[v][i], n[v][i], s2[v][i]);
          }
          R[v][i] = on[v] ? R[v][i] * ca[v][i] : 0.f;
        }
      norm_back<V>(R, n, on, inv_n, p.pre, 1.f / d, sum);
    }
    if (dr) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        unpack(rc[v], n[v]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) R[v][i] += n[v][i];
      }
    }
    const float a = y ? p.a : 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) n[v][i] = a * R[v][i];
      if (live && on[v]) store_vec(static_cast<TX*>(p.dx) + row * p.D + col[v], n[v]);
    }
    if (y) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if (live) su[v][i] = fmaf(R[v][i], m[v][i], su[v][i]);
          R[v][i] = on[v] ? R[v][i] * cg[v][i] : 0.f;
        }
      norm_back<V>(R, m, on, inv_m, p.post, 1.f / d, sum);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (live && on[v]) store_vec(static_cast<TY*>(p.dy) + row * p.D + col[v], R[v]);
    }
  }
  // The last group this worker had rows of; when it left through the end of
  // the last group, that group was flushed on the way.
  if (!first && g < p.G) flush();
}

struct SumArgs {
  const float* part;
  const float *gate, *scale, *weight, *bias, *post_weight;
  float *dgate, *dscale, *dshift, *dweight, *dbias, *dpost_weight;
  float* sums;  // [G][3][D] group sums, kept when a weight's gradient is wanted
};

constexpr int kSumLanes = 16;

// Column sums of one group: 32 columns per block, the group's slots dealt to
// 16 warps, their results added in warp order.
__global__ void __launch_bounds__(32 * kSumLanes) k_group_sums(const NormArgs p, const SumArgs q) {
  __shared__ float red[3][kSumLanes][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  for (int g = blockIdx.y; g < p.G; g += gridDim.y) {
    const int beg = g ? group_end(p, g - 1) : 0, end = group_end(p, g);
    float s[3] = {0.f, 0.f, 0.f};
    if (end > beg && col < p.D) {
      const long long c0 = beg / p.chunk + g, c1 = (end - 1) / p.chunk + g;
      for (long long c = c0 + w; c <= c1; c += kSumLanes) {
        const float* part = q.part + (size_t)c * 3 * p.D + col;
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += part[(size_t)k * p.D];
      }
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
      const size_t at = (size_t)g * p.D + col;
      const float wt = p.weight ? p.weight[col] : 1.f, b = p.bias ? p.bias[col] : 0.f;
      if (q.dshift) q.dshift[at] = s[0];
      if (q.dscale) q.dscale[at] = fmaf(wt, s[1], b * s[0]);
      if (q.dgate) q.dgate[at] = p.post_weight ? p.post_weight[col] * s[2] : s[2];
      if (q.sums)
#pragma unroll
        for (int k = 0; k < 3; ++k) q.sums[((size_t)g * 3 + k) * p.D + col] = s[k];
    }
    __syncthreads();
  }
}

// Gradients of the affine weights: the groups' sums weighted by 1 + s or g.
__global__ void __launch_bounds__(32 * kSumLanes) k_weight_sums(const NormArgs p, const SumArgs q) {
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

// Launch shape: threads per row, vectors per thread, rows per worker.
struct Shape {
  int V, tpr, block, chunk, grid;
  long long workers;
};

Shape norm_shape(int N, int D, bool back) {
  Shape s;
  const int nvec = D / kVec;
  s.V = nvec > 640 ? 2 : 1;
  if (nvec <= 32) {
    s.tpr = nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
    s.block = 128;
  } else {
    s.tpr = ((nvec + s.V - 1) / s.V + 31) / 32 * 32;
    s.block = s.tpr;
  }
  const int per = s.block / s.tpr;
  // Workers beyond what the SMs hold at once only add partial sums; the
  // backward pass of narrow rows is held to 2,048 of them for the same reason.
  const int ctas = back ? std::max(1, std::min(1024 / s.block, 8)) : std::max(1, std::min(2048 / s.block, 16));
  long long want = std::min<long long>(N, 148LL * ctas * per);
  if (back && nvec <= 32) want = std::min<long long>(want, 2048);
  s.chunk = (int)((N + want - 1) / want);
  s.workers = (N + s.chunk - 1) / s.chunk;
  s.grid = (int)((s.workers + per - 1) / per);
  return s;
}

NormArgs norm_args(const BlockNorm& b, const Shape& s) {
  NormArgs p{};
  p.x = b.x; p.y = b.y; p.dr = b.dr; p.dh = b.dh;
  p.gate = b.gate; p.scale = b.scale; p.shift = b.shift; p.weight = b.weight; p.bias = b.bias;
  p.post_weight = b.post_weight;
  p.offsets = b.offsets;
  p.N = b.p->N; p.D = b.p->D; p.G = b.p->G; p.pre = b.p->pre; p.post = b.p->post;
  p.tpr = s.tpr; p.chunk = s.chunk;
  p.eps = b.p->eps; p.a = b.p->res_scale;
  p.r = b.r; p.h = b.h; p.dx = b.dx; p.dy = b.dy;
  return p;
}

template <typename TX, typename TY>
void launch_norm(const NormArgs& p, const Shape& s, bool back, cudaStream_t st) {
  if (back) {
    if (s.V == 1) k_block_norm_back<TX, TY, 1><<<s.grid, s.block, 0, st>>>(p);
    else k_block_norm_back<TX, TY, 2><<<s.grid, s.block, 0, st>>>(p);
  } else {
    if (s.V == 1) k_block_norm<TX, TY, 1><<<s.grid, s.block, 0, st>>>(p);
    else k_block_norm<TX, TY, 2><<<s.grid, s.block, 0, st>>>(p);
  }
  note_launch();
}

void launch_typed(const BlockNorm& b, const NormArgs& p, const Shape& s, bool back, cudaStream_t st) {
  if (b.p->dtype == DT_F32) launch_norm<float, float>(p, s, back, st);
  else if (b.p->res_dtype == DT_F32) launch_norm<float, bf16>(p, s, back, st);
  else launch_norm<bf16, bf16>(p, s, back, st);
}

}  // namespace

size_t block_norm_back_ws_bytes(const svgear_norm_params* p) {
  const Shape s = norm_shape(p->N, p->D, true);
  Carve cv(nullptr);
  cv.take<float>((size_t)(s.workers + p->G) * 3 * p->D);
  cv.take<float>((size_t)p->G * 3 * p->D);
  return cv.used();
}

cudaError_t block_norm_run(const BlockNorm& b, cudaStream_t st) {
  const Shape s = norm_shape(b.p->N, b.p->D, false);
  launch_typed(b, norm_args(b, s), s, false, st);
  return cudaGetLastError();
}

cudaError_t block_norm_back_run(const BlockNorm& b, void* ws, cudaStream_t st) {
  const Shape s = norm_shape(b.p->N, b.p->D, true);
  NormArgs p = norm_args(b, s);
  Carve cv(ws);
  p.part = cv.take<float>((size_t)(s.workers + p.G) * 3 * p.D);
  SumArgs q{};
  q.part = p.part;
  q.dgate = b.dgate; q.dscale = b.dscale; q.dshift = b.dshift;
  q.dweight = b.dweight; q.dbias = b.dbias; q.dpost_weight = b.dpost_weight;
  if (q.dweight || q.dbias || q.dpost_weight) q.sums = cv.take<float>((size_t)p.G * 3 * p.D);
  launch_typed(b, p, s, true, st);
  cudaError_t e = cudaGetLastError();
  const int cols = (p.D + 31) / 32;
  if (e == cudaSuccess && (q.dgate || q.dscale || q.dshift || q.sums)) {
    k_group_sums<<<dim3(cols, std::min(p.G, 32768)), 32 * kSumLanes, 0, st>>>(p, q);
    note_launch();
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && q.sums) {
    k_weight_sums<<<cols, 32 * kSumLanes, 0, st>>>(p, q);
    note_launch();
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace svg
