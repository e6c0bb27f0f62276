// C ABI of the operators around the attention: validation and dispatch.  The
// declarations, with the argument contracts, are in include/svgear.h.
#include <cmath>

#include "../../include/svgear.h"
#include "common.cuh"
#include "internal.h"

namespace svg {
namespace {

template <typename... P>
inline bool aligned16(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 15u) == 0;
}
inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }
// A refused launch is reported here and does not stay behind as the thread's last error.
inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return SVGEAR_OK;
  cudaGetLastError();
  return SVGEAR_ERR_CUDA;
}
inline bool known_dtype(int t) { return t == SVGEAR_F32 || t == SVGEAR_BF16; }
inline int esize(int dtype) { return dtype == SVGEAR_BF16 ? 2 : 4; }

constexpr int kMaxNormCols = 8192;
constexpr int kMaxTokenCols = 16384;
constexpr int kMaxRows = 1 << 30;  // row counters are int, and run ahead by a few stages or a tile

int check_norm(const svgear_norm_params* p) {
  if (!p || p->N < 1 || p->D < 1 || p->G < 1) return SVGEAR_ERR_INVALID;
  const int pre = p->pre & ~SVGEAR_NORM_CLEAR_REST;
  if (pre < SVGEAR_NORM_NONE || pre > SVGEAR_NORM_LAYER) return SVGEAR_ERR_INVALID;
  if (p->post < SVGEAR_NORM_NONE || p->post > SVGEAR_NORM_LAYER) return SVGEAR_ERR_INVALID;
  if (!(p->eps > 0.f) || std::isinf(p->eps) || !std::isfinite(p->res_scale)) return SVGEAR_ERR_INVALID;
  if (!known_dtype(p->dtype) || !known_dtype(p->res_dtype)) return SVGEAR_ERR_UNSUPPORTED;
  if (p->res_dtype == SVGEAR_BF16 && p->dtype == SVGEAR_F32) return SVGEAR_ERR_UNSUPPORTED;
  if (p->D % 8 || p->D > kMaxNormCols || p->N > kMaxRows) return SVGEAR_ERR_UNSUPPORTED;
  return SVGEAR_OK;
}

// What forward and backward require of the inputs alike.
int check_norm_inputs(const BlockNorm& b) {
  const svgear_norm_params* p = b.p;
  if (!b.x || (!b.offsets && p->N % p->G)) return SVGEAR_ERR_INVALID;
  if (!b.y && (b.gate || b.post_weight || p->post != SVGEAR_NORM_NONE || p->res_scale != 1.f)) return SVGEAR_ERR_INVALID;
  if (!aligned16(b.x, b.y, b.gate, b.scale, b.shift, b.weight, b.bias, b.post_weight)) return SVGEAR_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(b.offsets) & 3u) return SVGEAR_ERR_INVALID;
  return SVGEAR_OK;
}

int check_rope(const svgear_rope_params* p) {
  if (!p || p->B < 1 || p->N < 1 || p->H < 1) return SVGEAR_ERR_INVALID;
  int turned = 0;
  for (int a = 0; a < 3; ++a) {
    if (p->axes[a] < 0 || p->axes[a] % 2 || p->axes[a] > p->d || p->grid[a] < 0) return SVGEAR_ERR_INVALID;
    if (!(p->theta[a] > 0.f) || std::isinf(p->theta[a]) || !std::isfinite(p->pos_scale[a])) return SVGEAR_ERR_INVALID;
    turned += p->axes[a];
  }
  if (p->pairing != SVGEAR_PAIR_ADJACENT && p->pairing != SVGEAR_PAIR_HALF) return SVGEAR_ERR_INVALID;
  if (p->norm < SVGEAR_QKNORM_NONE || p->norm > SVGEAR_QKNORM_TOKEN) return SVGEAR_ERR_INVALID;
  if (!(p->eps > 0.f) || std::isinf(p->eps)) return SVGEAR_ERR_INVALID;
  if (p->out_tokens < 0 || (p->out_tokens && p->out_tokens < p->N)) return SVGEAR_ERR_INVALID;
  if (!known_dtype(p->dtype)) return SVGEAR_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return SVGEAR_ERR_UNSUPPORTED;
  if (turned > p->d) return SVGEAR_ERR_INVALID;
  if ((long long)p->H * p->d > kMaxTokenCols) return SVGEAR_ERR_UNSUPPORTED;
  if ((long long)p->B * p->N > kMaxRows || (long long)p->B * p->H >= (1LL << 31)) return SVGEAR_ERR_UNSUPPORTED;
  return SVGEAR_OK;
}

// Rows start on 16-byte boundaries, and neighbours on either axis do not overlap.
bool row_strides_ok(const svgear_rope_params* p, int64_t ld, int64_t batch) {
  const int es = esize(p->dtype);
  const int64_t width = (int64_t)p->H * p->d;
  if (ld % (16 / es) || batch % (16 / es)) return false;
  if (p->N > 1 && ld < width) return false;
  return p->B == 1 || batch >= width;
}

// No two rows of an output overlap (row_strides_ok holds): either one axis lies
// within a step of the other, or no multiple of one stride comes nearer than a
// row to a multiple of the other, within the axes' lengths.
bool rows_apart(const svgear_rope_params* p, int64_t ld, int64_t batch) {
  typedef __int128 wide;  // the strides are the caller's, whatever they are
  const wide width = (wide)p->H * p->d;
  if (p->N == 1 || p->B == 1) return true;
  if (batch >= (p->N - 1) * (wide)ld + width || ld >= (p->B - 1) * (wide)batch + width) return true;
  const bool few = p->B <= p->N;
  const wide s1 = few ? batch : ld, s2 = few ? ld : batch;
  const int n1 = few ? p->B : p->N, n2 = few ? p->N : p->B;  // n1 <= 2^15
  for (int i = 1; i < n1; ++i) {
    const wide at = i * s1, j = at / s2;
    if ((j < n2 && at - j * s2 < width) || (j + 1 < n2 && (j + 1) * s2 - at < width)) return false;
  }
  return true;
}

int check_rope_inputs(const void* const in[3], const float* wq, const float* wk, const int32_t* pos,
                      const svgear_rope_params* p) {
  if (p->norm == SVGEAR_QKNORM_NONE && (wq || wk)) return SVGEAR_ERR_INVALID;
  if (!aligned16(in[0], in[1], in[2], wq, wk) || (reinterpret_cast<uintptr_t>(pos) & 3u)) return SVGEAR_ERR_INVALID;
  for (int k = 0; k < 3; ++k)
    if (in[k] && !row_strides_ok(p, p->ld[k], p->batch[k])) return SVGEAR_ERR_INVALID;
  if (!pos) {
    const long long plane = (long long)p->grid[1] * p->grid[2];
    if (plane > p->N || plane * p->grid[0] > p->N) return SVGEAR_ERR_INVALID;
  }
  return SVGEAR_OK;
}

int check_mx(int M, int K) {
  if (M < 1 || K < 1) return SVGEAR_ERR_INVALID;
  if (K % 32 || K > (1 << 20) || M > kMaxRows) return SVGEAR_ERR_UNSUPPORTED;
  if ((long long)M * K >= (1LL << 39)) return SVGEAR_ERR_UNSUPPORTED;  // one block of 2,048 elements per grid index
  return SVGEAR_OK;
}

int check_product(int M, int N, int K) {
  int rc = check_mx(M, K);
  if (!rc) rc = check_mx(N, K);
  if (rc) return rc;
  if (N % 8) return SVGEAR_ERR_UNSUPPORTED;
  // tile indices are int
  return ((long long)M / 16 + 1) * ((long long)N / 128 + 1) < (1LL << 31) ? SVGEAR_OK : SVGEAR_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace svg

using namespace svg;

extern "C" {

int svgear_block_norm(const void* x, const void* y, const float* gate, const float* scale, const float* shift,
                      const float* weight, const float* bias, const float* post_weight, const int32_t* offsets,
                      const svgear_norm_params* p, void* r, void* h, void* stream) {
  int rc = check_norm(p);
  if (rc) return rc;
  BlockNorm b{};
  b.p = p;
  b.x = x; b.y = y; b.gate = gate; b.scale = scale; b.shift = shift; b.weight = weight; b.bias = bias;
  b.post_weight = post_weight; b.offsets = offsets;
  b.r = r; b.h = h;
  rc = check_norm_inputs(b);
  if (rc) return rc;
  if (y ? !r : (r || !h)) return SVGEAR_ERR_INVALID;
  if (!aligned16(r, h)) return SVGEAR_ERR_INVALID;
  return cuda_status(block_norm_run(b, S(stream)));
}

size_t svgear_block_norm_backward_workspace_size(const svgear_norm_params* p) {
  if (check_norm(p)) return 0;
  return block_norm_back_ws_bytes(p);
}

int svgear_block_norm_backward(const void* x, const void* y, const void* dr, const void* dh, const float* gate,
                      const float* scale, const float* weight, const float* bias, const float* post_weight,
                      const int32_t* offsets, const svgear_norm_params* p, void* dx, void* dy, float* dgate,
                      float* dscale, float* dshift, float* dweight, float* dbias, float* dpost_weight, void* ws,
                      size_t ws_bytes, void* stream) {
  int rc = check_norm(p);
  if (rc) return rc;
  BlockNorm b{};
  b.p = p;
  b.x = x; b.y = y; b.dr = dr; b.dh = dh; b.gate = gate; b.scale = scale; b.weight = weight; b.bias = bias;
  b.post_weight = post_weight; b.offsets = offsets;
  b.dx = dx; b.dy = dy; b.dgate = dgate; b.dscale = dscale; b.dshift = dshift; b.dweight = dweight; b.dbias = dbias;
  b.dpost_weight = dpost_weight;
  rc = check_norm_inputs(b);
  if (rc) return rc;
  if ((!dr && !dh) || !dx || (y != nullptr) != (dy != nullptr)) return SVGEAR_ERR_INVALID;
  if (!y && (dgate || dpost_weight)) return SVGEAR_ERR_INVALID;
  if (!aligned16(dr, dh, dx, dy, dgate, dscale, dshift, dweight, dbias, dpost_weight)) return SVGEAR_ERR_INVALID;
  if (!ws || !aligned16(ws) || ws_bytes < block_norm_back_ws_bytes(p)) return SVGEAR_ERR_WORKSPACE;
  return cuda_status(block_norm_back_run(b, ws, S(stream)));
}

int svgear_qkv_rope(const void* q, const void* k, const void* v, const float* wq, const float* wk,
                    const int32_t* positions, const svgear_rope_params* p, void* Q, void* K, void* V, void* stream) {
  int rc = check_rope(p);
  if (rc) return rc;
  const void* in[3] = {q, k, v};
  void* out[3] = {Q, K, V};
  rc = check_rope_inputs(in, wq, wk, positions, p);
  if (rc) return rc;
  if (!q && !k && !v) return SVGEAR_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    if ((in[i] != nullptr) != (out[i] != nullptr)) return SVGEAR_ERR_INVALID;
  if (!aligned16(Q, K, V)) return SVGEAR_ERR_INVALID;
  return cuda_status(qkv_rope_run(in, wq, wk, positions, p, out, S(stream)));
}

size_t svgear_qkv_rope_backward_workspace_size(const svgear_rope_params* p) {
  if (check_rope(p)) return 0;
  return qkv_rope_back_ws_bytes(p);
}

int svgear_qkv_rope_backward(const void* dQ, const void* dK, const void* dV, const void* q, const void* k, const float* wq,
                    const float* wk, const int32_t* positions, const svgear_rope_params* p, void* dq, void* dk, void* dv,
                    float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_rope(p);
  if (rc) return rc;
  const bool normed = p->norm != SVGEAR_QKNORM_NONE;
  const void* grad[3] = {dQ, dK, dV};
  const void* in[3] = {normed ? q : nullptr, normed ? k : nullptr, nullptr};
  void* out[3] = {dq, dk, dv};
  rc = check_rope_inputs(in, wq, wk, positions, p);
  if (rc) return rc;
  if (!dQ && !dK && !dV) return SVGEAR_ERR_INVALID;
  for (int i = 0; i < 3; ++i) {
    if ((grad[i] != nullptr) != (out[i] != nullptr)) return SVGEAR_ERR_INVALID;
    if (normed && i < 2 && grad[i] && !in[i]) return SVGEAR_ERR_INVALID;
  }
  if ((dwq && (!normed || !dQ)) || (dwk && (!normed || !dK))) return SVGEAR_ERR_INVALID;
  if (!row_strides_ok(p, p->grad_ld, p->grad_batch) || !rows_apart(p, p->grad_ld, p->grad_batch)) return SVGEAR_ERR_INVALID;
  if (!aligned16(dQ, dK, dV, dq, dk, dv, dwq, dwk)) return SVGEAR_ERR_INVALID;
  if ((dwq || dwk) && (!ws || !aligned16(ws) || ws_bytes < qkv_rope_back_ws_bytes(p))) return SVGEAR_ERR_WORKSPACE;
  return cuda_status(qkv_rope_back_run(grad, in, wq, wk, positions, p, out, dwq, dwk, ws, S(stream)));
}

int svgear_mx_quantize(const void* X, int dtype, int M, int K, int head_d, uint8_t* codes, uint8_t* scales, void* stream) {
  const int rc = check_mx(M, K);
  if (rc) return rc;
  if (!known_dtype(dtype)) return SVGEAR_ERR_UNSUPPORTED;
  if (head_d < 0 || (head_d && (head_d % 8 || K % head_d))) return SVGEAR_ERR_INVALID;
  if (!X || !codes || !scales || !aligned16(X, codes, scales)) return SVGEAR_ERR_INVALID;
  return cuda_status(mx_quantize_run(X, dtype, M, K, head_d, codes, scales, S(stream)));
}

int svgear_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int M, int K, void* Y, int dtype, void* stream) {
  const int rc = check_mx(M, K);
  if (rc) return rc;
  if (!known_dtype(dtype)) return SVGEAR_ERR_UNSUPPORTED;
  if (!Y || !codes || !scales || !aligned16(Y, codes, scales)) return SVGEAR_ERR_INVALID;
  return cuda_status(mx_dequantize_run(codes, scales, M, K, Y, dtype, S(stream)));
}

int svgear_mx_product(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                      const float* bias, int M, int N, int K, void* Y, void* stream) {
  const int rc = check_product(M, N, K);
  if (rc) return rc;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !Y) return SVGEAR_ERR_INVALID;
  if (!aligned16(a_codes, a_scales, w_codes, w_scales, bias, Y)) return SVGEAR_ERR_INVALID;
  return cuda_status(mx_product_run(a_codes, a_scales, w_codes, w_scales, bias, M, N, K, Y, S(stream)));
}

}  // extern "C"
