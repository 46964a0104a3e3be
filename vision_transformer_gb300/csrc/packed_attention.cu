// Attention over packed documents (sv_attention_packed): document mask, causal mask with a
// visible prefix, tanh-capped scores, a bias that falls with distance, shared key heads.
//
// A query's visible keys are the keys j < lim of its document: lim = Lk, or with the prefix
// mask min(Lk, max(p_i + 1, prefix)), p_i = i + Lk - Lq. For these, in F32,
//   s_j = scale q . k_j;  s_j = cap tanh(s_j / cap);  s_j -= slope |p_i - j|,
//   o = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m),
// m following the running maximum. lim = 0 gives zeros.
#include <cuda_fp8.h>

#include <cmath>

#include "ptx.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct PackedParams {
  const __half *q, *k, *v;
  void* o;
  const int *q_off, *k_off, *prefix;
  const float* slopes;
  int docs, total_q, total_k, hq, hk, group, D;
  long long qs, ks, vs, os;
  float scale, cap;
  int causal, out_e4m3;
  int* err;
};

// Offset d of `docs` documents: the caller's, held to [0, total], or equal lengths.
__device__ __forceinline__ int offset_of(const int* off, int d, int docs, int total) {
  if (!off) return int(static_cast<long long>(total / docs) * d);
  return min(max(off[d], 0), total);
}

// Visible keys of a query at position `at` (p_i) of a document with lk keys.
__device__ __forceinline__ int limit_of(bool causal, int at, int lk, int prefix) {
  return causal ? min(lk, max(max(at + 1, prefix), 0)) : lk;
}

__device__ __forceinline__ float score_of(float s, float cap) { return cap > 0.0f ? cap * tanhf(s / cap) : s; }

// One warp per (query, head): 32 keys at a time, a lane's key dotted with q from shared
// memory, then a lane's output columns summed over the 32 keys.
__global__ void __launch_bounds__(128) packed_rows_kernel(const PackedParams p) {
  __shared__ float qs[4][128];
  __shared__ float ps[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && warp == 0)  // the documents' offsets, once
    for (int d = lane; d < p.docs; d += 32) {
      bool bad = false;
      if (p.q_off) bad |= p.q_off[d] < 0 || p.q_off[d + 1] < p.q_off[d] || p.q_off[d + 1] > p.total_q;
      if (p.k_off) bad |= p.k_off[d] < 0 || p.k_off[d + 1] < p.k_off[d] || p.k_off[d + 1] > p.total_k;
      if (bad) atomicOr(p.err, kDevErrOffsets);
    }
  const long long job = static_cast<long long>(blockIdx.x) * 4 + warp;
  const int row = int(job / p.hq), h = int(job % p.hq);
  if (row >= p.total_q) return;
  int doc = -1;
  for (int d0 = 0; d0 < p.docs && doc < 0; d0 += 32) {
    const int d = d0 + lane;
    const bool in = d < p.docs && offset_of(p.q_off, d, p.docs, p.total_q) <= row &&
                    row < offset_of(p.q_off, d + 1, p.docs, p.total_q);
    const unsigned hit = __ballot_sync(0xffffffffu, in);
    if (hit) doc = d0 + __ffs(hit) - 1;
  }
  if (doc < 0) return;
  const int q0 = offset_of(p.q_off, doc, p.docs, p.total_q), q1 = offset_of(p.q_off, doc + 1, p.docs, p.total_q);
  const int k0 = offset_of(p.k_off, doc, p.docs, p.total_k);
  const int lk = max(0, offset_of(p.k_off, doc + 1, p.docs, p.total_k) - k0);
  const int at = row - q0 + lk - (q1 - q0);
  const int lim = limit_of(p.causal, at, lk, p.prefix ? p.prefix[doc] : 0);
  const float slope = p.slopes ? p.slopes[h] : 0.0f;
  const __half* q = p.q + row * p.qs + h * p.D;
  for (int c = lane; c < p.D; c += 32) qs[warp][c] = __half2float(q[c]);
  __syncwarp();
  const __half* kb = p.k + k0 * p.ks + (h / p.group) * p.D;
  const __half* vb = p.v + k0 * p.vs + (h / p.group) * p.D;
  float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < lim; j0 += 32) {
    const int j = j0 + lane, n = min(32, lim - j0);
    float s = -INFINITY;
    if (j < lim) {
      const __half* kr = kb + j * p.ks;
      float dot = 0.0f;
      for (int c = 0; c < p.D; ++c) dot = fmaf(qs[warp][c], __half2float(kr[c]), dot);
      s = score_of(dot * p.scale, p.cap) - slope * fabsf(float(at - j));
      s *= kLog2e;
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.0f : mn;
    const float f = exp2f(m - ref);
    const float e = j < lim ? exp2f(s - ref) : 0.0f;
    float es = e;
    for (int o = 16; o; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
    l = l * f + es;
    m = mn;
    ps[warp][lane] = e;
    __syncwarp();
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      if (c >= p.D) break;
      float a = acc[i] * f;
      for (int jj = 0; jj < n; ++jj) a = fmaf(ps[warp][jj], __half2float(vb[(j0 + jj) * p.vs + c]), a);
      acc[i] = a;
    }
    __syncwarp();
  }
  const float inv = lim > 0 ? 1.0f / l : 0.0f;
  for (int i = 0; i < 4; ++i) {
    const int c = lane + 32 * i;
    if (c >= p.D) break;
    const size_t at_o = size_t(row) * size_t(p.os) + size_t(h) * size_t(p.D) + size_t(c);
    const float y = lim > 0 ? acc[i] * inv : 0.0f;
    if (p.out_e4m3)
      static_cast<uint8_t*>(p.o)[at_o] = __nv_cvt_float_to_fp8(16.0f * y, __NV_SATFINITE, __NV_E4M3);
    else
      static_cast<__half*>(p.o)[at_o] = __float2half_rn(y);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace sv

extern "C" {

size_t sv_attention_packed_workspace(int docs, int total_q, int total_k, int q_heads, int kv_heads, int head_dim) {
  (void)docs, (void)total_q, (void)total_k, (void)q_heads, (void)kv_heads, (void)head_dim;
  return 16;
}

sv_status sv_attention_packed(const void* q, const void* k, const void* v, void* o, const int* q_offsets,
                              const int* k_offsets, int docs, int total_q, int total_k, int q_heads, int kv_heads,
                              int head_dim, long long q_stride, long long k_stride, long long v_stride,
                              long long o_stride, const sv_attention_options* options, int out_dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  using namespace sv;
  const char* fn = "sv_attention_packed";
  if (docs < 1 || total_q < 0 || total_k < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
      (out_dtype != SV_DT_F16 && out_dtype != SV_DT_E4M3)) {
    set_error("%s: bad arguments (docs %d, total_q %d, total_k %d, heads %d over %d, out_dtype %d)", fn, docs, total_q,
              total_k, q_heads, kv_heads, out_dtype);
    return SV_ERR_INVALID_ARG;
  }
  if (head_dim < 8 || head_dim > 128 || head_dim % 8 || q_heads / kv_heads > 64 || q_heads > 65536) {
    set_error("%s: head_dim %d (a multiple of 8 in [8, 128]) or heads %d over %d are not supported", fn, head_dim,
              q_heads, kv_heads);
    return SV_ERR_UNSUPPORTED;
  }
  if ((!q_offsets && total_q % docs) || (!k_offsets && total_k % docs)) {
    set_error("%s: without offsets, %d queries and %d keys must divide by %d documents", fn, total_q, total_k, docs);
    return SV_ERR_INVALID_ARG;
  }
  const long long q_row = static_cast<long long>(q_heads) * head_dim, k_row = static_cast<long long>(kv_heads) * head_dim;
  if (q_stride == 0) q_stride = q_row;
  if (o_stride == 0) o_stride = q_row;
  if (k_stride == 0) k_stride = k_row;
  if (v_stride == 0) v_stride = k_row;
  if (q_stride < q_row || o_stride < q_row || k_stride < k_row || v_stride < k_row ||
      (q_stride | k_stride | v_stride | o_stride) % 8) {
    set_error("%s: row strides must be multiples of 8 that cover a row (q %lld, k %lld, v %lld, o %lld)", fn, q_stride,
              k_stride, v_stride, o_stride);
    return SV_ERR_INVALID_ARG;
  }
  if ((total_q && (!q || !o)) || (total_k && (!k || !v)) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(o) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(q_offsets) & 3) ||
      (reinterpret_cast<uintptr_t>(k_offsets) & 3)) {
    set_error("%s: q, k, v, o and workspace must be 16-byte aligned pointers, offsets 4-byte aligned", fn);
    return SV_ERR_INVALID_ARG;
  }
  if (workspace && workspace_bytes < sv_attention_packed_workspace(docs, total_q, total_k, q_heads, kv_heads, head_dim)) {
    set_error("%s: the workspace has %zu bytes, fewer than sv_attention_packed_workspace()", fn, workspace_bytes);
    return SV_ERR_INVALID_ARG;
  }
  sv_attention_options opt = {};
  if (options) opt = *options;
  if ((opt.mask != SV_MASK_DOCUMENT && opt.mask != SV_MASK_PREFIX) || !(opt.softcap >= 0.0f) ||
      !std::isfinite(opt.softcap) || !std::isfinite(opt.scale) ||
      (reinterpret_cast<uintptr_t>(opt.prefix) & 3) || (reinterpret_cast<uintptr_t>(opt.slopes) & 3)) {
    set_error("%s: bad options (mask %d, softcap %g, scale %g)", fn, opt.mask, double(opt.softcap), double(opt.scale));
    return SV_ERR_INVALID_ARG;
  }
  if (opt.scale <= 0.0f) opt.scale = 1.0f / std::sqrt(float(head_dim));
  if (total_q == 0) return SV_OK;
  sv_status st = ensure_runtime();
  if (st != SV_OK) return st;
  PackedParams p = {};
  p.q = static_cast<const __half*>(q);
  p.k = static_cast<const __half*>(k);
  p.v = static_cast<const __half*>(v);
  p.o = o;
  p.q_off = q_offsets;
  p.k_off = k_offsets;
  p.prefix = opt.prefix;
  p.slopes = opt.slopes;
  p.docs = docs;
  p.total_q = total_q;
  p.total_k = total_k;
  p.hq = q_heads;
  p.hk = kv_heads;
  p.group = q_heads / kv_heads;
  p.D = head_dim;
  p.qs = q_stride;
  p.ks = k_stride;
  p.vs = v_stride;
  p.os = o_stride;
  p.scale = opt.scale;
  p.cap = opt.softcap;
  p.causal = opt.mask == SV_MASK_PREFIX;
  p.out_e4m3 = out_dtype == SV_DT_E4M3;
  p.err = dev_err();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long blocks = (static_cast<long long>(total_q) * q_heads + 3) / 4;
  if (blocks > 0x7fffffffll) {
    set_error("%s: %d queries of %d heads are too many for one call", fn, total_q, q_heads);
    return SV_ERR_UNSUPPORTED;
  }
  LaunchScope L(kKindAttn, 0.0, 0.0, s);
  packed_rows_kernel<<<unsigned(blocks), 128, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "packed attention launch");
}

}  // extern "C"
