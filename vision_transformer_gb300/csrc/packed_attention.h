// What the two kernels of sv_attention_packed share (packed_attention.cu: tiles of 128 rows
// on the tensor cores; packed_few.cu: a few rows per document).
#pragma once
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "sv_internal.h"

namespace sv {
namespace packed {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSms = 152;  // SMs that a launch uses at most (the workspace is sized by it)
// Workspace: counters of arrivals first (zero before and after every call), then partial results.
constexpr int kTicket = 2 * kMaxSms * 8;  // the next item to hand out, behind the arrivals
constexpr size_t kCounterBytes = (size_t(kTicket) + 16) * sizeof(unsigned);

// The reference exponent of a row is set kHead below a tile's maximum when that maximum is
// more than kSlack above it: P <= 2^15 stays finite in F16, small probabilities stay above
// its subnormal range for longer, and O is rescaled rarely.
constexpr float kSlack = 15.0f, kHead = 8.0f;

struct Params {
  const __half *q, *k, *v;
  void* o;
  const int *q_off, *k_off, *prefix;
  const float* slopes;
  int docs, total_q, total_k, hq, hk, group, D;
  long long qs, ks, vs, os;
  float scale, cap;
  int causal, out_e4m3;
  int qt;              // queries of a 128-row tile: 128 / group
  int out_tma;         // whole warps' output rows go out by TMA
  unsigned* counters;  // workspace: arrivals; null: no key range is divided
  float* partial;      // workspace: partial results
  int* err;
};

// packed_few.cu, for few rows per document on average: bound by reading the keys and values, not by
// products
inline bool few_rows(int docs, int total_q, int group) {
  return static_cast<long long>(total_q) * group <= 16ll * docs;
}
sv_status few_launch(const Params& p, cudaStream_t s);
size_t few_workspace(int head_dim);

// Offset d of `docs` documents: the caller's, or equal lengths.
__device__ __forceinline__ int offset_of(const int* off, int d, int docs, int total) {
  return off ? __ldg(off + d) : (total / docs) * d;
}

// Visible keys of a query at position `at` (p_i) of a document with lk keys.
__device__ __forceinline__ int limit_of(int causal, int at, int lk, int prefix) {
  return causal ? min(lk, max(max(at + 1, prefix), 0)) : lk;
}

// Queries q0 .. q0 + lq - 1 and keys k0 .. k0 + lk - 1 of a document.
struct Document {
  int q0, lq, k0, lk, prefix;
};
// Document d (no queries and keys from `docs` on); false if its offsets decrease or leave [0, total].
__device__ __forceinline__ bool document(const Params& p, int d, int docs, Document& r) {
  r = {0, 0, 0, 0, 0};
  if (d >= docs) return true;
  r.q0 = offset_of(p.q_off, d, p.docs, p.total_q);
  r.k0 = offset_of(p.k_off, d, p.docs, p.total_k);
  const int q1 = offset_of(p.q_off, d + 1, p.docs, p.total_q), k1 = offset_of(p.k_off, d + 1, p.docs, p.total_k);
  r.prefix = p.prefix ? __ldg(p.prefix + d) : 0;
  if (r.q0 < 0 || q1 < r.q0 || q1 > p.total_q || r.k0 < 0 || k1 < r.k0 || k1 > p.total_k) return false;
  r.lq = q1 - r.q0;
  r.lk = k1 - r.k0;
  return true;
}

// cap tanh(s / cap) = cap - 2 cap / (2^x + 1), x = 2 s log2 e / cap, c = cap in any unit; exact
// limits for infinite s. The error, about 2^-22 cap, is that of the reciprocal of a number >= 1; from caps of
// kFarCap on, where that is more than 2^-14, scores that are small beside the cap are summed as a series.
constexpr float kFarCap = 256.0f;
__device__ __forceinline__ float capped(float x, float c) {
  const float u = ex2(x) + 1.0f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(u));
  return fmaf(-2.0f * c, r, c);
}
// The same for four values x y[i], with one reciprocal: 1 / u_0 = (u_1 (u_2 u_3)) / (u_0 u_1 u_2 u_3)
// and so on. Reciprocals run at a quarter of the exponentials' rate here, and the products on
// another pipe. x is held to 30, where 2 / (2^x + 1) is below the last bit of 1, so that the product
// of four stays finite; NaN passes through (into its neighbours too).
__device__ __forceinline__ void capped4(float* y, float x, float c) {
  float u[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    mul_x2(u[i], u[i + 1], y[i], y[i + 1], x, x);
    asm("min.NaN.f32 %0, %0, 0f41F00000;" : "+f"(u[i]));
    asm("min.NaN.f32 %0, %0, 0f41F00000;" : "+f"(u[i + 1]));
    u[i] = ex2(u[i]);
    u[i + 1] = ex2(u[i + 1]);
    add_x2(u[i], u[i + 1], u[i], u[i + 1], 1.0f, 1.0f);
  }
  const float a = u[0] * u[1], b = u[2] * u[3];
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
  r *= -2.0f * c;
  const float ra = r * b, rb = r * a;
  fma_x2(y[0], y[1], ra, ra, u[1], u[0], c, c);
  fma_x2(y[2], y[3], rb, rb, u[3], u[2], c, c);
}

// Factor of the scores' products for x above: 1e30 stands for more (the smallest product that is not 0 is 2^-48), so
// that a product of 0 stays 0 whatever the cap.
__device__ __forceinline__ float cap_factor(float scale, float cap) { return fminf(2.0f * kLog2e * scale / cap, 1e30f); }

// s: a score in units of log 2; x as above; big: what capped gives. Below |s / cap| = 1/4, where that cancels:
// s (1 - z^2 / 3 + 2 z^4 / 15 - 17 z^6 / 315 + 62 z^8 / 2835), z = x ln 2 / 2 (the next term is below 2^-26).
// The error is below 2^-18 of the score for any cap.
__device__ __forceinline__ float far_capped(float s, float x, float big) {
  const float z = x * 0.34657359f, y = z * z;
  float t = fmaf(y, 62.0f / 2835.0f, -17.0f / 315.0f);
  t = fmaf(y, t, 2.0f / 15.0f);
  t = fmaf(y, t, -1.0f / 3.0f);
  return fabsf(z) < 0.25f ? fmaf(s * y, t, s) : big;
}

// Eight values in the output's type at `to`.
__device__ __forceinline__ void put8(int e4m3, uint8_t* to, const float* y) {
  if (e4m3) {
    uint2 w;
    __nv_fp8x2_storage_t* h = reinterpret_cast<__nv_fp8x2_storage_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * y[2 * i], 16.0f * y[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(to) = w;
  } else {
    uint4 w;
    __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
    *reinterpret_cast<uint4*>(to) = w;
  }
}
// Eight values of an output row, `at` values into o.
__device__ __forceinline__ void store8(const Params& p, size_t at, const float* y) {
  put8(p.out_e4m3, static_cast<uint8_t*>(p.o) + (p.out_e4m3 ? at : 2 * at), y);
}

// Four values of an output row, on a multiple of four.
__device__ __forceinline__ void store4(const Params& p, size_t at, const float4& y) {
  if (p.out_e4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * y.x, 16.0f * y.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * y.z, 16.0f * y.w), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.o) + at) = lo | hi << 16;
  } else {
    __half2 h[2] = {__floats2half2_rn(y.x, y.y), __floats2half2_rn(y.z, y.w)};
    *reinterpret_cast<uint2*>(static_cast<__half*>(p.o) + at) = *reinterpret_cast<const uint2*>(h);
  }
}

// One value of an output row.
__device__ __forceinline__ void store1(const Params& p, size_t at, float y) {
  if (p.out_e4m3) static_cast<uint8_t*>(p.o)[at] = __nv_cvt_float_to_fp8(16.0f * y, __NV_SATFINITE, __NV_E4M3);
  else static_cast<__half*>(p.o)[at] = __float2half_rn(y);
}

// Rows whose result is not finite. A tile's product multiplies the probability 0 of a hidden key with its value,
// which is NaN for an infinite or NaN value. Keys behind the last one that any row of an item sees never reach a
// product, so only keys that some of its rows see and others do not can do this: a row is computed again where one
// of those keys that it does not see holds such a value, and a row that sees one itself keeps the products' result,
// which is not finite either.

// The last of the keys from .. to - 1 whose value row (D values at v, a document's first) holds an infinity or NaN, -1:
// none. By a whole warp.
static __device__ __noinline__ int last_spoiled(const Params& p, const __half* v, int from, int to, int lane) {
  const int chunks = p.D / 8;
  int last = -1;
  for (long long x = lane; x < static_cast<long long>(to - from) * chunks; x += 32) {
    const int key = from + int(x / chunks);
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(v + key * p.vs) + int(x % chunks));
    bool bad = false;
    const uint32_t pairs[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      bad |= (pairs[e] & 0x7c00u) == 0x7c00u || (pairs[e] & 0x7c000000u) == 0x7c000000u;
    if (bad) last = key;
  }
  return __reduce_max_sync(0xffffffffu, last);
}

// A row from its visible keys alone, by a whole warp: keys kb .. ke - 1 of the document, query position `at`. Four keys
// at a time, of which a lane holds the columns 4 lane .. 4 lane + 3 and then the score of key lane % 4. Unscaled sums,
// their exponent and denominator. 64 keys turn `beat` on (null: nobody waits for this). 31 rows over 20,000 keys of 128
// dimensions, the warp alone on its SM: 110 ms; a thread a row 370. (Four rows and eight keys at a time 30, with three
// times the registers, which the callers' loops need.)
static __device__ __noinline__ float4 row_again(const Params& p, const __half* q, const __half* k, const __half* v,
                                                int kb, int ke, int at, float slope, int lane, unsigned* beat,
                                                float& m_out, float& l_out) {
  constexpr int kKeys = 4;
  const bool mine = lane < p.D / 4;
  auto four = [&](const __half* row) {
    uint2 w = make_uint2(0u, 0u);
    if (mine) w = __ldg(reinterpret_cast<const uint2*>(row) + lane);
    return w;
  };
  auto wide = [](uint2 w) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  };
  const float4 qf = wide(four(q));
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float m = -INFINITY, l = 0.0f;
#pragma unroll 1
  for (int j0 = kb; j0 < ke; j0 += kKeys) {
    uint2 kx[kKeys], vx[kKeys];
#pragma unroll
    for (int b = 0; b < kKeys; ++b) {
      kx[b] = vx[b] = make_uint2(0u, 0u);
      if (j0 + b < ke) {
        kx[b] = four(k + (j0 + b) * p.ks);
        vx[b] = four(v + (j0 + b) * p.vs);
      }
    }
    float s[kKeys];
#pragma unroll
    for (int b = 0; b < kKeys; ++b) {
      const float4 kf = wide(kx[b]);
      s[b] = fmaf(qf.x, kf.x, fmaf(qf.y, kf.y, fmaf(qf.z, kf.z, qf.w * kf.w)));
    }
    // summed over the lanes, key j0 + lane % 4 left in each
#pragma unroll
    for (int x = 1; x < kKeys; x <<= 1)
#pragma unroll
      for (int b = 0; b < kKeys / (2 * x); ++b) {
        const bool odd = lane & x;
        const float give = odd ? s[2 * b] : s[2 * b + 1];
        s[b] = (odd ? s[2 * b + 1] : s[2 * b]) + __shfl_xor_sync(0xffffffffu, give, x);
      }
#pragma unroll
    for (int x = kKeys; x < 32; x <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], x);
    const int key = j0 + lane % kKeys;
    float x = s[0] * p.scale;
    if (p.cap > 0.0f) x = p.cap * tanhf(x / p.cap);
    x = key < ke ? (x - slope * fabsf(float(at - key))) * kLog2e : -INFINITY;
    float up = x;
#pragma unroll
    for (int o = 1; o < kKeys; o <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
    up = fmaxf(up, m);
    const float ref = up == -INFINITY ? 0.0f : up, back = exp2f(m - ref), e = exp2f(x - ref);
    m = up;
    float sum = e;
#pragma unroll
    for (int o = 1; o < kKeys; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = fmaf(l, back, sum);
    acc = make_float4(acc.x * back, acc.y * back, acc.z * back, acc.w * back);
#pragma unroll
    for (int b = 0; b < kKeys; ++b) {
      const float eb = __shfl_sync(0xffffffffu, e, b);
      const float4 vf = wide(vx[b]);
      acc.x = fmaf(eb, vf.x, acc.x);
      acc.y = fmaf(eb, vf.y, acc.y);
      acc.z = fmaf(eb, vf.z, acc.z);
      acc.w = fmaf(eb, vf.w, acc.w);
    }
    if (beat && lane == 0 && (j0 - kb) % 64 == 0) atomicAdd(beat, 1u);
  }
  m_out = m;
  l_out = l;
  return acc;
}

}  // namespace packed
}  // namespace sv
