// Rotary positions, and the norm of every query and key head with the rotation in the
// same pass (sv_rope, sv_qk_norm_rope).
//
// A head of head_dim values is D / 2 pairs (a, b). Pair p < rot_dim / 2 belongs to
// position axis x = p / n and has index i = p % n there (n pairs per axis); its angle is
// t = pos_x f_i and it becomes g (a cos t - b sin t, b cos t + a sin t). The pairs behind
// the rotated part keep their values (they are the two halves of a run of 2 V values).
// The norm comes first: RMS x / sqrt(mean x^2 + eps) gamma, or LayerNorm without a bias,
// (x - mean) / sqrt(mean (x - mean)^2 + eps) gamma, statistics and arithmetic in F32, one
// rounding to F16 at the end.
//
// Angles: a position may be millions of radians away, where a F32 angle has lost its
// fraction. The plan holds each frequency as a 64-bit fixed-point fraction of a turn per
// position, so position x frequency modulo 2^64 is the phase with whole turns dropped
// exactly (error below 2^-22 turns at 2^31 positions, 2^-33 at a million); its upper 32
// bits, as a signed fraction of half a turn, go to sincospif.
//
// Bound: DRAM, every value read and written once (4 bytes a value). The cosines of a row
// are the same for all of its heads: a warp computes them once and walks heads with them.
// A head is spread over L lanes (a power of two >= head_dim / 16), each holding eight
// pairs in runs of V values whose partners lie n values on (V = 8, 4, 2 or 1 by what
// divides n, so that every run is one aligned load); neighbouring lanes hold neighbouring
// runs. Statistics are xor-shuffle sums over the L lanes.
#include <cmath>

#include "ptx.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kRopeThreads = 256;
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

struct RopeParams {
  const __half* x[2];      // queries, keys (or the one tensor of sv_rope)
  __half* y[2];
  const __half* gamma[2];  // [head_dim] or null (ones)
  long long xs[2], ys[2];  // row strides in values
  int heads0, heads;       // heads of x[0], of both
  const int* pos;          // [axes, rows]
  int rows, head_dim, lanes, per_warp;  // heads a warp walks: per_warp x (32 / lanes)
  int chunks;              // warps per row
  float eps, inv_dim, gain;
  int pairs, n;            // rotated pairs, pairs per axis
  unsigned long long turns[SV_ROPE_MAX_PAIRS];
};

// One lane's runs: V values at `a`, V more at `b`; V = 0 (neighbouring pairs): eight
// values at `a`, four pairs. Run g of a head; returns its first pair.
template <int V>
__device__ __forceinline__ int run_at(int g, int pairs, int n, int& a, int& b) {
  if constexpr (V == 0) {
    a = 8 * g;
    b = a;
    return 4 * g;
  } else {
    const int p = g * V;
    if (p < pairs) {
      const int axis = p / n;
      a = p + axis * n;  // 2 n axis + (p - n axis)
      b = a + n;
    } else {
      a = 2 * p;
      b = a + V;
    }
    return p;
  }
}

template <int V>
struct Runs {
  static constexpr int kPer = V == 0 ? 4 : V;  // pairs per run
  static constexpr int kRuns = 8 / kPer;
};

template <int V>
__device__ __forceinline__ void load_half(const __half* p, __half2* h) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(p);
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(p);
  else *reinterpret_cast<unsigned*>(h) = *reinterpret_cast<const unsigned*>(p);
}
template <int V>
__device__ __forceinline__ void store_half(__half* p, const __half2* h) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
  else *reinterpret_cast<unsigned*>(p) = *reinterpret_cast<const unsigned*>(h);
}

// The kPer pairs of a run at p + a, p + b.
template <int V>
__device__ __forceinline__ void load_run(const __half* p, int a, int b, float* fa, float* fb) {
  if constexpr (V == 0) {
    __half2 h[4];
    load_half<8>(p + a, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      fa[i] = f.x;
      fb[i] = f.y;
    }
  } else if constexpr (V == 1) {
    fa[0] = __half2float(p[a]);
    fb[0] = __half2float(p[b]);
  } else {
    __half2 h[V / 2], k[V / 2];
    load_half<V>(p + a, h);
    load_half<V>(p + b, k);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = __half22float2(h[i]), g = __half22float2(k[i]);
      fa[2 * i] = f.x;
      fa[2 * i + 1] = f.y;
      fb[2 * i] = g.x;
      fb[2 * i + 1] = g.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void store_run(__half* p, int a, int b, const float* fa, const float* fb) {
  if constexpr (V == 0) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(fa[i], fb[i]);
    store_half<8>(p + a, h);
  } else if constexpr (V == 1) {
    p[a] = __float2half_rn(fa[0]);
    p[b] = __float2half_rn(fb[0]);
  } else {
    __half2 h[V / 2], k[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      h[i] = __floats2half2_rn(fa[2 * i], fa[2 * i + 1]);
      k[i] = __floats2half2_rn(fb[2 * i], fb[2 * i + 1]);
    }
    store_half<V>(p + a, h);
    store_half<V>(p + b, k);
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int V, int NORM>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = Runs<V>::kPer, kRuns = Runs<V>::kRuns;
  __shared__ unsigned long long turns[SV_ROPE_MAX_PAIRS];
  for (int i = threadIdx.x; i < p.n; i += kRopeThreads) turns[i] = p.turns[i];
  pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long job = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + warp;
  const long long row_ll = job / p.chunks;
  if (row_ll >= p.rows) return;
  const int row = int(row_ll), chunk = int(job - row_ll * p.chunks);
  const int slots = 32 / p.lanes, slot = lane / p.lanes, l = lane - slot * p.lanes;
  const int runs = p.head_dim / (2 * kPer);  // of one head

  float cs[8], sn[8];
  int at_a[kRuns], at_b[kRuns];
#pragma unroll
  for (int s = 0; s < kRuns; ++s) {
    const int pair = run_at<V>(s * p.lanes + l, p.pairs, p.n, at_a[s], at_b[s]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      cs[s * kPer + i] = 1.0f;
      sn[s * kPer + i] = 0.0f;
      if (pair + i < p.pairs) {
        const int axis = (pair + i) / p.n;
        const long long pos = p.pos[static_cast<long long>(axis) * p.rows + row];
        const unsigned long long phase = turns[pair + i - axis * p.n] * static_cast<unsigned long long>(pos);
        float a, b;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &a, &b);
        sn[s * kPer + i] = a * p.gain;
        cs[s * kPer + i] = b * p.gain;
      }
    }
  }

  float ga[8], gb[8];
  int gamma_of = -1;
  for (int it = 0; it < p.per_warp; ++it) {
    const int h = (chunk * p.per_warp + it) * slots + slot;
    if ((chunk * p.per_warp + it) * slots >= p.heads) break;
    const bool live = h < p.heads;
    const int which = live && h >= p.heads0 ? 1 : 0;
    const int head = which ? h - p.heads0 : h;
    const __half* x = p.x[which] + row * p.xs[which] + static_cast<long long>(head) * p.head_dim;
    float a[8], b[8];
#pragma unroll
    for (int s = 0; s < kRuns; ++s) {
      if (live && s * p.lanes + l < runs) load_run<V>(x, at_a[s], at_b[s], a + s * kPer, b + s * kPer);
      else
#pragma unroll
        for (int i = 0; i < kPer; ++i) a[s * kPer + i] = b[s * kPer + i] = 0.0f;
    }
    if constexpr (NORM != kNormNone) {
      if (gamma_of != which) {
        gamma_of = which;
        const __half* g = p.gamma[which];
#pragma unroll
        for (int s = 0; s < kRuns; ++s) {
          if (g && s * p.lanes + l < runs) load_run<V>(g, at_a[s], at_b[s], ga + s * kPer, gb + s * kPer);
          else
#pragma unroll
            for (int i = 0; i < kPer; ++i) ga[s * kPer + i] = gb[s * kPer + i] = 1.0f;
        }
      }
      if constexpr (NORM == kNormLayer) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += a[i] + b[i];
        const float mean = lanes_sum(sum, p.lanes) * p.inv_dim;
#pragma unroll
        for (int s = 0; s < kRuns; ++s)
          if (s * p.lanes + l < runs)
#pragma unroll
            for (int i = 0; i < kPer; ++i) a[s * kPer + i] -= mean, b[s * kPer + i] -= mean;
      }
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
      const float r = rsqrtf(lanes_sum(sq, p.lanes) * p.inv_dim + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] *= r * ga[i], b[i] *= r * gb[i];
    }
    if (!live) continue;
    __half* y = p.y[which] + row * p.ys[which] + static_cast<long long>(head) * p.head_dim;
#pragma unroll
    for (int s = 0; s < kRuns; ++s) {
      if (s * p.lanes + l >= runs) continue;
      float ya[kPer], yb[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int k = s * kPer + i;
        ya[i] = a[k] * cs[k] - b[k] * sn[k];
        yb[i] = b[k] * cs[k] + a[k] * sn[k];
      }
      store_run<V>(y, at_a[s], at_b[s], ya, yb);
    }
  }
}

template <int V>
cudaError_t rope_launch_v(const RopeParams& p, int norm, unsigned grid, cudaStream_t s) {
  if (norm == kNormRms) return launch_pdl(rope_kernel<V, kNormRms>, dim3(grid), dim3(kRopeThreads), 0, s, p);
  if (norm == kNormLayer) return launch_pdl(rope_kernel<V, kNormLayer>, dim3(grid), dim3(kRopeThreads), 0, s, p);
  return launch_pdl(rope_kernel<V, kNormNone>, dim3(grid), dim3(kRopeThreads), 0, s, p);
}

sv_status rope_launch(RopeParams& p, const sv_rope_plan* plan, int norm, cudaStream_t s) {
  const int D = p.head_dim;
  p.pairs = plan ? plan->rot_dim / 2 : 0;
  p.n = plan ? plan->pairs : 8;  // (no plan: no rotated pair, runs as wide as the head allows)
  p.gain = plan ? plan->gain : 1.0f;
  p.inv_dim = 1.0f / float(D);
  for (int i = 0; i < (plan ? plan->pairs : 0); ++i) p.turns[i] = plan->turns[i];
  p.lanes = 1;
  while (p.lanes * 16 < D) p.lanes *= 2;
  const int slots = 32 / p.lanes;
  const int trips = (p.heads + slots - 1) / slots;
  // heads per warp: enough to spread the row's cosines over, while the warps still fill
  // the GPU (about 32 warps on each SM)
  const long long want = 32ll * num_sms();
  p.per_warp = 1;
  while (p.per_warp < trips && p.per_warp < 8 &&
         static_cast<long long>(p.rows) * ((trips + p.per_warp) / (p.per_warp + 1)) >= want)
    ++p.per_warp;
  p.chunks = (trips + p.per_warp - 1) / p.per_warp;
  const long long warps = static_cast<long long>(p.rows) * p.chunks;
  const long long blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 0x7fffffffll) {
    set_error("rope: %d rows of %d heads are too many for one call", p.rows, p.heads);
    return SV_ERR_UNSUPPORTED;
  }
  const unsigned grid = unsigned(blocks);
  LaunchScope L(kKindOther, 0.0, 4.0 * p.rows * double(p.heads) * D, s);
  cudaError_t e;
  if (plan && plan->layout == SV_ROPE_INTERLEAVED) e = rope_launch_v<0>(p, norm, grid, s);
  else if (p.n % 8 == 0 && D % 16 == 0) e = rope_launch_v<8>(p, norm, grid, s);
  else if (p.n % 4 == 0) e = rope_launch_v<4>(p, norm, grid, s);
  else if (p.n % 2 == 0) e = rope_launch_v<2>(p, norm, grid, s);
  else e = rope_launch_v<1>(p, norm, grid, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "rope launch");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The checks both entry points share; 0 strides become contiguous rows.
sv_status rope_args(const char* fn, const sv_rope_plan* plan, const int* pos, int rows, int heads, int head_dim) {
  if (rows < 0 || heads < 1 || head_dim < 8 || head_dim > 256 || head_dim % 8) {
    set_error("%s: bad sizes (rows %d, heads %d, head_dim %d: a multiple of 8 in [8, 256])", fn, rows, heads, head_dim);
    return SV_ERR_INVALID_ARG;
  }
  if (plan) {
    if (plan->rot_dim < 2 || plan->rot_dim > head_dim || plan->axes < 1 || plan->axes > 2 ||
        plan->pairs < 1 || plan->pairs > SV_ROPE_MAX_PAIRS || plan->pairs * 2 * plan->axes != plan->rot_dim ||
        (plan->layout != SV_ROPE_HALF && plan->layout != SV_ROPE_INTERLEAVED)) {
      set_error("%s: the plan rotates %d of %d values (use sv_rope_plan_init)", fn, plan->rot_dim, head_dim);
      return SV_ERR_INVALID_ARG;
    }
    if (!pos || (reinterpret_cast<uintptr_t>(pos) & 3)) {
      set_error("%s: positions must be a 4-byte aligned device pointer", fn);
      return SV_ERR_INVALID_ARG;
    }
  }
  return SV_OK;
}

sv_status rope_tensor(const char* fn, const char* what, const void* p, long long* stride, int heads, int head_dim) {
  const long long row = static_cast<long long>(heads) * head_dim;
  if (*stride == 0) *stride = row;
  if (!p || !aligned16(p) || *stride < row || *stride % 8) {
    set_error("%s: %s must be 16-byte aligned with a row stride (%lld) that is a multiple of 8 and at least %lld", fn,
              what, *stride, row);
    return SV_ERR_INVALID_ARG;
  }
  return SV_OK;
}

}  // namespace
}  // namespace sv

extern "C" {

sv_status sv_rope_plan_init(sv_rope_plan* plan, int rot_dim, int axes, int layout, double base, int scaling,
                            double factor, int original_len) {
  using namespace sv;
  if (!plan || axes < 1 || axes > 2 || rot_dim < 2 || rot_dim % (2 * axes) || rot_dim / 2 > SV_ROPE_MAX_PAIRS ||
      (layout != SV_ROPE_HALF && layout != SV_ROPE_INTERLEAVED) || !(base >= 1.0) || !std::isfinite(base)) {
    set_error("sv_rope_plan_init: bad arguments (rot_dim %d, axes %d, layout %d, base %g)", rot_dim, axes, layout,
              base);
    return SV_ERR_INVALID_ARG;
  }
  const int n = rot_dim / 2 / axes;
  if (scaling < SV_ROPE_SCALE_NONE || scaling > SV_ROPE_SCALE_BY_PARTS ||
      (scaling != SV_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) ||
      (scaling == SV_ROPE_SCALE_BASE && n < 2) || (scaling == SV_ROPE_SCALE_BY_PARTS && original_len < 1)) {
    set_error("sv_rope_plan_init: bad scaling (%d, factor %g, original length %d)", scaling, factor, original_len);
    return SV_ERR_INVALID_ARG;
  }
  const double two_pi = 6.283185307179586476925;
  if (scaling == SV_ROPE_SCALE_BASE) base *= std::pow(factor, double(n) / double(n - 1));
  plan->rot_dim = rot_dim;
  plan->axes = axes;
  plan->layout = layout;
  plan->pairs = n;
  plan->gain = scaling == SV_ROPE_SCALE_BY_PARTS ? float(0.1 * std::log(factor) + 1.0) : 1.0f;
  for (int i = 0; i < n; ++i) {
    double f = std::pow(base, -double(i) / double(n));
    if (scaling == SV_ROPE_SCALE_LINEAR) f /= factor;
    if (scaling == SV_ROPE_SCALE_BY_PARTS) {
      const double keep = std::fmin(1.0, std::fmax(0.0, (original_len * f / two_pi - 1.0) / 31.0));
      f *= keep + (1.0 - keep) / factor;
    }
    plan->turns[i] = static_cast<unsigned long long>(std::ldexp(f / two_pi, 64));  // f <= 1: below 2^62
  }
  for (int i = n; i < SV_ROPE_MAX_PAIRS; ++i) plan->turns[i] = 0;
  return SV_OK;
}

sv_status sv_rope(const void* x, void* y, const int* positions, const sv_rope_plan* plan, int rows, int heads,
                  int head_dim, long long x_stride, long long y_stride, void* stream) {
  using namespace sv;
  if (!plan) {
    set_error("sv_rope: plan is NULL");
    return SV_ERR_INVALID_ARG;
  }
  sv_status st = rope_args("sv_rope", plan, positions, rows, heads, head_dim);
  if (st == SV_OK) st = rope_tensor("sv_rope", "x", x, &x_stride, heads, head_dim);
  if (st == SV_OK) st = rope_tensor("sv_rope", "y", y, &y_stride, heads, head_dim);
  if (st == SV_OK && x == y && x_stride != y_stride) {
    set_error("sv_rope: in place, x and y must have the same row stride");
    st = SV_ERR_INVALID_ARG;
  }
  if (st != SV_OK || rows == 0) return st;
  st = ensure_runtime();
  if (st != SV_OK) return st;
  RopeParams p = {};
  p.x[0] = p.x[1] = static_cast<const __half*>(x);
  p.y[0] = p.y[1] = static_cast<__half*>(y);
  p.xs[0] = p.xs[1] = x_stride;
  p.ys[0] = p.ys[1] = y_stride;
  p.heads0 = p.heads = heads;
  p.pos = positions;
  p.rows = rows;
  p.head_dim = head_dim;
  return rope_launch(p, plan, kNormNone, static_cast<cudaStream_t>(stream));
}

sv_status sv_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* q_gamma,
                          const void* k_gamma, int norm, float eps, const int* positions, const sv_rope_plan* plan,
                          int rows, int q_heads, int kv_heads, int head_dim, long long q_stride, long long k_stride,
                          long long q_out_stride, long long k_out_stride, void* stream) {
  using namespace sv;
  const char* fn = "sv_qk_norm_rope";
  if ((norm != SV_NORM_RMS && norm != SV_NORM_LAYER) || !(eps >= 0.0f) || kv_heads < 1 || q_heads < 1 ||
      q_heads > (1 << 20) || kv_heads > (1 << 20)) {
    set_error("%s: bad arguments (norm %d, eps %g, heads %d and %d)", fn, norm, double(eps), q_heads, kv_heads);
    return SV_ERR_INVALID_ARG;
  }
  sv_status st = rope_args(fn, plan, positions, rows, q_heads, head_dim);
  if (st == SV_OK) st = rope_tensor(fn, "q", q, &q_stride, q_heads, head_dim);
  if (st == SV_OK) st = rope_tensor(fn, "k", k, &k_stride, kv_heads, head_dim);
  if (st == SV_OK) st = rope_tensor(fn, "q_out", q_out, &q_out_stride, q_heads, head_dim);
  if (st == SV_OK) st = rope_tensor(fn, "k_out", k_out, &k_out_stride, kv_heads, head_dim);
  if (st == SV_OK && (!aligned16(q_gamma) || !aligned16(k_gamma))) {
    set_error("%s: gammas must be 16-byte aligned", fn);
    st = SV_ERR_INVALID_ARG;
  }
  if (st == SV_OK && ((q == q_out && q_stride != q_out_stride) || (k == k_out && k_stride != k_out_stride))) {
    set_error("%s: in place, input and output must have the same row stride", fn);
    st = SV_ERR_INVALID_ARG;
  }
  if (st != SV_OK || rows == 0) return st;
  st = ensure_runtime();
  if (st != SV_OK) return st;
  RopeParams p = {};
  p.x[0] = static_cast<const __half*>(q);
  p.x[1] = static_cast<const __half*>(k);
  p.y[0] = static_cast<__half*>(q_out);
  p.y[1] = static_cast<__half*>(k_out);
  p.gamma[0] = static_cast<const __half*>(q_gamma);
  p.gamma[1] = static_cast<const __half*>(k_gamma);
  p.xs[0] = q_stride;
  p.xs[1] = k_stride;
  p.ys[0] = q_out_stride;
  p.ys[1] = k_out_stride;
  p.heads0 = q_heads;
  p.heads = q_heads + kv_heads;
  p.pos = positions;
  p.rows = rows;
  p.head_dim = head_dim;
  p.eps = eps;
  return rope_launch(p, plan, norm == SV_NORM_RMS ? kNormRms : kNormLayer, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
