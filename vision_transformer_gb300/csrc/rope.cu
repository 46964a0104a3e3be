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
// Bound: DRAM, every value read and written once (4 bytes a value). A lane holds eight
// values, four pairs, so that few registers keep many warps and their loads in flight: a run of
// V values and the run n values on with their partners (V = 4, 2 or 1 by what divides n, so
// that every run is one aligned load), or one run of eight for neighbouring pairs. A head takes
// head_dim / 8 lanes, a warp as many whole heads as fit (72 values: 3 heads on 27 lanes), and
// neighbouring lanes hold neighbouring runs. The cosines of a row are the same for all of its
// heads: a block computes those of its rows once into shared memory, one to eight warps walk a
// row's heads with their share of them in registers, the next heads' loads ahead of the
// arithmetic. (Sixteen values a lane, a power of two of lanes a head, cosines in every warp:
// 23,328 rows of 32 heads of 72, 97 us, 337 instructions per warp and step.)
#include <cmath>

#include "ptx.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

struct RopeParams {
  const __half* x[2];      // queries, keys (or the one tensor of sv_rope)
  __half* y[2];
  const __half* gamma[2];  // [head_dim] or null (ones)
  long long xs[2], ys[2];  // row strides in values
  int heads0, heads;       // heads of x[0], of both
  const int* pos;          // [axes, rows]
  int rows, head_dim;
  int lanes, fold;         // lanes of a head, the largest power of two of them
  int slots;               // heads of a warp at a time
  int warps_row;           // warps that share a row (1, 2, 4 or 8)
  float eps, inv_dim, gain;
  int pairs, n;            // rotated pairs, pairs per axis
  unsigned long long turns[SV_ROPE_MAX_PAIRS];
};

// Runs of a lane: V > 0: kRuns runs of V values at a[] with their partners at b[]; V = 0
// (neighbouring pairs): eight values at a[0].
template <int V>
struct Runs {
  static constexpr int kPer = V == 0 ? 4 : V;  // pairs per run
  static constexpr int kRuns = 4 / kPer;
};

// A lane's eight values, as loaded: pairs of halves, for V = 1 (first, second) of each pair.
template <int V>
__device__ __forceinline__ void load_runs(const __half* p, const int* a, const int* b, __half2 (&h)[4]) {
  if constexpr (V == 0) {
    *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(p + a[0]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(p + a[0]);
    *reinterpret_cast<uint2*>(h + 2) = *reinterpret_cast<const uint2*>(p + b[0]);
  } else if constexpr (V == 2) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      h[s] = *reinterpret_cast<const __half2*>(p + a[s]);
      h[2 + s] = *reinterpret_cast<const __half2*>(p + b[s]);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) h[s] = __halves2half2(p[a[s]], p[b[s]]);
  }
}
template <int V>
__device__ __forceinline__ void store_runs(__half* p, const int* a, const int* b, const __half2 (&h)[4]) {
  if constexpr (V == 0) {
    *reinterpret_cast<uint4*>(p + a[0]) = *reinterpret_cast<const uint4*>(h);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p + a[0]) = *reinterpret_cast<const uint2*>(h);
    *reinterpret_cast<uint2*>(p + b[0]) = *reinterpret_cast<const uint2*>(h + 2);
  } else if constexpr (V == 2) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      *reinterpret_cast<__half2*>(p + a[s]) = h[s];
      *reinterpret_cast<__half2*>(p + b[s]) = h[2 + s];
    }
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      p[a[s]] = __low2half(h[s]);
      p[b[s]] = __high2half(h[s]);
    }
  }
}
// Between the loaded form and the four pairs (fa, fb).
template <int V>
__device__ __forceinline__ void unpack(const __half2 (&h)[4], float (&fa)[4], float (&fb)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    if constexpr (V <= 1) fa[i] = f.x, fb[i] = f.y;
    else if (i < 2) fa[2 * i] = f.x, fa[2 * i + 1] = f.y;
    else fb[2 * i - 4] = f.x, fb[2 * i - 3] = f.y;
  }
}
template <int V>
__device__ __forceinline__ void pack(const float (&fa)[4], const float (&fb)[4], __half2 (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (V <= 1) h[i] = __floats2half2_rn(fa[i], fb[i]);
    else h[i] = i < 2 ? __floats2half2_rn(fa[2 * i], fa[2 * i + 1]) : __floats2half2_rn(fb[2 * i - 4], fb[2 * i - 3]);
  }
}

// Sum over a head's lanes, the same bits in each. Where the lanes are no power of two, those
// behind the largest one (`fold`) are folded onto the first ones, which then sum by exchange.
struct HeadSum {
  int fold, from_fold, from[4], from_low;  // source lanes
  bool folds, has_fold;
  __device__ __forceinline__ HeadSum(const RopeParams& p, int first, int l) {
    fold = p.fold;
    folds = p.fold < p.lanes;
    has_fold = l + p.fold < p.lanes;
    from_fold = (first + l + p.fold) & 31;
    from_low = first + (l & (p.fold - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) from[i] = first + ((l & (p.fold - 1)) ^ (8 >> i));
  }
  __device__ __forceinline__ float operator()(float v) const {
    if (folds) {
      const float t = __shfl_sync(0xffffffffu, v, from_fold);
      if (has_fold) v += t;
    }
    if (fold == 32) v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (fold > (8 >> i)) v += __shfl_sync(0xffffffffu, v, from[i]);
    if (folds) v = __shfl_sync(0xffffffffu, v, from_low);
    return v;
  }
};

template <int V, int NORM>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = Runs<V>::kPer, kRuns = Runs<V>::kRuns;
  __shared__ float2 table[kRopeWarps * SV_ROPE_MAX_PAIRS];  // [row of the block][rotated pair]
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows_block = kRopeWarps / p.warps_row;
  const int row0 = int(blockIdx.x) * rows_block;
  const int r = warp / p.warps_row, sub = warp & (p.warps_row - 1);
  const int row = min(row0 + r, p.rows - 1);
  const int slot = lane / p.lanes, first = slot * p.lanes, l = lane - first;

  // this lane's runs: run g = s lanes + l of the head
  int at_a[kRuns], at_b[kRuns];
#pragma unroll
  for (int s = 0; s < kRuns; ++s) {
    const int g = s * p.lanes + l, pair = g * kPer;
    const int axis = pair >= p.n ? 1 : 0;
    if (V == 0) at_a[s] = 8 * g, at_b[s] = 8 * g;
    else if (pair < p.pairs) at_a[s] = pair + axis * p.n, at_b[s] = at_a[s] + p.n;
    else at_a[s] = 2 * pair, at_b[s] = 2 * pair + V;
  }
  const int head_step = p.warps_row * p.slots, step = head_step * p.head_dim;
  const int h_first = slot < p.slots ? sub * p.slots + slot : 0x40000000;  // (a lane of no head)
  __half2 next[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) next[i] = __float2half2_rn(0.0f);
  // the first heads are on their way while the cosines are worked out
  if (h_first < p.heads0) load_runs<V>(p.x[0] + row * p.xs[0] + h_first * p.head_dim, at_a, at_b, next);

  for (int i = threadIdx.x; i < rows_block * p.pairs; i += kRopeThreads) {
    const int tr = i / p.pairs, pair = i - tr * p.pairs, axis = pair >= p.n ? 1 : 0;
    if (row0 + tr >= p.rows) break;
    const long long pos = p.pos[static_cast<long long>(axis) * p.rows + row0 + tr];
    const unsigned long long phase = p.turns[pair - axis * p.n] * static_cast<unsigned long long>(pos);
    float sn, cs;
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &sn, &cs);
    table[i] = make_float2(cs * p.gain, sn * p.gain);
  }
  __syncthreads();
  if (row0 + r >= p.rows) return;
  const HeadSum head_sum(p, first, l);
  float cs[4], sn[4];
#pragma unroll
  for (int s = 0; s < kRuns; ++s)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int pair = (s * p.lanes + l) * kPer + i;
      const float2 t = pair < p.pairs ? table[r * p.pairs + pair] : make_float2(1.0f, 0.0f);
      cs[s * kPer + i] = t.x;
      sn[s * kPer + i] = t.y;
    }

#pragma unroll 1
  for (int part = 0; part < (NORM == kNormNone ? 1 : 2); ++part) {  // queries, keys
    const int heads = part ? p.heads - p.heads0 : p.heads0;
    // with a norm the weights go into the rotation: (a, b) -> rs (a ga cs - b gb sn, b gb cs + a ga sn)
    float aa[4], ab[4], bb[4], ba[4];
    if constexpr (NORM != kNormNone) {
      __half2 g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = __float2half2_rn(1.0f);
      if (p.gamma[part] && slot < p.slots) load_runs<V>(p.gamma[part], at_a, at_b, g);
      float ga[4], gb[4];
      unpack<V>(g, ga, gb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        aa[i] = ga[i] * cs[i];
        ab[i] = gb[i] * sn[i];
        bb[i] = gb[i] * cs[i];
        ba[i] = ga[i] * sn[i];
      }
    }
    int h = h_first;
    const int h_at = slot < p.slots ? h : 0;
    const __half* x = p.x[part] + row * p.xs[part] + h_at * p.head_dim;
    __half* y = p.y[part] + row * p.ys[part] + h_at * p.head_dim;
    if (part && h < heads) load_runs<V>(x, at_a, at_b, next);
#pragma unroll 1
    for (int h0 = sub * p.slots; h0 < heads; h0 += head_step) {
      float a[4], b[4];
      unpack<V>(next, a, b);
      const bool live = h < heads;
      h += head_step;
      x += step;
      if (h < heads) load_runs<V>(x, at_a, at_b, next);
      float ya[4], yb[4];
      if constexpr (NORM == kNormNone) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ya[i] = a[i] * cs[i] - b[i] * sn[i];
          yb[i] = b[i] * cs[i] + a[i] * sn[i];
        }
      } else {
        if constexpr (NORM == kNormLayer) {
          const float mean =
              head_sum(((a[0] + b[0]) + (a[1] + b[1])) + ((a[2] + b[2]) + (a[3] + b[3]))) * p.inv_dim;
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] -= mean, b[i] -= mean;
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) fma_x2(s0, s1, a[i], b[i], a[i], b[i], s0, s1);
        const float rs = rsqrtf(head_sum(s0 + s1) * p.inv_dim + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ya[i] = rs * (a[i] * aa[i] - b[i] * ab[i]);
          yb[i] = rs * (b[i] * bb[i] + a[i] * ba[i]);
        }
      }
      if (live) {
        __half2 out[4];
        pack<V>(ya, yb, out);
        store_runs<V>(y, at_a, at_b, out);
      }
      y += step;
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
  p.n = plan ? plan->pairs : 4;  // (no plan: no rotated pair, runs as wide as they get)
  p.gain = plan ? plan->gain : 1.0f;
  p.inv_dim = 1.0f / float(D);
  for (int i = 0; i < (plan ? plan->pairs : 0); ++i) p.turns[i] = plan->turns[i];
  p.lanes = D / 8;
  p.fold = 1;
  while (2 * p.fold <= p.lanes) p.fold *= 2;
  p.slots = 32 / p.lanes;
  const int trips = (p.heads + p.slots - 1) / p.slots;
  // warps per row: one (a row's cosines and gammas are then loaded into registers once) where
  // that fills the GPU with 32 warps an SM, more where rows are few
  p.warps_row = 1;
  while (p.warps_row < kRopeWarps && p.warps_row < trips &&
         static_cast<long long>(p.rows) * p.warps_row < 32ll * num_sms())
    p.warps_row *= 2;
  const int rows_block = kRopeWarps / p.warps_row;
  const long long blocks = (static_cast<long long>(p.rows) + rows_block - 1) / rows_block;
  const unsigned grid = unsigned(blocks);
  LaunchScope L(kKindOther, 0.0, 4.0 * p.rows * double(p.heads) * D, s);
  cudaError_t e;
  if (plan && plan->layout == SV_ROPE_INTERLEAVED) e = rope_launch_v<0>(p, norm, grid, s);
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
