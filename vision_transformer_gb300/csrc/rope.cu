// Rotary positions, and the norm of every query and key head with the rotation in the
// same pass (sv_rope, sv_qk_norm_rope).
//
// A head of head_dim values is D / 2 pairs (a, b). Pair p < rot_dim / 2 belongs to
// position axis x = p / n and has index i = p % n there (n pairs per axis); its angle is
// t = pos_x f_i and it becomes g (a cos t - b sin t, b cos t + a sin t). The pairs behind
// the rotated part keep their values (they are the two halves of a run of 2 V values).
// The norm comes first: RMS x / sqrt(mean x^2 + eps) gamma, or LayerNorm without a bias,
// (x - mean) / sqrt(mean (x - mean)^2 + eps) gamma, statistics and arithmetic in F32, one
// rounding to F16 at the end. Values behind the rotated part never meet their run's partners (cosine 1
// and sine 0 would spoil them with a partner's infinity or NaN): without a norm they are not
// touched at all, with one they are scaled alone.
//
// Angles: a position may be millions of radians away, where a F32 angle has lost its
// fraction. The plan holds each frequency as a 64-bit fixed-point fraction of a turn per
// position, so position x frequency modulo 2^64 is the phase with whole turns dropped
// exactly (error below 2^-22 turns at 2^31 positions, 2^-33 at a million); its upper 32
// bits, as a signed fraction of half a turn, go to sincospif.
//
// Bound: DRAM, every value read and written once (4 bytes a value). What it takes to get there
// is bytes in flight and few instructions: the heads of a row lie one behind another, so a warp
// copies up to 4 KB of them at a time to shared memory and back with one bulk copy each way, two
// ahead of the arithmetic, and works on them in place. (Loads and stores by the lanes, any
// layout and prefetch tried: 64 us at best for 23,328 rows of 32 heads of 72, at 170
// instructions per 216 values and 13 KB in flight per SM.)
// 23,328 rows of 32 heads of 72 in pairs 18 values apart, RMS norm: 50 us, 4.3 TB/s (2 values an
// access: 56% of all cycles issue, from 16 warps an SM); 8,191 rows of 40 heads of 128, RMS norm: 31 us, 5.4 TB/s; 16,411 rows of 8 heads of
// 128, half of each rotated, neighbouring pairs, no norm: 14.4 us, 4.7 TB/s (start and end of the launch).
// A lane holds eight pairs: runs of V values and the runs n values on with their partners
// (V = 4, 2 or 1 by what divides n, so that every run is one aligned access), or runs of eight
// for neighbouring pairs. A head takes head_dim / 16 lanes, a warp as many whole heads as fit
// (72 values: 6 heads on 30 lanes), and neighbouring lanes hold neighbouring runs.
// The cosines of a row are the same for all of its heads: a warp works them out once per row,
// the norm's weights multiplied in.
#include <cfloat>
#include <cmath>

#include "ptx.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

constexpr int kBufBytes = 4096, kBufs = 3;  // of a warp

struct RopeParams {
  const __half* x[2];      // queries, keys (or the one tensor of sv_rope)
  __half* y[2];
  const __half* gamma[2];  // [head_dim] or null (ones)
  long long xs[2], ys[2];  // row strides in values
  int heads[2];            // keys: 0 for the one tensor of sv_rope
  const int* pos;          // [axes, rows]
  int rows, head_dim;
  int lanes, fold;         // lanes of a head, the largest power of two of them
  int slots;               // heads of a warp at a time
  int chunk, chunks0, chunks;  // heads of a job, jobs of a row's queries, of a row
  float eps, inv_dim, gain;
  int pairs, n;            // rotated pairs, pairs per axis
  int* err;
  unsigned long long turns[SV_ROPE_MAX_PAIRS];
};

// Runs of a lane: V > 0: kRuns runs of V values at a with their partners at b; V = 0
// (neighbouring pairs): runs of eight values at a.
template <int V>
struct Runs {
  static constexpr int kPer = V == 0 ? 4 : V;  // pairs per run
  static constexpr int kRuns = 8 / kPer;
};

// The pairs (fa, fb) of a run.
template <int V>
__device__ __forceinline__ void load_run(const __half* p, int a, int b, float* fa, float* fb) {
  if constexpr (V == 0) {
    __half2 h[4];
    *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(p + a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      fa[i] = f.x, fb[i] = f.y;
    }
  } else if constexpr (V == 1) {
    fa[0] = __half2float(p[a]);
    fb[0] = __half2float(p[b]);
  } else {
    __half2 h[V / 2], k[V / 2];
    if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(p + a);
      *reinterpret_cast<uint2*>(k) = *reinterpret_cast<const uint2*>(p + b);
    } else {
      h[0] = *reinterpret_cast<const __half2*>(p + a);
      k[0] = *reinterpret_cast<const __half2*>(p + b);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = __half22float2(h[i]), g = __half22float2(k[i]);
      fa[2 * i] = f.x, fa[2 * i + 1] = f.y;
      fb[2 * i] = g.x, fb[2 * i + 1] = g.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void store_run(__half* p, int a, int b, const float* fa, const float* fb) {
  if constexpr (V == 0) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(fa[i], fb[i]);
    *reinterpret_cast<uint4*>(p + a) = *reinterpret_cast<const uint4*>(h);
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
    if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(p + a) = *reinterpret_cast<const uint2*>(h);
      *reinterpret_cast<uint2*>(p + b) = *reinterpret_cast<const uint2*>(k);
    } else {
      *reinterpret_cast<__half2*>(p + a) = h[0];
      *reinterpret_cast<__half2*>(p + b) = k[0];
    }
  }
}

// Sum over a head's lanes, the same bits in each. Where the lanes are no power of two, those
// behind the largest one (`fold`) are folded onto the first ones, which then sum by exchange.
struct HeadSum {
  int fold, from_fold, from[4], from_low;  // source lanes (a head has at most 16)
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
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (fold > (8 >> i)) v += __shfl_sync(0xffffffffu, v, from[i]);
    if (folds) v = __shfl_sync(0xffffffffu, v, from_low);
    return v;
  }
};

__host__ __device__ constexpr size_t rope_smem(int head_dim, int parts) {
  return size_t(kRopeWarps) * kBufs * kBufBytes + size_t(kRopeWarps + parts) * (head_dim / 2) * sizeof(float2);
}

// PART: a norm, and pairs that are not rotated (a kernel of its own: looking for them costs the others 7%).
template <int V, int NORM, bool PART>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPer = Runs<V>::kPer, kRuns = Runs<V>::kRuns;
  extern __shared__ __align__(128) uint8_t rope_shared[];
  __shared__ unsigned long long turns[SV_ROPE_MAX_PAIRS];
  __shared__ __align__(8) unsigned long long full[kRopeWarps][kBufs];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int all = p.head_dim / 2;  // pairs, with those behind the rotated part
  uint8_t* bufs = rope_shared + warp * kBufs * kBufBytes;
  // the row's (cosine, sine) of every pair; the norm's weights of its two values
  float2* tables = reinterpret_cast<float2*>(rope_shared + kRopeWarps * kBufs * kBufBytes);
  float2* weights = tables + kRopeWarps * all;
  float2* table = tables + warp * all;
  // the values of pair i of a head
  auto first_of = [&](int i) {
    if (V == 0) return 2 * i;
    if (i < p.pairs) return i + (i >= p.n ? p.n : 0);
    return 2 * i - i % kPer;
  };
  auto second_of = [&](int i) { return V == 0 ? 2 * i + 1 : first_of(i) + (i < p.pairs ? p.n : kPer); };
  for (int i = threadIdx.x; i < p.n && p.pairs; i += kRopeThreads) turns[i] = p.turns[i];
  if (lane == 0) {
    for (int b = 0; b < kBufs; ++b) mbar_init(smem_u32(&full[warp][b]), 1);
    if (warp == 0) abort_flag = 0;
    fence_barrier_init();
  }
  const int slot = lane / p.lanes, first = slot * p.lanes, l = lane - first;
  const HeadSum head_sum(p, first, l);
  const bool in = slot < p.slots;  // (a lane of no head otherwise)
  // this lane's runs: run g = s lanes + l of the head
  int at_a[kRuns], at_b[kRuns], pair_of[kRuns];
  bool has[kRuns];
  uint32_t behind = 0;  // pairs that are not rotated (without a norm they are neither loaded nor stored)
#pragma unroll
  for (int s = 0; s < kRuns; ++s) {
    has[s] = in && (s * p.lanes + l) * kPer < (NORM == kNormNone ? p.pairs : all);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int pair = (s * p.lanes + l) * kPer + i;
      behind |= uint32_t(pair >= p.pairs && pair < all) << (s * kPer + i);
    }
    pair_of[s] = min((s * p.lanes + l) * kPer, all - kPer);
    at_a[s] = first_of(pair_of[s]) + slot * p.head_dim;
    at_b[s] = V == 0 ? at_a[s] : second_of(pair_of[s]) + slot * p.head_dim;
  }
  pdl_launch_dependents();
  pdl_wait();
  if constexpr (NORM != kNormNone)
    for (int i = threadIdx.x; i < 2 * all; i += kRopeThreads) {
      const int part = i >= all, pair = part ? i - all : i;
      const __half* g = p.gamma[part];
      weights[i] =
          g ? make_float2(__half2float(g[first_of(pair)]), __half2float(g[second_of(pair)])) : make_float2(1.0f, 1.0f);
    }
  __syncthreads();

  // Jobs: chunk c of row r is job r x chunks + c; a warp takes a contiguous share of them.
  const long long jobs = static_cast<long long>(p.rows) * p.chunks, warps = static_cast<long long>(gridDim.x) * kRopeWarps;
  const long long me = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
  const long long begin = jobs * me / warps;
  const int count = int(jobs * (me + 1) / warps - begin);
  struct Job {
    int row, chunk, part, h0, heads;
  };
  auto fill = [&](Job& j) {
    j.part = j.chunk >= p.chunks0 ? 1 : 0;
    j.h0 = (j.part ? j.chunk - p.chunks0 : j.chunk) * p.chunk;
    j.heads = min(p.chunk, (j.part ? p.heads[1] : p.heads[0]) - j.h0);
  };
  auto advance = [&](Job& j) {
    if (++j.chunk == p.chunks) j.chunk = 0, ++j.row;
    fill(j);
  };
  Job now, load;
  now.row = int(begin / p.chunks);
  now.chunk = int(begin - static_cast<long long>(now.row) * p.chunks);
  fill(now);
  load = now;
  auto copy_in = [&](int n) {  // job `load`, the warp's n-th, into its buffer (lane 0)
    const uint32_t bar = smem_u32(&full[warp][n % kBufs]), bytes = uint32_t(load.heads * p.head_dim * 2);
    const __half* src = (load.part ? p.x[1] + load.row * p.xs[1] : p.x[0] + load.row * p.xs[0]) + load.h0 * p.head_dim;
    mbar_arrive_expect_tx(bar, bytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(bufs + (n % kBufs) * kBufBytes)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
  };
  for (int n = 0; n < kBufs - 1 && n < count; ++n) {
    if (lane == 0) copy_in(n);
    advance(load);
  }
  int table_row = -1, pos_row = now.row;
  auto position = [&](int axis, int row) {
    return p.pairs > axis * p.n ? p.pos[static_cast<long long>(axis) * p.rows + row] : 0;
  };
  int pos0 = count ? position(0, now.row) : 0, pos1 = count ? position(1, now.row) : 0;

  for (int n = 0; n < count; ++n, advance(now)) {
    if (now.row != table_row) {  // the row's cosines, each once for all heads
      table_row = now.row;
      if (pos_row != now.row) {
        pos_row = now.row;
        pos0 = position(0, pos_row);
        pos1 = position(1, pos_row);
      }
      __syncwarp();
      for (int i = lane; i < all; i += 32) {
        float sn = 0.0f, cs = 1.0f;
        if (i < p.pairs) {
          const bool second = i >= p.n;
          const unsigned long long phase =
              turns[second ? i - p.n : i] * static_cast<unsigned long long>(static_cast<long long>(second ? pos1 : pos0));
          sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &sn, &cs);
          sn *= p.gain;
          cs *= p.gain;
        }
        table[i] = make_float2(cs, sn);
      }
      __syncwarp();
      if (table_row + 1 < p.rows) {  // the next row's positions are on their way
        pos_row = table_row + 1;
        pos0 = position(0, pos_row);
        pos1 = position(1, pos_row);
      }
    }
    // a' = a aa + b ab, b' = b bb + a ba, the norm's weights in them
    float aa[8], ab[8], bb[8], ba[8];
#pragma unroll
    for (int s = 0; s < kRuns; ++s)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float2 t = table[pair_of[s] + i];
        const float2 g = NORM == kNormNone ? make_float2(1.0f, 1.0f) : weights[(now.part ? all : 0) + pair_of[s] + i];
        const int k = s * kPer + i;
        aa[k] = g.x * t.x, ab[k] = -g.y * t.y, bb[k] = g.y * t.x, ba[k] = g.x * t.y;
      }
    uint8_t* buf = bufs + (n % kBufs) * kBufBytes;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[warp][n % kBufs]), (n / kBufs) & 1, &abort_flag, p.err))) {
      // (the copies behind this one land before the block can exit)
      for (int i = n; lane == 0 && i < count && i < n + kBufs - 1; ++i)
        mbar_wait_bounded(smem_u32(&full[warp][i % kBufs]), (i / kBufs) & 1, p.err);
      break;
    }
    __half* xb = reinterpret_cast<__half*>(buf);
    for (int h = 0; h < now.heads; h += p.slots, xb += p.slots * p.head_dim) {
      const bool live = h + slot < now.heads;
      float a[8], b[8];
#pragma unroll
      for (int s = 0; s < kRuns; ++s) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) a[s * kPer + i] = b[s * kPer + i] = 0.0f;
        if (live && has[s]) load_run<V>(xb, at_a[s], at_b[s], a + s * kPer, b + s * kPer);
      }
      float rs = 1.0f;
      if constexpr (NORM != kNormNone) {
        if constexpr (NORM == kNormLayer) {
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            add_x2(s0, s1, s0, s1, a[i], a[i + 1]);
            add_x2(s0, s1, s0, s1, b[i], b[i + 1]);
          }
          // (Rounded as a division. The product with 1 / D, which may also be fused into the differences, misses the
          // value of a constant head where D is no power of two, and the norm divides what is left by next to nothing.)
          const float sum = head_sum(s0 + s1), near = sum * p.inv_dim;
          const float mean = fmaf(fmaf(-near, float(p.head_dim), sum), p.inv_dim, near);
#pragma unroll
          for (int s = 0; s < kRuns; ++s)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (has[s]) a[s * kPer + i] -= mean, b[s * kPer + i] -= mean;
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          fma_x2(s0, s1, a[i], a[i + 1], a[i], a[i + 1], s0, s1);
          fma_x2(s0, s1, b[i], b[i + 1], b[i], b[i + 1], s0, s1);
        }
        const float var = fmaf(head_sum(s0 + s1), p.inv_dim, p.eps);
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(var));
      }
      float ya[8], yb[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        mul_x2(ya[i], ya[i + 1], a[i], a[i + 1], aa[i], aa[i + 1]);
        mul_x2(yb[i], yb[i + 1], b[i], b[i + 1], bb[i], bb[i + 1]);
        if constexpr (!PART) {
          fma_x2(ya[i], ya[i + 1], b[i], b[i + 1], ab[i], ab[i + 1], ya[i], ya[i + 1]);
          fma_x2(yb[i], yb[i + 1], a[i], a[i + 1], ba[i], ba[i + 1], yb[i], yb[i + 1]);
        } else {
#pragma unroll
          for (int k = i; k < i + 2; ++k)
            if (!(behind >> k & 1)) {
              ya[k] = fmaf(b[k], ab[k], ya[k]);
              yb[k] = fmaf(a[k], ba[k], yb[k]);
            }
        }
        if constexpr (NORM != kNormNone) {
          mul_x2(ya[i], ya[i + 1], ya[i], ya[i + 1], rs, rs);
          mul_x2(yb[i], yb[i + 1], yb[i], yb[i + 1], rs, rs);
        }
      }
#pragma unroll
      for (int s = 0; s < kRuns; ++s) {
        if (!live || !has[s]) continue;
        if (NORM != kNormNone || V != 0 || !(behind >> (s * kPer) & 15)) {
          store_run<V>(xb, at_a[s], at_b[s], ya + s * kPer, yb + s * kPer);
        } else {
          for (int i = 0; i < kPer; ++i)
            if (!(behind >> (s * kPer + i) & 1))
              *reinterpret_cast<__half2*>(xb + at_a[s] + 2 * i) = __floats2half2_rn(ya[s * kPer + i], yb[s * kPer + i]);
        }
      }
    }
    fence_proxy_async_smem();  // the lanes' writes, before the copy out reads them
    __syncwarp();
    if (lane == 0) {
      __half* dst = (now.part ? p.y[1] + now.row * p.ys[1] : p.y[0] + now.row * p.ys[0]) + now.h0 * p.head_dim;
      bulk_store(dst, smem_u32(buf), uint32_t(now.heads * p.head_dim * 2));
      bulk_commit();
      if (n + kBufs - 1 < count) {
        bulk_wait_read<1>();  // the buffer of the job before has been read out
        copy_in(n + kBufs - 1);
      }
    }
    if (n + kBufs - 1 < count) advance(load);
  }
  if (lane == 0) bulk_wait_all();
}

template <int V, int NORM, bool PART>
cudaError_t rope_launch_as(const RopeParams& p, cudaStream_t s) {
  const size_t smem = rope_smem(p.head_dim, NORM == kNormNone ? 1 : 2);
  static unsigned long long attr_set = 0;  // the attribute is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < kMaxAttrDevices) ? 1ull << dev : 0ull;
  if (!(attr_set & bit) || !bit) {
    e = cudaFuncSetAttribute(rope_kernel<V, NORM, PART>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(rope_smem(256, 2)));
    if (e != cudaSuccess) return e;
    attr_set |= bit;
  }
  const long long jobs = static_cast<long long>(p.rows) * p.chunks, most = 2ll * num_sms();
  const long long blocks = (jobs + kRopeWarps - 1) / kRopeWarps;
  return launch_pdl(rope_kernel<V, NORM, PART>, dim3(unsigned(blocks < most ? blocks : most)), dim3(kRopeThreads), smem, s, p);
}

template <int V>
cudaError_t rope_launch_v(const RopeParams& p, int norm, cudaStream_t s) {
  const bool part = 2 * p.pairs < p.head_dim;
  if (norm == kNormRms) return part ? rope_launch_as<V, kNormRms, true>(p, s) : rope_launch_as<V, kNormRms, false>(p, s);
  if (norm == kNormLayer)
    return part ? rope_launch_as<V, kNormLayer, true>(p, s) : rope_launch_as<V, kNormLayer, false>(p, s);
  return rope_launch_as<V, kNormNone, false>(p, s);
}

sv_status rope_launch(RopeParams& p, const sv_rope_plan* plan, int norm, cudaStream_t s) {
  const int D = p.head_dim;
  p.pairs = plan ? plan->rot_dim / 2 : 0;
  p.n = plan ? plan->pairs : 4;  // (no plan: no rotated pair, runs as wide as they get)
  p.gain = plan ? plan->gain : 1.0f;
  p.inv_dim = 1.0f / float(D);
  p.err = dev_err();
  for (int i = 0; i < (plan ? plan->pairs : 0); ++i) p.turns[i] = plan->turns[i];
  p.lanes = (D + 15) / 16;
  p.fold = 1;
  while (2 * p.fold <= p.lanes) p.fold *= 2;
  p.slots = 32 / p.lanes;
  // heads of a job: what a buffer holds, less where the GPU's warps would not all get one,
  // down to the heads that a warp takes at a time
  p.chunk = kBufBytes / (2 * D);
  auto split = [&]() {
    p.chunks0 = (p.heads[0] + p.chunk - 1) / p.chunk;
    p.chunks = p.chunks0 + (p.heads[1] + p.chunk - 1) / p.chunk;
  };
  split();
  while (p.chunk > p.slots && static_cast<long long>(p.rows) * p.chunks < 2ll * kRopeWarps * num_sms()) {
    p.chunk = p.chunk / 2 > p.slots ? p.chunk / 2 : p.slots;
    split();
  }
  LaunchScope L(kKindOther, 0.0, 4.0 * p.rows * (double(p.heads[0]) + p.heads[1]) * D, s);
  cudaError_t e;
  if (plan && plan->layout == SV_ROPE_INTERLEAVED) e = rope_launch_v<0>(p, norm, s);
  else if (p.n % 4 == 0) e = rope_launch_v<4>(p, norm, s);
  else if (p.n % 2 == 0) e = rope_launch_v<2>(p, norm, s);
  else e = rope_launch_v<1>(p, norm, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "rope launch");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The checks both entry points share; 0 strides become contiguous rows.
sv_status rope_args(const char* fn, const sv_rope_plan* plan, const int* pos, int rows, int heads, int head_dim) {
  if (rows < 0 || heads < 1 || heads > (1 << 20) || head_dim < 8 || head_dim > 256 || head_dim % 8) {
    set_error("%s: bad sizes (rows %d, heads %d of at most 2^20, head_dim %d: a multiple of 8 in [8, 256])", fn, rows, heads, head_dim);
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
  p.heads[0] = heads;
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
  if ((norm != SV_NORM_RMS && norm != SV_NORM_LAYER) || !(eps >= 0.0f) || kv_heads < 1 || kv_heads > (1 << 20)) {
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
  p.heads[0] = q_heads;
  p.heads[1] = kv_heads;
  p.pos = positions;
  p.rows = rows;
  p.head_dim = head_dim;
  p.eps = eps > 0.0f && eps < FLT_MIN ? FLT_MIN : eps;  // (the reciprocal root takes subnormal numbers for 0)
  return rope_launch(p, plan, norm == SV_NORM_RMS ? kNormRms : kNormLayer, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
