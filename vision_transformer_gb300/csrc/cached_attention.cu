// Attention over a paged key/value cache (sv_attention_cached): the sequences' own tokens, a few rows each, and the
// prefix that they share; the entry point.
//
// A row is a query and one of the `group` query heads of a key head. Its visible keys are the prefix and the first
// lim of its sequence's own; with the stored numbers c and factors 2^ek, 2^ev of a key and its value
//   s_j = scale 2^ek_j q . ck_j, capped;  x_j = s_j log2 e + ev_j,
//   o = sum_j 2^(x_j - m) cv_j / sum_j 2^(x_j - m - ev_j),
// m following the running maximum of the x_j: the values' factors go into the exponents, which are in F32, and the
// products take the codes as they are (2^(x_j - m), rounded to F16, is then small only where the key's part in the
// result is small). A marked key or value (byte 255) makes s_j NaN for the rows that see it, and with it the whole row;
// its codes are 0, and every stored number is finite, so that the probability 0 of a hidden key keeps it out.
//
// Two passes where there is a prefix: first all rows of the batch over its keys (here in blocks of 8 or 16 rows), sums,
// exponents and denominators to the workspace; then every sequence's rows over its own tokens, which finish with
// the prefix's parts. Without a prefix the second alone.
//
// Bound: DRAM, every key and value read once for up to 8 or 16 rows. The arithmetic runs on warp-level matrix
// instructions (mma.sync m16n8k16, F32 accumulation): few rows fill no tcgen05 tile, and codes go from global memory to
// the registers of the instruction with a conversion between them (E4M3 to F16 in pairs, 64 a cycle and SM):
//   S^T = K Q^T: 16 keys x 8 rows. A lane's 8 neighbouring dimensions of a key serve as its operand values of two
//     instructions (the order of the summed dimensions is free); four lanes read 32 of them.
//   O^T += V^T P^T: 16 dimensions x 8 rows. Eight lanes read 64 neighbouring dimensions of a value, a lane has the same
//     8 of the keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; the bytes of two keys are interleaved before the conversion, which
//     so gives pairs of keys. P^T goes from the accumulator's layout to the operand's by a transposing 8 x 8 move.
// A warp takes 32 keys at a time (F16: 16), the registers of K loaded again as soon as S^T is done, those of V as soon as
// O^T is: these hold what is in flight. The four warps of a CTA take neighbouring keys of one head; 16 keys lie in one
// page.
//
// Work: the (sequence, key head, block of rows) items are laid out one behind another in steps of a CTA, and every CTA
// takes an equal, contiguous share of the steps, so that any distribution of lengths fills the GPU. An item inside one
// share is finished there; one that is cut goes in parts to the workspace, and the last CTA of its parts joins them in
// order.
#include <cmath>
#include <type_traits>

#include "cached.h"
#include "packed_attention.h"

namespace sv {
namespace cached {
namespace {

using packed::capped;
using packed::cap_factor;
using packed::far_capped;
using packed::kFarCap;
using packed::kHead;
using packed::kLog2e;
using packed::kMaxSms;
using packed::kSlack;

constexpr int kThreads = 128;
constexpr int kMostPerSm = 3;
constexpr int kMaxGrid = kMaxSms * kMostPerSm;
constexpr size_t kCounterBytes = (size_t(kMaxGrid) * sizeof(unsigned) + 127) / 128 * 128;
// CTAs an SM, by what the registers of a warp allow
constexpr int per_sm(int nt) { return nt > 1 ? 2 : 3; }
constexpr int step_keys(bool e4m3) { return e4m3 ? 128 : 64; }  // of a CTA

// Where the partial results of the prefix pass are: items (key head, block of rows) one behind another, each of `steps`
// steps, `chunk` steps a CTA. Item i and CTA c meet in part i + c: `rows` rows of D sums, then exponent and denominator
// of each.
struct PrefixParts {
  float* base;
  int rows, blocks, steps;
  long long chunk;
};

struct Params {
  View c;
  const __half* q;
  void* o;
  const int* q_off;
  int total_q, hq, group;
  long long qs, os;
  float scale, cap;
  int causal, out_e4m3;
  unsigned* counters;  // arrivals at cut items
  float* partial;      // two parts a CTA: of the item cut at the start of its share, at its end
  PrefixParts pre;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Two pairs of E4M3 codes as pairs of F16.
__device__ __forceinline__ void two_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Eight stored numbers in the registers that they are loaded into. ALONE: no other access needs the sectors that this one
// touches (they are not kept in L1).
template <bool E4M3>
struct Eight;
template <>
struct Eight<true> {
  uint2 w;
  template <bool ALONE>
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (ALONE) asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
    else asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
  }
  __device__ __forceinline__ void clear() { w = make_uint2(0u, 0u); }
};
template <>
struct Eight<false> {
  uint4 w;
  template <bool ALONE>
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (ALONE)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "l"(p));
    else
      asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "l"(p));
  }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
};

// Sixteen E4M3 codes in one access.
__device__ __forceinline__ void load_two(Eight<true>& a, Eight<true>& b, const uint8_t* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(a.w.x), "=r"(a.w.y), "=r"(b.w.x), "=r"(b.w.y)
               : "l"(p));
}
[[maybe_unused]] __device__ __forceinline__ void load_two(Eight<false>&, Eight<false>&, const uint8_t*) {}

// 2^(byte - 16) and its reciprocal, for bytes of factors.
__device__ __forceinline__ float power_of(int byte) { return __uint_as_float(uint32_t(byte + (127 - kNoScale)) << 23); }
__device__ __forceinline__ float reciprocal_of(int byte) {
  return __uint_as_float(uint32_t(127 + kNoScale - byte) << 23);
}

// A sequence of the call: its first row of q, its queries, own tokens. False if the offsets or the length are bad.
struct Sequence {
  int q0, n, have;
};
__device__ __forceinline__ bool sequence(const Params& p, int s, int count, Sequence& r) {
  r = {0, 0, 0};
  if (s >= count) return true;
  r.q0 = row_offset(p.q_off, s, p.c.count, p.total_q);
  const int q1 = row_offset(p.q_off, s + 1, p.c.count, p.total_q);
  r.have = __ldg(p.c.lengths + s);
  if (r.q0 < 0 || q1 < r.q0 || q1 > p.total_q || r.have < 0 ||
      r.have > (static_cast<long long>(p.c.stride) << p.c.shift)) {
    r = {0, 0, 0};
    return false;
  }
  r.n = q1 - r.q0;
  return true;
}

// Own tokens that query i of n sees.
__device__ __forceinline__ int limit_of(int causal, int i, int n, int have) {
  return causal ? max(0, min(have, have - n + i + 1)) : have;
}

// A run of steps of one item that falls into this CTA's share.
struct Segment {
  Sequence seq;
  const int* pages;       // of its keys
  int kvh, row0;          // key head, first of the item's rows (query x group + head) in the sequence
  int s0, s1, steps;      // steps of the item: this segment's, all
  long long base;         // place of the item's first step among all steps
  int item;               // (prefix pass)
};

// The items of the sequences in order: sequences, key heads, blocks of rows. 32 sequences at a time, one per lane,
// with their steps summed by shuffles; every warp works it out for itself. What it knows lies in shared memory (`st`, the
// warp's own): in registers it was in the way of the keys in flight.
struct ShareState {
  long long incl[32];  // steps of the sequences up to this one
  Sequence seq[32];
  int blocks[32], steps[32];
  long long chunk, at, end, base, total;
  int d0, count;
};
template <int ROWS, int STEP>
class Share {
 public:
  __device__ __forceinline__ Share(const Params& p, int lane, ShareState& st) : p_(p), lane_(lane), st_(st) {
    int count = p.c.count;
    long long work = 0;
    bool bad = false;
    for (int d0 = 0; d0 < p.c.count; d0 += 32) {
      Sequence q;
      int blocks, steps;
      bad |= !load(d0, count, q, blocks, steps);
      work += static_cast<long long>(blocks) * p.c.hk * steps;
    }
    for (int o = 16; o; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
    // bad offsets or lengths: reported, and nothing is computed
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0) atomicOr(p.c.err, kDevErrCache);
      count = 0;
      work = 0;
    }
    const long long chunk = max(1ll, (work + gridDim.x - 1) / gridDim.x), at = chunk * blockIdx.x;
    if (lane == 0) {
      st_.chunk = chunk;
      st_.at = at;
      st_.end = min(at + chunk, work);  // (a share may begin behind the last step)
      st_.base = 0;
      st_.count = count;
    }
    __syncwarp();
    open(0);
  }
  // The next segment of this CTA's share.
  __device__ __forceinline__ bool get(Segment& r) {
    const long long at = st_.at;
    if (at >= st_.end) return false;
    while (at >= st_.base + st_.total) {
      __syncwarp();
      if (lane_ == 0) st_.base += st_.total;
      __syncwarp();
      open(st_.d0 + 32);
    }
    const long long base = st_.base;
    const int src = __ffs(__ballot_sync(0xffffffffu, base + st_.incl[lane_] > at)) - 1;
    const int steps = st_.steps[src], blocks = st_.blocks[src];
    const long long first = base + st_.incl[src] - static_cast<long long>(blocks) * p_.c.hk * steps;
    const long long item = (at - first) / steps;
    Segment x;
    x.seq = st_.seq[src];
    x.pages = p_.c.table + static_cast<long long>(st_.d0 + src) * p_.c.stride;
    x.steps = steps;
    x.base = first + item * steps;
    x.kvh = int(item / blocks);
    x.row0 = int(item - static_cast<long long>(x.kvh) * blocks) * ROWS;
    x.s0 = int(at - x.base);
    x.s1 = int(min(st_.end - x.base, static_cast<long long>(steps)));
    x.item = 0;
    __syncwarp();
    if (lane_ == 0) {
      st_.at = x.base + x.s1;
      r = x;
    }
    __syncwarp();
    return true;
  }
  __device__ __forceinline__ int cta_of(long long step) const { return int(step / st_.chunk); }

 private:
  __device__ __forceinline__ bool load(int d0, int count, Sequence& q, int& blocks, int& steps) {
    const bool good = sequence(p_, d0 + lane_, count, q);
    blocks = int((static_cast<long long>(q.n) * p_.group + ROWS - 1) / ROWS);
    steps = max(1, (q.have + STEP - 1) / STEP);  // (a step without keys writes the prefix's result, or zeros)
    return good;
  }
  __device__ __forceinline__ void open(int d0) {
    Sequence q;
    int blocks, steps;
    load(d0, st_.count, q, blocks, steps);
    long long incl = static_cast<long long>(blocks) * p_.c.hk * steps;
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane_ >= o) incl += a;
    }
    st_.seq[lane_] = q;
    st_.blocks[lane_] = blocks;
    st_.steps[lane_] = steps;
    st_.incl[lane_] = incl;
    if (lane_ == 31) {
      st_.total = incl;
      st_.d0 = d0;
    }
    __syncwarp();
  }
  const Params& p_;
  const int lane_;
  ShareState& st_;
};

// The same for the prefix pass: all rows of the batch over one run of keys.
template <int ROWS>
class PrefixShare {
 public:
  __device__ __forceinline__ PrefixShare(const Params& p, int lane, ShareState& st) : p_(p), lane_(lane), st_(st) {
    const long long work = static_cast<long long>(p.pre.blocks) * p.c.hk * p.pre.steps;
    if (lane == 0) {
      st_.at = p.pre.chunk * blockIdx.x;
      st_.end = min(st_.at + p.pre.chunk, work);
    }
    __syncwarp();
  }
  __device__ __forceinline__ bool get(Segment& r) {
    const long long at = st_.at, end = st_.end;
    if (at >= end) return false;
    const long long item = at / p_.pre.steps;
    Segment x;
    x.seq = {0, p_.total_q, p_.c.prefix_len};
    x.pages = p_.c.prefix_pages;
    x.kvh = int(item / p_.pre.blocks);
    x.row0 = int(item - static_cast<long long>(x.kvh) * p_.pre.blocks) * ROWS;
    x.steps = p_.pre.steps;
    x.base = item * p_.pre.steps;
    x.s0 = int(at - x.base);
    x.s1 = int(min(end - x.base, static_cast<long long>(x.steps)));
    x.item = int(item);
    __syncwarp();
    if (lane_ == 0) {
      st_.at = x.base + x.s1;
      r = x;
    }
    __syncwarp();
    return true;
  }

 private:
  const Params& p_;
  const int lane_;
  ShareState& st_;
};

// Sums of a row with their exponent and denominator: four columns a lane.
struct RowSums {
  float4 y;
  float m, l;
  __device__ __forceinline__ void add(const float4& v, float mv, float lv) {
    const float up = fmaxf(m, mv), ref = up == -INFINITY ? 0.0f : up;
    const float a = ex2(m - ref), b = ex2(mv - ref);
    m = up;
    l = fmaf(a, l, b * lv);
    y = make_float4(fmaf(a, y.x, b * v.x), fmaf(a, y.y, b * v.y), fmaf(a, y.z, b * v.z), fmaf(a, y.w, b * v.w));
  }
  // Adds `n` parts in order, sixteen on their way at a time (they come from L2, and nothing else hides its latency):
  // at(w) is part w's place, [rows][D] sums and [rows] exponents and denominators.
  template <typename F>
  __device__ __forceinline__ void add_parts(int n, int row, int rows, int D, int lane, F at) {
    for (int w0 = 0; w0 < n; w0 += 16) {
      float4 v[16];
      float2 ml[16];
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        ml[b] = make_float2(-INFINITY, 0.0f);
        v[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (w0 + b < n) {
          const float* part = at(w0 + b);
          ml[b] = __ldcg(reinterpret_cast<const float2*>(part + size_t(rows) * D) + row);
          v[b] = __ldcg(reinterpret_cast<const float4*>(part + size_t(row) * D) + min(lane, D / 4 - 1));
        }
      }
      float up = m;
#pragma unroll
      for (int b = 0; b < 16; ++b) up = fmaxf(up, ml[b].x);
      const float ref = up == -INFINITY ? 0.0f : up, back = ex2(m - ref);
      m = up;
      l *= back;
      y = make_float4(y.x * back, y.y * back, y.z * back, y.w * back);
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        const float e = ex2(ml[b].x - ref);
        l = fmaf(e, ml[b].y, l);
        y.x = fmaf(e, v[b].x, y.x);
        y.y = fmaf(e, v[b].y, y.y);
        y.z = fmaf(e, v[b].z, y.z);
        y.w = fmaf(e, v[b].w, y.w);
      }
    }
  }
};

// Row r of the item at row0 of a sequence (sums so far: its own keys'), by one warp: with the prefix's parts, in the
// output's type.
__device__ __forceinline__ void finish_row(const Params& p, const Segment& sg, int r, int lane, RowSums a) {
  const int i = (sg.row0 + r) / p.group, head = sg.kvh * p.group + (sg.row0 + r - i * p.group);
  if (p.c.prefix_len > 0) {
    const PrefixParts& f = p.pre;
    const long long row = static_cast<long long>(sg.seq.q0 + i) * p.group + (head - sg.kvh * p.group);  // of the key head
    const int block = int(row / f.rows), at = int(row - static_cast<long long>(block) * f.rows);
    const long long item = static_cast<long long>(sg.kvh) * f.blocks + block, first = item * f.steps;
    const long long c0 = first / f.chunk, c1 = (first + f.steps - 1) / f.chunk;
    const float* part = f.base + size_t(item + c0) * (size_t(f.rows) * size_t(p.c.D + 2));
    a.add_parts(int(c1 - c0) + 1, at, f.rows, p.c.D, lane,
                [&](int w) { return part + size_t(w) * (size_t(f.rows) * size_t(p.c.D + 2)); });
  }
  const bool none = p.c.prefix_len == 0 && limit_of(p.causal, i, sg.seq.n, sg.seq.have) == 0;
  const float inv = 1.0f / a.l;
  if (lane >= p.c.D / 4) return;
  const size_t to = size_t(sg.seq.q0 + i) * size_t(p.os) + size_t(head) * size_t(p.c.D) + size_t(4 * lane);
  const float4 y = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                        : make_float4(a.y.x * inv, a.y.y * inv, a.y.z * inv, a.y.w * inv);
  if (p.out_e4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * y.x, 16.0f * y.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * y.z, 16.0f * y.w), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.o) + to) = lo | hi << 16;
  } else {
    __half2 h[2] = {__floats2half2_rn(y.x, y.y), __floats2half2_rn(y.z, y.w)};
    *reinterpret_cast<uint2*>(static_cast<__half*>(p.o) + to) = *reinterpret_cast<const uint2*>(h);
  }
}

// KI: 32-dimension groups of a key, VI: 64-dimension groups of a value; FULL: heads of just so many dimensions.
// NT: 8-row tiles of an item. PREFIX: all rows over the prefix, results left in parts; else the sequences' rows over their
// own tokens.
template <int KI, int VI, bool FULL, int NT, bool E4M3, bool PREFIX>
__global__ void __launch_bounds__(kThreads, per_sm(NT)) cached_few_kernel(const __grid_constant__ Params p) {
  constexpr int kRows = 8 * NT, kStep = step_keys(E4M3), kSub = kStep / 64;  // kSub: 16-key groups of a warp's step
  constexpr int kEs = E4M3 ? 1 : 2;
  constexpr int kOut = 64 * VI + 4;  // row pitch of the merge buffer (floats)
  static_assert(!FULL || 32 * KI == 64 * VI, "full heads");
  // A lane's runs of dimensions: 16 of a key (value) where four (eight) lanes then hold a whole head, else 8.
  constexpr bool kWideK = E4M3 && FULL, kWideV = kWideK && VI == 2;
  auto key_run = [](int k, int t) { return kWideK ? 64 * (k >> 1) + 16 * t + 8 * (k & 1) : 32 * k + 8 * t; };
  auto value_run = [](int k, int g) { return kWideV ? 16 * g + 8 * k : 64 * k + 8 * g; };
  __shared__ __align__(16) float red[4][kRows][kOut];
  __shared__ float red_m[4][kRows], red_l[4][kRows];
  __shared__ unsigned seen;
  __shared__ ShareState state[4];
  __shared__ Segment segment[4];  // of each warp, all the same
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  pdl_wait();
  const View& c = p.c;
  const int D = FULL ? 32 * KI : c.D;
  const int chunks = D / 8;
  const float sl2 = p.cap > 0.0f ? cap_factor(p.scale, p.cap) : kLog2e * p.scale;
  const int to_values = value_bytes(c), to_scales = scale_bytes(c), page_mask = (1 << c.shift) - 1;
  typename std::conditional<PREFIX, PrefixShare<kRows>, Share<kRows, kStep>>::type share(p, lane, state[warp]);

  Segment& sg = segment[warp];
  while (share.get(sg)) {
    const int rows_all = sg.seq.n * p.group;  // of the sequence (for this key head)
    // keys of this segment that one of its rows sees end here (the last row sees the most)
    int last = min(sg.s1 * kStep, sg.seq.have);
    if constexpr (!PREFIX)
      last = min(last, limit_of(p.causal, (min(sg.row0 + kRows, rows_all) - 1) / p.group, sg.seq.n, sg.seq.have));
    // and the keys that all of them see end here
    const int clear = PREFIX ? last : min(last, limit_of(p.causal, sg.row0 / p.group, sg.seq.n, sg.seq.have));

    // this lane's two rows of each tile as columns of S^T: visible keys
    int lim[NT][2];
    uint32_t q[NT][KI][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = sg.row0 + 8 * n + 2 * t + e;
        lim[n][e] = PREFIX || r >= rows_all ? last : min(last, limit_of(p.causal, r / p.group, sg.seq.n, sg.seq.have));
      }
      const int r = sg.row0 + 8 * n + g;  // Q^T: this lane's column
      const int i = r / p.group;
      const __half* qr = p.q + static_cast<long long>(sg.seq.q0 + i) * p.qs + (sg.kvh * p.group + r - i * p.group) * D;
#pragma unroll
      for (int k = 0; k < KI; ++k) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows_all && (FULL || 4 * k + t < chunks)) x = __ldg(reinterpret_cast<const uint4*>(qr + key_run(k, t)));
        q[n][k][0] = x.x, q[n][k][1] = x.y, q[n][k][2] = x.z, q[n][k][3] = x.w;
      }
    }

    // Pages of the segment's keys, a lane each: 32 from number first_page on, and the 32 behind them. (Looked up key by
    // key, a step's loads waited for L2 first: 107 us for one token of 16 requests over up to 32768 keys.)
    auto page_of = [&](int number) -> int {
      if (number >= (last + page_mask) >> c.shift) return 0;
      const int page = __ldg(sg.pages + number);
      if (unsigned(page) < unsigned(c.n_pages)) return page;
      atomicOr(c.err, kDevErrCache);
      return 0;
    };
    int first_page = (sg.s0 * kStep) >> c.shift;
    int here = page_of(first_page + lane), there = page_of(first_page + 32 + lane);
    const uint8_t* const head_at = c.pages + static_cast<long long>(sg.kvh << c.shift) * (D * kEs);
    const uint8_t* const scales_at = c.pages + to_scales + ((sg.kvh + (lane >> 4) * c.hk) << c.shift) + (lane & 15);
    Eight<E4M3> kx[kSub][2][KI], vx[kSub][4][VI];
    int scale[kSub];  // lane < 16: the byte of key lane, else of value lane - 16
    int page[kSub];   // of the keys that are loaded next
    auto load_k = [&](int key0) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int at = (key0 + 16 * u) & page_mask;
        const long long base = page[u] * c.page_bytes;
        const uint8_t* row = head_at + base + ((at + g) * D + key_run(0, t)) * kEs;
        const uint8_t* byte = scales_at + base + at;
        auto load = [&](auto live) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < KI; ++k) {
              const uint8_t* from = row + (8 * h * D + key_run(k, 0)) * kEs;
              if (kWideK && (k & 1)) continue;
              if (live(g + 8 * h) && (FULL || 4 * k + t < chunks)) {
                if constexpr (kWideK) load_two(kx[u][h][k], kx[u][h][k + 1 < KI ? k + 1 : 0], from);
                else kx[u][h][k].template load<FULL>(from);
              } else {
                kx[u][h][k].clear();
                if constexpr (kWideK) kx[u][h][k + 1 < KI ? k + 1 : 0].clear();
              }
            }
          scale[u] = live(lane & 15) ? __ldg(byte) : kNoScale;
        };
        const int left = last - (key0 + 16 * u);
        if (left >= 16) load([](int) { return true; });
        else load([&](int key) { return key < left; });
      }
    };
    auto load_v = [&](int key0) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const uint8_t* row = head_at + page[u] * c.page_bytes + to_values +
                             ((((key0 + 16 * u) & page_mask) + 2 * t) * D + value_run(0, g)) * kEs;
        auto load = [&](auto live) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int k = 0; k < VI; ++k) {
              const int key = (h & 1) + 8 * (h >> 1);
              const uint8_t* from = row + (key * D + value_run(k, 0)) * kEs;
              if (kWideV && (k & 1)) continue;
              if (live(2 * t + key) && (FULL || 8 * k + g < chunks)) {
                if constexpr (kWideV) load_two(vx[u][h][k], vx[u][h][k + 1 < VI ? k + 1 : 0], from);
                else vx[u][h][k].template load<FULL>(from);
              } else {
                vx[u][h][k].clear();
                if constexpr (kWideV) vx[u][h][k + 1 < VI ? k + 1 : 0].clear();
              }
            }
        };
        const int left = last - (key0 + 16 * u);
        if (left >= 16) load([](int) { return true; });
        else load([&](int key) { return key < left; });
      }
    };
    float o[NT][4 * VI][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 4 * VI; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    int key0 = sg.s0 * kStep + 16 * kSub * warp;
    auto look_up = [&](int key) {
      if ((key >> c.shift) - first_page >= 32) {
        first_page += 32;
        here = there;
        there = page_of(first_page + 32 + lane);
      }
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int n = ((key + 16 * u) >> c.shift) - first_page;
        page[u] = __shfl_sync(0xffffffffu, n < 32 ? here : there, n & 31);
      }
    };
    look_up(key0);
    load_k(key0);
    load_v(key0);
    for (; key0 < last; key0 += kStep) {
      float s[kSub][NT][4];
      int byte[kSub];
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        byte[u] = scale[u];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < KI; ++k) {
          uint4 a, b;  // eight dimensions of the keys g and g + 8
          if constexpr (E4M3) {
            a = e4m3_to_f16(kx[u][0][k].w);
            b = e4m3_to_f16(kx[u][1][k].w);
          } else {
            a = kx[u][0][k].w;
            b = kx[u][1][k].w;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(s[u][n], a.x, b.x, a.y, b.y, q[n][k][0], q[n][k][1]);
            mma16816(s[u][n], a.z, b.z, a.w, b.w, q[n][k][2], q[n][k][3]);
          }
        }
      }
      look_up(key0 + kStep);
      load_k(key0 + kStep);
      uint32_t b[kSub][NT][2];
      float up[kSub][2], back[kSub][2];  // of keys g and g + 8: ev, and what a probability counts in the denominator, 2^-ev
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kb = __shfl_sync(0xffffffffu, byte[u], g + 8 * h), vb = __shfl_sync(0xffffffffu, byte[u], 16 + g + 8 * h);
          // (a marked one counts NaN; 31 keeps the other bits a number)
          const float unit = max(kb, vb) == kMarked ? __uint_as_float(0x7fc00000u) : power_of(min(kb, 31));
          up[u][h] = float(min(vb, 31) - kNoScale);
          back[u][h] = reciprocal_of(min(vb, 31));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[u][n][2 * h] *= unit;
            s[u][n][2 * h + 1] *= unit;
          }
        }
      if (p.cap > 0.0f) {
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = s[u][n][e] * sl2, big = capped(y, p.cap * kLog2e);
              s[u][n][e] = (p.cap < kFarCap ? big : far_capped(s[u][n][e] * (kLog2e * p.scale), y, big)) + up[u][e >> 1];
            }
      } else {
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][n][e] = fmaf(s[u][n][e], sl2, up[u][e >> 1]);
      }
      if (key0 + 16 * kSub > clear)
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)  // e & 1: the row, e >> 1: keys g, g + 8
              if (key0 + 16 * u + g + 8 * (e >> 1) >= lim[n][e & 1]) s[u][n][e] = -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[2];
        bool raise = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[0][n][e], s[0][n][e + 2]);
          if constexpr (kSub == 2) mx = fmax3(mx, s[kSub - 1][n][e], s[kSub - 1][n][e + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const bool higher = mx > m[n][e] + kSlack;
          const float mn = higher ? mx - kHead : m[n][e];
          f[e] = higher ? ex2(m[n][e] - mn) : 1.0f;
          m[n][e] = mn;
          raise |= higher;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int j = 0; j < 4 * VI; ++j) {
            o[n][j][0] *= f[0];
            o[n][j][1] *= f[1];
            o[n][j][2] *= f[0];
            o[n][j][3] *= f[1];
          }
          l[n][0] *= f[0];
          l[n][1] *= f[1];
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[n][e] == -INFINITY ? 0.0f : m[n][e];
            s[u][n][e] = ex2(s[u][n][e] - ref);
            s[u][n][e + 2] = ex2(s[u][n][e + 2] - ref);
            l[n][e] = fmaf(s[u][n][e], back[u][0], fmaf(s[u][n][e + 2], back[u][1], l[n][e]));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // (F16, what the products take: 2^-11 of each probability; their sum l is of the unrounded ones)
            const __half2 w = __floats2half2_rn(s[u][n][2 * h], s[u][n][2 * h + 1]);
            b[u][n][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&w));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int k = 0; k < VI; ++k) {
          uint32_t a[4][4];  // [dimensions 2 j and 2 j + 1 of this lane's eight][operand register]
          if constexpr (E4M3) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {  // keys 2 t and 2 t + 1, then 2 t + 8 and 2 t + 9
              const uint2 w0 = vx[u][2 * hh][k].w, w1 = vx[u][2 * hh + 1][k].w;
              two_pairs(__byte_perm(w0.x, w1.x, 0x5140), a[0][2 * hh], a[0][2 * hh + 1]);
              two_pairs(__byte_perm(w0.x, w1.x, 0x7362), a[1][2 * hh], a[1][2 * hh + 1]);
              two_pairs(__byte_perm(w0.y, w1.y, 0x5140), a[2][2 * hh], a[2][2 * hh + 1]);
              two_pairs(__byte_perm(w0.y, w1.y, 0x7362), a[3][2 * hh], a[3][2 * hh + 1]);
            }
          } else {
            const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vx[u][0][k].w);
            const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vx[u][1][k].w);
            const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vx[u][2][k].w);
            const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vx[u][3][k].w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a[j][0] = __byte_perm(v0[j], v1[j], 0x5410), a[j][1] = __byte_perm(v0[j], v1[j], 0x7632);
              a[j][2] = __byte_perm(v2[j], v3[j], 0x5410), a[j][3] = __byte_perm(v2[j], v3[j], 0x7632);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(o[n][4 * k + j], a[j][0], a[j][1], a[j][2], a[j][3], b[u][n][0], b[u][n][1]);
        }
      load_v(key0 + kStep);
    }

    // the four warps' sums, brought to one exponent
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[n][e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (g == 0) {
          red_m[warp][8 * n + 2 * t + e] = m[n][e];
          red_l[warp][8 * n + 2 * t + e] = y;
        }
      }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4 * VI; j += 2)  // four neighbouring dimensions of a row
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(&red[warp][8 * n + 2 * t + e][value_run(j >> 2, g) + 2 * (j & 3)]) =
              make_float4(o[n][j][e], o[n][j][e + 2], o[n][j + 1][e], o[n][j + 1][e + 2]);
    __syncthreads();
    const int rows = min(kRows, rows_all - sg.row0);
    auto sums_of = [&](int r) {  // of row r, four columns a lane
      RowSums a = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, 0.0f};
#pragma unroll
      for (int w = 0; w < 4; ++w)
        a.add(*reinterpret_cast<const float4*>(&red[w][r][4 * min(lane, 16 * VI - 1)]), red_m[w][r], red_l[w][r]);
      return a;
    };
    auto put_part = [&](float* part, int r, const RowSums& a) {
      if (lane < c.D / 4) __stcg(reinterpret_cast<float4*>(part + size_t(r) * c.D) + lane, a.y);
      if (lane == 0) __stcg(reinterpret_cast<float2*>(part + size_t(kRows) * c.D) + r, make_float2(a.m, a.l));
    };
    const size_t part_size = size_t(kRows) * size_t(c.D + 2);
    if constexpr (PREFIX) {
      float* part = p.pre.base + size_t(sg.item + blockIdx.x) * part_size;
      for (int r = warp; r < rows; r += 4) put_part(part, r, sums_of(r));
      __syncthreads();  // the merge buffers are free again
    } else {
      if (sg.s0 == 0 && sg.s1 == sg.steps) {
        for (int r = warp; r < rows; r += 4) finish_row(p, sg, r, lane, sums_of(r));
        __syncthreads();
        continue;
      }
      auto part_of = [&](int cta, int end) { return p.partial + (size_t(cta) * 2 + end) * part_size; };
      float* mine = part_of(int(blockIdx.x), sg.s0 == 0 ? 1 : 0);
      for (int r = warp; r < rows; r += 4) put_part(mine, r, sums_of(r));
      // the last CTA of the item's parts joins them, in order
      const int c0 = share.cta_of(sg.base), c1 = share.cta_of(sg.base + sg.steps - 1);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) seen = atomicInc(p.counters + c0, unsigned(c1 - c0));  // 0 .. c1 - c0, then 0 again
      __syncthreads();
      if (seen == unsigned(c1 - c0)) {
        __threadfence();
        for (int r = warp; r < rows; r += 4) {
          RowSums a = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, 0.0f};
          a.add_parts(c1 - c0 + 1, r, kRows, c.D, lane, [&](int w) { return part_of(c0 + w, w == 0 ? 1 : 0); });
          finish_row(p, sg, r, lane, a);
        }
      }
      __syncthreads();  // `seen` and the merge buffers are free again
    }
  }
}

template <int KI, int VI, bool FULL, int NT, bool PREFIX>
cudaError_t few_launch_as(const Params& p, int grid, cudaStream_t s) {
  return launch_pdl(p.c.e4m3 ? cached_few_kernel<KI, VI, FULL, NT, true, PREFIX>
                             : cached_few_kernel<KI, VI, FULL, NT, false, PREFIX>,
                    dim3(unsigned(grid)), dim3(kThreads), 0, s, p);
}

template <int NT, bool PREFIX>
cudaError_t few_launch(const Params& p, int grid, cudaStream_t s) {
  if (p.c.D == 64) return few_launch_as<2, 1, true, NT, PREFIX>(p, grid, s);
  if (p.c.D == 128) return few_launch_as<4, 2, true, NT, PREFIX>(p, grid, s);
  if (p.c.D < 64) return few_launch_as<2, 1, false, NT, PREFIX>(p, grid, s);
  if (p.c.D <= 96) return few_launch_as<3, 2, false, NT, PREFIX>(p, grid, s);
  return few_launch_as<4, 2, false, NT, PREFIX>(p, grid, s);
}

// What the host alone decides of a call.
struct Plan {
  int nt, grid;          // the sequences' pass: 8-row tiles of an item, CTAs at most
  int pre_nt, pre_grid;  // the prefix's
  PrefixParts pre;       // (its base is an offset in floats)
  size_t bytes;          // workspace
};
Plan plan_of(const View& c, int total_q, int group, int sms) {
  Plan r = {};
  const long long rows = static_cast<long long>(total_q) * group;  // of a key head
  r.nt = rows <= 8ll * c.count ? 1 : 2;
  r.grid = sms * per_sm(r.nt);
  const size_t own = size_t(kMaxSms * per_sm(r.nt)) * 2 * size_t(8 * r.nt) * size_t(c.D + 2);
  r.bytes = kCounterBytes + own * sizeof(float);
  if (c.prefix_len > 0) {
    r.pre_nt = rows <= 8 ? 1 : 2;
    r.pre.rows = 8 * r.pre_nt;
    r.pre.blocks = int((rows + r.pre.rows - 1) / r.pre.rows);
    const int step = step_keys(c.e4m3);
    r.pre.steps = (c.prefix_len + step - 1) / step;
    const long long items = static_cast<long long>(r.pre.blocks) * c.hk, work = items * r.pre.steps;
    const int most = sms * per_sm(r.pre_nt);
    r.pre.chunk = (work + most - 1) / most;
    r.pre_grid = int((work + r.pre.chunk - 1) / r.pre.chunk);
    r.bytes += size_t(items + kMaxSms * per_sm(r.pre_nt)) * size_t(r.pre.rows) * size_t(c.D + 2) * sizeof(float);
  }
  return r;
}
constexpr long long kMostRows = 1ll << 26;  // of a call: query rows times heads (see check)

sv_status check(const char* fn, const sv_cache* cache, const sv_cache_batch* batch, const int* q_offsets, int total_q,
                int q_heads, View* c) {
  const sv_status st = make_view(fn, cache, batch, q_offsets, total_q, c);
  if (st != SV_OK) return st;
  if (q_heads < 1 || q_heads % c->hk) {
    set_error("%s: %d query heads over %d key heads", fn, q_heads, c->hk);
    return SV_ERR_INVALID_ARG;
  }
  if (q_heads / c->hk > 64 || q_heads > 65536 || c->count > (1 << 24) ||
      static_cast<long long>(total_q) * q_heads > kMostRows) {
    set_error("%s: heads %d over %d, %d sequences or %d queries are too many for one call", fn, q_heads, c->hk, c->count,
              total_q);
    return SV_ERR_UNSUPPORTED;
  }
  return SV_OK;
}

}  // namespace
}  // namespace cached
}  // namespace sv

extern "C" {

size_t sv_attention_cached_workspace(const sv_cache* cache, const sv_cache_batch* batch, int total_q, int q_heads) {
  using namespace sv::cached;
  View c = {};
  static const int none = 0;  // (any offsets)
  if (check("sv_attention_cached_workspace", cache, batch, &none, total_q, q_heads, &c) != SV_OK) return 0;
  if (total_q == 0) return 0;
  return plan_of(c, total_q, q_heads / c.hk, kMaxSms).bytes;
}

sv_status sv_attention_cached(const sv_cache* cache, const sv_cache_batch* batch, const void* q, void* o,
                              const int* q_offsets, int total_q, int q_heads, long long q_stride, long long o_stride,
                              const sv_attention_options* options, int out_dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  using namespace sv;
  using namespace sv::cached;
  const char* fn = "sv_attention_cached";
  Params p = {};
  sv_status st = check(fn, cache, batch, q_offsets, total_q, q_heads, &p.c);
  if (st != SV_OK) return st;
  const long long row = static_cast<long long>(q_heads) * p.c.D;
  p.qs = q_stride ? q_stride : row;
  p.os = o_stride ? o_stride : row;
  if (p.qs < row || p.os < row || (p.qs | p.os) % 8) {
    set_error("%s: row strides must be multiples of 8 that cover a row (q %lld, o %lld)", fn, p.qs, p.os);
    return SV_ERR_INVALID_ARG;
  }
  if (out_dtype != SV_DT_F16 && out_dtype != SV_DT_E4M3) {
    set_error("%s: bad out_dtype %d", fn, out_dtype);
    return SV_ERR_INVALID_ARG;
  }
  sv_attention_options opt = {};
  if (options) opt = *options;
  if ((opt.mask != SV_MASK_DOCUMENT && opt.mask != SV_MASK_PREFIX) || !(opt.softcap >= 0.0f) ||
      !std::isfinite(opt.softcap) || !std::isfinite(opt.scale)) {
    set_error("%s: bad options (mask %d, softcap %g, scale %g)", fn, opt.mask, double(opt.softcap), double(opt.scale));
    return SV_ERR_INVALID_ARG;
  }
  if (opt.prefix || opt.slopes) {
    set_error("%s: the options' prefix and slopes are not supported here", fn);
    return SV_ERR_UNSUPPORTED;
  }
  if ((total_q && (!q || !o)) ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(workspace)) & 15)) {
    set_error("%s: q, o and workspace must be 16-byte aligned pointers", fn);
    return SV_ERR_INVALID_ARG;
  }
  const size_t need = sv_attention_cached_workspace(cache, batch, total_q, q_heads);
  if (need && (!workspace || workspace_bytes < need)) {
    set_error("%s: the workspace has %zu bytes, fewer than sv_attention_cached_workspace() = %zu", fn,
              workspace ? workspace_bytes : size_t(0), need);
    return SV_ERR_INVALID_ARG;
  }
  if (total_q == 0) return SV_OK;
  st = ensure_runtime();
  if (st != SV_OK) return st;
  p.c.err = dev_err();
  p.q = static_cast<const __half*>(q);
  p.o = o;
  p.q_off = q_offsets;
  p.total_q = total_q;
  p.hq = q_heads;
  p.group = q_heads / p.c.hk;
  p.scale = opt.scale > 0.0f ? opt.scale : 1.0f / std::sqrt(float(p.c.D));
  p.cap = opt.softcap;
  p.causal = opt.mask == SV_MASK_PREFIX;
  p.out_e4m3 = out_dtype == SV_DT_E4M3;
  const Plan plan = plan_of(p.c, total_q, p.group, num_sms() < kMaxSms ? num_sms() : kMaxSms);
  p.counters = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  p.pre = plan.pre;
  p.pre.base = p.partial + size_t(kMaxSms * per_sm(plan.nt)) * 2 * size_t(8 * plan.nt) * size_t(p.c.D + 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (p.c.prefix_len > 0) {
    LaunchScope L(kKindAttn, 0.0, 0.0, s);
    e = plan.pre_nt == 1 ? few_launch<1, true>(p, plan.pre_grid, s) : few_launch<2, true>(p, plan.pre_grid, s);
  }
  if (e == cudaSuccess) {
    LaunchScope L(kKindAttn, 0.0, 0.0, s);
    e = plan.nt == 1 ? few_launch<1, false>(p, plan.grid, s) : few_launch<2, false>(p, plan.grid, s);
  }
  return e == cudaSuccess ? SV_OK : cuda_fail(e, fn);
}

}  // extern "C"
