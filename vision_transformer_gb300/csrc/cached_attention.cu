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
// Two passes where there is a prefix: first all rows of the batch over its keys (blocks of 8 or 16 rows here, more in
// cached_tiles.cu), sums, exponents and denominators to the workspace; then every sequence's rows over its own tokens,
// which finish with the prefix's parts. Without a prefix the second alone. Sequences of more than 32 rows on average go
// through cached_tiles.cu too, and cached_join_kernel puts their parts together. The second pass here needs the first
// only where it finishes rows: it begins while the first still runs (256 samples behind 32768 keys: 189 us to 176).
//
// Bound: DRAM, every key and value read once for up to 8 or 16 rows. The arithmetic runs on warp-level matrix
// instructions (mma.sync m16n8k16, F32 accumulation): few rows fill no tcgen05 tile, and codes go from global memory to
// the registers of the instruction with a conversion between them (E4M3 to F16 in pairs, 64 a cycle and SM):
//   S^T = K Q^T: 16 keys x 8 rows. A lane's 8 neighbouring dimensions of a key serve as its operand values of two
//     instructions (the order of the summed dimensions is free); four lanes read 32 of them.
//   O^T += V^T P^T: 16 dimensions x 8 rows. Eight lanes read 64 neighbouring dimensions of a value, a lane has the same
//     8 of the keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; the bytes of two keys are interleaved before the conversion, which
//     so gives pairs of keys. P^T goes from the accumulator's layout to the operand's by a transposing 8 x 8 move.
// A warp takes 16 to 64 keys at a time (by the bytes of a key), the registers of K loaded again as soon as S^T is done,
// those of V as soon as O^T is: these hold what is in flight. 16 keys lie in one page.
//
// Work: the (sequence, key head, block of rows) items are laid out one behind another in steps of a warp, and every warp
// takes an equal, contiguous share of the steps, so that any distribution of lengths fills the GPU and the items of
// short sequences run side by side, a warp each. An item inside one share is finished there; the parts of others go to
// shared memory, where the CTA's warps join them when all are through, and the parts of items that are cut between CTAs
// to the workspace, where the last CTA of an item joins them in order.
//
// One token of 16 sequences of 900 to 32768 tokens, 32 heads of 128 over 8, E4M3 (490 MB): 87 us, 85% of the copy
// bandwidth. Short calls are a chain of latencies: shares 2,000 cycles, segment 2,000, a step 3,000, parts 1,500, fence and
// counter 2,000, the join 3,000 (4 sequences of up to 700 tokens: 11.9 us).
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
constexpr int kWarps = kThreads / 32;
// Keys that an accumulator sums up at most. The tensor cores add by truncation: the sums of 16384 keys lose 1e-4 (those of a
// million lost 6.6e-3); a warp's part in shared memory takes them in F32.
constexpr int kMostKeys = 16384;
// 16-key groups of a warp's step: what the registers of a key and a value in flight hold
constexpr int groups_of(bool e4m3, int head_dim) { return (e4m3 ? 2 : 1) * (head_dim > 64 ? 1 : 2); }

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

// Eight stored numbers in the registers that they are loaded into, and left as they were where `live` is false: what is
// there then are other stored numbers, or zeros, which are finite. ALONE: no other access needs the sectors that this
// one touches (they are not kept in L1).
template <bool E4M3>
struct Eight;
template <>
struct Eight<true> {
  uint2 w;
  template <bool ALONE>
  __device__ __forceinline__ void load(const uint8_t* p, bool live) {
    if constexpr (ALONE) {
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
                   : "+r"(w.x), "+r"(w.y)
                   : "l"(p), "r"(uint32_t(live)));
    } else {
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
                   : "+r"(w.x), "+r"(w.y)
                   : "l"(p), "r"(uint32_t(live)));
    }
  }
  __device__ __forceinline__ void clear() { w = make_uint2(0u, 0u); }
};
template <>
struct Eight<false> {
  uint4 w;
  template <bool ALONE>
  __device__ __forceinline__ void load(const uint8_t* p, bool live) {
    if constexpr (ALONE) {
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
          : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)
          : "l"(p), "r"(uint32_t(live)));
    } else {
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                   : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)
                   : "l"(p), "r"(uint32_t(live)));
    }
  }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
};

// Sixteen E4M3 codes in one access.
__device__ __forceinline__ void load_two(Eight<true>& a, Eight<true>& b, const uint8_t* p, bool live) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
               : "+r"(a.w.x), "+r"(a.w.y), "+r"(b.w.x), "+r"(b.w.y)
               : "l"(p), "r"(uint32_t(live)));
}
[[maybe_unused]] __device__ __forceinline__ void load_two(Eight<false>&, Eight<false>&, const uint8_t*, bool) {}

// byte - 16 as a number, 2^(byte - 16) and its reciprocal, for bytes of factors.
__device__ __forceinline__ float exponent_of(int byte) {  // (2^23 + byte, less 2^23 + 16)
  return __uint_as_float(0x4b000000u | uint32_t(byte)) - float((1 << 23) + kNoScale);
}
__device__ __forceinline__ float power_of(int byte) { return __uint_as_float(uint32_t(byte + (127 - kNoScale)) << 23); }
__device__ __forceinline__ float reciprocal_of(int byte) {
  return __uint_as_float(uint32_t(127 + kNoScale - byte) << 23);
}

// A run of steps of one item that falls into a warp's share. (Steps are counted in 32 bits: the host has seen to that.)
struct Segment {
  Sequence seq;
  const int* pages;   // of its keys
  int kvh, row0;      // key head, first of the item's rows (query x group + head) in the sequence
  int s0, s1, steps;  // steps of the item: this segment's, all
  int at;             // first of the present piece's, kMostKeys keys of the segment
  int base;           // place of the item's first step among all steps
  int item;           // prefix pass: its number; else that of the sequence
};

// A warp's share of the steps. The items of the sequences in order: sequences, key heads, blocks of rows. 32 sequences at
// a time, one per lane, with their steps summed by shuffles; every warp works it out for itself. What it knows lies in
// shared memory (`st`, the warp's own): in registers it was in the way of the keys in flight.
struct ShareState {
  int incl[32];  // steps of the sequences up to this one
  Sequence seq[32];
  int blocks[32], steps[32];
  int chunk, at, end, base, total;
  int d0, count;
};
struct ShareTotals {  // of the CTA's warps together
  int part[32];       // steps of the sequences, 32 and 32
  unsigned work[kWarps];
  int bad[kWarps];
};
template <int ROWS, int STEP>
class Share {
 public:
  __device__ __forceinline__ Share(const Params& p, int warp, int lane, ShareState& st, ShareTotals& all)
      : p_(p), lane_(lane), st_(st) {
    int count = p.c.count;
    unsigned work;
    bool bad;
    Sequence q;
    int blocks, steps;
    if (count <= 32) {
      bad = !load(0, count, q, blocks, steps);
      work = __reduce_add_sync(0xffffffffu, unsigned(blocks * p.c.hk * steps));
      bad = __any_sync(0xffffffffu, bad);
    } else {  // the CTA's warps share them out
      work = 0;
      bad = false;
      for (int d0 = 32 * warp; d0 < count; d0 += 32 * kWarps) {
        bad |= !load(d0, count, q, blocks, steps);
        const unsigned some = __reduce_add_sync(0xffffffffu, unsigned(blocks * p.c.hk * steps));
        if (lane == 0 && d0 < 32 * 32) all.part[d0 / 32] = int(some);
        work += some;
      }
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) {
        all.work[warp] = work;
        all.bad[warp] = bad;
      }
      __syncthreads();
      work = all.work[0] + all.work[1] + all.work[2] + all.work[3];
      bad = all.bad[0] | all.bad[1] | all.bad[2] | all.bad[3];
      static_assert(kWarps == 4, "sums of four");
    }
    // bad offsets or lengths: reported, and nothing is computed
    if (bad) {
      if (lane == 0) atomicOr(p.c.err, kDevErrCache);
      count = 0;
      work = 0;
    }
    const unsigned warps = gridDim.x * kWarps, chunk = max(1u, (work + warps - 1) / warps);
    const int at = int(min(chunk * (blockIdx.x * kWarps + warp), work));  // (a share may begin behind the last step)
    // the 32 sequences that the share begins in; the first ones where there are more than 32 times 32
    int d0 = 0, base = 0;
    if (count > 32 && count <= 32 * 32) {
      const int mine = 32 * lane < count ? all.part[lane] : 0;
      int incl = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += a;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, incl > at);
      if (behind) {
        const int src = __ffs(int(behind)) - 1;
        d0 = 32 * src;
        base = __shfl_sync(0xffffffffu, incl - mine, src);
      }
    }
    if (lane == 0) {
      st_.chunk = int(chunk);
      st_.at = at;
      st_.end = int(min(unsigned(at) + chunk, work));
      st_.base = base;
      st_.count = count;
    }
    if (p.c.count > 32 || count == 0) load(d0, count, q, blocks, steps);
    open(d0, q, blocks, steps);
  }
  // The next segment of the share.
  __device__ __forceinline__ bool get(Segment& r) {
    const int at = st_.at;
    if (at >= st_.end) return false;
    while (at >= st_.base + st_.total) {
      __syncwarp();
      if (lane_ == 0) st_.base += st_.total;
      __syncwarp();
      Sequence q;
      int blocks, steps;
      const int d0 = st_.d0 + 32;
      load(d0, st_.count, q, blocks, steps);
      open(d0, q, blocks, steps);
    }
    const int base = st_.base;
    const int src = __ffs(__ballot_sync(0xffffffffu, base + st_.incl[lane_] > at)) - 1;
    const unsigned steps = unsigned(st_.steps[src]), blocks = unsigned(st_.blocks[src]);
    const int first = base + st_.incl[src] - int(blocks * unsigned(p_.c.hk) * steps);
    const unsigned item = unsigned(at - first) / steps;
    Segment x;
    x.seq = st_.seq[src];
    x.pages = p_.c.table + static_cast<long long>(st_.d0 + src) * p_.c.stride;
    x.steps = int(steps);
    x.base = first + int(item * steps);
    x.kvh = blocks == 1 ? int(item) : int(item / blocks);
    x.row0 = int(item - unsigned(x.kvh) * blocks) * ROWS;
    x.s0 = at - x.base;
    x.s1 = min(st_.end - x.base, x.steps);
    x.at = x.s0;
    x.item = st_.d0 + src;
    __syncwarp();
    if (lane_ == 0) {
      st_.at = x.base + x.s1;
      r = x;
    }
    __syncwarp();
    return true;
  }

 private:
  __device__ __forceinline__ bool load(int d0, int count, Sequence& q, int& blocks, int& steps) {
    const bool good = sequence(p_, d0 + lane_, count, q);
    blocks = (q.n * p_.group + ROWS - 1) / ROWS;
    steps = 1;
    if constexpr (STEP > 0) steps = max(1, (q.have + STEP - 1) / STEP);  // (one without keys writes the prefix's result, or zeros)
    return good;
  }
  __device__ __forceinline__ void open(int d0, const Sequence& q, int blocks, int steps) {
    __syncwarp();
    int incl = blocks * p_.c.hk * steps;
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, incl, o);
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
  __device__ __forceinline__ PrefixShare(const Params& p, int warp, int lane, ShareState& st, ShareTotals&) : p_(p), lane_(lane), st_(st) {
    const int work = p.pre.blocks * p.c.hk * p.pre.steps, chunk = p.pre.chunk / kWarps;
    if (lane == 0) {
      st_.at = min(chunk * (int(blockIdx.x) * kWarps + warp), work);
      st_.end = min(st_.at + chunk, work);
    }
    __syncwarp();
  }
  __device__ __forceinline__ bool get(Segment& r) {
    const int at = st_.at, end = st_.end;
    if (at >= end) return false;
    Segment x;
    x.item = at / p_.pre.steps;
    x.seq = {0, p_.total_q, p_.c.prefix_len};
    x.pages = p_.c.prefix_pages;
    x.kvh = x.item / p_.pre.blocks;
    x.row0 = (x.item - x.kvh * p_.pre.blocks) * ROWS;
    x.steps = p_.pre.steps;
    x.base = x.item * p_.pre.steps;
    x.s0 = at - x.base;
    x.s1 = min(end - x.base, x.steps);
    x.at = x.s0;
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

// Parts of a row's sums: part 0 at `first`, the others at `rest` and every `stride` floats on; a part has rows of `pitch`
// floats, and behind `ml` floats exponent and denominator of each. In shared memory (few parts, joined one by one) or in
// the workspace. (One form for both, by generic addresses, took 1,800 cycles for two parts in shared memory.)
struct Source {
  const float *first, *rest;
  int stride, n, pitch, ml;
  bool shared;
};

__device__ __forceinline__ float4 read_shared4(uint32_t at) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ float2 read_shared2(uint32_t at) {
  float2 r;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(at) : "memory");
  return r;
}

// A pair in F16, at most its largest number: a mean of stored numbers is within them, and what the probabilities' rounding
// puts above 65504 (2^-11 of it) is not an infinity. NaN stays.
__device__ __forceinline__ uint32_t f16_within(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Rows r, r + step, ... (up to four, `rows` of them) of an item, by one warp: the parts of their own keys' sums joined, and
// with the prefix's parts written in the output's type, or (put) kept as one part of part_rows rows. Eight lanes a row, 16
// columns each; with fewer rows the lanes share out the parts. Four parts are on their way at a time: they come from L2,
// and nothing else hides its latency. One function for all of the kernel's ends: its code, run once an item, comes from
// beyond the instruction caches.
__device__ __noinline__ void settle(const Params& p, const Segment& sg, const Source own, int r, int step, int rows, float* put,
                                    int part_rows) {
  constexpr int kBatch = 4;
  if (rows <= 0) return;
  const int lane = int(threadIdx.x) & 31, D = p.c.D;
  const int share = rows > 2 ? 4 : rows;  // rows at a time: 1, 2 or 4
  const int k = (lane >> 3) & (share - 1), every = 4 / share, turn = (lane >> 3) / share;
  const bool live = k < rows;
  const int in_item = r + (live ? k : 0) * step, row = sg.row0 + in_item;  // of the item, of the sequence (for this key head)
  float4 y[4];
  float m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < 4; ++c) y[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto column = [&](int c) { return min((lane & 7) + 8 * c, D / 4 - 1) * 4; };

  auto scale = [&](float f) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mul_x2(y[c].x, y[c].y, y[c].x, y[c].y, f, f);
      mul_x2(y[c].z, y[c].w, y[c].z, y[c].w, f, f);
    }
    l *= f;
  };
  auto add = [&](const float4 (&v)[4], float lv, float f) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      fma_x2(y[c].x, y[c].y, v[c].x, v[c].y, f, f, y[c].x, y[c].y);
      fma_x2(y[c].z, y[c].w, v[c].z, v[c].w, f, f, y[c].z, y[c].w);
    }
    l = fmaf(f, lv, l);
  };
  Source from = own;
  int at = in_item;
  if (own.shared) {
#pragma unroll 1
    for (int w = turn; w < own.n; w += every) {
      const uint32_t part = smem_u32(w == 0 ? own.first : own.rest + (w - 1) * own.stride);
      const float2 e = read_shared2(part + 4u * uint32_t(own.ml + 2 * at));
      float4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = read_shared4(part + 4u * uint32_t(at * own.pitch + column(c)));
      const float up = fmaxf(m, e.x), ref = up == -INFINITY ? 0.0f : up;
      scale(ex2(m - ref));
      m = up;
      add(v, e.y, ex2(e.x - ref));
    }
  }
#pragma unroll 1
  for (int pass = own.shared; pass < 2; ++pass) {
    if (pass == 1) {
      if (put || p.c.prefix_len == 0) break;
      const PrefixParts& f = p.pre;
      const unsigned all = unsigned(sg.seq.q0 * p.group + row), block = all / unsigned(f.rows);
      const unsigned item = unsigned(sg.kvh * f.blocks) + block, begin = item * unsigned(f.steps), c0 = begin / unsigned(f.chunk);
      from.stride = f.rows * (D + 2);
      from.first = f.base + size_t(item + c0) * size_t(from.stride);
      from.rest = from.first + from.stride;
      from.n = int((begin + unsigned(f.steps) - 1) / unsigned(f.chunk) - c0) + 1;
      from.pitch = D;
      from.ml = f.rows * D;
      at = int(all - block * unsigned(f.rows));
    }
#pragma unroll 1
    for (int w0 = turn; w0 < from.n; w0 += kBatch * every) {
      float4 v[kBatch][4];
      float2 e[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int w = w0 + b * every;
        e[b] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[b][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (w < from.n) {
          const float* part = w == 0 ? from.first : from.rest + (w - 1) * static_cast<long long>(from.stride);
          e[b] = __ldcg(reinterpret_cast<const float2*>(part + from.ml + 2 * at));
#pragma unroll
          for (int c = 0; c < 4; ++c) v[b][c] = __ldcg(reinterpret_cast<const float4*>(part + at * from.pitch + column(c)));
        }
      }
      float up = m;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) up = fmaxf(up, e[b].x);
      const float ref = up == -INFINITY ? 0.0f : up;
      scale(ex2(m - ref));
      m = up;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) add(v[b], e[b].y, ex2(e[b].x - ref));
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int o = 8 * share; o < 32; o <<= 1) {  // the lanes that have shared out the parts of a row
    const float mo = __shfl_xor_sync(0xffffffffu, m, o), lo = __shfl_xor_sync(0xffffffffu, l, o);
    const float up = fmaxf(m, mo), ref = up == -INFINITY ? 0.0f : up, fa = ex2(m - ref), fb = ex2(mo - ref);
    m = up;
    l = fa * l + fb * lo;  // (both lanes: the same two products)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float* x = reinterpret_cast<float*>(&y[c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fa * x[e] + fb * __shfl_xor_sync(0xffffffffu, x[e], o);
    }
  }
  if (!live || turn) return;
  if (put) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if ((lane & 7) + 8 * c < D / 4) __stcg(reinterpret_cast<float4*>(put + size_t(in_item) * D + column(c)), y[c]);
    if ((lane & 7) == 0) __stcg(reinterpret_cast<float2*>(put + size_t(part_rows) * D) + in_item, make_float2(m, l));
    return;
  }
  const int i = query_of(p, row), head = sg.kvh * p.group + (row - i * p.group);
  const bool none = p.c.prefix_len == 0 && limit_of(p.causal, i, sg.seq.n, sg.seq.have) == 0;
  const float inv = 1.0f / l;
  const size_t to = size_t(sg.seq.q0 + i) * size_t(p.os) + size_t(head) * size_t(D);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if ((lane & 7) + 8 * c >= D / 4) continue;
    const float4 z = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                          : make_float4(y[c].x * inv, y[c].y * inv, y[c].z * inv, y[c].w * inv);
    if (p.out_e4m3) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * z.x, 16.0f * z.y), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(16.0f * z.z, 16.0f * z.w), __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.o) + to + column(c)) = lo | hi << 16;
    } else {
      *reinterpret_cast<uint2*>(static_cast<__half*>(p.o) + to + column(c)) =
          make_uint2(f16_within(z.x, z.y), f16_within(z.z, z.w));
    }
  }
}

// A warp's part of an item.
template <int ROWS, int VI>
struct Part {
  float y[ROWS][64 * VI + 4];
  float2 ml[ROWS];
};
template <int ROWS, int VI>
struct FewShared {
  Part<ROWS, VI> part[kWarps][2];  // of the item cut at the start of the warp's share, at its end (and whole items, in turn)
  Segment cut[kWarps][2];          // these items; no steps: none
  Segment segment[kWarps];         // the warp's present one
  ShareState state[kWarps];
  ShareTotals totals;
  Params p;  // for settle(): the parameters' own place is far from a function that is not inlined
  unsigned seen[2];
};

// KI: 32-dimension groups of a key, VI: 64-dimension groups of a value; FULL: heads of just so many dimensions.
// NT: 8-row tiles of an item. PREFIX: all rows over the prefix, results left in parts; else the sequences' rows over their
// own tokens.
template <int KI, int VI, bool FULL, int NT, bool E4M3, bool PREFIX>
__global__ void __launch_bounds__(kThreads, per_sm(NT)) cached_few_kernel(const __grid_constant__ Params p) {
  constexpr int kRows = 8 * NT, kSub = groups_of(E4M3, 32 * KI), kStep = 16 * kSub;
  constexpr int kEs = E4M3 ? 1 : 2;
  using Mem = FewShared<kRows, VI>;
  static_assert(!FULL || 32 * KI == 64 * VI, "full heads");
  // A lane's runs of dimensions: 16 of a key (value) where four (eight) lanes then hold a whole head, else 8.
  constexpr bool kWideK = E4M3 && FULL, kWideV = kWideK && VI == 2;
  auto key_run = [](int k, int t) { return kWideK ? 64 * (k >> 1) + 16 * t + 8 * (k & 1) : 32 * k + 8 * t; };
  auto value_run = [](int k, int g) { return kWideV ? 16 * g + 8 * k : 64 * k + 8 * g; };
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Mem& mem = *reinterpret_cast<Mem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // Behind the prefix pass this kernel may begin before that one has ended, and needs nothing of it until its rows are
  // joined; what the calls before have written (queries, cache, lengths) is in place, since the prefix pass lets others
  // begin only after its own wait for them. Until the next wait nothing in global memory is written.
  if (PREFIX || p.c.prefix_len == 0) pdl_wait();
  pdl_launch_dependents();
  const View& c = p.c;
  const int D = FULL ? 32 * KI : c.D;
  const int chunks = D / 8;
  const float sl2 = p.cap > 0.0f ? cap_factor(p.scale, p.cap) : kLog2e * p.scale;
  const int to_values = value_bytes(c), to_scales = scale_bytes(c), page_mask = (1 << c.shift) - 1;
  typename std::conditional<PREFIX, PrefixShare<kRows>, Share<kRows, kStep>>::type share(p, warp, lane, mem.state[warp], mem.totals);
  if (lane < 2) mem.cut[warp][lane].steps = 0;  // (none)
  if (threadIdx.x < sizeof(Params) / 4) reinterpret_cast<int*>(&mem.p)[threadIdx.x] = reinterpret_cast<const int*>(&p)[threadIdx.x];
  static_assert(sizeof(Params) % 4 == 0 && sizeof(Params) / 4 <= kThreads, "a thread a word");
  __syncthreads();

  // parts in the workspace, and of the warps from `part` on
  auto kept_at = [&](int part) { return (PREFIX ? p.pre.base : p.partial) + size_t(part) * (size_t(kRows) * size_t(D + 2)); };
  auto shared_source = [](const Part<kRows, VI>* part, int n) -> Source {
    constexpr int kPitch = 64 * VI + 4;
    static_assert(sizeof(Part<kRows, VI>) % 16 == 0, "parts on 16 bytes");
    return {part->y[0], part->y[0], int(2 * sizeof(Part<kRows, VI>) / sizeof(float)), n, kPitch, kRows * kPitch, true};
  };

  Segment& sg = mem.segment[warp];
  constexpr int kMostSteps = kMostKeys / kStep;
  bool more_pieces = false;
  auto next = [&]() -> bool {  // the segment's next piece, or the next segment
    if (!more_pieces) return share.get(sg);
    __syncwarp();
    if (lane == 0) sg.at += kMostSteps;
    __syncwarp();
    return true;
  };
  while (next()) {
    more_pieces = sg.at + kMostSteps < sg.s1;
    const int rows_all = sg.seq.n * p.group;  // of the sequence (for this key head)
    // keys of this piece that one of its rows sees end here (the last row sees the most)
    int last = min(min(sg.s1, sg.at + kMostSteps) * kStep, sg.seq.have);
    if constexpr (!PREFIX)
      last = min(last, limit_of(p.causal, query_of(p, min(sg.row0 + kRows, rows_all) - 1), sg.seq.n, sg.seq.have));
    // and the keys that all of them see end here
    const int clear = PREFIX ? last : min(last, limit_of(p.causal, query_of(p, sg.row0), sg.seq.n, sg.seq.have));

    // this lane's two rows of each tile as columns of S^T: visible keys
    int lim[NT][2];
    uint32_t q[NT][KI][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = sg.row0 + 8 * n + 2 * t + e;
        lim[n][e] = PREFIX || r >= rows_all ? last : min(last, limit_of(p.causal, query_of(p, r), sg.seq.n, sg.seq.have));
      }
      const int r = sg.row0 + 8 * n + g;  // Q^T: this lane's column
      const int i = query_of(p, r);
      const __half* qr = p.q + static_cast<long long>(sg.seq.q0 + i) * p.qs + (sg.kvh * p.group + r - i * p.group) * D;
#pragma unroll
      for (int k = 0; k < KI; ++k) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows_all && (FULL || 4 * k + t < chunks)) x = __ldg(reinterpret_cast<const uint4*>(qr + key_run(k, t)));
        q[n][k][0] = x.x, q[n][k][1] = x.y, q[n][k][2] = x.z, q[n][k][3] = x.w;
      }
    }

    // Pages of the piece's keys, a lane each: 32 from number first_page on, and the 32 behind them. (Looked up key by
    // key, a step's loads waited for L2 first: 107 us for one token of 16 requests over up to 32768 keys.)
    auto page_of = [&](int number) -> int {
      if (number >= (last + page_mask) >> c.shift) return 0;
      const int page = __ldg(sg.pages + number);
      if (unsigned(page) < unsigned(c.n_pages)) return page;
      atomicOr(c.err, kDevErrCache);
      return 0;
    };
    int first_page = (sg.at * kStep) >> c.shift;
    int here = page_of(first_page + lane), there = page_of(first_page + 32 + lane);
    const uint8_t* const head_at = c.pages + static_cast<long long>(sg.kvh << c.shift) * (D * kEs);
    const uint8_t* const scales_at = c.pages + to_scales + ((sg.kvh + (lane >> 4) * c.hk) << c.shift) + (lane & 15);
    Eight<E4M3> kx[kSub][2][KI], vx[kSub][4][VI];
    int scale[kSub];  // lane < 16: the byte of key lane, else of value lane - 16
    int page[kSub];   // of the keys that are loaded next
    auto load_k = [&](int key0) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int at = (key0 + 16 * u) & page_mask, left = last - (key0 + 16 * u);  // (behind the last key nothing is live)
        const long long base = page[u] * c.page_bytes;
        const uint8_t* row = head_at + base + ((at + g) * D + key_run(0, t)) * kEs;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < KI; ++k) {
            const uint8_t* from = row + (8 * h * D + key_run(k, 0)) * kEs;
            const bool live = g + 8 * h < left && (FULL || 4 * k + t < chunks);
            if constexpr (kWideK) {
              if (!(k & 1)) load_two(kx[u][h][k], kx[u][h][k + 1 < KI ? k + 1 : 0], from, live);
            } else {
              kx[u][h][k].template load<FULL>(from, live);
            }
          }
        scale[u] = kNoScale;
        if ((lane & 15) < left) scale[u] = __ldg(scales_at + base + at);
      }
    };
    auto load_v = [&](int key0) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int left = last - (key0 + 16 * u);
        const uint8_t* row = head_at + page[u] * c.page_bytes + to_values +
                             ((((key0 + 16 * u) & page_mask) + 2 * t) * D + value_run(0, g)) * kEs;
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int k = 0; k < VI; ++k) {
            const int key = (h & 1) + 8 * (h >> 1);
            const uint8_t* from = row + (key * D + value_run(k, 0)) * kEs;
            const bool live = 2 * t + key < left && (FULL || 8 * k + g < chunks);
            if constexpr (kWideV) {
              if (!(k & 1)) load_two(vx[u][h][k], vx[u][h][k + 1 < VI ? k + 1 : 0], from, live);
            } else {
              vx[u][h][k].template load<FULL>(from, live);
            }
          }
      }
    };
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
#pragma unroll
      for (int k = 0; k < KI; ++k) kx[u][0][k].clear(), kx[u][1][k].clear();
#pragma unroll
      for (int k = 0; k < VI; ++k) vx[u][0][k].clear(), vx[u][1][k].clear(), vx[u][2][k].clear(), vx[u][3][k].clear();
    }
    float o[NT][4 * VI][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 4 * VI; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    int key0 = sg.at * kStep;
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
    // (the first step's loads and the others' are one piece of code: a short segment waits for its instructions)
#pragma unroll 1
    for (key0 -= kStep;; key0 += kStep) {
      const bool some = key0 >= sg.at * kStep, more = key0 + kStep < last;
      float s[kSub][NT][4];
      int byte[kSub];
      if (some) {
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
      }
      if (more) {
        look_up(key0 + kStep);
        load_k(key0 + kStep);
      }
      if (some) {
        uint32_t b[kSub][NT][2];
        int vbyte[kSub][2];  // the bytes of values g and g + 8 (31 at most)
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kb = __shfl_sync(0xffffffffu, byte[u], g + 8 * h), vb = __shfl_sync(0xffffffffu, byte[u], 16 + g + 8 * h);
            // (a marked one counts NaN)
            const float unit = max(kb, vb) == kMarked ? __uint_as_float(0x7fc00000u) : power_of(min(kb, 31));
            vbyte[u][h] = min(vb, 31);
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
                s[u][n][e] = (p.cap < kFarCap ? big : far_capped(s[u][n][e] * (kLog2e * p.scale), y, big)) +
                             exponent_of(vbyte[u][e >> 1]);
              }
        } else {
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][n][e] = fmaf(s[u][n][e], sl2, exponent_of(vbyte[u][e >> 1]));
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
#pragma unroll
            for (int u = 1; u < kSub; ++u) mx = fmax3(mx, s[u][n][e], s[u][n][e + 2]);
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
              l[n][e] = fmaf(s[u][n][e], reciprocal_of(vbyte[u][0]), fmaf(s[u][n][e + 2], reciprocal_of(vbyte[u][1]), l[n][e]));
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
      }
      if (!more) break;
      load_v(key0 + kStep);
    }

    // the rows' sums, to shared memory
    const bool whole = sg.s0 == 0 && sg.s1 == sg.steps;
    const int rows = min(kRows, rows_all - sg.row0);
    Part<kRows, VI>& mine = mem.part[warp][sg.s0 == 0 ? 1 : 0];
    if (sg.at > sg.s0) {  // to those of the pieces before, which this lane has written (m and l: the lanes of a row)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * t + e;
          const float2 before = mine.ml[r];
          const float up = fmaxf(m[n][e], before.x), ref = up == -INFINITY ? 0.0f : up;
          const float f = ex2(m[n][e] - ref), keep = ex2(before.x - ref);
          m[n][e] = up;
          l[n][e] = f * l[n][e] + (g == 0 ? keep * before.y : 0.0f);
#pragma unroll
          for (int j = 0; j < 4 * VI; j += 2) {
            const float4 z = *reinterpret_cast<const float4*>(&mine.y[r][value_run(j >> 2, g) + 2 * (j & 3)]);
            o[n][j][e] = fmaf(keep, z.x, f * o[n][j][e]);
            o[n][j][e + 2] = fmaf(keep, z.y, f * o[n][j][e + 2]);
            o[n][j + 1][e] = fmaf(keep, z.z, f * o[n][j + 1][e]);
            o[n][j + 1][e + 2] = fmaf(keep, z.w, f * o[n][j + 1][e + 2]);
          }
        }
      __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        float y = l[n][e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (g == 0) mine.ml[r] = make_float2(m[n][e], y);
#pragma unroll
        for (int j = 0; j < 4 * VI; j += 2)  // four neighbouring dimensions
          *reinterpret_cast<float4*>(&mine.y[r][value_run(j >> 2, g) + 2 * (j & 3)]) =
              make_float4(o[n][j][e], o[n][j][e + 2], o[n][j + 1][e], o[n][j + 1][e + 2]);
      }
    if (!whole && lane == 0) mem.cut[warp][sg.s0 == 0 ? 1 : 0] = sg;
    __syncwarp();
    if (whole && !more_pieces) {
      pdl_wait();
#pragma unroll 1
      for (int r = 0; r < rows; r += 4)
        settle(mem.p, sg, shared_source(&mine, 1), r, 1, min(4, rows - r), PREFIX ? kept_at(sg.item + int(blockIdx.x)) : nullptr, kRows);
      __syncwarp();
    }
  }

  // Items that were cut between the warps: the one that the CTA before has begun, and those that go on behind each warp's
  // share; four rows a warp in turn.
  pdl_wait();
  __syncthreads();
  auto cta_of = [&](int step) { return int(unsigned(step) / unsigned(mem.state[warp].chunk * kWarps)); };
  int open[2] = {-1, -1};  // first warps of the items that are cut at the start and at the end of the CTA's share
  int task = 0;
#pragma unroll 1
  for (int x = 0; x <= kWarps; ++x) {
    const int w0 = max(x - 1, 0), slot = x > 0;
    const Segment& first = mem.cut[w0][slot];
    if (first.steps == 0) continue;
    int n = 1, s1 = first.s1;
    while (s1 < first.steps && w0 + n < kWarps) s1 = mem.cut[w0 + n++][0].s1;
    Source from = shared_source(&mem.part[w0][slot], n);
    if (w0 + 1 < kWarps) from.rest = mem.part[w0 + 1][0].y[0];
    float* put = nullptr;
    if (PREFIX) {
      put = kept_at(first.item + int(blockIdx.x));
    } else if (first.s0 > 0 || s1 < first.steps) {
      const int end = first.s0 == 0;
      open[end] = w0;
      put = kept_at(2 * int(blockIdx.x) + end);
    }
    const int rows = min(kRows, first.seq.n * p.group - first.row0);
    for (int r = 0; r < rows; r += 4, ++task)
      if (task % kWarps == warp) settle(mem.p, first, from, r, 1, min(4, rows - r), put, kRows);
  }
  if (PREFIX || (open[0] < 0 && open[1] < 0)) return;

  // Items that were cut between CTAs: the last CTA of an item's parts joins them, every fourth row a warp.
  static_assert(kRows <= 4 * kWarps, "rows of a warp");
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2 && open[threadIdx.x] >= 0) {
    const Segment& cut = mem.cut[open[threadIdx.x]][threadIdx.x];
    const int c0 = cta_of(cut.base), c1 = cta_of(cut.base + cut.steps - 1);
    mem.seen[threadIdx.x] = atomicInc(p.counters + c0, unsigned(c1 - c0)) == unsigned(c1 - c0);  // then 0 again
  }
  __syncthreads();
#pragma unroll 1
  for (int end = 0; end < 2; ++end) {
    if (open[end] < 0 || !mem.seen[end]) continue;
    __threadfence();
    const Segment& cut = mem.cut[open[end]][end];
    const int c0 = cta_of(cut.base), c1 = cta_of(cut.base + cut.steps - 1);
    const int rows = min(kRows, cut.seq.n * p.group - cut.row0);
    const Source from = {kept_at(2 * c0 + 1), kept_at(2 * c0 + 2), 2 * kRows * (D + 2), c1 - c0 + 1, D, kRows * D, false};
    settle(mem.p, cut, from, warp, kWarps, (rows - warp + kWarps - 1) / kWarps, nullptr, kRows);
  }
}

// Behind the sequences' pass through tiles: every row's parts joined, four rows a warp at a time. Latency: offsets, places
// of the parts, parts, one after another (840 rows of 4 heads of 128, two parts of each pass: 9 us alone; 4 CTAs an SM
// instead of 8: 1 us more, 16: as much more).
struct JoinShared {
  Segment segment[kWarps];
  ShareState state[kWarps];
  ShareTotals totals;
  Params p;
};
__global__ void __launch_bounds__(kThreads) cached_join_kernel(const __grid_constant__ Params p) {
  __shared__ JoinShared mem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(sizeof(Params) / 4 <= kThreads, "a word a thread");
  if (threadIdx.x < sizeof(Params) / 4)
    reinterpret_cast<int*>(&mem.p)[threadIdx.x] = reinterpret_cast<const int*>(&p)[threadIdx.x];
  __syncthreads();
  Share<4, 0> share(p, warp, lane, mem.state[warp], mem.totals);  // (items of four rows, a step each)
  // Offsets and lengths are in place, since the tiles let others begin only after a wait for them (their own, or the prefix
  // pass's); the parts are not yet.
  pdl_wait();
  pdl_launch_dependents();
  Segment& sg = mem.segment[warp];
  while (share.get(sg)) {
    const int rows_all = sg.seq.n * p.group, row = sg.row0;
    const int2 first = __ldcg(p.firsts + sg.item);
    const int chunk = __ldcg(p.firsts + p.c.count).x;
    const int blocks = (rows_all + kTileRows - 1) / kTileRows;
    const int steps = max(1, (sg.seq.have + 2 * kTileRows - 1) / (2 * kTileRows));
    const int k = sg.kvh * blocks + row / kTileRows, begin = first.y + k * steps;
    const int c0 = begin / chunk, c1 = (begin + steps - 1) / chunk, D = p.c.D, size = kTileRows * (D + 2);
    const float* part = p.tiles + size_t(first.x + k + c0) * size_t(size);
    __syncwarp();
    if (lane == 0) sg.row0 = row / kTileRows * kTileRows;
    __syncwarp();
    settle(mem.p, sg, {part, part + size, size, c1 - c0 + 1, D, kTileRows * D, false}, row % kTileRows, 1,
           min(4, rows_all - row), nullptr, 0);
    __syncwarp();
  }
}

template <int KI, int VI, bool FULL, int NT, bool E4M3, bool PREFIX>
cudaError_t few_launch_type(const Params& p, int grid, cudaStream_t s) {
  auto kern = cached_few_kernel<KI, VI, FULL, NT, E4M3, PREFIX>;
  constexpr int kBytes = int(sizeof(FewShared<8 * NT, VI>));
  static unsigned long long set = 0;
  // L1 brings the sectors of a key's line together that lanes ask for one after another. Behind a tile kernel an SM kept
  // that one's 228 KB of shared memory where it was not told: 256 samples behind 32768 keys 177 us, now 170; 16 sequences
  // of 900 to 32768 tokens (490 MB) take 118 us beside so little L1, and 86 like this.
  const cudaError_t e = allow_shared(kern, kBytes, &set, per_sm(NT));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(kThreads), size_t(kBytes), s, p);
}
template <int KI, int VI, bool FULL, int NT, bool PREFIX>
cudaError_t few_launch_as(const Params& p, int grid, cudaStream_t s) {
  return p.c.e4m3 ? few_launch_type<KI, VI, FULL, NT, true, PREFIX>(p, grid, s)
                  : few_launch_type<KI, VI, FULL, NT, false, PREFIX>(p, grid, s);
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
  int nt, grid;          // the sequences' pass: 8-row tiles of an item (0: tiles of 128 rows, cached_tiles.cu), CTAs at most
  size_t own;            // bytes of its parts
  int pre_nt, pre_grid;  // the prefix's (pre_nt 0: tiles of 128 rows, cached_tiles.cu)
  PrefixParts pre;       // (its base is an offset in floats)
  size_t bytes;          // workspace
  bool too_much;         // steps (counted in 32 bits)
};
Plan plan_of(const View& c, int total_q, int group, int sms) {
  Plan r = {};
  const long long rows = static_cast<long long>(total_q) * group;  // of a key head
  // Blocks of 16 rows read a sequence's keys once each, tiles of 128 rows with a slower start. 64 sequences of 2250 tokens
  // (32 heads over 8 of 128, E4M3), blocks and tiles: 24 rows each 135 and 130 us, 32 137 and 135, 40 194 and 133; the
  // same with 225 tokens 32 and 46, 33 and 52, 40 and 50.
  r.nt = rows <= 8ll * c.count ? 1 : rows <= 32ll * c.count ? 2 : 0;
  r.grid = r.nt ? sms * per_sm(r.nt) : sms;
  const long long tokens = static_cast<long long>(c.stride) << c.shift;
  const int block = r.nt ? 8 * r.nt : kTileRows, keys = r.nt ? 16 * groups_of(c.e4m3, c.D) : 2 * kTileRows;
  const long long items = (rows / block + (c.count < total_q ? c.count : total_q)) * c.hk;  // (every sequence rounds up)
  r.too_much = items * (tokens / keys + 1) >= (1ll << 30);
  if (r.nt) {
    r.own = size_t(kMaxSms * per_sm(r.nt)) * 2 * size_t(8 * r.nt) * size_t(c.D + 2) * sizeof(float);
  } else {
    r.own = size_t(items + kMaxSms) * size_t(kTileRows) * size_t(c.D + 2) * sizeof(float) +
            (size_t(c.count + 1) * sizeof(int2) + 127) / 128 * 128;
  }
  r.bytes = kCounterBytes + 128 + r.own;  // (parts begin on 128 bytes)
  if (c.prefix_len > 0) {
    r.pre_nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 0;
    int step = 16 * groups_of(c.e4m3, c.D), most = sms * per_sm(r.pre_nt), at_most = kMaxSms * per_sm(r.pre_nt);
    int parts = kWarps;  // of a CTA's share: a whole number of steps each
    r.pre.rows = 8 * r.pre_nt;
    if (r.pre_nt == 0) {
      r.pre.rows = rows <= kTileRows ? kTileRows : 2 * kTileRows;
      step = rows <= kTileRows ? 2 * kTileRows : kTileRows;
      most = sms;
      at_most = kMaxSms;
      parts = 1;
    }
    r.pre.blocks = int((rows + r.pre.rows - 1) / r.pre.rows);
    r.pre.steps = (c.prefix_len + step - 1) / step;
    const long long pre_items = static_cast<long long>(r.pre.blocks) * c.hk, work = pre_items * r.pre.steps;
    if (work >= (1ll << 30)) {  // (behind it 32 bits would not hold the share)
      r.too_much = true;
      return r;
    }
    r.pre.chunk = int((work + static_cast<long long>(most) * parts - 1) / (static_cast<long long>(most) * parts) * parts);
    r.pre_grid = int((work + r.pre.chunk - 1) / r.pre.chunk);
    r.bytes += size_t(pre_items + at_most) * size_t(r.pre.rows) * size_t(c.D + 2) * sizeof(float);
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
  if (plan_of(*c, total_q, q_heads / c->hk, 1).too_much) {
    set_error("%s: %d queries of %d heads over a prefix of %d and %d pages of %d are too many for one call", fn, total_q, q_heads,
              c->prefix_len, c->stride, 1 << c->shift);
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
  p.group = q_heads / p.c.hk;
  p.per_group = unsigned((0xffffffffull + unsigned(p.group)) / unsigned(p.group));
  p.scale = opt.scale > 0.0f ? opt.scale : 1.0f / std::sqrt(float(p.c.D));
  p.cap = opt.softcap;
  p.causal = opt.mask == SV_MASK_PREFIX;
  p.out_e4m3 = out_dtype == SV_DT_E4M3;
  const Plan plan = plan_of(p.c, total_q, p.group, num_sms() < kMaxSms ? num_sms() : kMaxSms);
  p.counters = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + kCounterBytes + 127) & ~uintptr_t(127));
  p.pre = plan.pre;
  p.firsts = reinterpret_cast<int2*>(p.partial);
  p.tiles = p.partial + (size_t(p.c.count + 1) * sizeof(int2) + 127) / 128 * 128 / sizeof(float);
  p.pre.base = p.partial + plan.own / sizeof(float);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (p.c.prefix_len > 0) {
    LaunchScope L(kKindAttn, 0.0, 0.0, s);
    if (plan.pre_nt == 0) {
      st = prefix_launch(fn, p, plan.pre_grid, s);
      if (st != SV_OK) return st;
    } else {
      e = plan.pre_nt == 1 ? few_launch<1, true>(p, plan.pre_grid, s) : few_launch<2, true>(p, plan.pre_grid, s);
    }
  }
  if (e == cudaSuccess && plan.nt > 0) {
    LaunchScope L(kKindAttn, 0.0, 0.0, s);
    e = plan.nt == 1 ? few_launch<1, false>(p, plan.grid, s) : few_launch<2, false>(p, plan.grid, s);
  } else if (e == cudaSuccess) {
    {
      LaunchScope L(kKindAttn, 0.0, 0.0, s);
      st = own_tiles_launch(fn, p, plan.grid, s);
      if (st != SV_OK) return st;
    }
    LaunchScope L(kKindAttn, 0.0, 0.0, s);
    const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
    e = launch_pdl(cached_join_kernel, dim3(unsigned(8 * sms)), dim3(kThreads), 0, s, p);
  }
  return e == cudaSuccess ? SV_OK : cuda_fail(e, fn);
}

}  // extern "C"
