// sv_attention_packed for a few rows (queries x heads of a key head) per document: one new
// token of many requests over long caches, pooling probes over many images.
//
// Bound: DRAM, every key and value read once for (up to) 8 or 16 rows. The arithmetic runs on
// warp-level matrix instructions (mma.sync m16n8k16, F32 accumulation) because the rows fill
// no tcgen05 tile and keys and values can then go from global memory straight to the
// registers of the instruction, with nothing to wait for but the loads themselves:
//   S^T = K Q^T: 16 keys x 8 rows. The order of the summed dimensions is free as long as K
//     and Q agree, so a lane's 16 contiguous bytes of a key row (8 dimensions) serve as its
//     operand values of two instructions; four lanes read 64 contiguous bytes of a key.
//   O^T += V^T P^T: 16 dimensions x 8 rows. The order of O's dimensions is free as well: eight
//     lanes read 128 contiguous bytes of a value row, a lane holds the same 8 dimensions of the
//     keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9, and byte permutes pair the keys. P^T goes from the
//     accumulator's layout to the operand's by a transposing 8 x 8 move.
// A warp takes 16 keys at a time (its registers of K are reloaded as soon as S^T is done, those
// of V as soon as O^T is). The four warps of a CTA take four neighbouring key heads where their
// number allows and a row is no whole number of 64 bytes (or two heads and alternate keys, or one
// head): the rows of a key lie side by side, DRAM's sectors hold parts of two of them, and so these
// are asked for at the same time (64 probes, 16 heads of 72: 252 MB read for 163 MB of keys and
// values with a head per CTA). Two or three CTAs run per SM, by their registers: these hold what is in
// flight.
//
// Work: the (document, group of key heads, block of rows) items are laid out one behind another
// in steps of 64 keys of one head or 16 of four, and every CTA takes an equal, contiguous share of
// the steps, so that any distribution of lengths fills the GPU. An item inside one share is
// finished there; one that is cut goes in parts to the workspace, and the last CTA of its parts
// joins them in order. A CTA has at most two such parts, at the start and at the end of its share.
// One long range makes many parts (one query, 8 key heads of 128, 32768 keys: 57 a head), and what
// joins them is alone on the GPU by then, bound by the latency of L2: sixteen parts are on their
// way at a time (two at a time: 48 us for that call, now 31, its 134 MB being 20 us).
#include "packed_attention.h"

namespace sv {
namespace packed {
namespace {

constexpr int kFewThreads = 128;
constexpr int kMinShare = 64;       // keys of a CTA's share at least
constexpr int kMostPerSm = 3;
constexpr int kMaxFewGrid = kMaxSms * kMostPerSm;
// CTAs an SM, by what the registers of a warp allow: four of 8 rows spill inside their loop (64 probes, 16 heads of 72:
// 65 against 40 us; 16 ranges of 8192 keys, 7 heads of 72: 115 against 47).
constexpr int per_sm(int nt) { return nt > 1 ? 2 : 3; }

__device__ __forceinline__ uint4 load16(const __half* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ uint32_t load4(const __half* p) {
  uint32_t r;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t load2(const __half* p) {
  uint16_t r;
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
  return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A run of steps of one item that falls into this CTA's share.
struct Segment {
  Document doc;
  int kvh, row0;          // first key head, first of the item's rows (query x group + head) in the document
  int s0, s1, steps;      // steps of the item: this segment's, all
  long long base;         // place of the item's first step among all steps
};

// The items in order: documents, key heads, blocks of rows. 32 documents at a time, one per
// lane, with their steps summed by shuffles; every warp works it out for itself.
template <int ROWS, int HEADS>
class Share {
  static constexpr int kStep = 64 / HEADS;  // keys of a step
 public:
  __device__ __forceinline__ Share(const Params& p, int lane) : p_(p), lane_(lane), docs_(p.docs) {
    long long work = 0;
    bool bad = false;
    for (int d0 = 0; d0 < p.docs; d0 += 32) {
      bad |= !load(d0);
      work += mine();
    }
    for (int o = 16; o; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
    // offsets that decrease or leave [0, total]: reported, and nothing is computed
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0) atomicOr(p.err, kDevErrOffsets);
      docs_ = 0;
      work = 0;
    }
    chunk_ = (work + gridDim.x - 1) / gridDim.x;
    if (chunk_ < kMinShare / kStep) chunk_ = kMinShare / kStep;
    at_ = chunk_ * blockIdx.x;
    end_ = min(at_ + chunk_, work);  // (a share may begin behind the last step)
    if (p.docs > 32 || docs_ == 0) load(0);
    open(0);
  }
  // The next segment of this CTA's share. Without a workspace nothing is cut: a CTA takes the
  // items that begin in its share, whole.
  __device__ __forceinline__ bool get(Segment& r) {
    while (at_ < end_) {
      while (at_ >= base_ + total_) {
        base_ += total_;
        load(d0_ + 32);
        open(d0_ + 32);
      }
      const int src = __ffs(__ballot_sync(0xffffffffu, base_ + incl_ > at_)) - 1;
      r.doc.q0 = of(doc_.q0, src);
      r.doc.lq = of(doc_.lq, src);
      r.doc.k0 = of(doc_.k0, src);
      r.doc.lk = of(doc_.lk, src);
      r.doc.prefix = of(doc_.prefix, src);
      r.steps = of(steps_, src);
      const int blocks = of(blocks_, src);
      const long long first = base_ + __shfl_sync(0xffffffffu, incl_ - mine(), src);
      const long long item = (at_ - first) / r.steps;
      r.base = first + item * r.steps;
      r.kvh = int(item / blocks);
      r.row0 = int(item - static_cast<long long>(r.kvh) * blocks) * ROWS;
      r.kvh *= HEADS;
      r.s0 = int(at_ - r.base);
      r.s1 = int(min(end_ - r.base, static_cast<long long>(r.steps)));
      if (!p_.counters) {
        r.s1 = r.steps;
        if (r.s0 > 0) {  // begun by the CTA before
          at_ = r.base + r.steps;
          continue;
        }
      }
      at_ = r.base + r.s1;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ int cta_of(long long step) const { return int(step / chunk_); }

 private:
  __device__ __forceinline__ static int of(int v, int src) { return __shfl_sync(0xffffffffu, v, src); }
  __device__ __forceinline__ long long mine() const {
    return static_cast<long long>(blocks_) * (p_.hk / HEADS) * steps_;
  }
  __device__ __forceinline__ bool load(int d0) {
    d0_ = d0;
    const bool good = document(p_, d0 + lane_, docs_, doc_);
    blocks_ = int((static_cast<long long>(doc_.lq) * p_.group + ROWS - 1) / ROWS);
    steps_ = max(1, (doc_.lk + kStep - 1) / kStep);  // (a step without keys writes the zeros)
    return good;
  }
  __device__ __forceinline__ void open(int d0) {
    incl_ = mine();
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, incl_, o);
      if (lane_ >= o) incl_ += a;
    }
    total_ = __shfl_sync(0xffffffffu, incl_, 31);
  }
  const Params& p_;
  int lane_, docs_, d0_ = 0, blocks_, steps_;
  Document doc_;
  long long chunk_, at_, end_, base_ = 0, total_ = 0, incl_;
};

// The parts c0, c0 + 1, ... of a cut item: `rows_all` rows of D sums, then exponent and denominator of each.
struct Parts {
  const float* base;
  size_t slot;  // values of a part's place; a CTA has two, at the start of its share and at its end
  int n, D, rows_all;
  __device__ __forceinline__ const float* at(int w) const { return base + (w == 0 ? 1 : 2 * w) * slot; }
  // A row over the parts first, first + step, ... in order, sixteen of them on their way at a time (they
  // come from L2, and nothing else hides its latency): the lane's columns 4 lane .. 4 lane + 3, and the
  // row's exponent and denominator.
  __device__ __forceinline__ float4 sums(int row, int lane, int first, int step, float& mx, float& sum) const {
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    mx = -INFINITY;
    sum = 0.0f;
    for (int w0 = first; w0 < n; w0 += 16 * step) {
      float4 v[16];
      float2 ml[16];
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        const int w = w0 + b * step;
        ml[b] = make_float2(-INFINITY, 0.0f);
        v[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (w < n) {
          ml[b] = __ldcg(reinterpret_cast<const float2*>(at(w) + rows_all * D) + row);
          v[b] = __ldcg(reinterpret_cast<const float4*>(at(w) + row * D) + min(lane, D / 4 - 1));
        }
      }
      float up = mx;
#pragma unroll
      for (int b = 0; b < 16; ++b) up = fmaxf(up, ml[b].x);
      const float ref = up == -INFINITY ? 0.0f : up, back = ex2(mx - ref);
      mx = up;
      sum *= back;
      y = make_float4(y.x * back, y.y * back, y.z * back, y.w * back);
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        const float e = ex2(ml[b].x - ref);
        sum = fmaf(e, ml[b].y, sum);
        y.x = fmaf(e, v[b].x, y.x);
        y.y = fmaf(e, v[b].y, y.y);
        y.z = fmaf(e, v[b].z, y.z);
        y.w = fmaf(e, v[b].w, y.w);
      }
    }
    return y;
  }
};

// Eight sums of a part, as they are.
__device__ __forceinline__ void put_part(float* to, const float* y) {
  __stcg(reinterpret_cast<float4*>(to), make_float4(y[0], y[1], y[2], y[3]));
  __stcg(reinterpret_cast<float4*>(to) + 1, make_float4(y[4], y[5], y[6], y[7]));
}

// What rows of a segment need to be computed again: of its document the first query, the first key, queries, keys and
// prefix; its key head, its first row, its keys; rows of a head, and their place in a part (null: they are results).
struct Again {
  int q0, k0, lq, lk, prefix, kvh, row0, begin, end, rows;
  float *part, *part_ml;
};
// Those of the rows `todo` (a bit a row) of head hw that a hidden key's value has spoiled, again from their visible
// keys alone, by one warp. (Not inlined: it took the registers of the loop.)
__device__ __noinline__ void few_again(const Params& p, const Again sg, int hw, unsigned todo) {
  const int lane = int(threadIdx.x) & 31;
  const __half* k = p.k + sg.k0 * p.ks + (sg.kvh + hw) * p.D;
  const __half* v = p.v + sg.k0 * p.vs + (sg.kvh + hw) * p.D;
  auto limit = [&](int r) {
    return max(sg.begin, limit_of(p.causal, (sg.row0 + r) / p.group + sg.lk - sg.lq, sg.lk, sg.prefix));
  };
  const int low = limit(__ffs(int(todo)) - 1);  // (later rows see no fewer keys)
  const int last = low < sg.end ? last_spoiled(p, v, low, sg.end, lane) : -1;
  __syncwarp();  // (what other lanes have stored of the rows comes first)
#pragma unroll 1
  for (; todo; todo &= todo - 1) {
    const int r = __ffs(int(todo)) - 1, row = hw * sg.rows + r, lim = limit(r);
    if (lim > last) break;  // (its result, and the later ones', are the products')
    const int i = (sg.row0 + r) / p.group, head = (sg.kvh + hw) * p.group + (sg.row0 + r - i * p.group);
    float m, l;
    const float4 y = row_again(p, p.q + static_cast<long long>(sg.q0 + i) * p.qs + head * p.D, k, v, sg.begin,
                               min(sg.end, lim), i + sg.lk - sg.lq, p.slopes ? __ldg(p.slopes + head) : 0.0f, lane,
                               nullptr, m, l);
    if (sg.part) {
      if (lane < p.D / 4) __stcg(reinterpret_cast<float4*>(sg.part + row * p.D) + lane, y);
      if (lane == 0) __stcg(reinterpret_cast<float2*>(sg.part_ml) + row, make_float2(m, l));
    } else if (lane < p.D / 4) {
      store4(p, size_t(sg.q0 + i) * size_t(p.os) + size_t(head) * size_t(p.D) + size_t(4 * lane),
             make_float4(y.x / l, y.y / l, y.z / l, y.w / l));
    }
  }
}

// KI: 32-dimension groups of a key row, VI: 64-dimension groups of a value row, NT: 8-row
// tiles of an item, HEADS: key heads of an item (4 / HEADS warps share a head's keys). TAIL: eight
// more dimensions behind the groups (72), in instructions of their own: another group of each
// would hold registers for 96 and 128 dimensions (64 probes, 16 heads of 72: 47.3 us, 39.8 so).
template <int KI, int VI, int NT, int HEADS, bool TAIL>
__global__ void __launch_bounds__(kFewThreads, per_sm(NT)) few_kernel(const __grid_constant__ Params p) {
  constexpr int kRows = 8 * NT, kSplit = 4 / HEADS, kStep = 16 * kSplit;
  constexpr int kOut = 64 * VI + (TAIL ? 12 : 4);  // row pitch of the merge buffer (floats)
  __shared__ __align__(16) float red[4][kRows][kOut];
  __shared__ float red_m[4][kRows], red_l[4][kRows];
  __shared__ int row_bad[HEADS * kRows];
  __shared__ unsigned seen;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  pdl_wait();
  const int my_head = warp % HEADS, my_keys = warp / HEADS;
  Share<kRows, HEADS> share(p, lane);
  const int chunks = p.D / 8;  // 16-byte chunks of a row
  const float sl2 = p.cap > 0.0f ? cap_factor(p.scale, p.cap) : kLog2e * p.scale;

  Segment sg;
  while (share.get(sg)) {
    const int rows_all = sg.doc.lq * p.group;  // of the document (for this key head)
    const int lk = sg.doc.lk;
    const int kvh = sg.kvh + my_head;
    const __half* kb = p.k + sg.doc.k0 * p.ks + kvh * p.D;
    const __half* vb = p.v + sg.doc.k0 * p.vs + kvh * p.D;
    // keys of this segment that one of its rows sees end here (the last row sees the most)
    const int last = min(sg.s1 * kStep, limit_of(p.causal, (min(sg.row0 + kRows, rows_all) - 1) / p.group + lk - sg.doc.lq,
                                                 lk, sg.doc.prefix));

    // this lane's two rows of each tile as columns of S^T: visible keys, position, slope
    int lim[NT][2];
    int at[NT][2];
    float slope[NT][2];
    uint32_t q[NT][KI][4], q_tail[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = sg.row0 + 8 * n + 2 * t + e;
        const int i = r / p.group, pos = i + lk - sg.doc.lq;
        lim[n][e] = r < rows_all ? limit_of(p.causal, pos, lk, sg.doc.prefix) : lk;
        at[n][e] = pos;
        slope[n][e] = p.slopes && r < rows_all ? __ldg(p.slopes + kvh * p.group + (r - i * p.group)) * kLog2e : 0.0f;
      }
      const int r = sg.row0 + 8 * n + g;  // Q^T: this lane's column
      const int i = r / p.group;
      const __half* qr = p.q + static_cast<long long>(sg.doc.q0 + i) * p.qs + (kvh * p.group + r - i * p.group) * p.D;
#pragma unroll
      for (int c = 0; c < KI; ++c) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows_all && 4 * c + t < chunks) x = load16(qr + 8 * (4 * c + t));
        q[n][c][0] = x.x, q[n][c][1] = x.y, q[n][c][2] = x.z, q[n][c][3] = x.w;
      }
      q_tail[n] = TAIL && r < rows_all ? load4(qr + 32 * KI + 2 * t) : 0u;
    }

    uint4 kx[2][KI], vx[4][VI];
    uint32_t k_tail[2], v_tail[4];
    auto load_k = [&](int key0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = key0 + g + 8 * h;
        const __half* row = kb + key * p.ks;
#pragma unroll
        for (int c = 0; c < KI; ++c)
          kx[h][c] = key < last && 4 * c + t < chunks ? load16(row + 8 * (4 * c + t)) : make_uint4(0u, 0u, 0u, 0u);
        if (TAIL) k_tail[h] = key < last ? load4(row + 32 * KI + 2 * t) : 0u;
      }
    };
    auto load_v = [&](int key0) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int key = key0 + 2 * t + (h & 1) + 8 * (h >> 1);
        const __half* row = vb + key * p.vs;
#pragma unroll
        for (int c = 0; c < VI; ++c)
          vx[h][c] = key < last && 8 * c + g < chunks ? load16(row + 8 * (8 * c + g)) : make_uint4(0u, 0u, 0u, 0u);
        if (TAIL) v_tail[h] = key < last ? load2(row + 64 * VI + g) : 0u;
      }
    };
    float o[NT][4 * VI][4], o_tail[NT][4];  // the tail: dimension 64 VI + g of rows 2 t and 2 t + 1
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 4 * VI; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
      o_tail[n][0] = o_tail[n][1] = o_tail[n][2] = o_tail[n][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    int key0 = sg.s0 * kStep + 16 * my_keys;
    load_k(key0);
    load_v(key0);
    for (; key0 < last; key0 += kStep) {
      uint32_t b[NT][2];
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < KI; ++c) {
          mma16816(s[n], kx[0][c].x, kx[1][c].x, kx[0][c].y, kx[1][c].y, q[n][c][0], q[n][c][1]);
          mma16816(s[n], kx[0][c].z, kx[1][c].z, kx[0][c].w, kx[1][c].w, q[n][c][2], q[n][c][3]);
        }
        if (TAIL) mma1688(s[n], k_tail[0], k_tail[1], q_tail[n]);
      }
      load_k(key0 + kStep);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[4];
        float f[2];
        bool raise = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // e & 1: the row, e >> 1: keys g, g + 8
          const int key = key0 + g + 8 * (e >> 1);
          float y = s[n][e] * sl2;
          if (p.cap > 0.0f) {
            const float big = capped(y, p.cap * kLog2e);
            y = p.cap < kFarCap ? big : far_capped(s[n][e] * (kLog2e * p.scale), y, big);
          }
          if (p.slopes) y = fmaf(-slope[n][e & 1], fabsf(float(at[n][e & 1] - key)), y);  // (positions pass 2^24)
          x[e] = key < min(lim[n][e & 1], last) ? y : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[e], x[e + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const bool up = mx > m[n][e] + kSlack;
          const float mn = up ? mx - kHead : m[n][e];
          f[e] = up ? ex2(m[n][e] - mn) : 1.0f;
          m[n][e] = mn;
          raise |= up;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int j = 0; j < 4 * VI; ++j) {
            o[n][j][0] *= f[0];
            o[n][j][1] *= f[1];
            o[n][j][2] *= f[0];
            o[n][j][3] *= f[1];
          }
          o_tail[n][0] *= f[0];
          o_tail[n][1] *= f[1];
          l[n][0] *= f[0];
          l[n][1] *= f[1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[n][e] == -INFINITY ? 0.0f : m[n][e];
          x[e] = ex2(x[e] - ref);
          x[e + 2] = ex2(x[e + 2] - ref);
          l[n][e] += x[e] + x[e + 2];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (F16, what the products take: 2^-11 of each probability; their sum l is of the unrounded ones)
          const __half2 w = __floats2half2_rn(x[2 * h], x[2 * h + 1]);
          b[n][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&w));
        }
      }
#pragma unroll
      for (int c = 0; c < VI; ++c) {
        const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vx[0][c]);
        const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vx[1][c]);
        const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vx[2][c]);
        const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vx[3][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // dimensions 2 j and 2 j + 1 of this lane's eight
          const uint32_t a0 = __byte_perm(v0[j], v1[j], 0x5410), a1 = __byte_perm(v0[j], v1[j], 0x7632);
          const uint32_t a2 = __byte_perm(v2[j], v3[j], 0x5410), a3 = __byte_perm(v2[j], v3[j], 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[n][4 * c + j], a0, a1, a2, a3, b[n][0], b[n][1]);
        }
      }
      if constexpr (TAIL) {
        const uint32_t a0 = __byte_perm(v_tail[0], v_tail[1], 0x5410), a2 = __byte_perm(v_tail[2], v_tail[3], 0x5410);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(o_tail[n], a0, 0u, a2, 0u, b[n][0], b[n][1]);
      }
      load_v(key0 + kStep);
    }

    const bool whole = sg.s0 == 0 && sg.s1 == sg.steps;
    const int rows = min(kRows, rows_all - sg.row0);
    // a part's place: at the start of this CTA's share (0) or at its end (1)
    auto part = [&](int cta, int end) {
      return p.partial + (size_t(cta) * 2 + end) * size_t(HEADS * kRows) * size_t(p.D + 2);
    };
    float* mine = whole ? nullptr : part(int(blockIdx.x), sg.s0 == 0 ? 1 : 0);  // [row][D], then [row] exponent, denominator
    float* mine_ml = mine + HEADS * kRows * p.D;
    const int c0 = share.cta_of(sg.base), c1 = share.cta_of(sg.base + sg.steps - 1);  // the item's parts
    const Parts parts{part(c0, 0), size_t(HEADS * kRows) * size_t(p.D + 2), c1 - c0 + 1, p.D, HEADS * kRows};

    // Row r of head hw of the item from all its parts, by one warp.
    auto join_row = [&](int hw, int r) {
      float mx, sum;
      const float4 a = parts.sums(hw * rows + r, lane, 0, 1, mx, sum);
      const int i = (sg.row0 + r) / p.group, head = (sg.kvh + hw) * p.group + (sg.row0 + r - i * p.group);
      const bool none = limit_of(p.causal, i + lk - sg.doc.lq, lk, sg.doc.prefix) == 0;
      const float inv = 1.0f / sum;
      float y[8] = {a.x, a.y, a.z, a.w};  // and the next lane's four
#pragma unroll
      for (int j = 0; j < 4; ++j) y[4 + j] = __shfl_down_sync(0xffffffffu, y[j], 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = none ? 0.0f : y[j] * inv;
      if (!(lane & 1) && lane < p.D / 4)
        store8(p, size_t(sg.doc.q0 + i) * size_t(p.os) + size_t(head) * size_t(p.D) + size_t(4 * lane), y);
    };

    if constexpr (kSplit == 1) {
      // A warp has its head's rows to itself: they go out from its registers, and the warps of the
      // CTA need not wait for one another. A lane holds eight neighbouring columns of two rows.
      unsigned redo = 0;  // rows that are not finite
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * t + e, i = (sg.row0 + r) / p.group;
          const int head = kvh * p.group + (sg.row0 + r - i * p.group);
          const bool live = r < rows;
          const size_t to = size_t(sg.doc.q0 + i) * size_t(p.os) + size_t(head) * size_t(p.D);
          float* at_p = mine + (my_head * rows + r) * p.D;
          float* at_ml = mine_ml + 2 * (my_head * rows + r);
          float sum = l[n][e];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const bool none = lim[n][e] == 0;
          const float inv = whole ? 1.0f / sum : 1.0f;
          float bad = 0.0f;
#pragma unroll
          for (int v = 0; v < VI; ++v) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[2 * j] = none ? 0.0f : o[n][4 * v + j][e] * inv;
              y[2 * j + 1] = none ? 0.0f : o[n][4 * v + j][e + 2] * inv;
              bad = fmaf(y[2 * j], 0.0f, fmaf(y[2 * j + 1], 0.0f, bad));
            }
            if (!live || 8 * v + g >= chunks) continue;
            if (whole) store8(p, to + 8 * (8 * v + g), y);
            else put_part(at_p + 8 * (8 * v + g), y);
          }
          if constexpr (TAIL) {
            const float y = none ? 0.0f : o_tail[n][e] * inv;
            bad = fmaf(y, 0.0f, bad);
            if (live && whole) store1(p, to + 64 * VI + g, y);
            else if (live) __stcg(at_p + 64 * VI + g, y);
          }
          if (live && !whole && g == 0) __stcg(reinterpret_cast<float2*>(at_ml), make_float2(m[n][e], sum));
          const unsigned rows_bad = __ballot_sync(0xffffffffu, live && bad != 0.0f);
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)  // (the columns of a row are in the lanes of one t)
            if (rows_bad & (0x11111111u << tt)) redo |= 1u << (8 * n + 2 * tt + e);
        }
      if (redo)
        few_again(p, {sg.doc.q0, sg.doc.k0, sg.doc.lq, lk, sg.doc.prefix, sg.kvh, sg.row0, sg.s0 * kStep, last, rows, mine,
                      mine_ml}, my_head, redo);
      if (whole) continue;
      __threadfence();
      __syncwarp();
      unsigned arrived = 0;
      if (lane == 0) arrived = atomicInc(p.counters + c0 * 4 + warp, unsigned(c1 - c0));  // 0 .. c1 - c0, then 0 again
      if (__shfl_sync(0xffffffffu, arrived, 0) != unsigned(c1 - c0)) continue;
      __threadfence();
      for (int r = 0; r < rows; ++r) join_row(my_head, r);
    } else {
      // the four warps' sums, brought to one exponent
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[n][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          if (g == 0) {
            red_m[warp][8 * n + 2 * t + e] = m[n][e];
            red_l[warp][8 * n + 2 * t + e] = x;
          }
        }
      if (threadIdx.x < HEADS * kRows) row_bad[threadIdx.x] = 0;
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * t + e;
          float mx = red_m[my_head][r];
#pragma unroll
          for (int k = 1; k < kSplit; ++k) mx = fmaxf(mx, red_m[my_head + k * HEADS][r]);
          f[e] = ex2(m[n][e] - (mx == -INFINITY ? 0.0f : mx));
        }
#pragma unroll
        for (int j = 0; j < 4 * VI; j += 2)  // four neighbouring dimensions of a row
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(&red[warp][8 * n + 2 * t + e][64 * (j >> 2) + 8 * g + 2 * (j & 3)]) =
                make_float4(o[n][j][e] * f[e], o[n][j][e + 2] * f[e], o[n][j + 1][e] * f[e], o[n][j + 1][e + 2] * f[e]);
      }
      if constexpr (TAIL) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            float mx = red_m[my_head][r];
#pragma unroll
            for (int k = 1; k < kSplit; ++k) mx = fmaxf(mx, red_m[my_head + k * HEADS][r]);
            red[warp][r][64 * VI + g] = o_tail[n][e] * ex2(m[n][e] - (mx == -INFINITY ? 0.0f : mx));
          }
      }
      __syncthreads();
      // row x of the item's HEADS x rows: which head and row, query and query head
      auto row_of = [&](int x, int& hw, int& r, int& i, int& head) {
        hw = x / rows;
        r = x - hw * rows;
        i = (sg.row0 + r) / p.group;
        head = (sg.kvh + hw) * p.group + (sg.row0 + r - i * p.group);
      };
      int any_bad = 0;
      for (int x = int(threadIdx.x); x < HEADS * rows * chunks; x += kFewThreads) {
        const int row = x / chunks, c = 8 * (x - row * chunks);
        int hw, r, i, head;
        row_of(row, hw, r, i, head);
        float mx = red_m[hw][r], sum = 0.0f;
#pragma unroll
        for (int k = 1; k < kSplit; ++k) mx = fmaxf(mx, red_m[hw + k * HEADS][r]);
        const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
        for (int k = 0; k < kSplit; ++k) sum += ex2(red_m[hw + k * HEADS][r] - ref) * red_l[hw + k * HEADS][r];
        const bool none = limit_of(p.causal, i + lk - sg.doc.lq, lk, sg.doc.prefix) == 0;
        const float inv = whole ? 1.0f / sum : 1.0f;
        float y[8], bad = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = red[hw][r][c + e];
#pragma unroll
          for (int k = 1; k < kSplit; ++k) y[e] += red[hw + k * HEADS][r][c + e];
          y[e] = none ? 0.0f : y[e] * inv;
          bad = fmaf(y[e], 0.0f, bad);
        }
        if (bad != 0.0f) row_bad[row] = any_bad = 1;
        if (whole) {
          store8(p, size_t(sg.doc.q0 + i) * size_t(p.os) + size_t(head) * size_t(p.D) + size_t(c), y);
        } else {
          put_part(mine + row * p.D + c, y);
          if (c == 0) __stcg(reinterpret_cast<float2*>(mine_ml) + row, make_float2(mx, sum));
        }
      }
      if (__syncthreads_or(any_bad)) {
        // (with one head every fourth row a warp, with two every second)
        const int hw = warp % HEADS;
        unsigned redo = 0;
        for (int r = warp / HEADS; r < rows; r += kSplit)
          if (row_bad[hw * rows + r]) redo |= 1u << r;
        if (redo)
          few_again(p, {sg.doc.q0, sg.doc.k0, sg.doc.lq, lk, sg.doc.prefix, sg.kvh, sg.row0, sg.s0 * kStep, last, rows, mine,
                      mine_ml}, hw, redo);
        __syncthreads();  // row_bad is free again
      }
      if (whole) continue;

      // the last CTA of the item's parts joins them, in order
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) seen = atomicInc(p.counters + c0 * 4, unsigned(c1 - c0));  // 0 .. c1 - c0, then 0 again
      __syncthreads();
      if (seen == unsigned(c1 - c0)) {
        __threadfence();
        if (HEADS * rows >= 4) {  // a warp a row
          for (int row = warp; row < HEADS * rows; row += 4) join_row(row / rows, row % rows);
        } else {  // every fourth part a warp
          for (int row = 0; row < HEADS * rows; ++row) {
            float mx, sum;
            const float4 a = parts.sums(row, lane, warp, 4, mx, sum);
            if (lane == 0) red_m[warp][row] = mx, red_l[warp][row] = sum;
            if (lane < p.D / 4) *reinterpret_cast<float4*>(&red[warp][row][4 * lane]) = a;
          }
          __syncthreads();
          for (int x = int(threadIdx.x); x < HEADS * rows * chunks; x += kFewThreads) {
            const int row = x / chunks, c = 8 * (x - row * chunks);
            int hw, r, i, head;
            row_of(row, hw, r, i, head);
            float mx = red_m[0][row], sum = 0.0f, y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 1; k < 4; ++k) mx = fmaxf(mx, red_m[k][row]);
            const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f = ex2(red_m[k][row] - ref);
              sum = fmaf(f, red_l[k][row], sum);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = fmaf(f, red[k][row][c + e], y[e]);
            }
            const bool none = limit_of(p.causal, i + lk - sg.doc.lq, lk, sg.doc.prefix) == 0;
            const float inv = 1.0f / sum;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = none ? 0.0f : y[e] * inv;
            store8(p, size_t(sg.doc.q0 + i) * size_t(p.os) + size_t(head) * size_t(p.D) + size_t(c), y);
          }
        }
      }
      __syncthreads();  // `seen` and the merge buffers are free again
    }
  }
}

template <int KI, int VI, int NT, int HEADS, bool TAIL = false>
cudaError_t few_launch_as(const Params& p, cudaStream_t s) {
  const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  return launch_pdl(few_kernel<KI, VI, NT, HEADS, TAIL>, dim3(unsigned(sms * per_sm(NT))), dim3(kFewThreads), 0, s,
                    p);
}

template <int NT, int HEADS>
cudaError_t few_launch_rows(const Params& p, cudaStream_t s) {
  if (p.D <= 64) return few_launch_as<2, 1, NT, HEADS>(p, s);
  // (eight behind whole groups of 32 of a key row and of 64 of a value row; of 40 and 104 the value row's groups are
  // the same with a tail and without)
  if (p.D == 64 + 8) return few_launch_as<2, 1, NT, HEADS, true>(p, s);
  if (p.D <= 96) return few_launch_as<3, 2, NT, HEADS>(p, s);
  return few_launch_as<4, 2, NT, HEADS>(p, s);
}

template <int NT>
cudaError_t few_launch_heads(const Params& p, cudaStream_t s) {
  // Neighbouring heads in a CTA where a head's row is no whole number of 64 bytes (64 probes over
  // images, 16 heads of 72: 40 us against 58 with a head per CTA and 46 with two); else a head per CTA, whose
  // warps then share its long run of keys (one token of 16 requests, 8 key heads of 128: 162 us
  // against 178). Also where there is so little to read that a head's keys had better be spread
  // over as many warps as there are.
  const bool little = static_cast<long long>(p.total_k) * p.hk <= 64ll * 8 * kMaxSms;
  if (p.D % 32 && !little && p.hk % 4 == 0) return few_launch_rows<NT, 4>(p, s);
  if (p.D % 32 && !little && p.hk % 2 == 0) return few_launch_rows<NT, 2>(p, s);
  return few_launch_rows<NT, 1>(p, s);
}

}  // namespace

size_t few_workspace(int head_dim) {
  // two parts a CTA of up to four heads of 8 rows (three CTAs an SM) or 16 (two CTAs)
  const size_t rows = size_t(kMaxSms) * (kMostPerSm * 8 > 2 * 16 ? kMostPerSm * 8 : 2 * 16);
  return kCounterBytes + rows * 2 * 4 * size_t(head_dim + 2) * sizeof(float);
}

sv_status few_launch(const Params& p, cudaStream_t s) {
  static_assert(kMaxFewGrid * 4 * sizeof(unsigned) <= kTicket * sizeof(unsigned), "counters");
  // rows of the documents on average decide between one and two 8-row tiles
  const bool small = static_cast<long long>(p.total_q) * p.group <= 8ll * p.docs;
  const cudaError_t e = small ? few_launch_heads<1>(p, s) : few_launch_heads<2>(p, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "packed attention launch (few rows)");
}

}  // namespace packed
}  // namespace sv
