// The passes of sv_attention_cached for many rows, on the tensor cores, scores never leaving the SM: all rows of the batch
// over the keys that its sequences share (the prefix pass), and sequences of several queries each over their own tokens
// (OWN).
//
// A row is a query and one of the query heads of a key head (row = query x group + head). Of the prefix every row sees
// every key, so that nothing but the last tile's end is masked; of its sequence's own tokens a row sees the first
// limit_of(). For each row, in F32,
//   s_j = scale q . k_j, capped;  O = sum_j 2^(s_j log2 e - m) v_j,  l = sum_j 2^(s_j log2 e - m),
// m following the running maximum, go to the workspace, a part for each CTA that has worked on the row's item;
// cached_attention.cu joins them.
//
// A CTA (one per SM) has two tiles of 128 rows, or (SOLO: at most 128 rows in the batch, and OWN) one whose key tiles two
// groups take in turn. 16 warps:
//   warps 0..3, 4..7   softmax of group 0 and 1: a thread per row turns its S row into P (F16, over S in tensor memory);
//   warp 8             the MMA issuer: S_w = Q_w K^T (shared memory, 128-byte swizzle), O_w += P_w V (P from tensor memory);
//   warp 9             copies keys and values in turn, with their scale bytes, page by page (a lane each): E4M3 codes as
//                      they lie into a ring of their own, F16 numbers by TMA into the operands' ring. OWN: it also works
//                      out the CTA's share of the sequences, run by run, and hands the runs to the others;
//   warps 10..13       the operands, 32 rows of every tile a warp: codes in F16 with their factors applied (exactly, as
//                      sv_cache_read does). Marked ones become NaN, and with them every row; OWN, where not every row sees
//                      every key: the key of a marked value becomes NaN in its place (the value's numbers stay 0, so
//                      that a probability of 0 keeps it out). Keys and values behind the last one become zeros.
//   warps 14, 15       bring Q, all of it on its way at once (eight 16-byte loads a thread at a time, by way of registers:
//                      256 samples 170 us, now 162; 32 requests of 4 rows behind 8192 keys 32, now 30).
// Tensor memory: S_0, S_1, O_0, O_1 of 128 columns each.
//
// Two tiles of rows and 128 keys of 128 dimensions take 3,700 cycles: the products 2,048, the exponentials 2,048, shared
// memory's traffic 2,560, and what bounds it: the softmax of a group, its products and the next scores, one behind the
// other, 3,400 (256 samples of 32 heads over 32768 shared keys: 107 us of 160, 1,280 TFLOP/s). One tile of rows takes
// 3,000: the copies of codes on their way (four tiles of 16 KB instead of two: 3,360 before) and the same chain (8
// sequences of 15000 keys, 128 rows of 8 key heads each: 97 us, 2.6 TB/s, 650 TFLOP/s).
#include "cached.h"
#include "packed_attention.h"

namespace sv {
namespace cached {
namespace {

using packed::capped4;
using packed::cap_factor;
using packed::far_capped;
using packed::kFarCap;
using packed::kHead;
using packed::kLog2e;
using packed::kSlack;

constexpr int kTile = kTileRows;
constexpr int kBoxBytes = kTile * 128;  // 128 rows of 64 values
// Four warpgroups, whose registers are shared out anew at the start: 2 x 128 x 176 + 2 x 128 x 80 = 512 x 128.
constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
constexpr int kLoadWarps = 4;           // warps 10..13
constexpr int kQueryThreads = 64;       // of warps 14, 15
constexpr uint32_t kTmemCols = 512;
constexpr int kRunSlots = 2;            // runs between warp 9 and the others
constexpr int kOwnTotals = 32;
// Steps of a run at most. The tensor cores add to O by truncation: up to 16384 keys an accumulator its sums lose 1e-4 (with
// 2^20 they lost 6.6e-3, and with 2^28 equal ones stopped growing). What an item's runs leave behind is added up in F32.
constexpr int kMostSteps = 128;

// Operand tiles and, of E4M3, tiles of codes on their way. One tile of rows (SOLO) asks less of the tensor cores, and what
// it waits for is the copies: more of them, fewer operands.
template <int NB, bool E4M3, bool SOLO>
struct Smem {
  static constexpr int kOp = NB * kBoxBytes;  // one operand tile
  static constexpr int kStages = E4M3 && SOLO ? (NB == 1 ? 5 : 3) : (NB == 1 ? 8 : 4);
  static constexpr int kRaws = E4M3 ? (SOLO ? 8 : 4) / NB : kStages;  // tiles of codes; F16: of scale bytes alone
  static constexpr int kRaw = E4M3 ? kTile * 64 * NB : 0;
  static constexpr int kOffRing = 2 * kOp;                      // behind Q
  static constexpr int kOffRaw = kOffRing + kStages * kOp;
  static constexpr int kOffScales = kOffRaw + kRaws * kRaw;     // scale bytes of each tile; of keys, their values' behind
  // SOLO: exponents and sums of both groups' rows, then 4 KB a softmax warp; in place of a second tile of Q where that is
  // large enough
  static constexpr int kOffJoin = NB == 2 ? kOp : kOffScales + 2 * kRaws * kTile;
  static constexpr int kOffBar = kOffScales + 2 * kRaws * kTile + (NB == 2 ? 0 : 8 * 4096);
  static constexpr int kOffRuns = kOffBar + 448;
  static constexpr int kOffTotals = kOffRuns + kRunSlots * 64;
  static constexpr int kBytes = 1024 + kOffTotals + kOwnTotals * 8;
  static_assert(kBytes <= 232448, "shared memory budget");
};

enum {
  kBarFull = 0,    // +stage: the operand tile is written
  kBarEmpty = 8,   // +stage: products that read it have finished
  kBarRaw = 16,    // +tile of the copies' ring: it has arrived
  kBarRawFree = 24,
  kBarQFull = 32,
  kBarQEmpty = 33,
  kBarSFull = 34,  // +group: S_w has finished (and with it the P V products before it)
  kBarPFull = 36,  // +group: P_w (and any O rescale) is in tensor memory
  kBarOFull = 38,  // +group: the segment's last P V product has finished
  kBarJoin = 40,   // SOLO: both groups' exponents and sums are in shared memory
  kBarRead = 41,   // SOLO: both have read O
  kBarDrain = 42,
  kBarJoined = 43,  // SOLO: both groups have read the other's exponents and sums
  kBarRun = 44,     // OWN, +slot: warp 9 has written the run
  kBarRunDone = 46, // OWN, +slot: the other warps have read it
  kNumBars = 48
};

// A run of steps of one item that falls into this CTA's share.
struct Run {
  int item, s0, s1, kvh;  // (s1 0: there are no more)
  int row0;               // first of the item's rows among those of the sequence, or of the batch
  int q0, n, have;        // first row of q, queries, keys
  int again;              // the CTA's run before was of the same item: its sums are in the part
  const int* pages;
};
// The prefix pass: all rows of the batch over one run of keys.
struct Runs {
  int at, end, begin;
  __device__ __forceinline__ Runs(const Params& p) {
    const int work = p.pre.blocks * p.c.hk * p.pre.steps;
    begin = at = p.pre.chunk * int(blockIdx.x);
    end = min(at + p.pre.chunk, work);
  }
  __device__ __forceinline__ bool get(const Params& p, Run& r) {
    if (at >= end) return false;
    r.item = at / p.pre.steps;
    const int base = r.item * p.pre.steps;
    r.s0 = at - base;
    r.s1 = min(min(end - base, p.pre.steps), r.s0 + kMostSteps);
    r.again = r.s0 > 0 && at > begin;
    r.kvh = r.item / p.pre.blocks;
    r.row0 = (r.item - r.kvh * p.pre.blocks) * p.pre.rows;
    r.q0 = 0;
    r.n = p.total_q;
    r.have = p.c.prefix_len;
    r.pages = p.c.prefix_pages;
    at = base + r.s1;
    return true;
  }
};
// The sequences' pass, worked out by one warp: sequences, key heads, blocks of rows in order, 32 sequences at a time, one
// per lane; every CTA has an equal, contiguous share of the steps. totals: steps and items of the first sequences, 32
// and 32 (shared memory).
class OwnRuns {
 public:
  __device__ __forceinline__ OwnRuns(const Params& p, int lane, int2* totals) : p_(p), lane_(lane), count_(p.c.count) {
    unsigned work = 0;
    bool bad = false;
#pragma unroll 4
    for (int d0 = 0; d0 < count_; d0 += 32) {
      bad |= !load(d0);
      const unsigned steps = __reduce_add_sync(0xffffffffu, unsigned(blocks_ * p.c.hk * steps_));
      const unsigned items = __reduce_add_sync(0xffffffffu, unsigned(blocks_ * p.c.hk));
      if (lane == 0 && d0 < 32 * kOwnTotals) totals[d0 / 32] = make_int2(int(steps), int(items));
      work += steps;
    }
    // bad offsets or lengths: reported, and nothing is computed
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0) atomicOr(p.c.err, kDevErrCache);
      count_ = 0;
      work = 0;
    }
    const unsigned chunk = max(1u, (work + gridDim.x - 1) / gridDim.x);
    if (blockIdx.x == 0 && lane == 0) p.firsts[p.c.count] = make_int2(int(chunk), 0);
    begin_ = at_ = int(min(chunk * blockIdx.x, work));
    end_ = int(min(unsigned(at_) + chunk, work));
    __syncwarp();
    int d0 = 0;
    while (d0 + 32 < count_ && d0 < 32 * kOwnTotals && base_ + totals[d0 / 32].x <= at_) {
      base_ += totals[d0 / 32].x;
      items_base_ += totals[d0 / 32].y;
      d0 += 32;
    }
    load(d0);
    open();
  }
  __device__ __forceinline__ void get(Run& r) {
    r = {};
    if (at_ >= end_) return;
    while (at_ >= base_ + total_) {
      base_ += total_;
      items_base_ += items_total_;
      load(d0_ + 32);
      open();
    }
    const int src = __ffs(int(__ballot_sync(0xffffffffu, base_ + incl_ > at_))) - 1;
    auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
    const int blocks = of(blocks_), steps = of(steps_), items = blocks * p_.c.hk;
    const int first = base_ + of(incl_) - items * steps, item0 = items_base_ + of(items_) - items;
    const int k = (at_ - first) / steps;  // among the sequence's items
    r.item = item0 + k;
    r.kvh = k / blocks;
    r.row0 = (k - r.kvh * blocks) * kTileRows;
    r.s0 = at_ - (first + k * steps);
    r.s1 = min(min(end_ - (first + k * steps), steps), r.s0 + kMostSteps);
    r.again = r.s0 > 0 && at_ > begin_;
    r.q0 = of(seq_.q0);
    r.n = of(seq_.n);
    r.have = of(seq_.have);
    r.pages = p_.c.table + static_cast<long long>(d0_ + src) * p_.c.stride;
    if (at_ == first && lane_ == 0) p_.firsts[d0_ + src] = make_int2(item0, first);  // (one run of the launch is this one)
    at_ = first + k * steps + r.s1;
  }

 private:
  __device__ __forceinline__ bool load(int d0) {
    d0_ = d0;
    const bool good = sequence(p_, d0 + lane_, count_, seq_);
    blocks_ = (seq_.n * p_.group + kTileRows - 1) / kTileRows;
    steps_ = max(1, (seq_.have + 2 * kTileRows - 1) / (2 * kTileRows));  // (a step without keys leaves sums of 0)
    return good;
  }
  __device__ __forceinline__ void open() {
    items_ = blocks_ * p_.c.hk;
    incl_ = items_ * steps_;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, incl_, o), b = __shfl_up_sync(0xffffffffu, items_, o);
      if (lane_ >= o) incl_ += a, items_ += b;
    }
    total_ = __shfl_sync(0xffffffffu, incl_, 31);
    items_total_ = __shfl_sync(0xffffffffu, items_, 31);
  }
  const Params& p_;
  int lane_, count_, d0_, blocks_, steps_, incl_, items_, total_, items_total_;
  int at_, end_, begin_, base_ = 0, items_base_ = 0;
  Sequence seq_;
};

// `bytes` (a multiple of 16, both addresses on 16) from global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
               "r"(bytes), "r"(bar)
               : "memory");
}

// 16 bytes to shared memory, `some` of them (16 or 0) from global memory and zeros else; on its way until cp.async.wait_all.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, uint32_t some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(some) : "memory");
}

// Eight words on 32 bytes: a whole sector a lane (by 16 bytes the sums of a CTA's rows took twice as long to leave).
__device__ __forceinline__ void store8(float* to, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// 16-byte chunk of row `row` of an operand tile (64 values a box, 128-byte swizzle).
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  return uint32_t((chunk >> 3) * kBoxBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// pages: F16 pages as a tensor of [n_pages, 2 * kv_heads * page_size (keys, then values), head_dim].
// OWN (with SOLO): the sequences' rows over their own tokens; else all rows over the prefix. FULL: heads of 64 NB dimensions.
template <int NB, bool E4M3, bool SOLO, bool OWN, bool CAP, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
    cached_tile_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap pages_map) {
  using L = Smem<NB, E4M3, SOLO>;
  constexpr int kOp = L::kOp, kStages = L::kStages, kRaws = L::kRaws;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::kOffBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(8 * kNumBars + 8 <= 448 && sizeof(Run) <= 64, "barrier area");
  static_assert(!OWN || SOLO, "one tile of rows an item");
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const View& c = p.c;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), kLoadWarps);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int s = 0; s < kRaws; ++s) {
      mbar_init(bar(kBarRaw + s), 1);
      mbar_init(bar(kBarRawFree + s), kLoadWarps);
    }
    mbar_init(bar(kBarQFull), kQueryThreads);
    mbar_init(bar(kBarQEmpty), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(kBarSFull + w), 1);
      mbar_init(bar(kBarPFull + w), 128);
      mbar_init(bar(kBarOFull + w), 1);
    }
    mbar_init(bar(kBarJoin), 256);
    mbar_init(bar(kBarJoined), 256);
    mbar_init(bar(kBarRead), 256);
    mbar_init(bar(kBarDrain), 1);
    for (int s = 0; s < kRunSlots; ++s) {
      mbar_init(bar(kBarRun + s), 1);
      mbar_init(bar(kBarRunDone + s), kThreads / 32 - 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // Dimensions between D and the next multiple of 16 are read by the products and never written: zeros for good.
  if (!FULL && c.D % 16)
    for (int x = int(threadIdx.x); x < (2 + kStages) * kTile; x += kThreads)
      *reinterpret_cast<uint4*>(smem + x / kTile * kOp + chunk_at(x % kTile, c.D / 8)) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The sequences' pass behind a prefix pass begins as soon as SMs come free of that one, whose results it does not need: what
  // came before the two is complete, since the prefix pass lets others begin only after its own wait. It waits before it
  // ends, for the kernel that joins the parts of both. (24 requests of 35 rows behind 2047 keys: 55 us without, 51 so.)
  const bool early = OWN && c.prefix_len > 0;
  if (!early) pdl_wait();
  pdl_launch_dependents();
  auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, abort_flag, p.c.err); };
  auto wait_all = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };

  Runs runs(p);
  Run run = {};
  Run* ring = reinterpret_cast<Run*>(smem + L::kOffRuns);
  auto next_run = [&](int n) -> bool {  // run n of the CTA; false: there is none (or a wait has run out)
    if constexpr (!OWN) return runs.get(p, run);
    const int slot = n % kRunSlots;
    if (!wait_all(kBarRun + slot, (n / kRunSlots) & 1)) return false;
    run = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarRunDone + slot));
    return run.s1 > 0;
  };
  // Operand tile x of a run of `count` tiles from jb on: keys, values, keys, ... of one tile after another; SOLO: the keys
  // of two tiles, their values, ...
  auto is_values = [](int x) { return ((SOLO ? x >> 1 : x) & 1) != 0; };
  auto tile_of = [](int x) { return SOLO ? (x >> 2) * 2 + (x & 1) : x >> 1; };
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int w = warp >> 2;             // group
    const int r = (warp & 3) * 32 + lane;  // row of the tile == lane of tensor memory
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + uint32_t(w * 128) + lane_off;
    const uint32_t o_tm = tmem + uint32_t(256) + lane_off;  // of group 0
    const int Dn = (c.D + 15) / 16 * 16;
    const float sl2 = CAP ? cap_factor(p.scale, p.cap) : kLog2e * p.scale;
    const float on = CAP ? 1.0f : sl2;  // factor on the (capped) scores before the exponentials
    const float cap2 = p.cap * kLog2e;
    float2* join = reinterpret_cast<float2*>(smem + L::kOffJoin);
    bool ok = true;
    uint32_t t = 0;  // parity of the tiles so far
    for (int n = 0; ok && next_run(n); ++n) {
      const int j0 = SOLO ? 2 * run.s0 + w : run.s0, je = SOLO ? 2 * run.s1 : run.s1;
      const int rows_all = run.n * p.group, row = run.row0 + (SOLO ? 0 : w * kTile) + r;  // of the sequence, or of the batch
      // keys that the row sees
      const int seen = OWN && row < rows_all ? limit_of(p.causal, query_of(p, row), run.n, run.have) : run.have;
      float m = -INFINITY, l = 0.0f;
      for (int j = j0; j < je; j += SOLO ? 2 : 1, t ^= 1) {
        if (!(ok = wait_all(kBarSFull + w, t))) break;
        tc_fence_after();
        const int valid = seen - j * kTile;  // keys of the tile
        // (scores stay the words that tensor memory gives: the compiler may order accesses of two types as it likes)
        auto prepare = [&](uint32_t* s, int first) {  // 32 scores from column `first` on: capped, hidden ones -inf
          if constexpr (CAP) {
            if (OWN && valid < first + 32) {  // four scores share a reciprocal: a hidden NaN must not reach the others
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (first + e >= valid) s[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float big[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) big[k] = __uint_as_float(s[e + k]);
              capped4(big, sl2, cap2);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float x = __uint_as_float(s[e + k]);
                s[e + k] = __float_as_uint(p.cap < kFarCap ? big[k] : far_capped(x * (kLog2e * p.scale), x * sl2, big[k]));
              }
            }
          }
          if (valid < first + 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (first + e >= valid) s[e] = 0xff800000u;
          }
        };
        auto top_of = [&](const uint32_t* s, float mx) {
          auto f = [&](int e) { return __uint_as_float(s[e]); };
          float a = fmax3(mx, f(0), f(1)), b = fmaxf(f(2), f(3));
#pragma unroll
          for (int e = 4; e < 32; e += 4) {
            a = fmax3(a, f(e), f(e + 1));
            b = fmax3(b, f(e + 2), f(e + 3));
          }
          return fmaxf(a, b);
        };
        // Four scores share a reciprocal, and behind the prefix's last key a zero times an infinite query is NaN: the hidden ones
        // beside visible ones become 0 in tensor memory. (In registers, as above, 64 requests behind 4096 keys: 51 us, so 45.)
        if constexpr (CAP && !OWN) {
          if (valid > 0 && valid < kTile && (valid & 3)) {  // (the same for all rows)
            uint32_t e[8];
            tmem_ld8(s_tm + uint32_t(valid & ~7), e);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              asm volatile("" : "+r"(e[k]));  // no use before the wait
              if (k >= (valid & 7)) e[k] = 0u;
            }
            tmem_st8(s_tm + uint32_t(valid & ~7), e);
            tmem_st_wait();
          }
        }
        uint32_t ua[4][32];
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(s_tm + 32 * k, ua[k]);
        tmem_ld_wait(ua[0]);
        reg_fence(ua[1]);
        reg_fence(ua[2]);
        reg_fence(ua[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          prepare(ua[k], 32 * k);
          mx = top_of(ua[k], mx);
        }
        mx *= on;
        const bool raise = mx > m + kSlack;
        const float m_new = raise ? mx - kHead : m;
        if (j > j0 && __any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2(m - m_new) : 1.0f;
          l *= f;
#pragma unroll 1
          for (int d = 0; d < Dn; d += 8) {
            uint32_t e[8];
            tmem_ld8(o_tm + uint32_t(128 * w + d), e);
            tmem_ld_wait();
            asm volatile("" : "+r"(e[0]), "+r"(e[1]), "+r"(e[2]), "+r"(e[3]), "+r"(e[4]), "+r"(e[5]), "+r"(e[6]), "+r"(e[7]));
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = __float_as_uint(__uint_as_float(e[k]) * f);
            tmem_st8(o_tm + uint32_t(128 * w + d), e);
          }
        }
        m = m_new;
        const float ref = m == -INFINITY ? 0.0f : m;
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
        auto exponentials = [&](const uint32_t* s, uint32_t* pk) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            fma_x2(x0, x1, __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), on, on, -ref, -ref);
            x0 = ex2(x0);
            x1 = ex2(x1);
            if (e & 1) add_x2(s2, s3, s2, s3, x0, x1);
            else add_x2(s0, s1, s0, s1, x0, x1);
            // F16, what the products take at full rate: 2^-11 of each probability; their sum l is of the unrounded ones
            const __half2 y = __floats2half2_rn(x0, x1);
            pk[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
        };
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          uint32_t pk[32];
          exponentials(ua[k], pk);
          exponentials(ua[k + 1], pk + 16);
          tmem_st32(s_tm + 16 * k, pk);
        }
        l += (s0 + s1) + (s2 + s3);
        tmem_st_wait();
        if (SOLO && n > 0 && j == j0) {  // both groups have read what the next P V overwrites
          if (!(ok = wait_all(kBarRead, (n - 1) & 1))) break;
        }
        tc_fence_before();
        mbar_arrive(bar(kBarPFull + w));
      }
      if (!ok) break;
      // the run's sums: a part of the row's result
      const int at = (SOLO ? 0 : w * kTile) + r, part_rows = SOLO ? kTile : 2 * kTile;  // in the part
      float* part = (OWN ? p.tiles : p.pre.base) + size_t(run.item + int(blockIdx.x)) * (size_t(part_rows) * size_t(c.D + 2));
      float2* exponents = reinterpret_cast<float2*>(part + size_t(part_rows) * c.D) + at;
      const bool live = row < rows_all;
      // factors on the groups' O (SOLO; else on the group's own) and on what the item's run before has left
      float f0 = 1.0f, f1 = 0.0f, keep = 0.0f;
      float2 before = make_float2(-INFINITY, 0.0f);
      if (run.again && live) before = __ldcg(exponents);
      if constexpr (SOLO) {
        join[w * kTile + r] = make_float2(m, l);
        mbar_arrive(bar(kBarJoin));
        if (!(ok = wait_all(kBarJoin, n & 1) && wait_all(kBarOFull, n & 1) && wait_all(kBarOFull + 1, n & 1))) break;
        const float2 a = join[r], b = join[kTile + r];
        m = fmax3(a.x, b.x, before.x);
        const float ref = m == -INFINITY ? 0.0f : m;
        f0 = ex2(a.x - ref);
        f1 = ex2(b.x - ref);
        keep = ex2(before.x - ref);
        l = fmaf(keep, before.y, fmaf(f1, b.y, f0 * a.y));
      } else {
        if (!(ok = wait_all(kBarOFull + w, n & 1))) break;
        if (run.again) {
          const float up = fmaxf(m, before.x), ref = up == -INFINITY ? 0.0f : up;
          f0 = ex2(m - ref);
          keep = ex2(before.x - ref);
          l = fmaf(keep, before.y, f0 * l);
          m = up;
        }
        if (live) __stcg(exponents, make_float2(m, l));
      }
      tc_fence_after();
      if constexpr (SOLO) {
        // Both groups have read the other's exponents and sums, and those of the run before: the place is the warps' to turn
        // rows round in, so that eight lanes write 128 bytes of a row (a row a lane: 6,000 cycles, more than two tiles of
        // keys take).
        mbar_arrive(bar(kBarJoined));
        if (!(ok = wait_all(kBarJoined, n & 1))) break;
        if (live && w == 0) __stcg(exponents, make_float2(m, l));
        uint8_t* stage = smem + L::kOffJoin + warp * 4096;
#pragma unroll 1
        for (int d = 32 * w; d < Dn; d += 64) {  // every second 32 columns
          uint32_t a[32], b[32];
          tmem_ld32(o_tm + uint32_t(d), a);
          tmem_ld32(o_tm + uint32_t(128 + d), b);
          tmem_ld_wait(a);
          reg_fence(b);
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(fmaf(f1, __uint_as_float(b[e]), f0 * __uint_as_float(a[e])));
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                make_uint4(a[4 * u], a[4 * u + 1], a[4 * u + 2], a[4 * u + 3]);
          __syncwarp();
          if (run.again)  // what this lane has written there, added in the place where it reads next
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const int x = 4 * i + (lane >> 3), u = lane & 7;
              const float k = __shfl_sync(0xffffffffu, keep, x);
              if (row - lane + x >= rows_all || d + 4 * u >= c.D) continue;
              const float4 z = __ldcg(reinterpret_cast<const float4*>(part + size_t(at - lane + x) * c.D + d + 4 * u));
              float4& y = *reinterpret_cast<float4*>(stage + x * 128 + ((u ^ (x & 7)) << 4));
              y = make_float4(fmaf(k, z.x, y.x), fmaf(k, z.y, y.y), fmaf(k, z.z, y.z), fmaf(k, z.w, y.w));
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int x = 4 * i + (lane >> 3), u = lane & 7;  // row of the warp, 16 bytes of it
            const uint4 y = *reinterpret_cast<const uint4*>(stage + x * 128 + ((u ^ (x & 7)) << 4));
            if (row - lane + x < rows_all && d + 4 * u < c.D)
              __stcg(reinterpret_cast<uint4*>(part + size_t(at - lane + x) * c.D + d + 4 * u), y);
          }
          __syncwarp();
        }
        tc_fence_before();
        mbar_arrive(bar(kBarRead));
      } else {
#pragma unroll 1
        for (int d = 0; d < Dn; d += 16) {
          uint32_t a[16];
          tmem_ld16(o_tm + uint32_t(128 * w + d), a);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(a[e]));  // no use before the wait
          if (run.again && live) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              if (e == 8 && d + 8 >= c.D) break;
              const float4 z = __ldcg(reinterpret_cast<const float4*>(part + size_t(at) * c.D + d + e));
              a[e] = __float_as_uint(fmaf(keep, z.x, f0 * __uint_as_float(a[e])));
              a[e + 1] = __float_as_uint(fmaf(keep, z.y, f0 * __uint_as_float(a[e + 1])));
              a[e + 2] = __float_as_uint(fmaf(keep, z.z, f0 * __uint_as_float(a[e + 2])));
              a[e + 3] = __float_as_uint(fmaf(keep, z.w, f0 * __uint_as_float(a[e + 3])));
            }
          }
          if (live) {
            store8(part + size_t(at) * c.D + d, a);
            if (d + 8 < c.D) store8(part + size_t(at) * c.D + d + 8, a + 8);
          }
        }
      }
    }
    tmem_ld_wait();
    tmem_st_wait();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 9) {
      const int page_mask = (1 << c.shift) - 1, run_rows = min(kTile, page_mask + 1);
      // The pages of a tile's keys, a lane each (8 at most; runs of run_rows keys).
      auto pages_of = [&](int tile) -> int {
        const int number = ((tile * kTile) >> c.shift) + lane;
        if (lane >= kTile / run_rows || number >= (run.have + page_mask) >> c.shift) return -1;
        const int page = __ldg(run.pages + number);
        if (unsigned(page) < unsigned(c.n_pages)) return page;
        atomicOr(c.err, kDevErrCache);
        return 0;
      };
      if (!E4M3 && lane == 0) prefetch_tmap(&pages_map);
      uint32_t issued = 0, issued_phase = 0;  // copies in flight per tile of the ring, and their phase bits
      int use = 0;
      bool ok = true;
      auto copies_of = [&]() {  // of the run
        const int jb = SOLO ? 2 * run.s0 : run.s0, count = 2 * (run.s1 - run.s0) * (SOLO ? 2 : 1);
        int page = pages_of(jb);
        for (int x = 0; x < count; ++x, ++use) {
          const int tile = jb + tile_of(x);
          const int next = x + 1 < count ? pages_of(jb + tile_of(x + 1)) : -1;
          const int slot = use % kRaws;
          if (!(ok = wait_all((E4M3 ? kBarRawFree : kBarEmpty) + slot, ((use / kRaws) & 1) ^ 1))) break;
          const int copies = __popc(__ballot_sync(0xffffffffu, page >= 0));
          const uint32_t full = bar(kBarRaw + slot);
          const bool values = is_values(x);
          if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(copies * run_rows * ((OWN && !values ? 2 : 1) + (E4M3 ? c.D : NB * 128))));
          issued |= 1u << slot;
          issued_phase = (issued_phase & ~(1u << slot)) | uint32_t((use / kRaws) & 1) << slot;
          __syncwarp();
          if (page >= 0) {
            const int at = (tile * kTile) & page_mask, row = ((run.kvh + (values ? c.hk : 0)) << c.shift) + at;
            const uint8_t* from = c.pages + page * c.page_bytes;
            const uint32_t to_scales = sbase + L::kOffScales + 2 * slot * kTile + lane * run_rows;
            bulk_load(to_scales, from + scale_bytes(c) + row, uint32_t(run_rows), full);
            if (OWN && !values)
              bulk_load(to_scales + kTile, from + scale_bytes(c) + (c.hk << c.shift) + row, uint32_t(run_rows), full);
            if constexpr (E4M3) {
              bulk_load(sbase + L::kOffRaw + slot * L::kRaw + lane * run_rows * c.D, from + row * c.D, uint32_t(run_rows * c.D), full);
            } else {
              for (int b = 0; b < NB; ++b)
                tma_load_3d(sbase + L::kOffRing + slot * kOp + b * kBoxBytes + lane * run_rows * 128, &pages_map, full, 64 * b, row, page);
            }
          }
          page = next;
        }
      };
      if constexpr (OWN) {
        OwnRuns own(p, lane, reinterpret_cast<int2*>(smem + L::kOffTotals));
        for (int n = 0; ok; ++n) {
          own.get(run);
          const int slot = n % kRunSlots;
          if (!(ok = wait_all(kBarRunDone + slot, ((n / kRunSlots) & 1) ^ 1))) break;
          if (lane == 0) {
            ring[slot] = run;
            mbar_arrive(bar(kBarRun + slot));
          }
          __syncwarp();
          if (run.s1 == 0) break;
          copies_of();
        }
      } else {
        while (ok && runs.get(p, run)) copies_of();
      }
      // (after a time-out: every copy issued lands before the CTA can exit)
      for (int i = 0; i < kRaws; ++i)
        if (issued & (1u << i)) mbar_wait_bounded(bar(kBarRaw + i), (issued_phase >> i) & 1, p.c.err);
    } else if (warp >= 14) {
      const int tid = int(threadIdx.x) - 14 * 32;
      const int per_row = FULL ? 8 * NB : c.D / 8;  // 16-byte chunks of a row
      bool ok = true;
      for (int n = 0; ok && next_run(n); ++n) {
        if (!(ok = wait_all(kBarQEmpty, (n & 1) ^ 1))) break;
        const int rows_all = run.n * p.group;
        const int row_step = kQueryThreads / per_row, chunk_step = kQueryThreads % per_row;
        int row = tid / per_row, chunk = tid % per_row;  // (rows of both tiles)
#pragma unroll 4
        for (; row < (SOLO ? 1 : 2) * kTile;) {
          const int r = run.row0 + row, q = query_of(p, r);
          const bool live = r < rows_all;  // (zeros elsewhere)
          const __half* from = p.q + (run.q0 + q) * p.qs + (run.kvh * p.group + (r - q * p.group)) * c.D + 8 * chunk;
          copy16(sbase + (row >= kTile ? kOp : 0) + chunk_at(row & (kTile - 1), chunk), live ? from : p.q, live ? 16u : 0u);
          row += row_step;
          chunk += chunk_step;
          if (chunk >= per_row) chunk -= per_row, ++row;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(bar(kBarQFull));
      }
    } else if (warp >= 10) {
      const int per_row = FULL ? 8 * NB : c.D / 8;
      const int first = 32 * (warp - 10);  // row of the warp's piece of every tile
      int use = 0;                         // operand tiles so far
      bool ok = true;
      for (int n = 0; ok && next_run(n); ++n) {
        const int jb = SOLO ? 2 * run.s0 : run.s0, count = 2 * (run.s1 - run.s0) * (SOLO ? 2 : 1);
        constexpr int kMost = 8 * NB;  // chunks of a lane: of the rows `row`, `row` + row_step, ...
        const int row0 = lane / per_row, chunk0 = lane % per_row, row_step = 32 / per_row, chunk_step = 32 % per_row;
#pragma unroll 1
        for (int x = 0; x < count; ++x, ++use) {
          const int slot = use % kRaws, st = use % kStages;
          const int left = run.have - (jb + tile_of(x)) * kTile - first;  // keys of the piece
          if (!(ok = wait_all(kBarRaw + slot, (use / kRaws) & 1))) break;
          // The scale byte of row `lane`. OWN: a marked value makes its key NaN, for the rows that see it.
          const uint8_t* scales = smem + L::kOffScales + 2 * slot * kTile + first + lane;
          int byte = lane < left ? scales[0] : kNoScale;
          if constexpr (OWN) {
            if (is_values(x)) byte = byte == kMarked ? kNoScale : byte;
            else if (lane < left && scales[kTile] == kMarked) byte = kMarked;
          }
          uint8_t* to = smem + L::kOffRing + st * kOp + first * 128;
          if constexpr (E4M3) {
            // The codes go to registers first: their ring is free for the next copy before this tile has its place.
            const uint2* raw = reinterpret_cast<const uint2*>(smem + L::kOffRaw + slot * L::kRaw + first * c.D) + lane;
            uint2 codes[kMost];
#pragma unroll
            for (int i = 0; i < kMost; ++i)
              if (FULL || i < per_row) codes[i] = raw[i * 32];
            const uint32_t power = byte == 1 ? 0x0200u : uint32_t(byte - 1) << 10;
            const uint32_t factor = byte == kMarked ? 0x7e007e00u : power << 16 | power;
            // The next copy writes by the async proxy, which an arrival alone does not hold back behind these reads: without
            // the fence one call of 100 (256 samples behind 32768 keys) took 32 factors from the tile behind.
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarRawFree + slot));
            if (!(ok = wait_all(kBarEmpty + st, ((use / kStages) & 1) ^ 1))) break;
            int row = row0, chunk = chunk0;
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
              if (!FULL && i >= per_row) continue;
              if (left < 32 && row >= left) codes[i] = make_uint2(0u, 0u);
              uint4 y = e4m3_to_f16(codes[i]);
              const uint32_t w = __shfl_sync(0xffffffffu, factor, row);
              const __half2 f = *reinterpret_cast<const __half2*>(&w);
              __half2* h = reinterpret_cast<__half2*>(&y);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = __hmul2(h[e], f);
              // (whole heads: the steps change bits of the row that row0 leaves 0)
              if constexpr (FULL)
                *reinterpret_cast<uint4*>(to + (chunk_at(row0, chunk0) ^ uint32_t((i * (4 / NB) & 7) << 4)) + i * (4 / NB) * 128) = y;
              else
                *reinterpret_cast<uint4*>(to + chunk_at(row, chunk)) = y;
              row += row_step;
              chunk += chunk_step;
              if (!FULL && chunk >= per_row) chunk -= per_row, ++row;
            }
          } else if (lane >= left || byte == kMarked) {
            const uint32_t y = lane >= left ? 0u : 0x7e007e00u;
            for (int i = 0; i < per_row; ++i) *reinterpret_cast<uint4*>(to + chunk_at(lane, i)) = make_uint4(y, y, y, y);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarFull + st));
        }
      }
    } else if (warp == 8) {
      constexpr uint32_t idesc_s = make_idesc(128, 128, 0, false);
      const uint32_t idesc_o = make_idesc(128, (c.D + 15) / 16 * 16, 0, true);
      const int steps = FULL ? 4 * NB : (c.D + 15) / 16;
      const uint32_t lead = elect_one();
      auto commit = [&](int b) { tc_commit_if(lead, bar(b)); };
      int use = 0;  // operand tiles that earlier runs have used
      auto full = [&](int ahead) {
        const int u = use + ahead;
        const bool got = wait_all(kBarFull + u % kStages, (u / kStages) & 1);
        tc_fence_after();
        return got;
      };
      auto issue_s = [&](int w, int ahead) {
        const uint64_t qd = make_sdesc(sbase + uint32_t(SOLO ? 0 : w) * kOp, 16, 1024, 2);
        const uint64_t kd = make_sdesc(sbase + L::kOffRing + uint32_t((use + ahead) % kStages) * kOp, 16, 1024, 2);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 bytes of each row a step
            if (4 * b + kk < steps)
              mma_f16_if(lead, tmem + uint32_t(128 * w), qd + uint64_t(b * (kBoxBytes >> 4) + 2 * kk),
                         kd + uint64_t(b * (kBoxBytes >> 4) + 2 * kk), idesc_s, b + kk > 0);
        commit(kBarSFull + w);
      };
      auto issue_pv = [&](int w, int ahead, uint32_t keep) {
        const uint64_t vd = make_sdesc(sbase + L::kOffRing + uint32_t((use + ahead) % kStages) * kOp, kBoxBytes, 1024, 2);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // 16 keys a step: 8 columns of P, 16 rows of V
          mma_f16_ts_if(lead, tmem + uint32_t(256 + 128 * w), tmem + uint32_t(128 * w + 8 * kk),
                        vd + uint64_t(kk * (2048 >> 4)), idesc_o, kk > 0 ? 1u : keep);
      };
      auto empty = [&](int ahead) { commit(kBarEmpty + (use + ahead) % kStages); };
      uint32_t tt = 0;  // parity of the groups' tiles
      bool ok = true;
      for (int n = 0; ok && next_run(n); ++n) {
        const int count = run.s1 - run.s0;
        if (!(ok = wait_all(kBarQFull, n & 1))) break;
        if constexpr (SOLO) {
          for (int w = 0; w < 2 && ok; ++w) {
            if (!(ok = full(w))) break;
            issue_s(w, w);
            empty(w);
          }
          if (count == 1) commit(kBarQEmpty);
          for (int j = 0; ok && j < count; ++j, tt ^= 1, use += 4) {
            const bool last = j + 1 == count;
            for (int w = 0; w < 2 && ok; ++w) {
              if (!(ok = full(2 + w) && wait_all(kBarPFull + w, tt))) break;
              tc_fence_after();
              issue_pv(w, 2 + w, j > 0);
              empty(2 + w);
              if (last) {
                commit(kBarOFull + w);
              } else {
                if (!(ok = full(4 + w))) break;
                issue_s(w, 4 + w);
                empty(4 + w);
                if (w == 1 && j + 2 == count) commit(kBarQEmpty);
              }
            }
          }
        } else {
          if (!(ok = full(0))) break;
          issue_s(0, 0);
          issue_s(1, 0);
          empty(0);
          if (count == 1) commit(kBarQEmpty);
          for (int j = 0; ok && j < count; ++j, tt ^= 1, use += 2) {
            const bool last = j + 1 == count;
            if (!(ok = full(1) && (last || full(2)))) break;
            for (int w = 0; w < 2 && ok; ++w) {
              if (!(ok = wait_all(kBarPFull + w, tt))) break;
              tc_fence_after();
              issue_pv(w, 1, j > 0);
              if (last) commit(kBarOFull + w);
              else issue_s(w, 2);
            }
            if (!ok) break;
            empty(1);
            if (!last) empty(2);
            if (j + 2 == count) commit(kBarQEmpty);
          }
        }
      }
      commit(kBarDrain);
      __syncwarp();
      mbar_wait_bounded(bar(kBarDrain), 0, p.c.err);
    }
  }
  if (early) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int NB, bool E4M3, bool SOLO, bool OWN, bool CAP>
cudaError_t launch_as(const Params& p, const CUtensorMap& pages, int grid, cudaStream_t s) {
  // (whole heads' chunks lie where a thread need not work them out; E4M3 alone is converted)
  const bool full = E4M3 && p.c.D == 64 * NB;
  auto kern = full ? cached_tile_kernel<NB, E4M3, SOLO, OWN, CAP, E4M3> : cached_tile_kernel<NB, E4M3, SOLO, OWN, CAP, false>;
  static unsigned long long set[2] = {0, 0};
  const cudaError_t e = allow_shared(kern, Smem<NB, E4M3, SOLO>::kBytes, &set[full]);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(kThreads), size_t(Smem<NB, E4M3, SOLO>::kBytes), s, p, pages);
}

template <int NB, bool E4M3, bool SOLO, bool OWN>
cudaError_t launch_cap(const Params& p, const CUtensorMap& pages, int grid, cudaStream_t s) {
  return p.cap > 0.0f ? launch_as<NB, E4M3, SOLO, OWN, true>(p, pages, grid, s)
                      : launch_as<NB, E4M3, SOLO, OWN, false>(p, pages, grid, s);
}

template <bool SOLO, bool OWN>
sv_status launch(const char* fn, const Params& p, int grid, cudaStream_t s) {
  CUtensorMap pages = {};
  cudaError_t e;
  if (p.c.e4m3) {
    e = p.c.D > 64 ? launch_cap<2, true, SOLO, OWN>(p, pages, grid, s) : launch_cap<1, true, SOLO, OWN>(p, pages, grid, s);
  } else {
    const uint64_t dims[3] = {uint64_t(p.c.D), uint64_t(2 * p.c.hk) << p.c.shift, uint64_t(p.c.n_pages)};
    const uint64_t strides[2] = {uint64_t(p.c.D) * 2u, uint64_t(p.c.page_bytes)};
    const uint32_t box[3] = {64u, uint32_t(1 << p.c.shift < kTile ? 1 << p.c.shift : kTile), 1u};
    const sv_status st =
        make_tmap(&pages, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p.c.pages, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != SV_OK) return st;
    e = p.c.D > 64 ? launch_cap<2, false, SOLO, OWN>(p, pages, grid, s) : launch_cap<1, false, SOLO, OWN>(p, pages, grid, s);
  }
  return e == cudaSuccess ? SV_OK : cuda_fail(e, fn);
}

}  // namespace

sv_status prefix_launch(const char* fn, const Params& p, int grid, cudaStream_t s) {
  return p.pre.rows == kTile ? launch<true, false>(fn, p, grid, s) : launch<false, false>(fn, p, grid, s);
}
sv_status own_tiles_launch(const char* fn, const Params& p, int grid, cudaStream_t s) {
  return launch<true, true>(fn, p, grid, s);
}

}  // namespace cached
}  // namespace sv
