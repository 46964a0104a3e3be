// Attention over packed documents (sv_attention_packed): document mask, causal mask with a
// visible prefix, tanh-capped scores, a bias that falls with distance, shared key heads.
//
// A query's visible keys are the keys j < lim of its document: lim = Lk, or with the prefix
// mask min(Lk, max(p_i + 1, prefix)), p_i = i + Lk - Lq. For these, in F32,
//   s_j = scale q . k_j;  s_j = cap tanh(s_j / cap);  s_j -= slope |p_i - j|,
//   o = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m),
// m following the running maximum. lim = 0 gives zeros.
//
// One pass over the keys on the tensor cores, scores never leaving the SM. A tile of 128
// rows holds 128 / group queries with the `group` query heads of one key head (row r =
// query r / group, head r % group), so shared key heads are read once for all of them, and
// a single query of many heads fills rows. Persistent CTAs (one per SM) walk work items of
// two such tiles against the document's key tiles of 128; 352 threads:
//   warp 0      works out the items from the documents' lengths on the device (the lengths
//               never visit the host) and copies: Q of an item, key and value tiles in turn
//               into a ring, all by TMA from the caller's strided rows (values past a head's
//               width arrive as zeros: no copy into a padded layout);
//   warp 1      the MMA issuer: S_w = Q_w K^T (both in shared memory, 128-byte swizzle),
//               O_w += P_w V (P from tensor memory);
//   warps 2..5  softmax of tile 0, warps 6..9 of tile 1: a thread per row turns its S row into
//               P (F16, over S in tensor memory), keeps the exponent and the sum in F32, and
//               rescales O in tensor memory when the exponent rises by more than 2^15;
//   warp 10     clears the value rows of an item's last tile that none of its rows sees.
// An item's rows go out behind the next item's first tile: O is loaded between that tile's
// softmax and the arrival of its P, and scaled, rounded and stored while the products run.
// Items are handed out by tickets, the longest documents of every 32 first. In launches of few
// items (SOLO) an item is one tile, and the two groups share out its key tiles. Key ranges are
// divided among CTAs when there are few items (Schedule); the parts' O, m and l go to the
// caller's workspace and are joined two and two.
// Tensor memory: S_0, S_1, O_0, O_1 of 128 columns each.
//
// What bounds it: the chain of one tile of 128 rows, softmax (about 1,400 cycles), the way of P
// to the issuer and of S back (500), the products P V and S (760 at 72 dimensions, 1,024 at 128);
// two tiles a CTA run half a period apart, so that a pair of tiles takes 2,700 to 3,000 cycles, of
// which the tensor cores work 1,331 (72) or 2,048 (128). Tried against it and slower: P handed over
// in two halves, two warps for 32 rows, one arrival a warp, two issuers, warps of their own for
// the output. The code of an item is as long as the instruction caches: what runs rarely is
// out of line.
// 32 images of 729 tokens, 16 heads of 72: 123 us (635 TFLOP/s of the products of visible keys);
// one sequence of 8192 tokens behind the prefix mask, 32 heads of 128 over 8: 377 to 403 us by the GPU's
// clock, 1,365 to 1,460 TFLOP/s.
#include <cmath>

#include "packed_attention.h"

namespace sv {
namespace packed {
namespace {

constexpr int kTile = 128;                  // rows of a query tile, keys of a key tile
constexpr int kBoxBytes = kTile * 128;      // 128 rows of 64 values: one box of an operand tile
constexpr int kThreads = 352;
constexpr int kBarBytes = 768;              // barriers, TMEM address slot, abort flag, items
constexpr int kOutBytes = 32 * 64;          // 32 rows of 32 output columns
constexpr int kItems = 4;                   // work items between the copy warp and the others
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSlots = 2 * kMaxSms;      // partial results of a launch at most (see Schedule)
// Key tiles of a part of a divided range at least: below, the parts' way through the workspace
// costs more than their length (40 queries over 2048 keys: two parts of 8 tiles 34 us, 16 tiles one
// behind another 32; one image of 729 tokens, 16 heads: 48 items of 6 tiles 16 us, 144 parts of 2 tiles 38 us).
constexpr int kMinSplit = 8;
static_assert(kCounterBytes >= size_t(kMaxSlots) * 8 * sizeof(unsigned), "counters");

template <int NB>
struct Smem {
  static constexpr int kQBufs = NB == 1 ? 2 : 1;
  static constexpr int kStages = NB == 1 ? 8 : 4;  // key and value tiles in turn
  static constexpr int kOp = NB * kBoxBytes;       // one operand tile
  static constexpr int kOffKV = 2 * kQBufs * kOp;
  static constexpr int kOffOut = kOffKV + kStages * kOp;  // output rows on their way out: two buffers a softmax warp
  static constexpr int kOffBar = kOffOut + 8 * 2 * kOutBytes;
  static constexpr int kBytes = 1024 + kOffBar + kBarBytes;
  static_assert(kBytes <= 232448, "shared memory budget");
};

enum {
  kBarQFull = 0,    // +buffer
  kBarQEmpty = 2,   // +buffer: the item's last S products have read Q
  kBarFull = 4,     // +stage
  kBarEmpty = 12,   // +stage
  kBarSFull = 20,   // +group: S_w has finished (and with it the P V products before it)
  kBarPFull = 22,   // +group: the group has written P_w (and any O rescale) to TMEM
  kBarDrain = 24,
  kBarItem = 25,       // +item slot: the copy warp has written the item
  kBarItemDone = 29,   // +item slot: the issuer, the eight softmax warps and warp 10 are through with it
  kBarOFull = 33,      // +group: the item's last P V product of the group has finished
  kBarJoin = 35,       // one tile an item: the second group's exponents and sums are in shared memory
  kBarRead = 36,       // and its O has been read
  kBarRest = 37,       // +stage: value rows that warp 10 has to clear have arrived
  kNumBars = 45
};

// One work item: up to 2 qt queries of a document with the query heads of one key head
// (two tiles of rows, row r = query r / group, head r % group), over key tiles jb .. je - 1.
struct Item {
  int q0, nq;           // first query (row of q), queries of the item
  int k0, lk;           // the document's keys
  int at, prefix, kvh;  // position of the first query among the keys
  int jb, je;           // key tiles
  int ke;               // keys that some row of the item sees end here
  int slot, splits, split;  // partial result; splits 1: none
  int live;             // 0: no more items
};
constexpr int kOffItems = 8 * kNumBars + 8;  // in the barrier area
constexpr int kOffProgress = kBarBytes - 8;
static_assert(kOffItems + kItems * sizeof(Item) <= kOffProgress && kBarBytes <= 1024, "barrier area");
// Steps of work whose length the inputs decide (rows that are computed again), counted for those who wait; at: any
// place in the barrier area, which starts on 1024 bytes.
__device__ __forceinline__ unsigned* progress(const volatile void* at) {
  return reinterpret_cast<unsigned*>((reinterpret_cast<uintptr_t>(at) & ~uintptr_t(1023)) + kOffProgress);
}

// The items in order, worked out by the copy warp from the documents' lengths: a
// chunk of 32 documents at a time, one per lane, with their item counts summed by shuffles.
// Within a document: pairs of tiles from the last (longest) on, then key heads, then parts of
// the key range. Where the launch has less work than its CTAs could share evenly, a
// document's key range is divided into parts of at most `chunk` tiles, chunk = the launch's
// key tiles per CTA: then a launch has at most 2 x grid parts in divided ranges, since a
// range of n > chunk tiles has ceil(n / chunk) <= 2 n / chunk parts.
class Schedule {
 public:
  // span: queries of an item; min_split: key tiles of a part at least.
  __device__ __forceinline__ Schedule(const Params& p, int lane, int span, int min_split)
      : p_(p), lane_(lane), docs_(p.docs), span_(span) {
    chunk_ = 0x7fffffff;
    float work = 0.0f;
    bool bad = false;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {  // the work, then the items that it makes
      int items = 0;
#pragma unroll 1
      for (int d0 = 0; d0 < docs_; d0 += 32) {
        load(d0);
        bad |= bad_;
        work += float(pairs_) * float(tiles_);
        items += count_;
      }
      items_ = int(__reduce_add_sync(0xffffffffu, unsigned(items)));
      if (pass == 0) {
#pragma unroll
        for (int o = 16; o; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
        // offsets that decrease or leave [0, total]: reported, and nothing is computed, since
        // the bounds on items and parts hold for documents that do not overlap
        if (__any_sync(0xffffffffu, bad)) {
          if (lane == 0) atomicOr(p.err, kDevErrOffsets);
          docs_ = 0;
        }
        if (!p.counters) break;  // nothing is divided, and no tickets are drawn
        // work x heads / grid, rounded up (F32 sums of up to 2^24 documents, 32 lanes apart: a little more
        // does no harm)
        const float share = work * float(p.hk) * (1.1f / float(gridDim.x));
        chunk_ = max(min_split, int(fminf(share, 1e9f)) + 1);
      }
    }
  }
  // The CTA's first item is its own number, the others go to whoever is free, by a ticket from
  // the workspace: CTAs draw until they are refused, `items` tickets in all, and the counter
  // is back at 0. Without a workspace every CTA takes every gridDim-th item.
  __device__ __forceinline__ unsigned draw() const {  // (one lane; the answer takes a microsecond)
    return p_.counters ? atomicInc(p_.counters + kTicket, unsigned(items_ - 1)) : 0u;
  }
  // The number of the item after `it`, with lane 0's ticket.
  __device__ __forceinline__ int after(int it, unsigned ticket) const {
    return int(gridDim.x) + (p_.counters ? int(__shfl_sync(0xffffffffu, ticket, 0)) : it);
  }
  // Item number `it` (increasing from call to call); false behind the last.
  __device__ __forceinline__ bool get(int it, Item& r) {
    while (it >= base_ + total_) {
      d0_ += 32;
      if (d0_ >= docs_) return false;
      base_ += total_;
      slot_base_ += slot_total_;
      load(d0_);
      longest_first();
      incl_ = count_;
      slot_incl_ = splits_ > 1 ? count_ : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, incl_, o);
        if (lane_ >= o) incl_ += a;
      }
      if (__any_sync(0xffffffffu, splits_ > 1))
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int a = __shfl_up_sync(0xffffffffu, slot_incl_, o);
          if (lane_ >= o) slot_incl_ += a;
        }
      total_ = __shfl_sync(0xffffffffu, incl_, 31);
      slot_total_ = __shfl_sync(0xffffffffu, slot_incl_, 31);
    }
    const int at = it - base_;
    const int src = __ffs(__ballot_sync(0xffffffffu, incl_ > at)) - 1;
    auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
    const int pairs = of(pairs_), splits = of(splits_), tiles = of(tiles_);
    int k = at - of(incl_ - count_);
    r.slot = slot_base_ + of(slot_incl_ - (splits_ > 1 ? count_ : 0)) + k;
    r.splits = splits;
    r.split = k % splits;
    k /= splits;
    const int back = k / p_.hk;
    r.kvh = k - back * p_.hk;
    const int pair = pairs - 1 - back;
    const int lq = of(doc_.lq);
    r.lk = of(doc_.lk);
    r.k0 = of(doc_.k0);
    r.prefix = of(doc_.prefix);
    const int i0 = pair * span_;
    r.q0 = of(doc_.q0) + i0;
    r.nq = min(lq - i0, span_);
    r.at = i0 + r.lk - lq;
    r.ke = limit_of(p_.causal, r.at + r.nq - 1, r.lk, r.prefix);  // (the last query sees the most)
    const int n = (r.ke + kTile - 1) / kTile;
    const int part = (tiles + splits - 1) / splits;
    r.jb = min(r.split * part, n);
    r.je = min(r.jb + part, n);
    return true;
  }

 private:
  __device__ __forceinline__ void load(int d0) {
    bad_ = !document(p_, d0 + lane_, docs_, doc_);
    pairs_ = (doc_.lq + span_ - 1) / span_;
    tiles_ = (doc_.lk + kTile - 1) / kTile;  // of the last query
    splits_ = tiles_ > chunk_ ? (tiles_ + chunk_ - 1) / chunk_ : 1;
    count_ = pairs_ * p_.hk * splits_;
  }
  // Lane i takes the document with the i-th most key tiles of the 32 (equal ones in order): long
  // items come early, and the last ones to be handed out are short.
  __device__ __forceinline__ void longest_first() {
    // (equal ones, or one alone, are in order; a bitonic sort of tiles and lane in one word otherwise: every
    // CTA of the launch waits for this)
    const int before = __shfl_up_sync(0xffffffffu, tiles_, 1);
    if (!__any_sync(0xffffffffu, lane_ > 0 && tiles_ > before)) return;
    int key = tiles_ << 5 | (31 - lane_);  // (at most 2^24 tiles)
#pragma unroll 1
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll 1
      for (int j = k / 2; j; j /= 2) {
        const int other = __shfl_xor_sync(0xffffffffu, key, j);
        key = ((lane_ & j) == 0) == ((lane_ & k) == 0) ? max(key, other) : min(key, other);
      }
    const int from = 31 - (key & 31);
    auto take = [&](int& v) { v = __shfl_sync(0xffffffffu, v, from); };
    take(doc_.q0);
    take(doc_.lq);
    take(doc_.k0);
    take(doc_.lk);
    take(doc_.prefix);
    take(pairs_);
    take(tiles_);
    take(splits_);
    take(count_);
  }
  const Params& p_;
  int lane_, docs_, span_, chunk_;
  bool bad_;
  int items_ = 0;
  int d0_ = -32, base_ = 0, total_ = 0, slot_base_ = 0, slot_total_ = 0;
  Document doc_;  // this lane's
  int pairs_, tiles_, splits_, count_, incl_, slot_incl_;
};

// A wait whose long form is one function for all of the kernel's waits: inlined, the waits alone
// were a sixth of the code, and code that runs once an item then came from beyond the
// instruction caches. It gives up (as mbar_wait does) after the limit without progress.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
  unsigned long long t0 = globaltimer();
  const volatile unsigned* steps = progress(abort);
  unsigned seen = *steps;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i & 255u) continue;
    if (*abort) return false;
    if (globaltimer() - t0 <= kWaitLimitNs) continue;
    const unsigned now = *steps;
    if (now == seen) {
      *abort = 1;
      atomicOr(err, kDevErrTimeout);
      return false;
    }
    seen = now;
    t0 = globaltimer();
  }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort, err);
}

// Joins the parts of a divided range for row r of tile w (out_to: its place, -1 none), two at a time
// along a binary tree over the parts: of two neighbours the warp that arrives second adds them, on
// the left one's place, and goes on with the sum; the last one of all writes the row. So the joins
// of a long range run on many SMs (by the last of all parts alone, in order: 40 queries of 8 heads
// over 32768 keys of 2, 64 parts, 184 us; so 67, 53 with the groups sharing tiles), and the order of the sums is the tree's, whoever is
// second.
__device__ __noinline__ void join_parts(const Params& p, const Item& it, long long out_to, int w, int r) {
  const int Dn = (p.D + 15) / 16 * 16, n = it.splits, first = it.slot - it.split;
  auto place = [&](int part) {  // exponent, denominator, then the columns, kTile rows each
    return p.partial + (size_t(first + part) * 2 + w) * size_t(Dn + 2) * kTile + r;
  };
  int left = it.split;  // the parts left .. left + step - 1 (below n) are summed at `left`
#pragma unroll 1
  for (int step = 1; step < n; step *= 2) {
    int right = left + step;
    if (left & step) right = left, left -= step;
    if (right >= n) continue;  // (no neighbour on this level)
    __threadfence();
    __syncwarp();
    unsigned seen = 0;
    if ((r & 31) == 0)  // 0, then 1, and 0 again
      seen = atomicInc(p.counters + size_t(first + right) * 8 + (w * 4 + (r >> 5)), 1u);
    if (__shfl_sync(0xffffffffu, seen, 0) == 0) return;
    __threadfence();
    float* a = place(left);
    const float* b = place(right);
    const float ma = __ldcg(a), mb = __ldcg(b), la = __ldcg(a + kTile), lb = __ldcg(b + kTile);
    const float mx = fmaxf(ma, mb), ref = mx == -INFINITY ? 0.0f : mx;
    const float fa = ex2(ma - ref), fb = ex2(mb - ref), l = fmaf(fb, lb, fa * la);
    const bool last = 2 * step >= n;
    const int i = w * p.qt + r / p.group;
    const bool none = limit_of(p.causal, it.at + i, it.lk, it.prefix) == 0;
    const float inv = 1.0f / l;
#pragma unroll 1
    for (int c = 0; c < Dn; c += 16) {  // (what lies between D and Dn is read and of no use)
      float y[16], yb[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        y[e] = __ldcg(a + (2 + c + e) * kTile);
        yb[e] = __ldcg(b + (2 + c + e) * kTile);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        y[e] = fmaf(fb, yb[e], fa * y[e]);
        if (last) y[e] = none ? 0.0f : y[e] * inv;
        else __stcg(a + (2 + c + e) * kTile, y[e]);
      }
      if (last && out_to >= 0) {
        store8(p, size_t(out_to) + c, y);
        if (c + 8 < p.D) store8(p, size_t(out_to) + c + 8, y + 8);
      }
    }
    if (!last) {
      __stcg(a, mx);
      __stcg(a + kTile, l);
    }
  }
}

// What a row of an item needs beside O / l: it sees no key; its item is a part of a divided range;
// its item has no keys at all.
enum { kNothing = 1, kPart = 2, kEmpty = 4 };

// The rows of tile w whose O is not finite (r: this lane's; out_to -1: no such row), again from the visible keys alone where a key that
// the row does not see has spoiled it; of a part, their sums, exponents and denominators. By a whole warp.
__device__ __noinline__ void rows_again(const Params& p, const Item& it, long long out_to, int how, int w, int r) {
  const int Dn = (p.D + 15) / 16 * 16, lane = r & 31;
  const __half* k = p.k + it.k0 * p.ks + it.kvh * p.D;
  const __half* v = p.v + it.k0 * p.vs + it.kvh * p.D;
  const int i = w * p.qt + r / p.group, head = it.kvh * p.group + r % p.group;
  const int kb = it.jb * kTile, ke = min(it.ke, it.je * kTile);  // the keys of the products
  const int lim = out_to >= 0 ? max(limit_of(p.causal, it.at + i, it.lk, it.prefix), kb) : ke;
  const int low = __reduce_min_sync(0xffffffffu, lim);
  const int last = low < ke ? last_spoiled(p, v, low, ke, lane) : -1;
  const float slope = p.slopes && lim < ke ? __ldg(p.slopes + head) : 0.0f;
  __syncwarp();  // (what the rows' own lanes have stored comes first)
#pragma unroll 1
  for (uint32_t todo = __ballot_sync(0xffffffffu, lim <= last); todo; todo &= todo - 1) {
    const int src = __ffs(int(todo)) - 1;
    auto of = [&](auto x) { return __shfl_sync(0xffffffffu, x, src); };
    const int row_i = of(i), row_head = of(head);
    float m, l;
    const float4 y = row_again(p, p.q + static_cast<long long>(it.q0 + row_i) * p.qs + row_head * p.D, k, v, kb, of(lim),
                               it.at + row_i, of(slope), lane, progress(&it), m, l);
    const long long to = of(out_to);
    if (of(how) & kPart) {
      float* pb = p.partial + (size_t(it.slot) * 2 + w) * size_t(Dn + 2) * kTile + (r - lane + src);
      if (lane == 0) {
        __stcg(pb, m);
        __stcg(pb + kTile, l);
      }
      if (lane < p.D / 4) {
        pb += size_t(2 + 4 * lane) * kTile;
        __stcg(pb, y.x);
        __stcg(pb + kTile, y.y);
        __stcg(pb + 2 * kTile, y.z);
        __stcg(pb + 3 * kTile, y.w);
      }
    } else if (lane < p.D / 4) {
      store4(p, size_t(to) + 4 * lane, make_float4(y.x / l, y.y / l, y.z / l, y.w / l));
    }
  }
}

// Row r of tile w where `how` is not 0 for its whole warp. Out of the way of the common case,
// whose code must stay in the instruction caches.
__device__ __noinline__ void write_special(const Params& p, const Item& it, uint32_t o_tm, float m, float l,
                                           long long out_to, int how, int w, int r) {
  const int Dn = (p.D + 15) / 16 * 16;
  const int i = w * p.qt + r / p.group;
  const int lim = out_to < 0 ? 0 : limit_of(p.causal, it.at + i, it.lk, it.prefix);
  const float inv = 1.0f / l;
  float* pb = p.partial + (size_t(it.slot) * 2 + w) * size_t(Dn + 2) * kTile + r;
  if (how & kPart) {
    const bool some = lim > it.jb * kTile && !(how & kEmpty);
    __stcg(pb, some ? m : -INFINITY);
    __stcg(pb + kTile, some ? l : 0.0f);
  }
  float bad = 0.0f;
  for (int c = 0; c < p.D; c += 8) {
    uint32_t o[8];
    tmem_ld8(o_tm + uint32_t(c), o);
    tmem_ld_wait();
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      asm volatile("" : "+r"(o[e]));  // no use before the wait
      y[e] = how & (kNothing | kEmpty) ? 0.0f : __uint_as_float(o[e]) * (how & kPart ? 1.0f : inv);
      bad = fmaf(y[e], 0.0f, bad);
    }
    if (out_to < 0) continue;
    if (how & kPart) {
#pragma unroll
      for (int e = 0; e < 8; ++e) __stcg(pb + size_t(2 + c + e) * kTile, y[e]);
    } else {
      store8(p, size_t(out_to) + c, y);
    }
  }
  if (__any_sync(0xffffffffu, out_to >= 0 && bad != 0.0f)) rows_again(p, it, bad != 0.0f ? out_to : -1, how, w, r);
  if (how & kPart) join_parts(p, it, out_to, w, r);
}

// Row r of an item of one tile whose key tiles the two groups have shared out: exponent, denominator and O of both.
__device__ __noinline__ void write_shared(const Params& p, const Item& it, uint32_t o_tm, float m0, float l0, float m1,
                                          float l1, long long out_to, int how, int r) {
  const int Dn = (p.D + 15) / 16 * 16;
  const float mx = fmaxf(m0, m1), ref = mx == -INFINITY ? 0.0f : mx;
  const float f0 = ex2(m0 - ref), f1 = ex2(m1 - ref), l = fmaf(f1, l1, f0 * l0);
  const float inv = how & kPart ? 1.0f : 1.0f / l;
  float* pb = p.partial + size_t(it.slot) * 2 * size_t(Dn + 2) * kTile + r;
  if (how & kPart) {
    __stcg(pb, mx);
    __stcg(pb + kTile, l);
  }
  float bad = 0.0f;
#pragma unroll 1
  for (int c = 0; c < p.D; c += 8) {
    uint32_t a[8], b[8];
    tmem_ld8(o_tm + uint32_t(c), a);
    tmem_ld8(o_tm + uint32_t(128 + c), b);
    tmem_ld_wait();
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      asm volatile("" : "+r"(a[e]), "+r"(b[e]));  // no use before the wait
      y[e] = how & kNothing ? 0.0f : fmaf(f1, __uint_as_float(b[e]), f0 * __uint_as_float(a[e])) * inv;
      bad = fmaf(y[e], 0.0f, bad);
    }
    if (out_to < 0) continue;
    if (how & kPart) {
#pragma unroll
      for (int e = 0; e < 8; ++e) __stcg(pb + size_t(2 + c + e) * kTile, y[e]);
    } else {
      store8(p, size_t(out_to) + c, y);
    }
  }
  if (__any_sync(0xffffffffu, out_to >= 0 && bad != 0.0f)) rows_again(p, it, bad != 0.0f ? out_to : -1, how, 0, r);
  if (how & kPart) join_parts(p, it, out_to, 0, r);
}

// Row r of tile w of an item, once its last P V has finished (o_tm: the row's O). `loaded` is called
// when O has left tensor memory. Where a warp's 32 rows are all the item's and make whole queries
// (p.out_tma) they go out by TMA from shared memory (`stage`: two buffers), 32 columns at a time;
// the rows of a part-filled warp are stored by their lanes (a bulk copy a row instead: 134 against
// 128 us then for 32 images of 729 tokens). E4M3 rows that do not start on 16 bytes are stored in runs,
// after four lanes, which hold four rows, have exchanged quarters of 32 columns. (All rows by their
// lanes: 24 us for 23,328 rows of 16 heads of 72 by itself, and the load-store unit held up for
// everything else meanwhile.)
template <int NB, bool E4M3, typename F>
__device__ __forceinline__ void write_rows(const Params& p, const Item& it, const CUtensorMap& to_map, uint8_t* stage,
                                           uint32_t o_tm, float m, float l, long long out_to, int how, int w, int r,
                                           F loaded) {
  if (__any_sync(0xffffffffu, how)) {
    write_special(p, it, o_tm, m, l, out_to, how, w, r);
    loaded();
    return;
  }
  uint32_t o[NB * 2][32];
#pragma unroll
  for (int c = 0; c < NB * 2; ++c) tmem_ld32(o_tm + uint32_t(32 * c), o[c]);
#pragma unroll
  for (int c = 0; c < NB * 2; ++c) tmem_ld_wait(o[c]);
  loaded();
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(l));
  if (E4M3) inv *= 16.0f;
  const int lane = r & 31;
  float bad0 = 0.0f, bad1 = 0.0f;  // NaN once a value of the row is not finite
#pragma unroll
  for (int c = 0; c < NB * 2; ++c) {  // in the output's type, over the first registers of o[c]
    if (32 * c < p.D) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float a, b;
        mul_x2(a, b, __uint_as_float(o[c][e]), __uint_as_float(o[c][e + 1]), inv, inv);
        fma_x2(bad0, bad1, a, b, 0.0f, 0.0f, bad0, bad1);
        if constexpr (E4M3) {
          const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
          o[c][e >> 2] = e & 2 ? o[c][e >> 2] | h << 16 : h;
        } else {
          const __half2 h = __floats2half2_rn(a, b);
          o[c][e >> 1] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
  }
  const bool bad = out_to >= 0 && bad0 + bad1 != 0.0f;
  bool again = false;
  constexpr int kRow = E4M3 ? 32 : 64;  // bytes of a staged row, swizzled for a TMA store
  if (p.out_tma && __all_sync(0xffffffffu, out_to >= 0 && !bad)) {
    const int turn = E4M3 ? (lane >> 2) & 1 : (lane >> 1) & 3;  // swizzle
    if (lane == 0) bulk_wait_read<0>();
#pragma unroll
    for (int c = 0; c < NB * 2; ++c) {
      if (32 * c < p.D) {
        if (c >= 2 && lane == 0) bulk_wait_read<1>();  // the buffer's columns before have been read out
        __syncwarp();
        uint8_t* buf = stage + (c & 1) * kOutBytes;
#pragma unroll
        for (int u = 0; u < kRow / 16; ++u)
          *reinterpret_cast<uint4*>(buf + lane * kRow + ((u ^ turn) << 4)) =
              make_uint4(o[c][4 * u], o[c][4 * u + 1], o[c][4 * u + 2], o[c][4 * u + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&to_map, smem_u32(buf), 32 * c, it.kvh * p.group, it.q0 + (w * kTile + r) / p.group);
          bulk_commit();
        }
      }
    }
  } else if constexpr (!E4M3) {
    again = __any_sync(0xffffffffu, bad);
    if (out_to >= 0)
#pragma unroll
      for (int g = 0; g < NB * 8; ++g)
        if (8 * g < p.D)
          *reinterpret_cast<uint4*>(static_cast<__half*>(p.o) + out_to + 8 * g) = make_uint4(
              o[g >> 2][4 * (g & 3)], o[g >> 2][4 * (g & 3) + 1], o[g >> 2][4 * (g & 3) + 2], o[g >> 2][4 * (g & 3) + 3]);
  } else if constexpr (E4M3) {
    again = __any_sync(0xffffffffu, bad);
    const int quarter = lane & 3;
    long long to[4];  // the four rows' places
#pragma unroll
    for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, out_to, (lane & 28) + k);
#pragma unroll
    for (int c = 0; c < NB * 2; ++c) {
      if (32 * c < p.D) {
        uint32_t v[4][2];
#pragma unroll
        for (int g = 0; g < 4; ++g) v[g][0] = o[c][2 * g], v[g][1] = o[c][2 * g + 1];
#pragma unroll
        for (int x = 1; x < 4; x <<= 1)  // transpose the quarters among the four lanes
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (!(g & x))
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const bool high = lane & x;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? v[g][e] : v[g ^ x][e], x);
                if (high) v[g][e] = got;
                else v[g ^ x][e] = got;
              }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (to[k] >= 0 && 32 * c + 8 * quarter < p.D)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.o) + to[k] + 32 * c + 8 * quarter) =
                make_uint2(v[k][0], v[k][1]);
      }
    }
  }
  if (again) rows_again(p, it, bad ? out_to : -1, how, w, r);
}

// Four capped scores share a reciprocal (capped4), where a hidden one must have no part: those behind a row's `valid`
// visible scores, up to the next multiple of eight, become -inf in tensor memory. The columns are the warp's, so the
// rows take turns. (In registers, by a select for each of the 128 scores as after the cap, this costs 9% of such calls.)
__device__ __forceinline__ void cut_scores(uint32_t s_tm, int valid) {
  const bool cut = valid > 0 && valid < kTile && (valid & 3);
  uint32_t todo = __ballot_sync(0xffffffffu, cut);
  if (!todo) return;
#pragma unroll 1
  do {
    const int at = __shfl_sync(0xffffffffu, valid, __ffs(int(todo)) - 1) & ~7;
    const bool mine = cut && (valid & ~7) == at;
    uint32_t s[8];
    tmem_ld8(s_tm + uint32_t(at), s);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      asm volatile("" : "+r"(s[e]));  // no use before the wait
      if (mine && at + e >= valid) s[e] = 0xff800000u;
    }
    tmem_st8(s_tm + uint32_t(at), s);
    tmem_st_wait();
    todo &= ~__ballot_sync(0xffffffffu, mine);
  } while (todo);
}

// SOLO: items of one tile, whose key tiles the two groups take in turn (for launches of few items: half the chain, and
// an end at which the groups' sums are joined). The output's type is then read from the parameters.
// CAP: 0 none, 1 below kFarCap, 2 from there on (with BIAS, whose slopes may then be null, and without SOLO).
template <int NB, int CAP, bool BIAS, bool E4M3, bool SOLO>
// 11 warps: three share each of three SM sub-partitions, so a thread may hold at most
// 16384 / (3 x 32) registers, rounded down to the allocation granule.
__global__ void __maxnreg__(168)
    packed_tile_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ CUtensorMap to) {
  using L = Smem<NB>;
  constexpr int kOp = L::kOp, kStages = L::kStages, kQBufs = L::kQBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::kOffBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQBufs; ++s) {
      mbar_init(bar(kBarQFull + s), 1);
      mbar_init(bar(kBarQEmpty + s), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
      mbar_init(bar(kBarRest + s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(kBarSFull + w), 1);
      mbar_init(bar(kBarPFull + w), 128);  // every softmax thread of the group arrives
      mbar_init(bar(kBarOFull + w), 1);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(bar(kBarItem + s), 1);
      mbar_init(bar(kBarItemDone + s), 10);
    }
    mbar_init(bar(kBarJoin), 128);
    mbar_init(bar(kBarRead), 128);
    mbar_init(bar(kBarDrain), 1);
    *abort_flag = 0;
    *progress(abort_flag) = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();  // q, k, v, offsets, prefix and slopes may be written by the previous kernel
  Item* items = reinterpret_cast<Item*>(smem + L::kOffBar + kOffItems);
  auto item_wait = [&](int n) {
    return wait_bar(bar(kBarItem + n % kItems), (n / kItems) & 1, abort_flag, p.err);
  };

  if (warp == 0) {
    Schedule sched(p, lane, (SOLO ? 1 : 2) * p.qt, (SOLO ? 2 : 1) * kMinSplit);
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
    }
    // copies in flight per full barrier (bit b: Q buffer b, 4 + stage) and their phase bits
    uint32_t issued = 0, issued_phase = 0;
    uint32_t rest = 0, rest_phase = 0;  // stages whose last copy went to warp 10 first; the phase of the next that does
    auto note = [&](int bit, uint32_t ph) {
      issued |= 1u << bit;
      issued_phase = (issued_phase & ~(1u << bit)) | (ph << bit);
    };
    const uint32_t q_bytes = uint32_t(2 * NB * 128 * p.group * p.qt);
    int t = 0, n = 0;  // operand tiles and non-empty items so far
    int told = 0;      // items written for the other warps
    // The next item, written for the other warps. (It waits for the item four before to be
    // written out, so it must not come before copies that this depends on.)
    int number = int(blockIdx.x);  // of the next item
    unsigned ticket = 0;           // lane 0's, for the one after
    auto tell = [&](Item& r) -> int {
      if (told > 0) number = sched.after(number, ticket);
      r.live = sched.get(number, r);
      const int slot = told % kItems;
      int ok = wait_bar(bar(kBarItemDone + slot), ((told / kItems) & 1) ^ 1, abort_flag, p.err);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && lane == 0) {
        items[slot] = r;
        mbar_arrive(bar(kBarItem + slot));
      }
      ++told;
      return ok;
    };
    Item it;
    int ok = 1;
    while (ok && tell(it) && it.live) {
      if (it.jb >= it.je) {
        if (lane == 0) ticket = sched.draw();
        continue;
      }
      if (lane == 0) {
        // The next item is drawn late, so that the work stays balanced, but where the ring is short before
        // the last copies, whose room has to be waited for anyway (32 images: 124.5 -> 121.5 us; where it holds
        // four key tiles, earlier than behind the last copy costs 2%).
        const int copies = SOLO ? 4 * ((it.je - it.jb + 1) / 2) : 2 * (it.je - it.jb), draw_at = NB == 1 ? copies : copies - 2;
        const int clean = min(it.ke, it.je * kTile) / kTile;  // tiles with values of the item's keys alone
        auto kv = [&](bool values, int j) -> bool {
          const int st = t % kStages;
          const uint32_t ph = (t / kStages) & 1;
          if (!wait_bar(bar(kBarEmpty + st), ph ^ 1, abort_flag, p.err)) return false;
          const bool clear = values && j >= clean;
          const uint32_t full = bar((clear ? kBarRest : kBarFull) + st);
          mbar_arrive_expect_tx(full, kOp);
          for (int b = 0; b < NB; ++b)
            tma_load_3d(sbase + L::kOffKV + st * kOp + b * kBoxBytes, values ? &tv : &tk, full, 64 * b, it.kvh,
                        it.k0 + j * kTile);
          note(4 + st, ph);
          if (clear) rest |= 1u << st, rest_phase ^= 1u << st;
          else rest &= ~(1u << st);
          ++t;
          return true;
        };
#pragma unroll 1
        for (int x = 0; ok && x < copies; ++x) {  // a key tile, its values, the next key tile, ...
          if (x == draw_at) ticket = sched.draw();
          if constexpr (SOLO) ok = kv(x & 2, it.jb + 2 * (x >> 2) + (x & 1));  // two keys, their values, ...
          else ok = kv(x & 1, it.jb + (x >> 1));
          if (ok && x == 0) {
            const int qb = n % kQBufs;
            const uint32_t ph = (n / kQBufs) & 1;
            if ((ok = wait_bar(bar(kBarQEmpty + qb), ph ^ 1, abort_flag, p.err))) {
              mbar_arrive_expect_tx(bar(kBarQFull + qb), q_bytes);
#pragma unroll 1
              for (int w = 0; w < 2; ++w)
                for (int b = 0; b < NB; ++b)
                  tma_load_3d(sbase + (2 * qb + w) * kOp + b * kBoxBytes, &tq, bar(kBarQFull + qb), 64 * b,
                              it.kvh * p.group, it.q0 + (SOLO ? 0 : w * p.qt));
              note(qb, ph);
            }
          }
        }
        if (draw_at == copies) ticket = sched.draw();
      }
      ++n;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0)  // every copy this thread issued lands before the CTA can exit
      for (int i = 0; i < 4 + kStages; ++i)
        if (issued & (1u << i)) {
          const int st = i - 4;
          if (i >= 4 && (rest >> st & 1)) mbar_wait_bounded(bar(kBarRest + st), ~(rest_phase >> st) & 1, p.err);
          else mbar_wait_bounded(bar(i < 4 ? kBarQFull + i : kBarFull + st), (issued_phase >> i) & 1, p.err);
        }
  } else if (warp == 1) {
    // The MMA issuer: S_0(0), S_1(0), then per key tile t of all items: O_0 += P_0(t) V_t,
    // S_0(t+1), O_1 += P_1(t) V_t, S_1(t+1). MMAs run in issue order, so S_w(t+1)
    // overwrites P_w(t) only after the product has read it, and the completion of
    // S_w(t+1) also means that O_w holds the sum up to tile t. One issuer for both tiles keeps
    // them half a period apart, one's products under the other's softmax. The whole warp runs
    // this, in step (every condition is a vote), and one elected lane issues: descriptors
    // and addresses then stay in uniform registers, and an MMA takes few cycles to issue.
    constexpr uint32_t idesc_s = make_idesc(128, 128, 0, false);
    const uint32_t idesc_o = make_idesc(128, (p.D + 15) / 16 * 16, 0, true);
    const int steps = (p.D + 15) / 16;
    const uint32_t lead = elect_one();
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    auto commit = [&](int b) { tc_commit_if(lead, bar(b)); };
    auto wait = [&](int b, uint32_t parity) { return all(wait_bar(bar(b), parity, abort_flag, p.err)); };
    uint32_t kv = 0, kv_phase = 0;  // ring place and phase of the current key tile
    auto place = [&](uint32_t ahead, uint32_t& st, uint32_t& ph) {
      st = kv + ahead;
      ph = kv_phase;
      if (st >= kStages) st -= kStages, ph ^= 1;
    };
    auto wait_full = [&](uint32_t ahead) {
      uint32_t st, ph;
      place(ahead, st, ph);
      return wait(kBarFull + int(st), ph);
    };
    auto issue_s = [&](int w, int qb, uint32_t st) {
      uint64_t qd = make_sdesc(sbase + uint32_t(2 * qb + w) * kOp, 16, 1024, 2);
      uint64_t kd = make_sdesc(sbase + L::kOffKV + st * kOp, 16, 1024, 2);
      const uint32_t d = tmem + uint32_t(128 * w);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 bytes of each row a step
          if (4 * b + kk < steps)
            mma_f16_if(lead, d, qd + uint64_t(b * (kBoxBytes >> 4) + 2 * kk), kd + uint64_t(b * (kBoxBytes >> 4) + 2 * kk),
                       idesc_s, b + kk > 0);
      }
      commit(kBarSFull + w);
    };
    auto issue_pv = [&](int w, uint32_t st, uint32_t keep) {
      const uint64_t vd = make_sdesc(sbase + L::kOffKV + st * kOp, kBoxBytes, 1024, 2);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // 16 keys a step: 8 TMEM columns of P, 16 rows of V
        mma_f16_ts_if(lead, tmem + uint32_t(256 + 128 * w), tmem + uint32_t(128 * w + 8 * kk), vd + uint64_t(kk * (2048 >> 4)),
                      idesc_o, kk > 0 ? 1u : keep);
    };
    int read = 0;  // items so far
    // key tiles of the next item that has any (0: there is none); -1 after a time-out, or
    // where it is not there yet and `block` is false
    auto next = [&](bool block) -> int {
      for (;;) {
        const int b = kBarItem + read % kItems, ph = (read / kItems) & 1;
        if (block ? !wait(b, uint32_t(ph)) : !all(mbar_test(bar(b), uint32_t(ph)))) return -1;
        const Item& r = items[read % kItems];
        const int live = r.live, tiles = r.je - r.jb;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarItemDone + read % kItems));
        __syncwarp();
        if (!all(live)) return 0;
        ++read;
        if (all(tiles > 0)) return tiles;
      }
    };
    if constexpr (SOLO) {
      // S_0(0), S_1(1), then per two key tiles: O_0 += P_0 V, S_0 of the next two, O_1 += P_1 V, S_1
      uint32_t copied = 0, tt = 0, item = 0;  // copies used up, parity of the P, items with keys
      auto stage = [&](uint32_t k) { return (copied + k) % kStages; };
      auto full = [&](uint32_t k) {
        const bool got = wait(kBarFull + int(stage(k)), ((copied + k) / kStages) & 1);
        tc_fence_after();
        return got;
      };
      for (bool ok = true; ok; ++item) {
        const int tiles = next(true), steps = (tiles + 1) / 2, qb = int(item % kQBufs);
        if (!all(tiles > 0)) break;
        ok = wait(kBarQFull + qb, (item / kQBufs) & 1);
#pragma unroll 1
        for (uint32_t w = 0; w < 2 && ok; ++w) {
          if (!(ok = full(w))) break;
          issue_s(int(w), qb, stage(w));
          commit(kBarEmpty + int(stage(w)));
        }
        if (all(steps == 1)) commit(kBarQEmpty + qb);
#pragma unroll 1
        for (int s = 0; ok && all(s < steps); ++s, copied += 4, tt ^= 1) {
#pragma unroll 1
          for (uint32_t w = 0; w < 2 && ok; ++w) {
            if (!(ok = full(2 + w) && wait(kBarPFull + int(w), tt))) break;
            tc_fence_after();
            issue_pv(int(w), stage(2 + w), s > 0);
            commit(kBarEmpty + int(stage(2 + w)));
            if (all(s + 1 == steps)) {
              commit(kBarOFull + int(w));
            } else {
              if (!(ok = full(4 + w))) break;
              issue_s(int(w), qb, stage(4 + w));
              commit(kBarEmpty + int(stage(4 + w)));
              if (w == 1 && all(s + 2 == steps)) commit(kBarQEmpty + qb);
            }
          }
        }
      }
    }
    int tiles = SOLO ? 0 : next(true);
    bool ok = all(tiles > 0) && wait_full(0) && wait(kBarQFull, 0);
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int w = 0; w < 2; ++w) issue_s(w, 0, 0);
      commit(kBarEmpty);
      if (all(tiles == 1)) commit(kBarQEmpty);
    }
    uint32_t tt = 0;  // parity of the tiles so far
    int qb = 0, qph = 0;  // Q buffer and phase of the current item
    while (ok && all(tiles > 0)) {
      int more = 0;  // key tiles of the next item
      const int qb_next = qb + 1 == kQBufs ? 0 : qb + 1, qph_next = qb + 1 == kQBufs ? qph ^ 1 : qph;
      for (int j = 0; ok && all(j < tiles); ++j, tt ^= 1) {
        // ring: key tile at 0, its values at 1, the next key tile at 2
        const bool last = all(j + 1 == tiles);
        uint32_t st_v, st_k, ph;
        place(1, st_v, ph);
        place(2, st_k, ph);
        // (the copies are waited for before P, which is what the products really wait for)
        ok = wait_full(1) && (last || wait_full(2));
        bool late = false;  // the next item was not there for S_0
#pragma unroll 1
        for (int w = 0; w < 2 && ok; ++w) {
          if (!(ok = wait(kBarPFull + w, tt))) break;
          tc_fence_after();
          issue_pv(w, st_v, j > 0);
          int first = w;  // S products to issue: tiles first .. w
          if (last) {
            commit(kBarOFull + w);
            // The copy warp may need this item's slot for the next one (behind items without
            // keys): both tiles' O must be on their way before the issuer waits for it.
            if (w == 0 || late) {
              more = next(w == 1);
              if (w == 1) first = 0;
              late = all(more < 0);
              if (late && w == 1) ok = false;
            }
            if (late || all(more == 0)) first = 2;
            if (first == 0) {
              ok = wait_full(2) && wait(kBarQFull + qb_next, uint32_t(qph_next));
              tc_fence_after();
            }
          }
          const int q = last ? qb_next : qb;
#pragma unroll 1
          for (int s = first; s <= w && ok; ++s) {
            issue_s(s, q, st_k);
            if (s == 1) {
              commit(kBarEmpty + int(st_k));
              // the last S product of its item has read Q
              if (last ? all(more == 1) : all(j + 2 == tiles)) commit(kBarQEmpty + q);
            }
          }
          if (w == 1) commit(kBarEmpty + int(st_v));
        }
        kv += 2;
        if (kv >= kStages) kv -= kStages, kv_phase ^= 1;
      }
      tiles = more;
      qb = qb_next;
      qph = qph_next;
    }
    commit(kBarDrain);
    __syncwarp();
    mbar_wait_bounded(bar(kBarDrain), 0, p.err);
  } else if (warp == 10) {
    // Value rows of an item's last tile that none of its rows sees (the next document's, say) become zeros: their
    // probabilities are 0, but 0 times an infinity or NaN would spoil every row. The values of such a tile arrive
    // here, and go to the issuer from here. (A warp of its own: 1 to 2% of a call, in the issuer's or the softmax
    // warps' loops 2 to 5%.)
    uint32_t phase = 0;
    int pairs = 0;  // pairs of key and value tiles so far
    // (Its waits are long: it sleeps.)
    auto wait = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_try_wait<1000000>(bar(b), parity) || wait_bar(bar(b), parity, abort_flag, p.err));
    };
    for (int n = 0; wait(kBarItem + n % kItems, (n / kItems) & 1); ++n) {
      const Item& it = items[n % kItems];
      const int live = it.live, jb = it.jb, tiles = it.je - it.jb, end = min(it.ke, it.je * kTile);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarItemDone + n % kItems));
      if (!live) break;
      if (tiles <= 0) continue;
      bool ok = true;
      const int padded = SOLO ? (tiles + 1) / 2 * 2 : tiles;
      for (int j = max(end / kTile - jb, 0); ok && j < padded; ++j) {
        const int copy = 2 * pairs + (SOLO ? 4 * (j / 2) + 2 + j % 2 : 2 * j + 1), st = copy % kStages;
        if (!(ok = wait(kBarRest + st, (phase >> st) & 1))) break;
        phase ^= 1u << st;
        uint8_t* values = smem + L::kOffKV + st * kOp;
        for (int x = max(end - (jb + j) * kTile, 0) * 8 + lane; x < kTile * 8; x += 32)
          for (int b = 0; b < NB; ++b)
            *reinterpret_cast<uint4*>(values + b * kBoxBytes + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarFull + st));
      }
      if (!ok) break;
      pairs += padded;
    }
  } else {
    const int w = (warp - 2) >> 2;  // softmax group
    const int sub = warp & 3;       // TMEM lane quarter
    const int r = sub * 32 + lane;  // row of the group's tile == TMEM lane
    const uint32_t lane_off = uint32_t(sub * 32) << 16;
    const uint32_t s_tm = tmem + uint32_t(w * 128) + lane_off;
    const uint32_t o_tm = tmem + uint32_t(256 + w * 128) + lane_off;
    const int qi = r / p.group, head = r - qi * p.group;  // this row's query in the tile, head in the group
    const int Dn = (p.D + 15) / 16 * 16;
    const float sl2 = CAP ? cap_factor(p.scale, p.cap) : kLog2e * p.scale;
    const float cap2 = p.cap * kLog2e;
    // query of this row in an item: index, -1 if the row holds none
    auto query = [&](const Item& it) {
      const int i = (SOLO ? 0 : w * p.qt) + qi;
      return (qi < p.qt && i < it.nq) ? i : -1;
    };
    auto out_at = [&](const Item& it, int i) {
      return size_t(it.q0 + i) * size_t(p.os) + size_t(it.kvh * p.group + head) * size_t(p.D);
    };
    constexpr bool kUnits = CAP != 0 || BIAS;       // scores in units of log 2 before the exponentials
    // A tile of 128 keys in one step or in two of 64: then the second half of S is on its way while the first is
    // worked on, and only the first half's maximum stands before the first exponentials, but a row's exponent is
    // checked twice. 32 images of 729, 16 heads of 72, E4M3 out: 122 us in one step, 113 in two; 48 documents of up
    // to 1024, 16 heads of 64: 127 and 122. Wide F16 heads lose what they gain (8192 causal, 32 heads of 128: 370
    // and 377; 32 images, 72: 120.6 and 119.4), capped and biased scores more (106 and 124; 56 and 63).
    constexpr int kSteps = kUnits || (NB == 2 && !E4M3) ? 1 : 2;
    float m = -INFINITY, l = 0.0f;
    uint8_t* stage = smem + L::kOffOut + (w * 4 + sub) * 2 * kOutBytes;

    // The pending item's row: where it goes in o (-1: the row holds no query), and what to do.
    long long out_to = -1;
    int out_how = 0;
    // through with item n
    auto done = [&](int n) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarItemDone + n % kItems));
    };
    // Rows are loaded 32 columns at a time. The columns that no product writes hold what an earlier kernel has left;
    // a NaN among them would send every row the long way round (rows_again).
    for (int c = Dn; c < (p.D + 31) / 32 * 32; c += 8) {
      const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      tmem_st8(o_tm + uint32_t(c), zero);
    }
    tmem_st_wait();
    int pending = -1;  // the item whose rows are not written yet
    bool pending_keys = false;
    int full = 0;      // items with keys so far
    bool ok = true;
    int t = 0;  // S tiles so far
    for (int n = 0;; ++n) {
      if (!__all_sync(0xffffffffu, item_wait(n))) {
        ok = false;
        break;
      }
      const Item& it = items[n % kItems];
      const bool keys = it.live && it.jb < it.je;
      if (pending >= 0 && !keys) {  // nothing to hide the item before's rows under
        if (pending_keys && !__all_sync(0xffffffffu, wait_bar(bar(kBarOFull + w), (full - 1) & 1, abort_flag, p.err)))
          break;
        tc_fence_after();
        write_rows<NB, E4M3>(p, items[pending % kItems], to, stage, o_tm, m, l, out_to, out_how, w, r, [] {});
        done(pending);
        pending = -1;
      }
      if (!it.live) break;
      const int jb = it.jb, je = it.je;
      const int i = query(it);
      const int at = it.at + i;
      // rows without a query are computed like the others and never stored
      const int lim = i < 0 ? 0x7fffffff : limit_of(p.causal, at, it.lk, it.prefix);
      // the item before, whose rows go out behind this one's first tile
      const float m_before = m, l_before = l;
      const long long to_before = out_to;
      const int how_before = out_how;
      out_to = i < 0 ? -1 : static_cast<long long>(out_at(it, i));
      out_how = (lim == 0 ? kNothing : 0) | (it.splits > 1 ? kPart : 0) | (jb >= je ? kEmpty : 0);
      const float slope2 = BIAS && i >= 0 && (CAP != 2 || p.slopes) ? __ldg(p.slopes + it.kvh * p.group + head) * kLog2e : 0.0f;
      m = -INFINITY;
      l = 0.0f;
      const int j0 = SOLO ? jb + w : jb, j_end = SOLO ? jb + (je - jb + 1) / 2 * 2 : je;
      for (int j = j0; j < j_end; j += SOLO ? 2 : 1, ++t) {
        // S(t) has finished, and with it every P V product of the group before it
        if (!__all_sync(0xffffffffu, wait_bar(bar(kBarSFull + w), t & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // visible keys of this tile (shared out, the second group's last may lie behind the item's)
        const int valid = (SOLO ? min(lim, je * kTile) : lim) - j * kTile;
        if constexpr (CAP != 0) cut_scores(s_tm, valid);
        float sv[4][32];
        uint32_t(&su)[4][32] = reinterpret_cast<uint32_t(&)[4][32]>(sv);
        tmem_ld32(s_tm, su[0]);
        tmem_ld32(s_tm + 32, su[1]);
        if constexpr (kSteps == 2) {
          tmem_ld_wait(su[0]);
          reg_fence(su[1]);
        }
        tmem_ld32(s_tm + 64, su[2]);
        tmem_ld32(s_tm + 96, su[3]);
        if constexpr (kSteps == 1) {
          tmem_ld_wait(su[0]);
          reg_fence(su[1]);
          reg_fence(su[2]);
          reg_fence(su[3]);
        }
        const float d0 = float(at - j * kTile);
        // Where no visible key of the tile lies behind the query, or none before it, |d0 - e| is a line.
        // (A row without a query has nothing to say.)
        const bool none_behind = BIAS && __all_sync(0xffffffffu, i < 0 || at >= min(lim, j * kTile + kTile) - 1);
        const bool line = BIAS && (none_behind || __all_sync(0xffffffffu, i < 0 || at <= j * kTile));
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
        for (int h = 0; h < kSteps; ++h) {
          constexpr int kC = 4 / kSteps;  // 32-key groups of a step
          if (h == 1) {
            tmem_ld_wait(su[2]);
            reg_fence(su[3]);
          }
          if constexpr (CAP != 0)
#pragma unroll
            for (int c = kC * h; c < kC * h + kC; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float* s = &sv[c][e];
                if constexpr (CAP == 1) {
                  capped4(s, sl2, cap2);
                } else {
                  float big[4] = {s[0], s[1], s[2], s[3]};
                  capped4(big, sl2, cap2);
#pragma unroll
                  for (int k = 0; k < 4; ++k) s[k] = far_capped(s[k] * (kLog2e * p.scale), s[k] * sl2, big[k]);
                }
              }
          if constexpr (BIAS) {
            const float on = CAP ? 1.0f : sl2;
            if (line) {
              const float slope = none_behind ? slope2 : -slope2, first = -slope * d0;
#pragma unroll
              for (int c = kC * h; c < kC * h + kC; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                  fma_x2(sv[c][e], sv[c][e + 1], sv[c][e], sv[c][e + 1], on, on, fmaf(slope, float(32 * c + e), first),
                         fmaf(slope, float(32 * c + e + 1), first));
            } else {
#pragma unroll
              for (int c = kC * h; c < kC * h + kC; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  sv[c][e] = fmaf(-slope2, fabsf(d0 - float(32 * c + e)), CAP ? sv[c][e] : sv[c][e] * sl2);
            }
          }
          if (valid < 32 * kC * (h + 1)) {
#pragma unroll
            for (int c = kC * h; c < kC * h + kC; ++c)
              if (valid < 32 * c + 32)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (32 * c + e >= valid) sv[c][e] = -INFINITY;
          }
          float mq[2 * kC];
#pragma unroll
          for (int k = 0; k < 2 * kC; ++k) {
            const float* s = &sv[kC * h + (k >> 1)][(k & 1) * 16];
            mq[k] = fmaxf(s[0], s[1]);
          }
#pragma unroll
          for (int k = 0; k < 2 * kC; ++k)
#pragma unroll
            for (int e = 2; e < 16; e += 2) {
              const float* s = &sv[kC * h + (k >> 1)][(k & 1) * 16];
              mq[k] = fmax3(mq[k], s[e], s[e + 1]);
            }
          float mx = fmaxf(fmax3(mq[0], mq[1], mq[2]), mq[3]);
          if constexpr (kC == 4) mx = fmaxf(fmax3(mq[4], mq[5], mq[6]), fmaxf(mq[7], mx));
          const float m_half = kUnits ? mx : mx * sl2;
          const bool raise = m_half > m + kSlack;
          // (with two steps a whole number: the factor on the first one's P loses no bits)
          const float m_new = raise ? (kSteps == 2 ? floorf(m_half) : m_half) - kHead : m;
          if ((j > j0 || h == 1) && __any_sync(0xffffffffu, raise)) {
            const float f = raise ? ex2(m - m_new) : 1.0f;
            l *= f;
            if (h == 1) {  // what the first half has left
              s0 *= f, s1 *= f, s2 *= f, s3 *= f;
              tmem_st_wait();
              uint32_t pk[32];
              tmem_ld32(s_tm, pk);
              tmem_ld_wait(pk);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&pk[e]));
                // (f is a power of two: only what falls below 2^-14 loses bits, 2^-33 of the row's largest)
                const __half2 y = __floats2half2_rn(x.x * f, x.y * f);
                pk[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              tmem_st32(s_tm, pk);
            }
            if (j > j0)
#pragma unroll 1
              for (int c = 0; c < Dn; c += 8) {
                uint32_t e[8];
                tmem_ld8(o_tm + uint32_t(c), e);
                tmem_ld_wait();
                asm volatile("" : "+r"(e[0]), "+r"(e[1]), "+r"(e[2]), "+r"(e[3]), "+r"(e[4]), "+r"(e[5]), "+r"(e[6]),
                             "+r"(e[7]));
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = __float_as_uint(__uint_as_float(e[k]) * f);
                tmem_st8(o_tm + uint32_t(c), e);
              }
          }
          m = m_new;
          const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
          for (int c = kC * h; c < kC * h + kC; c += 2) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float* s = &sv[c + (e >> 4)][2 * (e & 15)];
              float x0, x1;
              if constexpr (kUnits) add_x2(x0, x1, s[0], s[1], -ref, -ref);
              else fma_x2(x0, x1, s[0], s[1], sl2, sl2, -ref, -ref);
              x0 = ex2(x0);
              x1 = ex2(x1);
              if (e & 1) add_x2(s2, s3, s2, s3, x0, x1);
              else add_x2(s0, s1, s0, s1, x0, x1);
              // F16, what the products take at full rate: 2^-11 of each probability (with TF32 or in two F16 parts
              // P V would take twice as long); their sum l is of the unrounded ones.
              const __half2 y = __floats2half2_rn(x0, x1);
              pk[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            tmem_st32(s_tm + 16 * c, pk);
          }
        }
        l += (s0 + s1) + (s2 + s3);
        auto arrive = [&]() {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(kBarPFull + w));
        };
        if (!SOLO && j == j0 && pending >= 0) {
          // The item before: this S followed its last P V, so its O is final, and the first P V
          // of this item, which overwrites O, waits for the arrival. Between the two O is only
          // loaded; its rows are written while the products run. (Written before the item's
          // first tile they took 4,000 to 6,000 cycles that nothing else ran in.)
          write_rows<NB, E4M3>(p, items[pending % kItems], to, stage, o_tm, m_before, l_before, to_before, how_before, w, r, arrive);
          done(pending);
          pending = -1;
        } else {
          arrive();
        }
      }
      if (!ok) break;
      if constexpr (SOLO) {
        if (jb < je) {
          float2* ml = reinterpret_cast<float2*>(smem + L::kOffOut) + r;
          auto wait = [&](int b) {
            const bool got = __all_sync(0xffffffffu, wait_bar(bar(b), full & 1, abort_flag, p.err));
            tc_fence_after();
            return got;
          };
          if (w == 1) {
            *ml = make_float2(m, l);
            mbar_arrive(bar(kBarJoin));
            if (!wait(kBarRead)) break;  // (the next item's P V writes O again)
          } else {
            if (!wait(kBarOFull) || !wait(kBarOFull + 1) || !wait(kBarJoin)) break;
            write_shared(p, it, o_tm, m, l, ml->x, ml->y, out_to, out_how, r);
            tc_fence_before();
            mbar_arrive(bar(kBarRead));
          }
          ++full;
        } else if (w == 0) {
          write_special(p, it, o_tm, m, l, out_to, out_how, 0, r);
        }
        done(n);
        continue;
      }
      pending = n;
      pending_keys = jb < je;
      full += pending_keys;
    }
    tmem_ld_wait();
    tmem_st_wait();
    if (lane == 0) bulk_wait_all();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Tensor map of [rows, heads * D] with a row stride: boxes of 64 values x `box_heads` heads x
// `box_rows` rows, 128-byte swizzle; values past a head's width and rows past the last read as 0.
sv_status packed_map(CUtensorMap* m, const void* ptr, int D, int heads, int rows, long long stride, int box_heads,
                     int box_rows) {
  const uint64_t dims[3] = {uint64_t(D), uint64_t(heads), uint64_t(rows)};
  const uint64_t strides[2] = {uint64_t(D) * 2u, uint64_t(stride) * 2u};
  const uint32_t box[3] = {64u, uint32_t(box_heads), uint32_t(box_rows)};
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int NB, int CAP, bool BIAS, bool E4M3, bool SOLO>
sv_status packed_launch_as(const Params& p, int grid, cudaStream_t s) {
  auto kern = packed_tile_kernel<NB, CAP, BIAS, E4M3, SOLO>;
  static unsigned long long attr_set = 0;  // the attribute is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice(packed attention)");
  const unsigned long long bit = (dev >= 0 && dev < kMaxAttrDevices) ? 1ull << dev : 0ull;
  if (!(attr_set & bit) || !bit) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<NB>::kBytes);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(packed attention)");
    attr_set |= bit;
  }
  CUtensorMap tq, tk, tv;
  sv_status st = packed_map(&tq, p.q, p.D, p.hq, p.total_q, p.qs, p.group, p.qt);
  // (without keys no item copies any; the maps then only need to be valid)
  const bool keys = p.total_k > 0;
  if (st == SV_OK) st = packed_map(&tk, keys ? p.k : p.q, p.D, p.hk, keys ? p.total_k : 1, p.ks, 1, kTile);
  if (st == SV_OK) st = packed_map(&tv, keys ? p.v : p.q, p.D, p.hk, keys ? p.total_k : 1, p.vs, 1, kTile);
  // the output: 32 columns of the rows of a softmax warp
  CUtensorMap to = tq;
  if (st == SV_OK && p.out_tma) {
    const uint64_t es = p.out_e4m3 ? 1 : 2;
    const uint64_t dims[3] = {uint64_t(p.D), uint64_t(p.hq), uint64_t(p.total_q)};
    const uint64_t strides[2] = {uint64_t(p.D) * es, uint64_t(p.os) * es};
    const uint32_t box[3] = {32u, uint32_t(p.group), uint32_t(32 / p.group)};
    st = make_tmap(&to, p.out_e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p.o, dims,
                   strides, box, p.out_e4m3 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (st != SV_OK) return st;
  e = launch_pdl(kern, dim3(unsigned(grid)), dim3(kThreads), size_t(Smem<NB>::kBytes), s, p, tq, tk, tv, to);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "packed attention launch");
}

template <int NB, bool E4M3, bool SOLO>
sv_status packed_launch(const Params& p, int grid, cudaStream_t s) {
  if constexpr (!SOLO)
    if (p.cap >= kFarCap) return packed_launch_as<NB, 2, true, E4M3, SOLO>(p, grid, s);
  if (p.cap > 0.0f)
    return p.slopes ? packed_launch_as<NB, 1, true, E4M3, SOLO>(p, grid, s)
                    : packed_launch_as<NB, 1, false, E4M3, SOLO>(p, grid, s);
  return p.slopes ? packed_launch_as<NB, 0, true, E4M3, SOLO>(p, grid, s)
                  : packed_launch_as<NB, 0, false, E4M3, SOLO>(p, grid, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

sv_status tile_launch(const Params& p, cudaStream_t s) {
  // items at most: every document rounds its pairs of tiles up
  const long long items = (p.total_q / (2 * p.qt) + p.docs) * static_cast<long long>(p.hk);
  int grid = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  if (!p.counters && items < grid) grid = int(items);
  // Few items of 8 key tiles and more on average: a tile each, its keys shared out between the groups. (256 queries of
  // 8 heads of 128 over 2: 1,024 keys 19.2 us in items of two tiles and 18.0 so, 2,048 keys 34 and 25, 9,000 keys
  // 58 and 48; one image of 729 tokens, 16 heads of 72: 16.0 and 16.9, the end costs what the chain has saved.)
  if (p.counters && p.cap < kFarCap && 2 * items <= grid && p.total_k >= static_cast<long long>(kMinSplit) * kTile * p.docs)
    return p.D > 64 ? packed_launch<2, false, true>(p, grid, s) : packed_launch<1, false, true>(p, grid, s);
  if (p.out_e4m3) return p.D > 64 ? packed_launch<2, true, false>(p, grid, s) : packed_launch<1, true, false>(p, grid, s);
  return p.D > 64 ? packed_launch<2, false, false>(p, grid, s) : packed_launch<1, false, false>(p, grid, s);
}

}  // namespace packed
}  // namespace sv

extern "C" {

size_t sv_attention_packed_workspace(int docs, int total_q, int total_k, int q_heads, int kv_heads, int head_dim) {
  using namespace sv::packed;
  if (docs < 1 || total_q < 0 || total_k < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
      q_heads / kv_heads > 64 || head_dim < 1)
    return kCounterBytes;  // (the call refuses these)
  const int group = q_heads / kv_heads, d = head_dim > 128 ? 128 : (head_dim + 15) / 16 * 16;
  if (few_rows(docs, total_q, group)) return few_workspace(d);
  // parts of divided ranges: twice the grid at most (see Schedule), and twice the key tiles over
  // the shortest part
  const double pairs = double(total_q / (2 * (kTile / group))) + docs, tiles = double(total_k / kTile) + 1.0;
  const double most = 2.0 * pairs * kv_heads * tiles / kMinSplit + 1.0;
  const size_t slots = total_k <= kMinSplit * kTile ? 0 : size_t(most < kMaxSlots ? most : kMaxSlots);
  return kCounterBytes + slots * 2 * size_t(d + 2) * kTile * sizeof(float);
}

sv_status sv_attention_packed(const void* q, const void* k, const void* v, void* o, const int* q_offsets,
                              const int* k_offsets, int docs, int total_q, int total_k, int q_heads, int kv_heads,
                              int head_dim, long long q_stride, long long k_stride, long long v_stride,
                              long long o_stride, const sv_attention_options* options, int out_dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  using namespace sv;
  using namespace sv::packed;
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
  constexpr int kMostRows = 0x7fffffff - 4096;  // (key and row numbers run past the last by less than that)
  if (total_q > kMostRows || total_k > kMostRows || docs > (1 << 24) ||
      (total_q / (2 * kTile * kv_heads / q_heads) + static_cast<long long>(docs)) * kv_heads >= (1ll << 30)) {
    // (items hold 2 (128 / group) queries, which may be a fifth fewer: their numbers stay below 2^31)
    set_error("%s: %d documents of %d queries with %d heads and %d keys are too many for one call", fn, docs, total_q,
              q_heads, total_k);
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
  Params p = {};
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
  p.qt = kTile / p.group;
  // a warp's 32 output rows go by TMA where they are whole queries on 16 bytes
  p.out_tma = 32 % p.group == 0 && (!p.out_e4m3 || (head_dim % 16 == 0 && o_stride % 16 == 0));
  if (workspace) {
    p.counters = static_cast<unsigned*>(workspace);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  }
  LaunchScope L(kKindAttn, 0.0, 0.0, s);
  return few_rows(docs, total_q, p.group) ? few_launch(p, s) : tile_launch(p, s);
}

}  // extern "C"
