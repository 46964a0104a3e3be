// What the kernels on a paged key/value cache share (cache.cu: writing and reading it; cached_attention.cu,
// cached_tiles.cu: attention over it).
#pragma once
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "sv_internal.h"

namespace sv {
namespace cached {

constexpr int kNoScale = 16;  // the byte of the factor 1
constexpr int kMarked = 255;  // the byte of a head that held an infinity or NaN

// A cache and the sequences of a call as the kernels read them.
struct View {
  uint8_t* pages;
  long long page_bytes;
  int n_pages, shift;  // page_size = 1 << shift
  int hk, D;
  int e4m3;
  int count, stride, prefix_len;
  const int *table, *lengths, *prefix_pages;
  int* err;
};

// Bytes in a page before the values, and before the keys' scale bytes, of which there are hk << shift, then as many
// of the values.
__host__ __device__ __forceinline__ int value_bytes(const View& c) {
  return (c.hk << c.shift) * c.D * (c.e4m3 ? 1 : 2);
}
__host__ __device__ __forceinline__ int scale_bytes(const View& c) { return 2 * value_bytes(c); }

// Offset s of the rows of the call's sequences: the caller's, or equal parts.
__device__ __forceinline__ int row_offset(const int* off, int s, int count, int total) {
  return off ? __ldg(off + s) : (total / count) * s;
}

// The eight F16 numbers of eight E4M3 codes (without their factor).
__device__ __forceinline__ uint4 e4m3_to_f16(uint2 w) {
  uint4 r;
  asm("{\n\t.reg .b16 a, b, c, d;\n\t"
      "mov.b32 {a, b}, %4;\n\t"
      "mov.b32 {c, d}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, c;\n\t"
      "cvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "r"(w.x), "r"(w.y));
  return r;
}

// 2^e as F16, twice, for e in -15 .. 15 (2^-15 is below the normal range).
__device__ __forceinline__ __half2 f16_power(int e) {
  const uint32_t h = e == -15 ? 0x0200u : uint32_t(e + 15) << 10;
  const uint32_t w = h | h << 16;
  return *reinterpret_cast<const __half2*>(&w);
}

// Where the partial results of the prefix pass are: items (key head, block of rows) one behind another, each of `steps`
// steps, `chunk` steps a CTA. Item i and CTA c meet in part i + c: `rows` rows of D sums, then exponent and denominator
// of each.
struct PrefixParts {
  float* base;
  int rows, blocks, steps, chunk;  // (all steps together: below 2^31)
};

struct Params {
  View c;
  const __half* q;
  void* o;
  const int* q_off;
  int total_q, group;
  unsigned per_group;  // ceil(2^32 / group)
  long long qs, os;
  float scale, cap;
  int causal, out_e4m3;
  unsigned* counters;  // arrivals at cut items
  float* partial;      // two parts a CTA: of the item cut at the start of its share, at its end
  PrefixParts pre;
  // Where the sequences' rows go through tiles: parts of kTileRows rows, part i + c of item i and CTA c; number and first
  // step of each sequence's first item, then (of one behind the last) the steps of a CTA.
  float* tiles;
  int2* firsts;
};

// Lets a kernel have that much dynamic shared memory (set: devices, by number, that have heard so already). ctas: so many
// an SM are to fit, and the rest of the SM's 228 KB is to be L1; 0: as it comes.
template <typename K>
cudaError_t allow_shared(K kern, int bytes, unsigned long long* set, int ctas = 0) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < kMaxAttrDevices ? 1ull << dev : 0ull;
  if ((*set & bit) && bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && ctas > 0) {
    constexpr int kAll = 228 * 1024;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, (ctas * (bytes + 1024) * 100 + kAll - 1) / kAll);
  }
  if (e == cudaSuccess) *set |= bit;
  return e;
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

// The query of row r of a key head (rows x group of a call are below 2^32).
__device__ __forceinline__ int query_of(const Params& p, int r) {
  return p.group == 1 ? r : int(__umulhi(unsigned(r), p.per_group));
}

// Many rows (cached_tiles.cu), in tiles of 128 rows and 128 keys, results left in parts. The prefix pass: items of `rows`
// 256 or 128 rows, steps of one key tile or two; grid: CTAs that have work. The sequences' pass: items of 128 rows,
// steps of two key tiles.
constexpr int kTileRows = 128;
sv_status prefix_launch(const char* fn, const Params& p, int grid, cudaStream_t s);
sv_status own_tiles_launch(const char* fn, const Params& p, int grid, cudaStream_t s);

// Host: checks a cache and a batch, of `total` rows with or without offsets, and fills the view (its device error
// word once the runtime is there).
sv_status make_view(const char* fn, const sv_cache* cache, const sv_cache_batch* batch, const int* offsets, int total,
                    View* v);

}  // namespace cached
}  // namespace sv
