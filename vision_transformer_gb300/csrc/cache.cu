// A key/value cache in pages (sv_cache_write, sv_cache_read): heads of tokens quantised into it and read back.
//
// A head x of a token (D values of F16) is stored as codes c = E4M3(x 2^-e) with the least e in -15 .. 8 for which
// max |x| <= 448 2^e. With max |x| = m 2^p (1 <= m < 2) that is p - 8, or p - 7 where m > 1.75: both are read off the
// bits of the largest magnitude, and no division or logarithm is needed. Two roundings do not meet: x 2^-e in F16 is
// exact but below 2^-14, where the code is 0 either way (it rounds to multiples of 2^-9). Reading gives c 2^e, an
// F16 number: c is 0 or a multiple of 2^-9 with four significant bits, and where c's own grid is finer than F16's
// (x a multiple of 2^-24), x was on that grid already.
//
// Bound: DRAM, every value read once and written once in its other form (D = 128: 3 bytes and 1/128 a value).
// A warp takes 16 consecutive tokens of one head of the keys (or values): 8 or 16 lanes a token, 16 bytes of F16 a
// lane, all of its loads on their way at once (8 KB of F16 at 128 dimensions), the largest magnitude by shuffles among
// the token's lanes. So the stored rows of a warp lie side by side in the page (as long as the tokens are of one
// sequence), and the 16 scale bytes go out in one access. The tokens' sequences and pages are looked up a lane a token
// (a binary search among the offsets), when writing behind the loads of the values, which do not depend on them.
// 14,174 tokens of 8 heads of 128 are written in 18.2 us (4.8 TB/s; 56% of all cycles issue), 23,328 of 16 heads of 72
// as F16 in 40.4 (80% of the copy bandwidth), 24,742 of 8 heads of 128 read back in 29.0 (90%). 64 or 512 threads a
// CTA, or registers for 8 or 10 of them an SM, change nothing or lose.
#include "cached.h"

namespace sv {
namespace cached {
namespace {

constexpr int kMoveThreads = 128;
constexpr int kTokens = 16;  // of a warp

struct MoveParams {
  View c;
  const __half *k, *v;  // written to when reading the cache
  long long ks, vs;
  const int* off;
  int total;
};

// Whether a sequence with n rows in the call, behind `first` tokens that count as its own, cannot have `have` tokens.
__device__ __forceinline__ bool bad_length(const View& c, int have, long long n, int first) {
  return have < 0 || have > (static_cast<long long>(c.stride) << c.shift) || n > static_cast<long long>(first) + have;
}

// Where token t of the call is kept: the first byte of its page, and its place there; false: nowhere.
template <bool READ>
__device__ __forceinline__ bool place_of(const MoveParams& p, int t, long long& base, int& at) {
  const View& c = p.c;
  int s = 0;
  if (p.off) {  // the number of offsets 1 .. count that are <= t
    int hi = c.count;
    while (s < hi) {
      const int mid = s + (hi - s + 1) / 2;
      if (__ldg(p.off + mid) <= t) s = mid;
      else hi = mid - 1;
    }
  } else {
    s = t / (p.total / c.count);
  }
  if (s >= c.count) return false;
  const int q0 = row_offset(p.off, s, c.count, p.total), q1 = row_offset(p.off, s + 1, c.count, p.total);
  if (t < q0 || t >= q1) return false;  // a row of no sequence
  const int have = __ldg(c.lengths + s), first = READ ? c.prefix_len : 0;
  const long long n = static_cast<long long>(q1) - q0;
  if (q0 < 0 || q1 > p.total || bad_length(c, have, n, first)) {
    atomicOr(c.err, kDevErrCache);
    return false;
  }
  int pos = int(have - n + (t - q0));  // among its own tokens
  const int* pages = c.table + static_cast<long long>(s) * c.stride;
  if (READ && pos < 0) {
    pages = c.prefix_pages;
    pos += first;
  }
  const int page = __ldg(pages + (pos >> c.shift));
  if (page < 0 || page >= c.n_pages) {
    atomicOr(c.err, kDevErrCache);
    return false;
  }
  base = page * c.page_bytes;
  at = pos & ((1 << c.shift) - 1);
  return true;
}

// LANES lanes hold a token's head, eight values each.
template <bool READ, bool E4M3, int LANES>
__global__ void __launch_bounds__(kMoveThreads) cache_kernel(const __grid_constant__ MoveParams p) {
  constexpr int kPer = 32 / LANES, kSteps = kTokens / kPer;  // tokens of a step, steps
  static_assert(LANES == 2 * kSteps, "a token's lanes are two for each step");
  constexpr int kEs = E4M3 ? 1 : 2;
  const View& c = p.c;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const unsigned unit = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);  // (below 2^31)
  // Sequences, 32 a warp: offsets that decrease or leave [0, total], and lengths, of those without rows too. (Without
  // offsets every sequence has rows.)
  if (p.off) {
    bool bad = false;
    for (long long s = 32ll * unit + lane; s < c.count; s += 32ll * (kMoveThreads / 32) * gridDim.x) {
      const int a = __ldg(p.off + s), b = __ldg(p.off + s + 1), have = __ldg(c.lengths + s);
      bad |= a < 0 || b < a || b > p.total || bad_length(c, have, static_cast<long long>(b) - a, READ ? c.prefix_len : 0);
    }
    if (bad) atomicOr(c.err, kDevErrCache);
  }
  const unsigned block = unit / unsigned(2 * c.hk);
  const int t0 = int(block) * kTokens;
  if (t0 >= p.total) return;
  const int which = int(unit - block * unsigned(2 * c.hk));  // heads of the keys, then of the values
  const bool values = which >= c.hk;
  const int head = values ? which - c.hk : which;
  const int group = lane / LANES, chunk = lane % LANES;
  const bool mine = 8 * chunk < c.D;
  const long long stride = values ? p.vs : p.ks;
  const __half* rows = (values ? p.v : p.k) + (t0 + group) * stride + head * c.D + 8 * chunk;  // of step 0
  const int last = p.total - t0 - group;  // this lane's tokens are steps i with i * kPer < last

  uint4 x[kSteps];
  if constexpr (!READ) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mine && i * kPer < last) x[i] = __ldg(reinterpret_cast<const uint4*>(rows + i * kPer * stride));
    }
  }
  // Lane r < 16: where token t0 + r is kept, its codes' and its scale byte's place (-1: nowhere).
  long long page = -1;
  int at = 0;
  if (lane < kTokens && t0 + lane < p.total && !place_of<READ>(p, t0 + lane, page, at)) page = -1;
  __syncwarp();
  const int codes = (values ? value_bytes(c) : 0) + (head << c.shift) * c.D * kEs;
  const long long code_place = page < 0 ? -1 : page + codes + at * c.D * kEs;
  const long long scale_place = page < 0 ? -1 : page + scale_bytes(c) + (which << c.shift) + at;
  // Mostly the sixteen lie one behind another in a page: then nobody needs to be asked for a place.
  const long long place0 = __shfl_sync(0xffffffffu, code_place, 0), scale0 = __shfl_sync(0xffffffffu, scale_place, 0);
  const bool in_line = place0 >= 0 && __all_sync(0xffffffffu, lane >= kTokens || scale_place == scale0 + lane);
  auto place_in = [&](int i) -> uint8_t* {  // of this lane's eight numbers of step i
    const long long at_row = in_line ? place0 + (i * kPer + group) * c.D * kEs
                                     : __shfl_sync(0xffffffffu, code_place, i * kPer + group);
    return mine && at_row >= 0 ? c.pages + at_row + 8 * chunk * kEs : nullptr;
  };

  if constexpr (READ) {
    int scale = kNoScale;
    if (page >= 0) scale = __ldg(c.pages + scale_place);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint8_t* from = place_in(i);
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (from) {
        if constexpr (E4M3) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(from));
          x[i].x = w.x, x[i].y = w.y;
        } else {
          x[i] = __ldg(reinterpret_cast<const uint4*>(from));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int byte = __shfl_sync(0xffffffffu, scale, i * kPer + group);
      const bool live = in_line || __shfl_sync(0xffffffffu, code_place, i * kPer + group) >= 0;
      uint4 y = x[i];
      if constexpr (E4M3) {
        y = e4m3_to_f16(make_uint2(x[i].x, x[i].y));
        const __half2 f = f16_power(min(byte, 31) - kNoScale);
        __half2* h = reinterpret_cast<__half2*>(&y);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = __hmul2(h[j], f);
      }
      if (byte == kMarked) y = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
      if (mine && live) *reinterpret_cast<uint4*>(const_cast<__half*>(rows) + i * kPer * stride) = y;
    }
  } else {
    // The largest magnitude's bits of every token (an infinity or NaN is at least 0x7c00): each exchange halves the
    // steps that a lane has a maximum of, until it has that of step lane % kSteps alone.
    uint32_t m[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      m[i] = __vimax3_u16x2(__vimax3_u16x2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu),
                            x[i].w & 0x7fff7fffu, 0u);
#pragma unroll
    for (int o = 1; o < kSteps; o <<= 1) {
      const bool high = lane & o;
#pragma unroll
      for (int i = 0; i < kSteps / (2 * o); ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? m[2 * i] : m[2 * i + 1], o);
        m[i] = __vimax3_u16x2(high ? m[2 * i + 1] : m[2 * i], got, 0u);
      }
    }
    m[0] = __vimax3_u16x2(m[0], __shfl_xor_sync(0xffffffffu, m[0], kSteps), 0u);
    const int top = int(max(m[0] & 0xffffu, m[0] >> 16));
    const bool bad = top >= 0x7c00;
    int e = 0;
    if constexpr (E4M3) e = bad ? 0 : max(-15, (top >> 10) - 23 + ((top & 0x3ff) > 0x300));
    // its scale byte
    const int r = (lane % kSteps) * kPer + group;
    const long long to = in_line ? scale0 + r : __shfl_sync(0xffffffffu, scale_place, r);
    if (to >= 0 && !(lane & kSteps)) c.pages[to] = uint8_t(bad ? kMarked : e + kNoScale);
    const bool some_bad = __any_sync(0xffffffffu, bad), some_large = __any_sync(0xffffffffu, e == 8);
    const uint32_t power = uint32_t(15 - e) << 10;  // 2^-e in F16, twice
    const uint32_t factor = power | power << 16;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int holder = (lane & ~(LANES - 1)) + i;
      if (some_bad && __shfl_sync(0xffffffffu, int(bad), holder)) x[i] = make_uint4(0u, 0u, 0u, 0u);
      uint8_t* to_row = place_in(i);
      if constexpr (E4M3) {
        const uint32_t fw = __shfl_sync(0xffffffffu, factor, holder);
        const __half2 f = *reinterpret_cast<const __half2*>(&fw);
        __half2* h = reinterpret_cast<__half2*>(&x[i]);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = __hmul2(h[j], f);
        if (some_large) {  // (at most 448 but for e = 8, where 256 is held to 240)
          const __half2 most = __float2half2_rn(__shfl_sync(0xffffffffu, e, holder) == 8 ? 240.0f : 448.0f);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = __hmax2(__hmin2(h[j], most), __hneg2(most));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h[j]), __NV_SATFINITE, __NV_E4M3);
        if (to_row) *reinterpret_cast<uint2*>(to_row) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      } else {
        if (to_row) *reinterpret_cast<uint4*>(to_row) = x[i];
      }
    }
  }
}

template <bool READ>
sv_status move(const char* fn, const sv_cache* cache, const sv_cache_batch* batch, const void* k, const void* v,
               const int* offsets, int total, long long k_stride, long long v_stride, cudaStream_t s) {
  MoveParams p = {};
  sv_status st = make_view(fn, cache, batch, offsets, total, &p.c);
  if (st != SV_OK) return st;
  const long long row = static_cast<long long>(p.c.hk) * p.c.D;
  p.ks = k_stride ? k_stride : row;
  p.vs = v_stride ? v_stride : row;
  if (p.ks < row || p.vs < row || (p.ks | p.vs) % 8) {
    set_error("%s: row strides must be multiples of 8 that cover a row (k %lld, v %lld)", fn, p.ks, p.vs);
    return SV_ERR_INVALID_ARG;
  }
  if ((total && (!k || !v)) || ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15)) {
    set_error("%s: k and v must be 16-byte aligned pointers", fn);
    return SV_ERR_INVALID_ARG;
  }
  if (total == 0) return SV_OK;
  st = ensure_runtime();
  if (st != SV_OK) return st;
  p.c.err = dev_err();
  p.k = static_cast<const __half*>(k);
  p.v = static_cast<const __half*>(v);
  p.off = offsets;
  p.total = total;
  const long long units = (static_cast<long long>(total) + kTokens - 1) / kTokens * (2 * p.c.hk);
  const dim3 grid(unsigned((units + kMoveThreads / 32 - 1) / (kMoveThreads / 32)));
  const double numbers = 2.0 * total * double(row);
  LaunchScope L(kKindOther, 0.0, numbers * (2 + (p.c.e4m3 ? 1 : 2)), s);
  void (*kern)(MoveParams);
  if (p.c.D > 64) kern = p.c.e4m3 ? cache_kernel<READ, true, 16> : cache_kernel<READ, false, 16>;
  else kern = p.c.e4m3 ? cache_kernel<READ, true, 8> : cache_kernel<READ, false, 8>;
  const cudaError_t e = launch_pdl(kern, grid, dim3(kMoveThreads), 0, s, p);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, fn);
}

bool cache_sizes(int page_size, int kv_heads, int head_dim, int dtype) {
  return page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0 && kv_heads >= 1 &&
         kv_heads <= 65536 && head_dim >= 8 && head_dim <= 128 && head_dim % 8 == 0 &&
         (dtype == SV_DT_F16 || dtype == SV_DT_E4M3) &&
         // (places in a page are 32-bit numbers)
         static_cast<long long>(page_size) * kv_heads * (2 * head_dim + 1) * 2 < (1ll << 31);
}

}  // namespace

sv_status make_view(const char* fn, const sv_cache* cache, const sv_cache_batch* batch, const int* offsets, int total,
                    View* v) {
  if (!cache || !batch) {
    set_error("%s: no cache or batch", fn);
    return SV_ERR_INVALID_ARG;
  }
  if (cache->n_pages < 1 || cache->kv_heads < 1 || (cache->dtype != SV_DT_F16 && cache->dtype != SV_DT_E4M3) ||
      batch->count < 1 || batch->table_stride < 0 || batch->prefix_len < 0 || total < 0) {
    set_error("%s: bad arguments (n_pages %d, kv_heads %d, dtype %d, count %d, table_stride %d, prefix_len %d, total %d)",
              fn, cache->n_pages, cache->kv_heads, cache->dtype, batch->count, batch->table_stride, batch->prefix_len,
              total);
    return SV_ERR_INVALID_ARG;
  }
  if (!cache_sizes(cache->page_size, cache->kv_heads, cache->head_dim, cache->dtype)) {
    set_error("%s: page_size %d (16, 32, 64, 128 or 256), head_dim %d (a multiple of 8 in [8, 128]) or %d heads are not "
              "supported", fn, cache->page_size, cache->head_dim, cache->kv_heads);
    return SV_ERR_UNSUPPORTED;
  }
  constexpr int kMost = 0x7fffffff - 4096;  // (token and row numbers run past the last by less than that)
  if (total > kMost || batch->count > kMost ||
      static_cast<long long>(batch->prefix_len) +
              static_cast<long long>(batch->table_stride) * cache->page_size > kMost ||
      static_cast<long long>(total) * cache->kv_heads >= (1ll << 33)) {
    set_error("%s: %d sequences of up to %d pages of %d behind %d tokens, %d rows, are too many for one call", fn,
              batch->count, batch->table_stride, cache->page_size, batch->prefix_len, total);
    return SV_ERR_UNSUPPORTED;
  }
  if (!offsets && total % batch->count) {
    set_error("%s: without offsets, %d rows must divide by %d sequences", fn, total, batch->count);
    return SV_ERR_INVALID_ARG;
  }
  if (!cache->pages || (reinterpret_cast<uintptr_t>(cache->pages) & 15) || !batch->lengths ||
      (batch->table_stride && !batch->page_table) || (batch->prefix_len && !batch->prefix_pages) ||
      ((reinterpret_cast<uintptr_t>(batch->page_table) | reinterpret_cast<uintptr_t>(batch->lengths) |
        reinterpret_cast<uintptr_t>(batch->prefix_pages) | reinterpret_cast<uintptr_t>(offsets)) & 3)) {
    set_error("%s: pages must be a 16-byte aligned pointer, page_table, lengths, prefix_pages and offsets 4-byte aligned "
              "ones", fn);
    return SV_ERR_INVALID_ARG;
  }
  v->pages = static_cast<uint8_t*>(cache->pages);
  v->page_bytes = static_cast<long long>(
      sv_cache_page_bytes(cache->page_size, cache->kv_heads, cache->head_dim, cache->dtype));
  v->n_pages = cache->n_pages;
  for (v->shift = 0; (1 << v->shift) < cache->page_size;) ++v->shift;
  v->hk = cache->kv_heads;
  v->D = cache->head_dim;
  v->e4m3 = cache->dtype == SV_DT_E4M3;
  v->count = batch->count;
  v->stride = batch->table_stride;
  v->prefix_len = batch->prefix_len;
  v->table = batch->page_table;
  v->lengths = batch->lengths;
  v->prefix_pages = batch->prefix_pages;
  return SV_OK;
}

}  // namespace cached
}  // namespace sv

extern "C" {

size_t sv_cache_page_bytes(int page_size, int kv_heads, int head_dim, int dtype) {
  if (!sv::cached::cache_sizes(page_size, kv_heads, head_dim, dtype)) return 0;
  const size_t heads = size_t(page_size) * size_t(kv_heads);
  return (heads * 2 * (size_t(head_dim) * (dtype == SV_DT_E4M3 ? 1 : 2) + 1) + 127) / 128 * 128;
}

sv_status sv_cache_write(const sv_cache* cache, const sv_cache_batch* batch, const void* k, const void* v,
                         const int* offsets, int total, long long k_stride, long long v_stride, void* stream) {
  return sv::cached::move<false>("sv_cache_write", cache, batch, k, v, offsets, total, k_stride, v_stride,
                                 static_cast<cudaStream_t>(stream));
}

sv_status sv_cache_read(const sv_cache* cache, const sv_cache_batch* batch, void* k, void* v, const int* offsets,
                        int total, long long k_stride, long long v_stride, void* stream) {
  return sv::cached::move<true>("sv_cache_read", cache, batch, k, v, offsets, total, k_stride, v_stride,
                                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
