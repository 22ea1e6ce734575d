// What the kernels that attend over a paged cache share: conversions, the
// exponential, and a call's sequences.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "token_ops.h"

namespace wan {

template <typename T>
__device__ __forceinline__ float val(T v);
template <>
__device__ __forceinline__ float val<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float val<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }
// bit masks of the exponent of a 16-bit value: all ones marks an infinity or a NaN
template <typename T>
struct Expo;
template <>
struct Expo<__nv_bfloat16> { static constexpr uint32_t m = 0x7F80u; };
template <>
struct Expo<__half> { static constexpr uint32_t m = 0x7C00u; };
template <typename T>
__device__ __forceinline__ bool odd16(uint32_t v) { return (v & Expo<T>::m) == Expo<T>::m; }
template <typename T>
__device__ __forceinline__ bool odd32(uint32_t v) { return odd16<T>(v) || odd16<T>(v >> 16); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(x - m); where m = -inf nothing but hidden keys (x = -inf) or a NaN was
// seen: 0, or the NaN
__device__ __forceinline__ float weight(float x, float m) { return m == -INFINITY ? (x == x ? 0.f : x) : ex2(x - m); }

struct Seq {
  int r0, n, len;  // first token row, tokens, keys
};
// Sequence b; one that its batch does not describe has no tokens (or no keys),
// and is told to the status word if `tell`.  X: rows may see by their place (calls
// with ranges take up to 1% longer if that is asked each time).
template <bool X = true>
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, bool tell) {
  Seq s;
  const bool ok = kv_rows(a.b.cu, a.b.T, b, &s.r0, &s.n);
  bool okl = kv_length(a.b.lengths[b], a.b.max_pages, a.c.page_size, &s.len);
  // its tokens have no places, or are more than a tree's may be
  if (X && a.mask != kMaskRanges && (s.n > s.len || (a.mask == kMaskTree && s.n > kMaxDrafts))) {
    okl = false;
    s.len = 0;
  }
  if (tell && !(ok && okl) && a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadLength);
  return s;
}

// Row r of a sequence and key head: token r / group, query head h * group + r %
// group.
template <typename T>
__device__ __forceinline__ T* out_row(const AttnArgs& a, const Seq& s, int h, int r) {
  const int t = r / a.group, g = r - t * a.group;
  return (T*)a.out + (long long)(s.r0 + t) * a.o_t + (long long)(h * a.group + g) * a.o_h;
}
// lse of a row whose weights 2^(x - m) sum to l
__device__ __forceinline__ void put_lse(const AttnArgs& a, const Seq& s, int h, int r, float m, float l) {
  if (!a.lse) return;
  const int t = r / a.group, g = r - t * a.group;
  a.lse[(long long)(s.r0 + t) * a.q_heads + h * a.group + g] =
      l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
// The keys that token row t sees, cut to the sequence's: [first, last), (0, 0) if none.
__device__ __forceinline__ void seen_range(const AttnArgs& a, int t, int len, int* first, int* last) {
  *first = 0;
  *last = len;
  if (a.ranges) {
    *first = max(0, a.ranges[2LL * t]);
    *last = min(len, a.ranges[2LL * t + 1]);
    if (*first >= *last) *first = *last = 0;
  }
}
// What the i-th token of a sequence sees by its place: [0, c) and [lo, hi), c <= lo, and in a tree the drafts of
// ancestors() too.  (c = 0 where the two meet.)
struct Sight {
  int c, lo, hi;
};
__device__ __forceinline__ Sight sight(const AttnArgs& a, const Seq& s, int i) {
  const int base = s.len - s.n;
  if (a.mask == kMaskTree) return Sight{0, 0, base};
  const uint32_t p = (uint32_t)(base + i);
  const uint32_t e = a.frame == 1 ? p + 1 : (p / a.frame + 1) * a.frame;  // below 2^32: p and a frame are below 2^31
  Sight v;
  v.lo = e > a.span ? (int)(e - a.span) : 0;
  v.hi = (int)min((uint32_t)s.len, e);
  v.c = min(a.sinks, v.lo);
  if (v.c == v.lo) v.c = v.lo = 0;
  return v;
}
// The drafts [from, from + 64) that draft i of a sequence sees: bit j - from for its ancestor j, and itself.  A parent that
// is none of the drafts before its child ends the walk, and is told.  A whole warp calls it, each lane for a draft of its own
// (i < 0: none).  Trees of up to 32 * kFamily drafts lie in the lanes' registers, and a step up takes a few shuffles; in
// larger ones each step waits for memory.  (26 drafts of one sequence against 2000 keys took 23.3 us with memory's steps.)
constexpr int kFamily = 4;
struct Family {
  int up[kFamily];  // lane l: parents of drafts l, l + 32, ..
};
__device__ __forceinline__ Family family(const AttnArgs& a, const Seq& s) {
  Family f;
#pragma unroll
  for (int k = 0; k < kFamily; ++k) {
    const int i = 32 * k + (threadIdx.x & 31);
    f.up[k] = i < s.n ? __ldg(a.parents + s.r0 + i) : -1;
  }
  return f;
}
__device__ __forceinline__ uint64_t ancestors(const AttnArgs& a, const Seq& s, const Family& f, int i, int from) {
  uint64_t bits = 0;
  bool bad = false;
  if (s.n <= 32 * kFamily) {
    while (__any_sync(0xffffffffu, i >= from && i >= 0)) {
      int p = __shfl_sync(0xffffffffu, f.up[0], i & 31);
#pragma unroll
      for (int k = 1; k < kFamily; ++k) {
        const int q = __shfl_sync(0xffffffffu, f.up[k], i & 31);
        if ((i >> 5) == k) p = q;
      }
      if (i >= from && i >= 0) {
        if (i - from < 64) bits |= 1ull << (i - from);
        if (p >= i || p < -1) bad = true, p = -1;
        i = p;
      }
    }
  } else {
    while (i >= from && i >= 0) {
      if (i - from < 64) bits |= 1ull << (i - from);
      int p = __ldg(a.parents + s.r0 + i);
      if (p >= i || p < -1) bad = true, p = -1;
      i = p;
    }
  }
  if (bad && a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadParent);
  return bits;
}
// The lowest n of 32 bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }
// Bit j: key k0 + j is in the row's two ranges.
__device__ __forceinline__ uint32_t sight_bits(const Sight& v, int k0) {
  return low_bits(v.c - k0) | (low_bits(v.hi - k0) & ~low_bits(v.lo - k0));
}
// Zeros for the rows of sequences without a key, and NaN for all others if `fault`:
// block `me` of `G` takes every G-th sequence.
template <typename T>
__device__ __forceinline__ void put_empty(const AttnArgs& a, int me, int G, bool fault = false) {
  for (int b = me; b < a.b.B; b += G) {
    const Seq s = sequence(a, b, true);
    if (s.len > 0 && !fault) continue;
    const float x = s.len > 0 ? __int_as_float(0x7fffffff) : 0.f, z = s.len > 0 ? x : -INFINITY;
    for (long long i = threadIdx.x; i < (long long)s.n * a.q_heads; i += blockDim.x) {
      const int t = (int)(i / a.q_heads), h = (int)(i - (long long)t * a.q_heads);
      T* o = (T*)a.out + (long long)(s.r0 + t) * a.o_t + (long long)h * a.o_h;
      for (int c = 0; c < a.c.D; ++c) o[c] = round_to<T>(x);
      if (a.lse) a.lse[(long long)(s.r0 + t) * a.q_heads + h] = z;
    }
  }
}

// A call's tiles form one line, sequence after sequence, that is cut into equal
// pieces of `least` tiles or more; a block takes PIECES of them in a row (one
// each for its warps, or one for all).
//
// 64-bit division takes a tenth of a microsecond; most operands fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((unsigned long long)a | (unsigned long long)b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
struct Piece {
  long long beg, end;  // tiles of the line (empty: beg == end)
  long long live;      // pieces that are not empty: each of `size` tiles, the first `longer` of them one more
  long long size, longer;
  int b;         // the sequence of tile beg
  long long at;  // and the tile's number in it
  __device__ __forceinline__ long long start(long long q) const { return q * size + min(q, longer); }
  // the piece that holds tile x of the line
  __device__ __forceinline__ int holder(long long x) const {
    const long long n = longer * (size + 1);
    return (int)(x < n ? quotient(x, size + 1) : longer + quotient(x - n, size));
  }
};
// All threads of the block call this; `of(b)` counts the tiles of sequence b;
// `scratch` is shared memory of WARPS + 2 PIECES values.
template <int WARPS, int PIECES, typename F>
__device__ __forceinline__ Piece cut_line(int B, int least, long long* scratch, F of) {
  static_assert(PIECES == 1 || PIECES == WARPS, "a piece for the block, or one for each warp");
  long long *s_scan = scratch, *s_b = scratch + WARPS, *s_at = s_b + PIECES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Piece p;
  p.beg = p.end = 0;
  p.b = 0;
  p.at = 0;
  const long long my_q = (long long)blockIdx.x * PIECES + (PIECES == 1 ? 0 : warp);
  long long total = 0;
  auto cut = [&] {
    p.live = min((long long)gridDim.x * PIECES, max(quotient(total, least), total > 0 ? 1LL : 0LL));
    p.size = total > 0 ? quotient(total, p.live) : 1;
    p.longer = total - p.size * p.live;
  };
  if (B <= 32) {
    // a sequence per lane, each warp for itself: no barrier (one sequence of 1000 keys 9.1 us, 9.9 with them)
    const long long mine = lane < B ? of(lane) : 0;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    cut();
    if (my_q < p.live) {
      p.beg = p.start(my_q);
      p.end = p.start(my_q + 1);
      const uint32_t here = __ballot_sync(0xffffffffu, p.beg >= incl - mine && p.beg < incl);
      p.b = __ffs(here) - 1;
      p.at = p.beg - __shfl_sync(0xffffffffu, incl - mine, p.b);
    }
    return p;
  }
  const int chunk = (B + 32 * WARPS - 1) / (32 * WARPS);
  const int b_lo = min(B, (int)threadIdx.x * chunk), b_hi = min(B, b_lo + chunk);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += of(b);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  cut();
#pragma unroll 1
  for (int w = 0; w < PIECES; ++w) {
    const long long q = (long long)blockIdx.x * PIECES + w;
    if (q >= p.live) break;
    const long long beg = p.start(q);
    if (beg >= before && beg < before + mine) {
      long long at = beg - before;
      int b = b_lo;
      for (; b < b_hi; ++b) {
        const long long n = of(b);
        if (at < n) break;
        at -= n;
      }
      s_b[w] = b;
      s_at[w] = at;
    }
  }
  __syncthreads();
  const int w = PIECES == 1 ? 0 : warp;
  if (my_q < p.live) {
    p.beg = p.start(my_q);
    p.end = p.start(my_q + 1);
    p.b = (int)s_b[w];
    p.at = s_at[w];
  }
  return p;
}

// What a piece leaves for the join: the row tile whose first part it holds.
struct Open {
  int parts;  // parts of it in the pieces after this one (0: nothing to join)
  int h, row0, cnt;
  Seq s;
  int pad;
};

}  // namespace wan
