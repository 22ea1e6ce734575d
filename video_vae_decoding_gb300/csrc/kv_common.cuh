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
// and is told to the status word if `tell`.
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, bool tell) {
  Seq s;
  const bool ok = kv_rows(a.b.cu, a.b.T, b, &s.r0, &s.n);
  const bool okl = kv_length(a.b.lengths[b], a.b.max_pages, a.c.page_size, &s.len);
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
    *first = max(0, a.ranges[2 * t]);
    *last = min(len, a.ranges[2 * t + 1]);
    if (*first >= *last) *first = *last = 0;
  }
}
// Zeros for the rows of sequences without a key: block `me` of `G` takes every
// G-th sequence.
template <typename T>
__device__ __forceinline__ void put_empty(const AttnArgs& a, int me, int G) {
  for (int b = me; b < a.b.B; b += G) {
    const Seq s = sequence(a, b, true);
    if (s.len > 0) continue;
    for (int i = threadIdx.x; i < s.n * a.q_heads; i += blockDim.x) {
      const int t = i / a.q_heads, h = i - t * a.q_heads;
      T* o = (T*)a.out + (long long)(s.r0 + t) * a.o_t + (long long)h * a.o_h;
      for (int c = 0; c < a.c.D; ++c) o[c] = round_to<T>(0.f);
      if (a.lse) a.lse[(long long)(s.r0 + t) * a.q_heads + h] = -INFINITY;
    }
  }
}

// A call's tiles form one line, sequence after sequence; block `me` of `G` takes
// an equal piece of it, of `least` tiles or more.  All threads call this; `of(b)` counts the tiles of
// sequence b.
struct Piece {
  long long beg, end;  // tiles of the line (empty: beg == end)
  long long total, live;  // all tiles, and the blocks that have a piece
  int b;               // the sequence of tile beg
  long long at;        // and the tile's number in it
  // the block that holds tile x of the line
  __device__ __forceinline__ int holder(long long x) const { return (int)(((x + 1) * live - 1) / total); }
};
template <int WARPS, typename F>
__device__ __forceinline__ Piece cut_line(int B, int me, int G, int least, long long* scratch, F of) {
  long long *s_scan = scratch + 2, *s_b = scratch, *s_at = scratch + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  Piece p;
  long long before = incl - mine;
  p.total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_scan[w];
    p.total += s_scan[w];
  }
  p.live = min((long long)G, max(p.total / least, p.total > 0 ? 1LL : 0LL));
  p.beg = p.end = 0;
  p.b = 0;
  p.at = 0;
  if (me >= p.live) return p;
  p.beg = p.total * me / p.live;
  p.end = p.total * (me + 1) / p.live;
  if (p.beg >= before && p.beg < before + mine) {
    long long at = p.beg - before;
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const long long n = of(b);
      if (at < n) break;
      at -= n;
    }
    *s_b = b;
    *s_at = at;
  }
  __syncthreads();
  p.b = (int)*s_b;
  p.at = *s_at;
  return p;
}

// What a block leaves for the join: a row tile whose first part it holds.
struct Open {
  int b, rt, h;
  int parts;  // blocks after this one that hold the rest (0: nothing to join)
};

}  // namespace wan
