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
    *first = max(0, a.ranges[2LL * t]);
    *last = min(len, a.ranges[2LL * t + 1]);
    if (*first >= *last) *first = *last = 0;
  }
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
