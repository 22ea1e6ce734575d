// Rotary positions with several axes, and the append to a paged key-value
// cache that applies them on the way.
//
// Pair j of a head's channels, (x, y), at a position p with coordinates
// p[0 .. axes): angle a = p[axis_j] * f_j, result (x cos a - y sin a,
// y cos a + x sin a).  The gradient turns by -a.  Channels past the pairs pass
// through.
//
// Bound: memory, each element read once and written once.  The angle is the
// part that could exceed it: cos and sin cost about 30 instructions a pair,
// against 8 bytes moved, so a thread forms them once for its channels of a
// token and applies them to several heads.  The angle itself is an integer
// product modulo one turn (RotaryPlan): exact to 2^-32 turns at any position,
// where a product in 32-bit floating point loses the fraction of a turn from a
// few thousand positions on, and 64-bit floating point runs at a small
// fraction of the rate here.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "token_ops.h"

namespace wan {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// E elements, as one access of W elements' bytes each.
template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using t = uint4; };
template <>
struct Raw<8> { using t = uint2; };
template <>
struct Raw<4> { using t = uint32_t; };
template <>
struct Raw<2> { using t = uint16_t; };

template <typename T, int E, int W>
struct Vec {
  static_assert(E % W == 0, "whole accesses");
  using R = typename Raw<W * (int)sizeof(T)>::t;
  union {
    R r[E / W];
    T e[E];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < E / W; ++i) r[i] = reinterpret_cast<const R*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < E / W; ++i) reinterpret_cast<R*>(p)[i] = r[i];
  }
};

__device__ __forceinline__ long long position(const void* pos, int pos64, long long i) {
  return pos64 ? ((const long long*)pos)[i] : (long long)((const int*)pos)[i];
}

// cos and sin of pair j's angle at the position whose coordinates start at
// value i of pos.
__device__ __forceinline__ void pair_angle(const RotaryPlan& plan, int j, const void* pos, int pos64, long long i,
                                           float* c, float* s) {
  const long long p = position(pos, pos64, i + plan.axis[j]);
  const uint64_t turn = (uint64_t)p * plan.turn[j];
  // the signed top word, -2^31 .. 2^31, is -1/2 .. 1/2 turns: -1 .. 1 half turns
  const float half_turns = (float)(int)(turn >> 32) * 0x1p-31f;
  sincospif(half_turns, s, c);
  if (plan.inverse) *s = -*s;
}

// The columns a thread handles in one head.  Interleaved: E consecutive
// channels, E / 2 pairs.  Halves: columns below pairs / E hold E pairs, the
// channels [E c, E c + E) and the ones `pairs` further on; the columns after
// them hold E channels that pass through.
template <typename T, int E, int W, bool INTER>
struct Column {
  static constexpr int NP = INTER ? E / 2 : E;
  float c[NP], s[NP];
  uint32_t on;  // interleaved: bit i set if pair i is turned (the others pass through)
  int c0, c1;   // first channel, and the second half's first channel (or -1)

  static __host__ __device__ __forceinline__ int count(int D, int pairs) {
    return INTER ? D / E : pairs / E + (D - 2 * pairs) / E;
  }
  __device__ __forceinline__ void place(int col, int pairs, bool turn) {
    on = 0;
    if (INTER) {
      c0 = col * E;
      c1 = -1;
      if (turn) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (col * NP + i < pairs) on |= 1u << i;
      }
    } else {
      const int rot = pairs / E;
      if (col < rot) {
        c0 = col * E;
        c1 = c0 + pairs;
        on = turn ? 1u : 0u;
      } else {
        c0 = 2 * pairs + (col - rot) * E;
        c1 = -1;
      }
    }
  }
  __device__ __forceinline__ void angles(const RotaryPlan& plan, int col, const void* pos, int pos64, long long i0) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (INTER ? (on >> i) & 1 : on) pair_angle(plan, col * NP + i, pos, pos64, i0, &c[i], &s[i]);
    }
  }
  __device__ __forceinline__ void turn(Vec<T, E, W>& a, Vec<T, E, W>& b) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      T& xr = INTER ? a.e[INTER ? 2 * i : i] : a.e[i];
      T& yr = INTER ? a.e[INTER ? 2 * i + 1 : i] : b.e[i];
      const float x = to_f(xr), y = to_f(yr);
      const T nx = from_f<T>(fmaf(x, c[i], -(y * s[i]))), ny = from_f<T>(fmaf(y, c[i], x * s[i]));
      if (INTER ? (on >> i) & 1 : on) {
        xr = nx;
        yr = ny;
      }
    }
  }
  // heads h0 .. h1-1 of one token, U of them in flight
  template <int U>
  __device__ __forceinline__ void run(const T* x, long long xh, T* out, long long oh, int h0, int h1) const {
    for (int h = h0; h < h1; h += U) {
      Vec<T, E, W> a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u < h1) {
          a[u].load(x + (h + u) * xh + c0);
          if (!INTER && c1 >= 0) b[u].load(x + (h + u) * xh + c1);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u < h1) {
          turn(a[u], b[u]);
          a[u].store(out + (h + u) * oh + c0);
          if (!INTER && c1 >= 0) b[u].store(out + (h + u) * oh + c1);
        }
    }
  }
};

constexpr int kRotaryThreads = 256;

template <typename T, int E, int W, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads)
    rotary_kernel(const __grid_constant__ RotaryArgs a, int cols, int tpb, int hpt) {
  const int tl = threadIdx.x / cols, col = threadIdx.x - tl * cols;
  const long long tok = (long long)blockIdx.x * tpb + tl;
  if (tok >= (long long)a.B * a.S) return;
  const int b = (int)(tok / a.S), t = (int)(tok - (long long)b * a.S);
  Column<T, E, W, INTER> cl;
  cl.place(col, a.plan.pairs, true);
  cl.angles(a.plan, col, a.pos, a.pos64, b * a.pos_b + (long long)t * a.plan.axes);
  const int h0 = blockIdx.y * hpt;
  cl.template run<4>((const T*)a.x + b * a.xb + t * a.xs, a.xh, (T*)a.out + b * a.ob + t * a.os, a.oh, h0,
                     min(a.H, h0 + hpt));
}

// Rows of k (turned), v (as they are) and q (turned): grid.y runs over groups
// of hpt heads of q, then of k, then of v.  A token whose slot does not exist
// (no sequence, a bad page, a position outside the table) leaves the cache as
// it is and says so in the status word; its q row is turned all the same when
// a sequence owns it.
template <typename T, int E, int W, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads)
    kv_append_kernel(const __grid_constant__ AppendArgs a, int cols, int tpb, int hpt, int nq, int nk) {
  const int tl = threadIdx.x / cols, col = threadIdx.x - tl * cols;
  const long long row = (long long)blockIdx.x * tpb + tl;
  if (row >= a.b.T) return;
  const int t = (int)row;
  // the sequence of the row: the last one that starts at or before it
  int b = t, r0 = t, n = 1;
  if (a.b.cu) {
    int lo = 0, hi = a.b.B;  // cu[lo] <= t (if anything is)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.b.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    if (!kv_rows(a.b.cu, a.b.T, b, &r0, &n)) {
      if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadLength);
      return;
    }
    if (t < r0 || t >= r0 + n) return;  // behind the last sequence
  } else if (t >= a.b.B) {
    return;
  }
  const int y = blockIdx.y;
  const int kind = y < nq ? 0 : y < nq + nk ? 1 : 2;  // q, k, v
  Column<T, E, W, INTER> cl;
  cl.place(col, a.plan.pairs, kind < 2);
  const T* src;
  T* dst;
  long long sh, dh;
  int h0, heads;
  if (kind == 0) {
    src = (const T*)a.q + t * a.q_t;
    dst = (T*)a.qo + t * a.qo_t;
    sh = a.q_h;
    dh = a.qo_h;
    h0 = y * hpt;
    heads = a.q_heads;
  } else {
    const long long i = (long long)a.b.lengths[b] - n + (t - r0);
    int len;
    if (!kv_length(a.b.lengths[b], a.b.max_pages, a.c.page_size, &len) || i < 0) {
      if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadLength);
      return;
    }
    const int p = kv_page(a.b.pages + b * a.b.page_stride, (int)i, a.c.page_size, a.c.pages);
    if (p < 0) {
      if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadPage);
      return;
    }
    const int off = (int)i % a.c.page_size;
    heads = a.c.heads;
    if (kind == 1) {
      src = (const T*)a.k + t * a.k_t;
      sh = a.k_h;
      dst = (T*)a.c.k + p * a.c.k_page + off * a.c.k_row;
      dh = a.c.k_head;
      h0 = (y - nq) * hpt;
    } else {
      src = (const T*)a.v + t * a.v_t;
      sh = a.v_h;
      dst = (T*)a.c.v + p * a.c.v_page + off * a.c.v_row;
      dh = a.c.v_head;
      h0 = (y - nq - nk) * hpt;
    }
  }
  if (kind < 2) cl.angles(a.plan, col, a.pos, a.pos64, (long long)t * a.plan.axes);
  cl.template run<4>(src, sh, dst, dh, h0, min(heads, h0 + hpt));
}

// Heads per thread: as many as leave two blocks of threads per SM (one angle
// serves them all), up to 8.
int heads_per_thread(long long rows, int cols, int heads) {
  int hpt = 8;
  while (hpt > 1 && rows * cols * ((heads + hpt - 1) / hpt) < 2LL * 152 * kRotaryThreads) hpt /= 2;
  return hpt;
}

template <typename T, int E, int W, bool INTER>
cudaError_t go_rotary(const RotaryArgs& a, cudaStream_t s) {
  const int cols = Column<T, E, W, INTER>::count(a.D, a.plan.pairs);
  const int tpb = kRotaryThreads / cols;
  const long long rows = (long long)a.B * a.S;
  const int hpt = heads_per_thread(rows, cols, a.H);
  const dim3 grid((unsigned)((rows + tpb - 1) / tpb), (a.H + hpt - 1) / hpt);
  rotary_kernel<T, E, W, INTER><<<grid, tpb * cols, 0, s>>>(a, cols, tpb, hpt);
  return cudaGetLastError();
}

template <typename T, int E, int W, bool INTER>
cudaError_t go_append(const AppendArgs& a, cudaStream_t s) {
  const int cols = Column<T, E, W, INTER>::count(a.c.D, a.plan.pairs);
  const int tpb = kRotaryThreads / cols;
  const int hpt = heads_per_thread(a.b.T, cols, 2 * a.c.heads + a.q_heads);
  const int nq = (a.q_heads + hpt - 1) / hpt, nk = (a.c.heads + hpt - 1) / hpt;
  const dim3 grid((unsigned)((a.b.T + tpb - 1) / tpb), nq + 2 * nk);
  kv_append_kernel<T, E, W, INTER><<<grid, tpb * cols, 0, s>>>(a, cols, tpb, hpt, nq, nk);
  return cudaGetLastError();
}

// Columns of E elements in accesses of W: 16-byte columns where the channel
// counts divide into them and the addresses allow it, narrower ones otherwise.
// Interleaved columns need D (even) a multiple of E (pairs past the turned ones
// pass through inside a column); halves also need `pairs` to be one.
template <typename T, template <typename, int, int, bool> class Go, typename Args>
cudaError_t by_width(const Args& a, int D, int pairs, int width, bool inter, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (inter) {
    if (D % V == 0 && width >= V) return Go<T, V, V, true>::go(a, s);
    if (D % 4 == 0 && width >= 4) return Go<T, 4, 4, true>::go(a, s);
    if (width >= 2) return Go<T, 2, 2, true>::go(a, s);
    return Go<T, 2, 1, true>::go(a, s);
  }
  const int g = pairs | D;  // a power of two divides both iff it divides their bitwise or
  if (g % V == 0 && width >= V) return Go<T, V, V, false>::go(a, s);
  if (g % 4 == 0 && width >= 4) return Go<T, 4, 4, false>::go(a, s);
  if (g % 2 == 0 && width >= 2) return Go<T, 2, 2, false>::go(a, s);
  return Go<T, 1, 1, false>::go(a, s);
}
template <typename T, int E, int W, bool INTER>
struct GoRotary {
  static cudaError_t go(const RotaryArgs& a, cudaStream_t s) { return go_rotary<T, E, W, INTER>(a, s); }
};
template <typename T, int E, int W, bool INTER>
struct GoAppend {
  static cudaError_t go(const AppendArgs& a, cudaStream_t s) { return go_append<T, E, W, INTER>(a, s); }
};

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  const bool in = a.plan.interleaved;
  if (a.elem == 0) return by_width<float, GoRotary>(a, a.D, a.plan.pairs, a.width, in, s);
  if (a.elem == 1) return by_width<__nv_bfloat16, GoRotary>(a, a.D, a.plan.pairs, a.width, in, s);
  return by_width<__half, GoRotary>(a, a.D, a.plan.pairs, a.width, in, s);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) {
  const bool in = a.plan.interleaved;
  if (a.c.elem == 1) return by_width<__nv_bfloat16, GoAppend>(a, a.c.D, a.plan.pairs, a.width, in, s);
  return by_width<__half, GoAppend>(a, a.c.D, a.plan.pairs, a.width, in, s);
}

}  // namespace wan
