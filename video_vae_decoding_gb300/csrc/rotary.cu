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
// token and applies them to up to eight heads, whose elements are on their way
// meanwhile (Column).  The angle itself is an integer product modulo one turn
// (RotaryPlan), whose top word is rounded to 24 bits of a half turn: off by pi 2^-25
// at any position, and by the position times what the frequency's rounding to 2^-52 of
// itself is.  A product in 32-bit floating point loses the fraction of a turn from a
// few thousand positions on, and 64-bit floating point runs at a small
// fraction of the rate here.
// 27,280 tokens of 16 heads of 128 in bf16 take 35.7 us, 6.3 TB/s (0.92 of a plain
// copy's rate); the gradient of 16,380 tokens of 12 heads of 80 in fp32 20.8 us
// (0.89).  (Cosines and sines formed once per block in shared memory, with a
// barrier for each group of tokens: 43 us; eight heads' loads with the tables of
// several tokens in registers: 62 us, at 121 registers.)
// The append is bound by the chain token range -> length -> page -> store at three
// waves of blocks: 3520 tokens with queries 16.4 us (0.78 of the copy's rate), seven
// ragged prompts, whose tokens search for their sequence, 22.5 us (0.69).  (Looked up
// once per block through shared memory: 17.8 and 26.5; ahead of the angles: 16.1 and
// 23.3.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "token_ops.h"

namespace wan {

namespace {

// N elements in accesses of W: 32-bit words of one fp32 or two 16-bit values.
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

template <typename T, int N, int W>
struct Vec {
  static_assert(N % W == 0, "whole accesses");
  using R = typename Raw<W * (int)sizeof(T)>::t;
  static constexpr int kWords = (N * (int)sizeof(T) + 3) / 4;
  union {
    R r[N / W];
    uint32_t w[kWords];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* p) {
    if (W * sizeof(T) == 2) w[kWords - 1] = 0;
#pragma unroll
    for (int i = 0; i < N / W; ++i) r[i] = reinterpret_cast<const R*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N / W; ++i) reinterpret_cast<R*>(p)[i] = r[i];
  }
};

// The two 16-bit values of a word, and back (one conversion for both).
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t repack(float x, float y);
template <>
__device__ __forceinline__ uint32_t repack<__nv_bfloat16>(float x, float y) { return pack_bf16x2(x, y); }
template <>
__device__ __forceinline__ uint32_t repack<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float turn_x(float x, float y, float c, float s) { return fmaf(x, c, -(y * s)); }
__device__ __forceinline__ float turn_y(float x, float y, float c, float s) { return fmaf(y, c, x * s); }

// Pairs of neighbouring channels: pair i is (2i, 2i + 1).  Bit i of `on`: turned.
template <typename T, int N, int W>
__device__ __forceinline__ void turn_pairs(Vec<T, N, W>& v, const float* c, const float* s, uint32_t on) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (sizeof(T) == 4) {
      const int e = sizeof(T) == 4 ? 2 * i : 0;
      const float x = __uint_as_float(v.w[e]), y = __uint_as_float(v.w[sizeof(T) == 4 ? e + 1 : 0]);
      if ((on >> i) & 1) {
        v.w[e] = __float_as_uint(turn_x(x, y, c[i], s[i]));
        v.w[sizeof(T) == 4 ? e + 1 : 0] = __float_as_uint(turn_y(x, y, c[i], s[i]));
      }
    } else {
      const float2 f = unpack<typename std::conditional<sizeof(T) == 4, __half, T>::type>(v.w[sizeof(T) == 4 ? 0 : i]);
      if ((on >> i) & 1)
        v.w[sizeof(T) == 4 ? 0 : i] = repack<typename std::conditional<sizeof(T) == 4, __half, T>::type>(
            turn_x(f.x, f.y, c[i], s[i]), turn_y(f.x, f.y, c[i], s[i]));
    }
  }
}
// Channels of the first half (a) with those of the second (b), all turned.
template <typename T, int N, int W>
__device__ __forceinline__ void turn_halves(Vec<T, N, W>& a, Vec<T, N, W>& b, const float* c, const float* s) {
  using H = typename std::conditional<sizeof(T) == 4, __half, T>::type;
#pragma unroll
  for (int i = 0; i < Vec<T, N, W>::kWords; ++i) {
    if (sizeof(T) == 4) {
      const float x = __uint_as_float(a.w[i]), y = __uint_as_float(b.w[i]);
      a.w[i] = __float_as_uint(turn_x(x, y, c[i], s[i]));
      b.w[i] = __float_as_uint(turn_y(x, y, c[i], s[i]));
    } else {
      const float2 x = unpack<H>(a.w[i]), y = unpack<H>(b.w[i]);
      const int p = 2 * i, q = 2 * i + 1 < N ? 2 * i + 1 : p;
      a.w[i] = repack<H>(turn_x(x.x, y.x, c[p], s[p]), turn_x(x.y, y.y, c[q], s[q]));
      b.w[i] = repack<H>(turn_y(x.x, y.x, c[p], s[p]), turn_y(x.y, y.y, c[q], s[q]));
    }
  }
}

constexpr int kRotaryThreads = 256;
constexpr long long kSms = 152;  // of the GB300; they only choose a launch's shape

// How a launch covers tokens x heads x columns.  A column is what a thread
// handles of one head: interleaved, E consecutive channels (E / 2 pairs);
// halves, below pairs / E the channels [E c, E c + E) and the ones `pairs`
// further on (E pairs), after that E channels that pass through.  A block takes
// tpb tokens at a time, `per` times, and one group of hpt heads (blockIdx.y).
struct Cover {
  int cols, tpb, per, hpt;
};

template <typename T, int E, int W, bool INTER>
struct Column {
  static constexpr int NP = INTER ? E / 2 : E;
  // heads per thread: 128 bytes (16-byte columns), asked for together
  static constexpr int U = INTER ? 8 : 4;
  int c0, c1;   // first channel, and the second half's first channel (or -1)
  int p0;       // first pair
  uint32_t on;  // bit i: pair p0 + i is turned
  float c[NP], s[NP];
  Vec<T, E, W> a[U], b[INTER ? 1 : U];

  static __host__ __device__ __forceinline__ int count(int D, int pairs) {
    return INTER ? D / E : pairs / E + (D - 2 * pairs) / E;
  }
  __device__ __forceinline__ void place(int col, int pairs) {
    on = 0;
    c1 = -1;
    if (INTER) {
      c0 = col * E;
      p0 = col * NP;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (p0 + i < pairs) on |= 1u << i;
    } else {
      const int rot = pairs / E;
      p0 = col * E;
      c0 = col < rot ? col * E : 2 * pairs + (col - rot) * E;
      if (col < rot) {
        c1 = c0 + pairs;
        on = (1u << NP) - 1u;
      }
    }
  }
  // `n` heads (at most U) of a token
  __device__ __forceinline__ void fetch(const T* x, long long xh, int n) {
    x += c0;
#pragma unroll
    for (int u = 0; u < U; ++u, x += xh)
      if (u < n) {
        a[u].load(x);
        if (!INTER && c1 >= 0) b[INTER ? 0 : u].load(x + (c1 - c0));
      }
  }
  // the angles at the position whose coordinates start at value i0 of pos
  __device__ __forceinline__ void angles(const uint64_t* turn, const uint8_t* axis, float sign, const void* pos,
                                         int pos64, long long i0) {
    if (!on) return;
    uint64_t p = 0;
    int ax = -1;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (!((on >> i) & 1)) continue;
      const int x = axis[p0 + i];
      if (x != ax) p = pos64 ? (uint64_t)((const long long*)pos)[i0 + x] : (uint64_t)(long long)((const int*)pos)[i0 + x];
      ax = x;
      // the product's signed top word, -2^31 .. 2^31, is -1/2 .. 1/2 turns: -1 .. 1 half turns
      sincospif((float)(int)((p * turn[p0 + i]) >> 32) * 0x1p-31f, &s[i], &c[i]);
      s[i] *= sign;
    }
  }
  __device__ __forceinline__ void put(T* out, long long oh, int n) {
    out += c0;
    const bool all = on == (1u << NP) - 1u;
#pragma unroll
    for (int u = 0; u < U; ++u, out += oh)
      if (u < n) {
        if (INTER) {
          if (all) turn_pairs(a[u], c, s, ~0u);
          else if (on) turn_pairs(a[u], c, s, on);
        } else if (on) {
          turn_halves(a[u], b[INTER ? 0 : u], c, s);
        }
        a[u].store(out);
        if (!INTER && c1 >= 0) b[INTER ? 0 : u].store(out + (c1 - c0));
      }
  }
};

// The plan's frequencies and axes in shared memory: lanes that ask the kernel's
// parameters for different ones are served one after the other.
struct Table {
  uint64_t turn[kMaxRotaryPairs];
  uint8_t axis[kMaxRotaryPairs];
  __device__ __forceinline__ void fill(const RotaryPlan& plan) {
    for (int j = threadIdx.x; j < plan.pairs; j += blockDim.x) {
      turn[j] = plan.turn[j];
      axis[j] = plan.axis[j];
    }
    __syncthreads();
  }
};

template <typename T, int E, int W, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads, 3)
    rotary_kernel(const __grid_constant__ RotaryArgs a, const Cover cv) {
  __shared__ Table table;
  table.fill(a.plan);
  const int tl = threadIdx.x / cv.cols, h0 = blockIdx.y * cv.hpt, n = min(a.H - h0, cv.hpt);
  Column<T, E, W, INTER> cl;
  cl.place(threadIdx.x - tl * cv.cols, a.plan.pairs);
  const float sign = a.plan.inverse ? -1.f : 1.f;
  const T* x = (const T*)a.x + h0 * a.xh;
  T* out = (T*)a.out + h0 * a.oh;
  const uint32_t S = a.S, rows = (uint32_t)a.B * S;
  uint32_t row = blockIdx.x * (uint32_t)(cv.tpb * cv.per) + tl;
  for (int k = 0; k < cv.per && row < rows; ++k, row += cv.tpb) {
    const uint32_t b = a.B == 1 ? 0 : row / S;
    const long long t = row - b * S;
    cl.fetch(x + b * a.xb + t * a.xs, a.xh, n);
    cl.angles(table.turn, table.axis, sign, a.pos, a.pos64, b * a.pos_b + t * a.plan.axes);
    cl.put(out + b * a.ob + t * a.os, a.oh, n);
  }
}

// The sequence that owns row t, and its first row and number of rows; false if
// none does (behind the last sequence, or a range that is none).
__device__ __forceinline__ bool owner(const AppendArgs& a, int t, int* b, int* r0, int* n) {
  *b = *r0 = t;
  *n = 1;
  if (!a.b.cu) return t < a.b.B;
  int lo = 0, hi = a.b.B;  // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.b.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  *b = lo;
  if (!kv_rows(a.b.cu, a.b.T, lo, r0, n)) {
    if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadLength);
    return false;
  }
  return t >= *r0 && t < *r0 + *n;
}

// Rows of q (turned), k (turned) and v (as they are): blockIdx.y runs over groups
// of hpt heads of q, then of k, then of v.  A token whose slot does not exist (a
// bad page, a position outside the table) leaves the cache as it is and says
// so in the status word; its q is turned all the same when a sequence owns it.
template <typename T, int E, int W, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads, 3)
    kv_append_kernel(const __grid_constant__ AppendArgs a, const Cover cv, const int nq, const int nk) {
  __shared__ Table table;
  table.fill(a.plan);
  const int y = blockIdx.y, kind = y < nq ? 0 : y < nq + nk ? 1 : 2;  // q, k, v
  const int tl = threadIdx.x / cv.cols;
  const int h0 = (kind == 0 ? y : kind == 1 ? y - nq : y - nq - nk) * cv.hpt;
  const int n = min((kind == 0 ? a.q_heads : a.c.heads) - h0, cv.hpt);
  const long long xt = kind == 0 ? a.q_t : kind == 1 ? a.k_t : a.v_t, xh = kind == 0 ? a.q_h : kind == 1 ? a.k_h : a.v_h;
  const long long oh = kind == 0 ? a.qo_h : kind == 1 ? a.c.k_head : a.c.v_head;
  const T* x = (const T*)(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + h0 * xh;
  T* out = (T*)(kind == 0 ? a.qo : kind == 1 ? a.c.k : a.c.v) + h0 * oh;
  Column<T, E, W, INTER> cl;
  cl.place(threadIdx.x - tl * cv.cols, a.plan.pairs);
  if (kind == 2) cl.on = 0;
  uint32_t row = blockIdx.x * (uint32_t)(cv.tpb * cv.per) + tl;
  for (int k = 0; k < cv.per && row < (uint32_t)a.b.T; ++k, row += cv.tpb) {
    const int t = (int)row;
    cl.fetch(x + t * xt, xh, n);
    cl.angles(table.turn, table.axis, 1.f, a.pos, a.pos64, (long long)t * a.plan.axes);
    int b, r0, m, len;
    if (!owner(a, t, &b, &r0, &m)) continue;
    long long to;
    if (kind == 0) {
      to = t * a.qo_t;
    } else {
      const long long i = (long long)a.b.lengths[b] - m + (t - r0);
      if (!kv_length(a.b.lengths[b], a.b.max_pages, a.c.page_size, &len) || i < 0) {
        if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadLength);
        continue;
      }
      const int p = kv_page(a.b.pages + b * a.b.page_stride, (int)i, a.c.page_size, a.c.pages);
      if (p < 0) {
        if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadPage);
        continue;
      }
      const int r = (int)i % a.c.page_size;
      to = kind == 1 ? p * a.c.k_page + r * a.c.k_row : p * a.c.v_page + r * a.c.v_row;
    }
    cl.put(out + to, oh, n);
  }
}

// Heads per thread: up to `most`, fewer where that leaves less than two blocks
// of threads per SM.  Tokens per thread: 4 where that leaves two waves of three
// blocks per SM (the table is then filled for four times the work), else 1.
Cover cover(long long rows, int cols, int heads, int most) {
  Cover c;
  c.cols = cols;
  c.tpb = kRotaryThreads / cols;
  c.hpt = most;
  while (c.hpt > 1 && rows * cols * ((heads + c.hpt - 1) / c.hpt) < 2 * kSms * kRotaryThreads) c.hpt /= 2;
  const long long threads = rows * cols * ((heads + c.hpt - 1) / c.hpt);
  c.per = threads >= kSms * 3 * 2 * 4 * kRotaryThreads ? 4 : 1;
  return c;
}
unsigned blocks(long long rows, const Cover& c) {
  const long long n = (long long)c.tpb * c.per;
  return (unsigned)((rows + n - 1) / n);
}

template <typename T, int E, int W, bool INTER>
cudaError_t go_rotary(const RotaryArgs& a, cudaStream_t s) {
  using Col = Column<T, E, W, INTER>;
  const long long rows = (long long)a.B * a.S;
  const Cover c = cover(rows, Col::count(a.D, a.plan.pairs), a.H, Col::U);
  rotary_kernel<T, E, W, INTER><<<dim3(blocks(rows, c), (a.H + c.hpt - 1) / c.hpt), c.tpb * c.cols, 0, s>>>(a, c);
  return cudaGetLastError();
}

template <typename T, int E, int W, bool INTER>
cudaError_t go_append(const AppendArgs& a, cudaStream_t s) {
  using Col = Column<T, E, W, INTER>;
  const Cover c = cover(a.b.T, Col::count(a.c.D, a.plan.pairs), 2 * a.c.heads + a.q_heads, Col::U);
  const int nq = (a.q_heads + c.hpt - 1) / c.hpt, nk = (a.c.heads + c.hpt - 1) / c.hpt;
  kv_append_kernel<T, E, W, INTER><<<dim3(blocks(a.b.T, c), nq + 2 * nk), c.tpb * c.cols, 0, s>>>(a, c, nq, nk);
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
