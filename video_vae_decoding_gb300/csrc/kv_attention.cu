// Attention of a few new tokens over a paged key-value cache, split over the
// cache's length and joined.
//
// Row r of a sequence and key head h (row r: token r / group, query head
// h * group + r % group): o = sum_j p_j v_j / sum_j p_j, p_j = 2^(s_j - m),
// s_j = scale log2(e) q . k_j over the keys the row sees, m their maximum.
//
// Bound: memory.  Every key and value is read once for up to 16 rows, 4 D
// bytes against 4 D operations a row, far below the tensor cores' rate; so
// mma.sync on fragments fetched by ldmatrix is enough, and what matters is
// that loads never wait for arithmetic:
//  - a warp owns 16 keys of each tile and a ring of its own (cp.async, kStages
//    deep), so warps never wait for one another inside a run;
//  - the whole call's tiles (sequence x row tile x head x key tile) are one
//    line that is cut into equal pieces, one per resident block, on the device
//    from the lengths themselves: any raggedness gives every SM the same
//    bytes, a captured graph follows its lengths, and one long sequence is
//    spread over the whole card;
//  - a row tile that a cut divides leaves partial (m, l, o) in the workspace,
//    and a second kernel, launched to start as the first drains, joins them in
//    the order of the keys: the result does not depend on timing.
// Sums, maxima and outputs are held in 32 bits; how the weights are rounded is
// told at Weights.
#include "kv_common.cuh"

namespace wan {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;            // rows of a tile: the MMA's M
constexpr int kWarpKeys = 16;        // keys per warp and tile
constexpr int kKeys = kWarps * kWarpKeys;

template <int DP>
struct Cfg {
  static constexpr int CH = DP / 8;                     // 16-byte chunks per row
  static constexpr int kStages = DP == 64 ? 6 : 3;
  static constexpr int kCtas = DP == 256 ? 1 : 2;       // resident blocks per SM
  static constexpr int kHalf = kWarpKeys * DP * 2;      // bytes of K (or V) per warp and stage
  static constexpr int kRing = kStages * 2 * kHalf;     // bytes per warp
  static constexpr int kSmem = kWarps * kRing + kRows * DP * 2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// How the weights p >= 0 of a pair of keys enter the product with v.
//  bfloat16: as hi + lo, hi the upper half of p's bits (so lo >= 0) and lo at
//  least p 2^-24: the result carries only its own rounding, and both products
//  with an infinite v have its sign, as p v has.
//  float16: rounded once, with all weights 2^kBias times larger, so that keys
//  down to 2^-36 of the largest weight still count; kBias leaves the largest
//  below 65504.
template <typename T>
struct Weights;
template <>
struct Weights<__nv_bfloat16> {
  static constexpr bool kTwo = true;
  static constexpr float kBias = 0.f;
  static __device__ __forceinline__ uint32_t hi(float x, float y) {
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  }
  static __device__ __forceinline__ uint32_t lo(float x, float y) {
    const float hx = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float hy = __uint_as_float(__float_as_uint(y) & 0xFFFF0000u);
    return pack_bf16x2(fmaxf(x - hx, x * 0x1p-24f), fmaxf(y - hy, y * 0x1p-24f));
  }
};
template <>
struct Weights<__half> {
  static constexpr bool kTwo = false;
  static constexpr float kBias = 12.f;
  static __device__ __forceinline__ uint32_t hi(float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint32_t lo(float, float) { return 0; }
};
// ------------------------------------------------------------ the line of tiles
// Tiles of a sequence on the line: row tiles x heads x key tiles.
struct Tiles {
  int key_tiles;
  long long all;
};
__device__ __forceinline__ Tiles tiles_of(const AttnArgs& a, const Seq& s) {
  Tiles t;
  t.key_tiles = (s.len + kKeys - 1) / kKeys;
  t.all = ((long long)s.n * a.group + kRows - 1) / kRows * a.c.heads * t.key_tiles;
  return t;
}

struct Space {  // the workspace: per block an Open and two parts (0: a row tile's later keys, 1: its first ones)
  Open* open;
  float2* ml;  // [2 G][kRows]: running max (log2 units) and sum
  float* o;    // [2 G][kRows][DP]
};
template <int DP>
__host__ __device__ inline Space space(void* w, int G) {
  Space s;
  s.open = (Open*)w;
  s.ml = (float2*)((char*)w + (size_t)G * sizeof(Open));
  s.o = (float*)((char*)s.ml + (size_t)2 * G * kRows * sizeof(float2));
  return s;
}
long long space_bytes(int DP, int G) {
  return (long long)G * (sizeof(Open) + 2 * kRows * (sizeof(float2) + (size_t)DP * sizeof(float)));
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, Cfg<DP>::kCtas)
    kv_split_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<DP>;
  constexpr int CH = C::CH, ST = C::kStages, NK = DP / 16;
  constexpr bool kQRegs = DP <= 128;  // q fragments in registers; at 256 channels they are fetched again
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_seen[kWarps][ST];
  __shared__ long long s_line[kWarps + 2];
  __shared__ float2 s_ml[kWarps][kRows];
  __shared__ float s_p[kWarps][kRows][kWarpKeys];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x, me = blockIdx.x;
  uint8_t* ring = smem + warp * C::kRing;
  uint8_t* sq = smem + kWarps * C::kRing;
  const uint32_t ring_a = smem_u32(ring), sq_a = smem_u32(sq);
  const Space ws = space<DP>(a.workspace, G);

  // the join's blocks may start as soon as every block of this grid runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  put_empty<T>(a, me, G);

  // --------------------------------------------- this block's piece of the line
  const Piece pc =
      cut_line<kWarps>(a.b.B, me, G, 1, s_line, [&](int b) { return tiles_of(a, sequence(a, b, false)).all; });
  if (threadIdx.x == 0) ws.open[me] = Open{0, 0, 0, 0};
  int b = pc.b;
  long long at = pc.at;
  const T* kbase = (const T*)a.c.k;
  const T* vbase = (const T*)a.c.v;

  for (long long line = pc.beg; line < pc.end;) {
    Seq s = sequence(a, b, false);
    Tiles tl = tiles_of(a, s);
    while (at >= tl.all) {  // the next sequence with a tile
      at -= tl.all;
      s = sequence(a, ++b, false);
      tl = tiles_of(a, s);
    }
    // the run: key tiles [kt0, kt1) of one row tile and head
    const int seg = (int)(at / tl.key_tiles), kt0 = (int)(at - (long long)seg * tl.key_tiles);
    const int kt1 = (int)min((long long)tl.key_tiles, kt0 + (pc.end - line));
    // heads of a row tile side by side, row tiles behind them
    const int rt = seg / a.c.heads, h = seg - rt * a.c.heads;
    const int row0 = rt * kRows, cnt = min(kRows, s.n * a.group - row0);

    // q into shared memory, 16-byte chunk c of row r at chunk c ^ (r & 7); zeros past the rows and channels
    for (int i = threadIdx.x; i < kRows * CH; i += kThreads) {
      const int r = i / CH, c = i - r * CH;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < cnt && c * 8 < a.c.D) {
        const int t = (row0 + r) / a.group, g = row0 + r - t * a.group;
        const T* src = (const T*)a.q + (long long)(s.r0 + t) * a.q_t + (long long)(h * a.group + g) * a.q_h + c * 8;
        if (((uintptr_t)src & 15) == 0) {
          v = *reinterpret_cast<const uint4*>(src);
        } else {
          uint32_t w[4];
          const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = (uint32_t)e[2 * j] | ((uint32_t)e[2 * j + 1] << 16);
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      *reinterpret_cast<uint4*>(sq + r * DP * 2 + ((c ^ (r & 7)) << 4)) = v;
    }
    // the keys that this thread's two rows see, and those that any row does
    const int r_a = lane >> 2, r_b = r_a + 8;
    int lo_a = 0, hi_a = 0, lo_b = 0, hi_b = 0;
    int lo = 0x7fffffff, hi = 0;
    for (int r = 0; r < cnt; ++r) {
      int f, e;
      seen_range(a, s.r0 + (row0 + r) / a.group, s.len, &f, &e);
      if (r == r_a) lo_a = f, hi_a = e;
      if (r == r_b) lo_b = f, hi_b = e;
      if (f < e) {
        lo = min(lo, f);
        hi = max(hi, e);
      }
      if (!a.ranges) {  // all rows alike
        if (r_a < cnt) lo_a = f, hi_a = e;
        if (r_b < cnt) lo_b = f, hi_b = e;
        break;
      }
    }
    // rows of one token, or of tokens that see the same keys, need no mask of their own
    const bool differ = (r_a < cnt && (lo_a != lo || hi_a != hi)) || (r_b < cnt && (lo_b != lo || hi_b != hi));
    const bool mixed = __any_sync(0xffffffffu, differ);
    __syncthreads();

    uint32_t qf[kQRegs ? NK : 1][4];
    const uint32_t q_row = sq_a + (lane & 15) * DP * 2;
    if (kQRegs) {
#pragma unroll
      for (int k = 0; k < NK; ++k) ldsm4(q_row + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4), qf[kQRegs ? k : 0]);
    }

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;

    const int* table = a.b.pages + b * a.b.page_stride;
    const int w0 = max(kt0, lo == 0x7fffffff ? kt1 : lo / kKeys), w1 = min(kt1, (hi + kKeys - 1) / kKeys);

    auto issue = [&](int kt) {
      const int st = kt % ST;
      const int key0 = kt * kKeys + warp * kWarpKeys;
      const uint32_t dk = ring_a + st * 2 * C::kHalf, dv = dk + C::kHalf;
      uint32_t seen = 0;
      // rows that hold a key some row sees
      const int key = key0 + (lane & 15);
      bool take = key >= lo && key < hi;
      long long ko = 0, vo = 0;
      if (take) {
        const int pi = key / a.c.page_size, off = key - pi * a.c.page_size;
        const int p = table[pi];
        if (p >= 0 && p < a.c.pages) {
          ko = p * a.c.k_page + h * a.c.k_head + off * a.c.k_row;
          vo = p * a.c.v_page + h * a.c.v_head + off * a.c.v_row;
        } else {
          take = false;
          if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadPage);
        }
      }
      seen = __ballot_sync(0xffffffffu, take) & 0xffffu;
      if (lane == 0) s_seen[warp][st] = seen;
      constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;  // rows per instruction
#pragma unroll
      for (int i = 0; i < kWarpKeys / RPI; ++i) {
        const int r = i * RPI + lane / CH, c = lane % CH;
        const long long kr = __shfl_sync(0xffffffffu, ko, r), vr = __shfl_sync(0xffffffffu, vo, r);
        const bool ok = ((seen >> r) & 1) && c * 8 < a.c.D;
        const uint32_t d = r * DP * 2 + ((c ^ (r & 7)) << 4);
        cp_async16(dk + d, kbase + (ok ? kr + c * 8 : 0), ok);
        cp_async16(dv + d, vbase + (ok ? vr + c * 8 : 0), ok);
      }
    };

#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      if (w0 + i < w1) issue(w0 + i);
      cp_commit();
    }
    for (int kt = w0; kt < w1; ++kt) {
      cp_wait<ST - 2>();
      __syncwarp();
      const int st = kt % ST;
      const uint32_t sk = ring_a + st * 2 * C::kHalf, sv = sk + C::kHalf;
      const uint32_t seen = s_seen[warp][st];
      if (seen) {
        const int key0 = kt * kKeys + warp * kWarpKeys;
        float sc[2][4] = {};
        const int kr = ((lane >> 4) << 3) + (lane & 7);
        const uint32_t krow = sk + kr * DP * 2;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          uint32_t bk[4];
          ldsm4(krow + (((2 * k + ((lane >> 3) & 1)) ^ (lane & 7)) << 4), bk);
          if (kQRegs) {
            mma16816<T>(sc[0], qf[kQRegs ? k : 0], bk[0], bk[1]);
            mma16816<T>(sc[1], qf[kQRegs ? k : 0], bk[2], bk[3]);
          } else {
            uint32_t qk[4];
            ldsm4(q_row + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4), qk);
            mma16816<T>(sc[0], qk, bk[0], bk[1]);
            mma16816<T>(sc[1], qk, bk[2], bk[3]);
          }
        }
        // mask: hidden keys to -inf
        bool part = seen != 0xffffu;  // some key hidden from every row
        if (mixed) part = part || __any_sync(0xffffffffu, (r_a < cnt && (key0 < lo_a || key0 + kWarpKeys > hi_a)) ||
                                                              (r_b < cnt && (key0 < lo_b || key0 + kWarpKeys > hi_b)));
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[n][i] *= a.scale_log2;
            if (part) {
              const int kk = n * 8 + (lane & 3) * 2 + (i & 1), key = key0 + kk;
              const int f = i < 2 ? lo_a : lo_b, e = i < 2 ? hi_a : hi_b;
              if (!((seen >> kk) & 1) || key < f || key >= e) sc[n][i] = -INFINITY;
            }
          }
        float x_a = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
        float x_b = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          x_a = fmaxf(x_a, __shfl_xor_sync(0xffffffffu, x_a, d));
          x_b = fmaxf(x_b, __shfl_xor_sync(0xffffffffu, x_b, d));
        }
        if (__any_sync(0xffffffffu, x_a > m_a || x_b > m_b)) {
          const float n_a = fmaxf(m_a, x_a), n_b = fmaxf(m_b, x_b);
          const float c_a = weight(m_a, n_a), c_b = weight(m_b, n_b);
          m_a = n_a;
          m_b = n_b;
          l_a *= c_a;
          l_b *= c_b;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            o[i][0] *= c_a;
            o[i][1] *= c_a;
            o[i][2] *= c_b;
            o[i][3] *= c_b;
          }
        }
        float p[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[n][i] = weight(sc[n][i], (i < 2 ? m_a : m_b) - Weights<T>::kBias);
        l_a += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
        l_b += (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]);
        uint32_t hi4[4], lo4[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            hi4[2 * n + j] = Weights<T>::hi(p[n][2 * j], p[n][2 * j + 1]);
            lo4[2 * n + j] = Weights<T>::lo(p[n][2 * j], p[n][2 * j + 1]);
          }
        // A value that some rows see and others do not must not reach the
        // others: 0 times an infinity or a NaN is a NaN.  Such values are
        // taken out of the tile and added to the rows that see them.
        bool odd = false;
        if (mixed && part) {
          for (int i = lane; i < kWarpKeys * CH; i += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(ring + (sv - ring_a) + i * 16);
            odd |= odd32<T>(v.x) || odd32<T>(v.y) || odd32<T>(v.z) || odd32<T>(v.w);
          }
          odd = __any_sync(0xffffffffu, odd);
          if (odd) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s_p[warp][(i < 2 ? r_a : r_b)][n * 8 + (lane & 3) * 2 + (i & 1)] = sc[n][i] == -INFINITY ? -1.f : p[n][i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int c = i * 8 + (lane & 3) * 2 + (j & 1);
                for (int k = 0; k < kWarpKeys; ++k) {
                  const float w = s_p[warp][j < 2 ? r_a : r_b][k];
                  const uint8_t* e = ring + (sv - ring_a) + k * DP * 2 + ((((c >> 3) ^ (k & 7)) << 4) | ((c & 7) * 2));
                  const T v = *reinterpret_cast<const T*>(e);
                  if (w >= 0.f && odd16<T>(*reinterpret_cast<const uint16_t*>(e))) o[i][j] += w * val<T>(v);
                }
              }
            __syncwarp();
            for (int i = lane; i < kWarpKeys * DP; i += 32) {
              uint16_t* e = reinterpret_cast<uint16_t*>(ring + (sv - ring_a)) + i;
              if (odd16<T>(*e)) *e = 0;
            }
            __syncwarp();
          }
        }
        const uint32_t vrow = sv + (lane & 15) * DP * 2;
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
          uint32_t bv[4];
          ldsm4t(vrow + (((2 * n + (lane >> 4)) ^ (lane & 7)) << 4), bv);
          mma16816<T>(o[2 * n], hi4, bv[0], bv[1]);
          mma16816<T>(o[2 * n + 1], hi4, bv[2], bv[3]);
          if (Weights<T>::kTwo) {
            mma16816<T>(o[2 * n], lo4, bv[0], bv[1]);
            mma16816<T>(o[2 * n + 1], lo4, bv[2], bv[3]);
          }
        }
      }
      __syncwarp();
      if (kt + ST - 1 < w1) issue(kt + ST - 1);
      cp_commit();
    }
    cp_wait<0>();

    // --------------------------------------------- the warps' parts into one
    if (Weights<T>::kBias != 0.f) {
      const float f = exp2f(-Weights<T>::kBias);
      l_a *= f;
      l_b *= f;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= f;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l_a += __shfl_xor_sync(0xffffffffu, l_a, d);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, d);
    }
    if ((lane & 3) == 0) {
      s_ml[warp][r_a] = make_float2(m_a, l_a);
      s_ml[warp][r_b] = make_float2(m_b, l_b);
    }
    __syncwarp();
    float* so = reinterpret_cast<float*>(ring);  // [kRows][DP], in the warp's own ring
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) {
      const int c = i * 8 + (lane & 3) * 2;
      if (r_a < cnt) *reinterpret_cast<float2*>(so + r_a * DP + c) = make_float2(o[i][0], o[i][1]);
      if (r_b < cnt) *reinterpret_cast<float2*>(so + r_b * DP + c) = make_float2(o[i][2], o[i][3]);
    }
    __syncthreads();
    const bool whole = kt0 == 0 && kt1 == tl.key_tiles;
    const int slot = 2 * me + (kt0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < cnt * DP; i += kThreads) {
      const int r = i / DP, c = i - r * DP;
      float m = -INFINITY, l = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w][r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = weight(s_ml[w][r].x, m);
        l += f * s_ml[w][r].y;
        v += f * reinterpret_cast<const float*>(smem + w * C::kRing)[r * DP + c];
      }
      if (whole) {
        if (c < a.c.D) out_row<T>(a, s, h, row0 + r)[c] = round_to<T>(l == 0.f ? 0.f : v / l);
        if (c == 0) put_lse(a, s, h, row0 + r, m, l);
      } else {
        ws.o[((long long)slot * kRows + r) * DP + c] = v;
        if (c == 0) ws.ml[slot * kRows + r] = make_float2(m, l);
      }
    }
    if (!whole && kt0 == 0 && threadIdx.x == 0) {
      const long long last = line + tl.key_tiles - 1;  // the row tile's last tile: its block is the last part's
      ws.open[me] = Open{b, rt, h, pc.holder(last) - me};
    }
    __syncthreads();
    at += kt1 - kt0;
    line += kt1 - kt0;
  }
}

// Joins the parts of the row tile that block `blockIdx.x` of the split kernel
// left open, in the order of the keys.
template <typename T, int DP>
__global__ void __launch_bounds__(DP) kv_join_kernel(const __grid_constant__ AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int me = blockIdx.x;
  const Space ws = space<DP>(a.workspace, gridDim.x);
  const Open op = ws.open[me];
  if (op.parts == 0) return;
  const Seq s = sequence(a, op.b, false);
  const int row0 = op.rt * kRows, cnt = min(kRows, s.n * a.group - row0);
  const int c = threadIdx.x;
  for (int r = blockIdx.y; r < cnt; r += gridDim.y) {
    float m = -INFINITY, l = 0.f, v = 0.f;
    for (int i = 0; i <= op.parts; ++i) {
      const long long slot = 2LL * (me + i) + (i == 0 ? 1 : 0);
      const float2 ml = ws.ml[slot * kRows + r];
      const float x = ws.o[(slot * kRows + r) * DP + c];
      const float n = fmaxf(m, ml.x);
      const float f = weight(m, n), g = weight(ml.x, n);
      l = l * f + ml.y * g;
      v = v * f + x * g;
      m = n;
    }
    if (c < a.c.D) out_row<T>(a, s, op.h, row0 + r)[c] = round_to<T>(l == 0.f ? 0.f : v / l);
    if (c == 0) put_lse(a, s, op.h, row0 + r, m, l);
  }
}

template <typename T, int DP>
cudaError_t go_split(const AttnArgs& a, int sms, cudaStream_t s) {
  using C = Cfg<DP>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem((const void*)kv_split_kernel<T, DP>, C::kSmem, &allowed);
  if (e != cudaSuccess) return e;
  const int G = sms * C::kCtas;
  kv_split_kernel<T, DP><<<G, kThreads, C::kSmem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G, min(kRows, 4));
  cfg.blockDim = dim3(DP);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<T, DP>, a);
}

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

template <typename T>
cudaError_t by_dim(const AttnArgs& a, int sms, cudaStream_t s) {
  switch (padded(a.c.D)) {
    case 64: return go_split<T, 64>(a, sms, s);
    case 128: return go_split<T, 128>(a, sms, s);
    default: return go_split<T, 256>(a, sms, s);
  }
}

}  // namespace

long long kv_attention_workspace(const AttnArgs& a, int sms) {
  const int DP = padded(a.c.D);
  return space_bytes(DP, sms * (DP == 256 ? Cfg<256>::kCtas : Cfg<128>::kCtas));
}

cudaError_t launch_kv_attention(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.c.elem == 1 ? by_dim<__nv_bfloat16>(a, sms, s) : by_dim<__half>(a, sms, s);
}

}  // namespace wan
