// Attention of many new tokens over a paged key-value cache: a flash kernel on
// the fifth-generation tensor cores.
//
// For 256 rows (row r of a sequence and key head h: token r / group, query head
// h * group + r % group) in two halves of 128, per block of up to 128 keys j:
//   S_t = Q_t K_j^T          (t = 0, 1: the halves; M = 128, N = 128)
//   P_t = 2^(scale S_t - m)  two threads per row: running maximum m, moved only
//                            when a block exceeds it by 8 (O is then rescaled)
//   O_t += P_t V_j           P_t read from tensor memory, in the half of S_t's
//                            columns that its own thread has already read
// and O_t / l at the end.  While one half's softmax runs, the tensor cores work
// for the other.  TMEM: S_0, S_1 (128 columns each), O_0, O_1 (DP each).
//
// Bound: the tensor cores, 4 D operations per row and key; K and V come through
// one ring in the order of their use and serve both halves, so a block of 128
// keys asks 64 KB (D = 128) for 33.6 MFLOP.
// V is taken as it lies in the cache, [key][channel]: the MMA's second operand
// with its N dimension contiguous, so nothing is transposed on the way.
//
// Pages: a block is as many whole pages as fit 128 keys (each one TMA box of
// its rows, rounded up to 8), or a part of a longer page.  Rows past a page's
// end, a page that the cache does not have and pages past the sequence read as
// zeros (the TMA's fill).
//
// The line of (sequence, row tile, head, key block) is cut into equal pieces,
// one per SM, as in the split kernel; the join adds up what a cut divides.
#include "kv_common.cuh"
#include "kv_chunk.h"

namespace wan {

namespace {

// Warps 0 loads, 1 MMA, 2 TMEM, 3 idle; 4-11 softmax of half 0, 12-19 of half 1:
// two threads per row, which share a block's keys (64 each) and the output's
// channels.
constexpr int kThreads = 640;
constexpr int kHalfRows = 128;
constexpr int kTileRows = 256;
constexpr int kBlock = 128;      // key columns of a block
constexpr int kBoxBytes = 16384;  // 128 rows x 64 channels
constexpr float kSlack = 8.f;    // log2 units that the reference maximum may lag behind

template <int DP>
struct Cfg {
  static constexpr int ND = DP / 64;
  static constexpr int kSlot = ND * kBoxBytes;          // K or V of a block
  static constexpr int kStages = DP == 128 ? 5 : 10;
  static constexpr int kQ = 2 * ND * kBoxBytes;
  static constexpr int kSmem = kQ + kStages * kSlot + 512 + 2048;
};

// Weights 2^(x - m) reach 2^kSlack; in float16 they are taken 2^7 times larger
// (65504 is the end), so that keys down to 2^-31 of the largest still count.
template <typename T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
  static constexpr float kBias = 0.f;
  static constexpr uint32_t kFormat = 1;
  static __device__ __forceinline__ uint32_t two(float x, float y) { return pack_bf16x2(x, y); }
};
template <>
struct Pack<__half> {
  static constexpr float kBias = 7.f;
  static constexpr uint32_t kFormat = 0;
  static __device__ __forceinline__ uint32_t two(float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// kind::f16, fp32 accumulator, operand format 1 (bf16) or 0 (fp16); b_mn: the
// second operand's N dimension is the contiguous one.
__device__ __forceinline__ constexpr uint32_t idesc(uint32_t format, bool b_mn, int N) {
  return (1u << 4) | (format << 7) | (format << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
// Shared-memory operand descriptors (ptx.cuh: sdesc_k128): the low word holds
// the address and the leading byte offset, the high word never changes.
//  first operand and K: K contiguous, leading offset unused (1)
//  V: N contiguous in the 128-byte swizzle: atoms of 64 channels x 8 keys (1024 B)
//     stacked by 8 keys (stride byte offset), the next 64 channels a box further
//     on (leading byte offset)
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_v(uint32_t saddr) { return (saddr >> 4) | ((uint32_t)(kBoxBytes >> 4) << 16); }
// One thread of the calling warp.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// D[tmem] (+)= A[smem] B[smem]^T
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(id), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t id,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(id), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}

// Two 32-bit products and sums, or sums, in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The two warps whose threads share their rows (named barriers 1-8).
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
// The same, and whether v holds for any of their 64 threads.
__device__ __forceinline__ bool pair_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------- pages and blocks
__device__ __forceinline__ int blocks_of(const ChunkGeo& g, int page_size, int len) {
  if (g.parts == 1) return ((len + page_size - 1) / page_size + g.pages - 1) / g.pages;
  return len / page_size * g.parts + (len % page_size + kBlock - 1) / kBlock;
}
__device__ __forceinline__ int block_of_key(const ChunkGeo& g, int page_size, int key) {
  if (g.parts == 1) return key / page_size / g.pages;
  return key / page_size * g.parts + key % page_size / kBlock;
}
// first key of block j, and the rows that its pages give it
__device__ __forceinline__ void block_keys(const ChunkGeo& g, int page_size, int j, int* base, int* rows) {
  if (g.parts == 1) {
    *base = j * g.pages * page_size;
    *rows = g.pages * page_size;
  } else {
    const int p = j / g.parts, off = (j - p * g.parts) * kBlock;
    *base = p * page_size + off;
    *rows = min(kBlock, page_size - off);
  }
}

struct Tiles {
  int blocks;
  long long all;
};
__device__ __forceinline__ Tiles tiles_of(const AttnArgs& a, const ChunkGeo& g, const Seq& s) {
  Tiles t;
  t.blocks = blocks_of(g, a.c.page_size, s.len);
  t.all = ((long long)s.n * a.group + kTileRows - 1) / kTileRows * a.c.heads * t.blocks;
  return t;
}

struct Space {
  Open* open;
  float2* ml;  // [2 G][kTileRows]
  float4* o;   // [2 G][DP / 4][kTileRows]: the rows side by side
};
template <int DP>
__host__ __device__ inline Space space(void* w, int G) {
  Space s;
  s.open = (Open*)w;
  s.ml = (float2*)((char*)w + (size_t)G * sizeof(Open));
  s.o = (float4*)((char*)s.ml + (size_t)2 * G * kTileRows * sizeof(float2));
  return s;
}

// A run: blocks [j0, j1) of one row tile and head, [k0, k1) of the line's.
struct Run {
  Seq s;
  int b, rt, h, row0, cnt;
  int k0, k1, blocks;
  int lo, hi;          // keys that some row sees
  int all_lo[2], all_hi[2];  // per half: keys that every row sees
  int odd_lo, odd_hi;  // blocks whose values were cleaned (below)
  int stop;
};

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    kv_chunk_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                    const __grid_constant__ AttnArgs a, const __grid_constant__ ChunkGeo geo) {
  using C = Cfg<DP>;
  constexpr int S = C::kStages, ND = C::ND;
  // the only shared memory of the kernel, so it starts on a 1024-byte boundary, as the swizzled boxes must
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(sizeof(Run) + 8 * (2 * S + 9) + 80 <= 512, "barriers and the run's description");
  uint8_t* sQ = smem;  // [half][64-channel box][128 rows]
  uint8_t* sR = sQ + C::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(sR + S * C::kSlot);
  uint64_t* empty = full + S;
  uint64_t* s_full = empty + S;   // [2] S_t in TMEM
  uint64_t* p_full = s_full + 2;  // [2] 256 arrivals: P_t in TMEM (S_t read, O_t rescaled)
  uint64_t* o_done = p_full + 2;  // [2] O_t += P_t V_j complete
  uint64_t* done = o_done + 2;
  if (smem_u32(smem) & 1023) {
    if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevTimeoutFull);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* hole = tmem_slot + 2;  // [16]: bit i of hole[j % 16]: page i of block j is none of the cache's
  Run* run = reinterpret_cast<Run*>(hole + 16);
  // [2 halves][2 key halves][128 rows]: what the two threads of a row tell each other.  One buffer: a block's values
  // are read before the block's P is complete, and the next block's come after.
  float* red = reinterpret_cast<float*>(run + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = gridDim.x, me = blockIdx.x;
  const Space ws = space<DP>(a.workspace, G);
  const int page_size = a.c.page_size;
  int* const err = a.b.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_full[t]), 256);
      mbar_init(smem_u32(&o_done[t]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *stop = 0;
    fence_mbar_init();
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
  }
  // rows of a slot that no box fills stay zero: their weights are zero, and 0 times a stray NaN would not be
  for (int i = threadIdx.x; i < S * C::kSlot / 16; i += kThreads)
    reinterpret_cast<uint4*>(sR)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  put_empty<T>(a, me, G);
  const Piece pc =
      cut_line<kThreads / 32>(a.b.B, me, G, reinterpret_cast<long long*>(red), [&](int b) { return tiles_of(a, geo, sequence(a, b, false)).all; });
  if (threadIdx.x == 0) ws.open[me] = Open{0, 0, 0, 0};
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 256;  // half t: S at tS + 128 t, P in its upper 64 columns, O at tO + DP t

  int b = pc.b;
  long long at = pc.at;
  int it = 0;                 // ring slots used so far (all roles count alike)
  int ns[2] = {0, 0};         // blocks of each half so far

  for (long long line = pc.beg; line < pc.end;) {
    // ------------------------------------------------------------- the next run
    if (threadIdx.x == 0) {
      Seq s = sequence(a, b, false);
      Tiles tl = tiles_of(a, geo, s);
      while (at >= tl.all) {
        at -= tl.all;
        s = sequence(a, ++b, false);
        tl = tiles_of(a, geo, s);
      }
      const int seg = (int)(at / tl.blocks);
      run->s = s;
      run->b = b;
      run->rt = seg / a.c.heads;
      run->h = seg - run->rt * a.c.heads;
      run->row0 = run->rt * kTileRows;
      run->cnt = min(kTileRows, s.n * a.group - run->row0);
      run->blocks = tl.blocks;
      run->k0 = (int)(at - (long long)seg * tl.blocks);
      run->k1 = (int)min((long long)tl.blocks, run->k0 + (pc.end - line));
      run->lo = 0x7fffffff;
      run->hi = 0;
      for (int t = 0; t < 2; ++t) {
        run->all_lo[t] = 0;
        run->all_hi[t] = 0x7fffffff;
      }
      run->odd_lo = 0x7fffffff;
      run->odd_hi = -1;
      at += run->k1 - run->k0;
    }
    __syncthreads();
    const int h = run->h, row0 = run->row0, cnt = run->cnt, k0 = run->k0, k1 = run->k1;
    const Seq s = run->s;
    const bool two = cnt > kHalfRows;
    // softmax threads: their row's keys, and its q
    const int half = (warp - 4) >> 3, hk = (warp - 4) >> 2 & 1;  // softmax warps: the half, and the half of its keys
    const int hrow = 32 * (warp & 3) + lane;                     // the row in its half: its TMEM lane
    const int row = half * kHalfRows + hrow;
    const bool mine = warp >= 4 && row < cnt;
    int lo = 0, hi = 0x40000000;  // rows past the tile's see everything: they need no mask
    if (mine) {
      seen_range(a, s.r0 + (row0 + row) / a.group, s.len, &lo, &hi);
      if (lo < hi) {
        atomicMin(&run->lo, lo);
        atomicMax(&run->hi, hi);
      }
      if (lo > 0) atomicMax(&run->all_lo[half], lo);
      atomicMin(&run->all_hi[half], hi);
    }
    if (warp >= 4 && (half == 0 || two)) {
      uint8_t* q = sQ + half * ND * kBoxBytes + hrow * 128;
      // q is negated for a negative scale (the maximum is then that of q . k) and cleared for a scale of zero
      // (whose product with a hidden key's -inf is none)
      const bool flip = a.scale_log2 < 0.f;
      const T* src = nullptr;
      if (mine) {
        const int t = (row0 + row) / a.group, g = row0 + row - t * a.group;
        src = (const T*)a.q + (long long)(s.r0 + t) * a.q_t + (long long)(h * a.group + g) * a.q_h;
      }
#pragma unroll 4
      for (int c = hk * (DP / 16); c < (hk + 1) * (DP / 16); ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (mine && c * 8 < a.c.D) {
          if (((uintptr_t)src & 15) == 0) {
            v = *reinterpret_cast<const uint4*>(src + c * 8);
          } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(src + c * 8);
            v = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                           e[6] | (uint32_t)e[7] << 16);
          }
          if (a.scale_log2 == 0.f) v = make_uint4(0, 0, 0, 0);
          if (flip) v = make_uint4(v.x ^ 0x80008000u, v.y ^ 0x80008000u, v.z ^ 0x80008000u, v.w ^ 0x80008000u);
        }
        *reinterpret_cast<uint4*>(q + (c >> 3) * kBoxBytes + (((c & 7) ^ (hrow & 7)) << 4)) = v;
      }
      fence_proxy_async_smem();
    }
    __syncthreads();
    const int j0 = run->hi > 0 ? max(k0, block_of_key(geo, page_size, run->lo)) : k1;
    const int j1 = run->hi > 0 ? min(k1, block_of_key(geo, page_size, run->hi - 1) + 1) : k1;
    const int nb = max(0, j1 - j0);
    bool ok = true;

    if (nb > 0) {
      if (warp == 0) {
        // ------------------------------------------------------------- loads
        const int* table = a.b.pages + run->b * a.b.page_stride;
        const int held = (s.len + page_size - 1) / page_size;  // pages of the sequence
        const int bytes = geo.parts == 1 ? geo.pages * geo.box_rows * 128 * ND : C::kSlot;
        int slot = it % S, lap = it / S;
        for (int j = j0; j < j1 && ok; ++j) {
          int idx, off = 0;
          if (geo.parts == 1) {
            idx = j * geo.pages + lane;
          } else {
            idx = j / geo.parts;
            off = (j - idx * geo.parts) * kBlock;
          }
          int page = (int)a.c.pages;  // past the sequence: past the cache, which reads as zeros
          bool none = false;
          if (lane < geo.pages && idx < held) {
            page = table[idx];
            none = page < 0 || page >= a.c.pages;
            if (none) {
              page = (int)a.c.pages;
              if (err) atomicCAS(err, 0, (int)kDevBadPage);
            }
          }
          const uint32_t nones = __ballot_sync(0xffffffffu, none);
          if (lane == 0) hole[j & 15] = nones;
          for (int kv = 0; kv < 2 && ok; ++kv) {
            int good = 1;
            if (lane == 0) {
              if (lap > 0) good = mbar_wait_bounded(smem_u32(&empty[slot]), (lap - 1) & 1, err, kDevTimeoutEmpty);
              if (*stop) good = 0;
              if (good) mbar_arrive_expect_tx(smem_u32(&full[slot]), bytes);
            }
            ok = __shfl_sync(0xffffffffu, good, 0);
            if (!ok) break;
            if (lane < geo.pages) {
              int c[3];
              c[geo.dim_row] = off;
              c[geo.dim_head] = h;
              c[geo.dim_page] = page;
              const uint32_t d = smem_u32(sR + slot * C::kSlot) + lane * geo.box_rows * 128;
#pragma unroll
              for (int u = 0; u < ND; ++u)
                tma_load_4d(d + u * kBoxBytes, kv ? &mapV : &mapK, smem_u32(&full[slot]), 64 * u, c[0], c[1], c[2]);
            }
            if (++slot == S) slot = 0, ++lap;
          }
        }
        if (!ok) *stop = 1;
      } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        // The whole warp walks the blocks (what it computes stays in uniform
        // registers, which the instructions take their operands from); one
        // thread issues.
        const uint32_t idS = idesc(Pack<T>::kFormat, false, kBlock);
        const int dn = (a.c.D + 15) / 16;  // k steps of S, N / 16 of O
        const uint32_t idO = idesc(Pack<T>::kFormat, true, 16 * dn);
        const int last = two ? 1 : 0;
        const bool one = elect();
        const uint32_t q0 = desc_k(smem_u32(sQ)), kd0 = desc_k(smem_u32(sR)), vd0 = desc_v(smem_u32(sR));
        int slot = it % S, phase = (it / S) & 1;
        auto next = [&] {
          if (++slot == S) slot = 0, phase ^= 1;
        };
        auto scores = [&](int t, int sl, bool done_with_slot) {
          const uint32_t q = q0 + t * (ND * kBoxBytes >> 4), k = kd0 + sl * (C::kSlot >> 4);
          if (one) {
#pragma unroll
            for (int u = 0; u < 4 * ND; ++u)
              if (u < dn)
                umma_ss(tS + kBlock * t, q + (u >> 2) * (kBoxBytes >> 4) + 2 * (u & 3),
                        k + (u >> 2) * (kBoxBytes >> 4) + 2 * (u & 3), idS, u > 0);
            umma_commit(smem_u32(&s_full[t]));
            if (done_with_slot) umma_commit(smem_u32(&empty[sl]));
          }
        };
        ok = mbar_wait_bounded(smem_u32(&full[slot]), phase, err, kDevTimeoutFull);
        tc_fence_after();
        for (int t = 0; t <= last && ok; ++t) scores(t, slot, t == last);
        next();
        for (int j = 0; j < nb && ok; ++j) {
          const int sv = slot, pv = phase;
          next();
          const bool more = j + 1 < nb;
          const int sk = slot, pk = phase;
          if (more) next();
          ok = mbar_wait_bounded(smem_u32(&full[sv]), pv, err, kDevTimeoutFull);
          if (more && ok) ok = mbar_wait_bounded(smem_u32(&full[sk]), pk, err, kDevTimeoutFull);
          for (int t = 0; t <= last && ok; ++t) {
            const uint32_t v = vd0 + sv * (C::kSlot >> 4);
            ok = mbar_wait_bounded(smem_u32(&p_full[t]), (ns[t] + j) & 1, err, kDevTimeoutAccum);
            if (!ok) break;
            tc_fence_after();
            if (one) {
#pragma unroll
              for (int u = 0; u < kBlock / 16; ++u)
                umma_ts(tO + DP * t, tS + kBlock * t + 64 + 8 * u, v + 128 * u, idO, j > 0 || u > 0);
              umma_commit(smem_u32(&o_done[t]));
              if (t == last) umma_commit(smem_u32(&empty[sv]));
            }
            if (more) scores(t, sk, t == last);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *stop = 1;
      } else if (warp >= 4 && (half == 0 || two)) {
        // ------------------------------------------------------ softmax, output
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t myS = tS + kBlock * half + lane_off, myO = tO + DP * half + lane_off;
        const float sc = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
        const int n0 = ns[half];
        const int all_lo = run->all_lo[half], all_hi = run->all_hi[half];
        const int pair = 1 + 4 * half + (warp & 3);
        float* rd = red + half * 256 + hrow;
        float m = -INFINITY, l = 0.f;
        float ref = -Pack<T>::kBias;  // what the weights are relative to: m, or 0 while it is -inf
        int base, rows, off = 0;  // first key of the block, rows that its pages give it, its place in a long page
        block_keys(geo, page_size, j0, &base, &rows);
        if (geo.parts > 1) off = base % page_size;
        for (int j = 0; j < nb; ++j) {
          if (j > 0) {  // the next block: the next pages, or the next part of one
            base += rows;
            if (geo.parts > 1) {
              off = off + kBlock < page_size ? off + kBlock : 0;
              rows = min(kBlock, page_size - off);
            }
          }
          // this thread's columns [d0, d1) are keys of its row; `part`: not all of them, for some row
          const int d0 = max(0, lo - base) - 64 * hk, d1 = min(rows, hi - base) - 64 * hk;
          const bool part = __any_sync(0xffffffffu, d0 > 0 || d1 < 64);
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&s_full[half]), (n0 + j) & 1, err, kDevTimeoutAccum));
          if (!ok) break;
          tc_fence_after();
          const uint32_t nones = hole[(j0 + j) & 15];
          float x[2][32];  // keys 64 hk ..
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld32(myS + 64 * hk + 32 * c, x[c]);
          tmem_ld_wait();
          if (__builtin_expect(part || nones != 0, 0)) {
            // by groups of 16 columns: most lie inside every row's range, or past a page's end
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (__any_sync(0xffffffffu, d0 > 16 * q || d1 < 16 * q + 16)) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (16 * q + i < d0 || 16 * q + i >= d1) x[q >> 1][16 * (q & 1) + i] = -INFINITY;
              }
            const int per = geo.parts == 1 ? page_size : kBlock;
            for (uint32_t left = nones; left; left &= left - 1) {
              const int p0 = (__ffs(left) - 1) * per - 64 * hk;
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (32 * c + i >= p0 && 32 * c + i < p0 + per) x[c][i] = -INFINITY;
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float* xp = &x[c >> 1][16 * (c & 1)];
            mx[c] = xp[0];
#pragma unroll
            for (int i = 1; i < 15; i += 2) mx[c] = max3(mx[c], xp[i], xp[i + 1]);
            mx[c] = fmaxf(mx[c], xp[15]);
          }
          float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
          // One barrier of the rows' two warps tells whether any row's maximum has
          // outgrown its reference; if so, the threads of a row agree on the new
          // one, and O and l are brought down to it.
          if (__builtin_expect(pair_any(pair, mb > m + kSlack), 0)) {
            rd[128 * hk] = mb;
            pair_sync(pair);
            mb = fmaxf(mb, rd[128 * (1 - hk)]);
            float alpha = 1.f;
            if (mb > m + kSlack) {
              alpha = weight(m, mb);
              m = mb;
              ref = (m == -INFINITY ? 0.f : m) - Pack<T>::kBias;
            }
            l *= alpha;
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
              ok = __all_sync(0xffffffffu,
                              mbar_wait_bounded(smem_u32(&o_done[half]), (n0 + j - 1) & 1, err, kDevTimeoutAccum));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = hk * (DP / 32); c < (hk + 1) * (DP / 32); ++c) {
                uint32_t r[16];
                tmem_ld16(myO + 16 * c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                tmem_st16(myO + 16 * c, r);
              }
              tmem_st_wait();
            }
          }
          // Keys that some row of this half does not see: an infinity or a NaN
          // among their values must not meet a weight of zero.  Such values
          // leave the block here, and the rows that see them get them at the
          // end.
          if (__builtin_expect(base < all_lo || base + rows > all_hi, 0)) {
            const int n = it + 2 * j + 1;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&full[n % S]), (n / S) & 1, err, kDevTimeoutFull));
            if (!ok) break;
            uint4* v = reinterpret_cast<uint4*>(sR + (n % S) * C::kSlot);
            for (int i = hrow + kHalfRows * hk; i < C::kSlot / 16; i += 2 * kHalfRows) {
              const uint4 w = v[i];
              if (odd32<T>(w.x) || odd32<T>(w.y) || odd32<T>(w.z) || odd32<T>(w.w)) {
                atomicMin(&run->odd_lo, j0 + j);
                atomicMax(&run->odd_hi, j0 + j);
                __threadfence_block();
                uint16_t* e = reinterpret_cast<uint16_t*>(v + i);
                for (int k = 0; k < 8; ++k)
                  if (odd16<T>(e[k])) e[k] = 0;
              }
            }
            fence_proxy_async_smem();
          }
          const float2 sc2 = make_float2(sc, sc), nr2 = make_float2(-ref, -ref);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 e = fma2(make_float2(x[c][2 * i], x[c][2 * i + 1]), sc2, nr2);
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              sum[i & 1] = add2(sum[i & 1], e);
              p[i] = Pack<T>::two(e.x, e.y);
            }
            tmem_st16(myS + 64 + 32 * hk + 16 * c, p);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(smem_u32(&p_full[half]));
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
        }
        if (ok)
          ok = __all_sync(0xffffffffu,
                          mbar_wait_bounded(smem_u32(&o_done[half]), (n0 + nb - 1) & 1, err, kDevTimeoutAccum));
        if (!ok) {
          *stop = 1;
        } else {
          tc_fence_after();
          const bool whole = k0 == 0 && k1 == run->blocks;
          const long long part = 2LL * me + (k0 == 0 ? 1 : 0);
          // the row's sum: both threads' keys
          rd[128 * hk] = l;
          pair_sync(pair);
          l += rd[128 * (1 - hk)];
          const float rl = l == 0.f ? 0.f : 1.f / l;
          const int odd_lo = max(run->odd_lo, j0), odd_hi = min(run->odd_hi, j1 - 1);
          T* dst = mine ? out_row<T>(a, s, h, row0 + row) : nullptr;
#pragma unroll 1
          for (int c = hk * (DP / 32); c < (hk + 1) * (DP / 32); ++c) {
            uint32_t r[16];
            __syncwarp();
            tmem_ld16(myO + 16 * c, r);
            tmem_ld_wait();
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 16 * c < a.c.D ? __uint_as_float(r[i]) : 0.f;
            if (odd_lo <= odd_hi && mine) {
              const int* table = a.b.pages + run->b * a.b.page_stride;
              int k_lo, k_hi, rows;
              block_keys(geo, page_size, odd_lo, &k_lo, &rows);
              block_keys(geo, page_size, odd_hi, &k_hi, &rows);
              k_hi += rows;
              for (int k = max(lo, k_lo); k < min(hi, k_hi); ++k) {
                const int page = kv_page(table, k, page_size, a.c.pages);
                if (page < 0) continue;
                const T* src = (const T*)a.c.v + page * a.c.v_page + h * a.c.v_head + (k % page_size) * a.c.v_row;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (16 * c + i < a.c.D && odd16<T>(reinterpret_cast<const uint16_t*>(src)[16 * c + i]))
                    v[i] += val<T>(src[16 * c + i]);
              }
            }
            if (mine && !whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                ws.o[(part * (DP / 4) + 4 * c + i) * kTileRows + row] =
                    make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else if (mine) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= rl;
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = Pack<T>::two(v[2 * i], v[2 * i + 1]);
              const int left = a.c.D - 16 * c;
              if (((uintptr_t)dst & 15) == 0) {
                if (left >= 8) *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
                if (left >= 16) *reinterpret_cast<uint4*>(dst + 16 * c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (i < left) reinterpret_cast<uint16_t*>(dst)[16 * c + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
              }
            }
          }
          if (mine && hk == 0) {
            if (whole) put_lse(a, s, h, row0 + row, ref, l);
            else ws.ml[part * kTileRows + row] = make_float2(ref, l);
          }
        }
      }
    } else if (mine && hk == 0) {
      // no block of this run holds a key that any row sees
      if (k0 == 0 && k1 == run->blocks) {
        T* dst = out_row<T>(a, s, h, row0 + row);
        for (int c = 0; c < a.c.D; ++c) dst[c] = round_to<T>(0.f);
        put_lse(a, s, h, row0 + row, 0.f, 0.f);
      } else {
        const long long part = 2LL * me + (k0 == 0 ? 1 : 0);
        for (int c = 0; c < DP / 4; ++c) ws.o[(part * (DP / 4) + c) * kTileRows + row] = make_float4(0.f, 0.f, 0.f, 0.f);
        ws.ml[part * kTileRows + row] = make_float2(0.f, 0.f);
      }
    }
    if (threadIdx.x == 0 && k0 == 0 && k1 < run->blocks)
      ws.open[me] = Open{run->b, run->rt, h, pc.holder(line + run->blocks - 1) - me};
    it += 2 * nb;
    ns[0] += nb;
    if (two) ns[1] += nb;
    line += k1 - k0;
    // TMEM reads of this run come before the next run's MMAs
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*stop) break;
  }

  // after a wait that ran out: the loads in flight arrive, and the MMAs complete, before the memory is given back
  if (*stop && warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_wait_bounded(smem_u32(&full[s]), 0, err, kDevTimeoutFull, 20000000);
      mbar_wait_bounded(smem_u32(&full[s]), 1, err, kDevTimeoutFull, 20000000);
    }
  }
  if (warp == 1 && lane == 0) {
    umma_commit(smem_u32(done));
    mbar_wait_bounded(smem_u32(done), 0, err, kDevTimeoutAccum);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the row tile that block `blockIdx.x` left open, in the
// order of the keys.  A warp takes 8 rows x 16 channels: 128-byte reads of the
// parts, 32-byte writes of the rows.
constexpr int kJoinThreads = 256;
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) kv_chunk_join_kernel(const __grid_constant__ AttnArgs a, const int G) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int me = blockIdx.x;
  const Space ws = space<DP>(a.workspace, G);
  const Open op = ws.open[me];
  if (op.parts == 0) return;
  const Seq s = sequence(a, op.b, false);
  const int row0 = op.rt * kTileRows, cnt = min(kTileRows, s.n * a.group - row0);
  const int lane = threadIdx.x & 31;
  for (int w = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); w < kTileRows / 8 * (DP / 16);
       w += gridDim.y * (kJoinThreads / 32)) {
    const int r = w / (DP / 16) * 8 + (lane & 7), c = w % (DP / 16) * 4 + (lane >> 3);
    if (r >= cnt) continue;
    float m = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i <= op.parts; ++i) {
      const long long part = 2LL * (me + i) + (i == 0 ? 1 : 0);
      const float2 ml = ws.ml[part * kTileRows + r];
      const float4 x = ws.o[(part * (DP / 4) + c) * kTileRows + r];
      if (ml.y == 0.f) continue;  // nothing seen there
      const float n = fmaxf(m, ml.x);
      const float f = weight(m, n), g = weight(ml.x, n);
      l = l * f + ml.y * g;
      v.x = v.x * f + x.x * g;
      v.y = v.y * f + x.y * g;
      v.z = v.z * f + x.z * g;
      v.w = v.w * f + x.w * g;
      m = n;
    }
    const float rl = l == 0.f ? 0.f : 1.f / l;
    if (4 * c < a.c.D) {
      T* dst = out_row<T>(a, s, op.h, row0 + r) + 4 * c;
      const uint32_t lo = Pack<T>::two(v.x * rl, v.y * rl), hi = Pack<T>::two(v.z * rl, v.w * rl);
      if (((uintptr_t)dst & 7) == 0) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
      } else {
        uint16_t* e = reinterpret_cast<uint16_t*>(dst);
        e[0] = (uint16_t)lo;
        e[1] = (uint16_t)(lo >> 16);
        e[2] = (uint16_t)hi;
        e[3] = (uint16_t)(hi >> 16);
      }
    }
    if (c == 0) put_lse(a, s, op.h, row0 + r, m, l);
  }
}

template <typename T, int DP>
cudaError_t go(const ChunkLaunch& L, int sms, cudaStream_t s) {
  using C = Cfg<DP>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem((const void*)kv_chunk_kernel<T, DP>, C::kSmem, &allowed);
  if (e != cudaSuccess) return e;
  kv_chunk_kernel<T, DP><<<sms, kThreads, C::kSmem, s>>>(L.k, L.v, L.a, L.geo);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms, 16);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_chunk_join_kernel<T, DP>, L.a, sms);
}

}  // namespace

bool kv_chunk_geometry(const AttnArgs& a, ChunkGeo* g) {
  const int ps = a.c.page_size;
  if (a.c.D > 128) return false;
  g->box_rows = ps >= kBlock ? kBlock : (ps + 7) / 8 * 8;
  g->parts = ps > kBlock ? (ps + kBlock - 1) / kBlock : 1;
  g->pages = g->parts > 1 ? 1 : kBlock / g->box_rows;
  // pages whose rows are no multiple of 8 leave gaps between them in a block: one such page to a block, or none
  return ps % 8 == 0 || g->pages == 1;
}

long long kv_chunk_workspace(const AttnArgs& a, int sms) {
  const int DP = a.c.D <= 64 ? 64 : 128;
  return (long long)sms * (sizeof(Open) + 2 * kTileRows * (sizeof(float2) + (size_t)DP * sizeof(float)));
}

cudaError_t launch_kv_chunk(const ChunkLaunch& L, int sms, cudaStream_t s) {
  if (L.a.c.elem == 1) return L.a.c.D <= 64 ? go<__nv_bfloat16, 64>(L, sms, s) : go<__nv_bfloat16, 128>(L, sms, s);
  return L.a.c.D <= 64 ? go<__half, 64>(L, sms, s) : go<__half, 128>(L, sms, s);
}

}  // namespace wan
