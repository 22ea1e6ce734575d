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
// that loads never wait for arithmetic, nor a warp for another:
//  - a warp has a ring of its own (cp.async, kStages deep, 16 keys a stage) and
//    works alone: while one starts or ends a row tile, the others of its SM keep
//    the memory busy;
//  - the whole call's tiles (sequence x row tile x head x 16 keys) are one line
//    that is cut into equal pieces, one per resident warp, on the device from the
//    lengths themselves: any raggedness gives every warp the same bytes, a
//    captured graph follows its lengths, and one long sequence is spread over
//    the whole card;
//  - a row tile that a cut divides leaves partial (m, l, o) in the workspace,
//    and a second kernel, launched to start as the first drains, joins them in
//    the order of the keys: the result does not depend on timing.
// Two sequences of up to 131k keys, 64 heads of 128 on 8 (0.96 GB), take 153 us, 6.3
// TB/s (0.92 of a plain copy's rate); 64 ragged ones of up to 8000 keys, 32 heads on 8
// (1.04 GB), 176 us, 5.9 TB/s; one of 1000 keys 9 us, of which the keys take 2.  (With a
// block's four warps on one row tile, merged through shared memory at its end, the
// first two took 11 and 2 us more.)
// Sums, maxima and outputs are held in 32 bits; how the weights are rounded is
// told at Weights.
//
// The kernel's second form (X) is for rows that see by their place: a window with
// first keys, or a tree of drafts.  Its line holds only the tiles that a row tile's
// rows see: 48 ragged sequences of up to 20,000 keys, windows of 4096 and 128 first
// keys, 32 heads of 128 on 8 (0.78 GB), take 130 us, 6.0 TB/s.
#include <algorithm>

#include "kv_common.cuh"

namespace wan {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;    // rows of a tile: the MMA's M
constexpr int kKeys = 16;    // keys of a tile
// Least tiles of a piece.  One, since a warp's wait for its next tile costs more than a further part in the join: with
// two, one sequence of 1000 keys takes 2.1 us more; long ones never come to the limit.
constexpr int kLeast = 1;

template <int DP>
struct Cfg {
  static constexpr int CH = DP / 8;                     // 16-byte chunks per row
  static constexpr int kStages = DP == 64 ? 6 : DP == 128 ? 3 : 2;
  static constexpr int kCtas = DP == 256 ? 1 : 2;       // resident blocks per SM
  static constexpr int kHalf = kKeys * DP * 2;          // bytes of K (or V) per stage
  static constexpr int kRing = kStages * 2 * kHalf;     // bytes per warp
  static constexpr bool kQRegs = DP <= 128;             // q fragments in registers; at 256 channels they are fetched again
  static constexpr int kQ = kRows * DP * 2;             // q, and then (or behind it) a tile's weights on a rare path
  static constexpr int kWarp = kRing + kQ + (kQRegs ? 0 : kRows * kKeys * 4);
  static constexpr int kSmem = kWarps * kWarp;
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

// How the weights p >= 0 of a pair of keys enter the product with v: as hi + lo, hi
// cut to the type's bits (so lo >= 0), and lo above zero where hi is, so that both
// products with an infinite v have its sign, as p v has.  The result then carries only
// its own rounding; with weights rounded once to float16, two sequences of 131k keys
// were off by 2.5e-4 instead of 2.1e-4.  A tile of at most 8 rows has its lower parts
// in the place of the upper rows, so the products stay as many (those two sequences
// take 154 us, with products of their own 157, with one part alone 152; 64 ragged ones
// of up to 8000 keys 177, 181, 181).
//  bfloat16: lo is at least p 2^-24.
//  float16: all weights are 2^kBias times larger, so that keys down to 2^-36 of the
//  largest weight still count; kBias leaves the largest below 65504.
template <typename T>
struct Weights;
template <>
struct Weights<__nv_bfloat16> {
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
  static constexpr float kBias = 12.f;
  static __device__ __forceinline__ uint32_t hi(float x, float y) {
    uint32_t v;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(y), "f"(x));
    return v;
  }
  static __device__ __forceinline__ uint32_t lo(float x, float y) {
    const uint32_t h = hi(x, y);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    // where hi is not zero x is 2^-24, float16's least, or more
    const __half2 v = __floats2half2_rn(fmaxf(x - f.x, fminf(x, 0x1p-24f)), fmaxf(y - f.y, fminf(y, 0x1p-24f)));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
// ------------------------------------------------------------ the line of tiles
// Tiles of a sequence on the line: row tiles x heads x key tiles.
struct Tiles {
  int key_tiles;
  long long runs, all;  // row tiles of all heads, their key tiles
};
// With X (rows see by their place) a row tile's key tiles are those that some row of it sees, numbered without the
// gap between the first keys and the window; as many as the widest row tile can have stand on the line, the others
// leave their last ones empty.
template <bool X>
__device__ __forceinline__ Tiles tiles_of(const AttnArgs& a, const Seq& s) {
  Tiles t;
  t.key_tiles = (s.len + kKeys - 1) / kKeys;
  if (X && a.mask == kMaskWindow) {
    // the tokens of 16 rows reach over 15 / group + 1 steps at most, each of which can begin a frame
    const uint32_t steps = s.n > 1 ? min((uint32_t)(s.n - 1), (uint32_t)((kRows - 1) / a.group + 1)) : 0;
    const uint32_t reach = steps == 0 ? 0 : a.frame >= steps ? a.frame : ((steps - 1) / a.frame + 1) * a.frame;
    const uint32_t most = (min(a.span, (uint32_t)s.len) + reach) / kKeys + 2 + ((uint32_t)a.sinks + kKeys - 1) / kKeys;
    t.key_tiles = (int)min((uint32_t)t.key_tiles, most);
  }
  t.runs = ((long long)s.n * a.group + kRows - 1) / kRows * a.c.heads;
  t.all = t.runs * t.key_tiles;
  return t;
}

// A call of few tiles, cut so that no warp has more than one run: one that ends a row tile and starts another takes 5 us
// longer than the others, and the call with it (26 drafts of 16 heads against 2000 keys 23.9 us by the line, 21.3 so; 8
// drafts 18.3 and 14.8; 32 single tokens with windows of 300 keys 23.2 and 21.1; 4 of 500 keys 11.7 and 12.3).  Each row
// tile is cut into equal parts of at most `size` tiles, the least size for which there are warps enough; false if there are
// more than kSmall tiles a warp, where a run's start counts less, or more than 32 sequences.  All warps find the same.
constexpr int kSmall = 12;
__device__ __forceinline__ float inverse(int d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((float)d));
  return r;
}
// x / d by d's inverse, of results below 2^20 (which the product is off by less than one from)
__device__ __forceinline__ int part_of(int x, int d, float inv) {
  int q = (int)((float)x * inv);
  if (q * d > x) --q;
  if ((q + 1) * d <= x) ++q;
  return q;
}
__device__ __forceinline__ bool cut_tiles(const AttnArgs& a, int me, int G, Piece* p, int* parts) {
  if (a.b.B > 32) return false;
  const int lane = threadIdx.x & 31;
  const long long most = (kSmall + 1) * G;  // (a sequence's numbers are cut to it: sums of 32 then fit 32 bits)
  Tiles t{0, 0, 0};
  if (lane < a.b.B) t = tiles_of<true>(a, sequence<true>(a, lane, false));
  const int total = (int)__reduce_add_sync(0xffffffffu, (uint32_t)min(t.all, most));
  if (total > kSmall * G) return false;
  const int runs = t.key_tiles > 0 ? (int)t.runs : 0;
  int size = max(1, (int)((float)total * inverse(G))), mine = 0, all;  // (one too few is one more round)
  for (;; ++size) {
    mine = runs * part_of(t.key_tiles + size - 1, size, inverse(size));
    all = (int)__reduce_add_sync(0xffffffffu, (uint32_t)mine);
    if (all <= G) break;
    if (size > 2 * kSmall) return false;  // (more row tiles than warps)
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  p->beg = p->end = 0;
  p->live = all;
  p->size = size;
  p->longer = 0;
  p->b = 0;
  p->at = 0;
  if (me >= all) return true;
  p->b = __ffs(__ballot_sync(0xffffffffu, me >= incl - mine && me < incl)) - 1;
  const int q = me - __shfl_sync(0xffffffffu, incl - mine, p->b);
  const int n = __shfl_sync(0xffffffffu, t.key_tiles, p->b), of = part_of(n + size - 1, size, inverse(size));
  const float inv = inverse(of);
  const int tile = part_of(q, of, inv), part = q - tile * of, t0 = part_of(n * part, of, inv), t1 = part_of(n * (part + 1), of, inv);
  *parts = of;
  p->at = (long long)tile * n + t0;
  p->end = t1 - t0;
  return true;
}

struct Space {  // the workspace: per piece an Open and two parts (0: a row tile's later keys, 1: its first ones)
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

template <typename T, int DP, bool X>
__global__ void __launch_bounds__(kThreads, Cfg<DP>::kCtas)
    kv_split_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<DP>;
  constexpr int CH = C::CH, ST = C::kStages, NK = DP / 16;
  constexpr bool kQRegs = C::kQRegs;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_seen[kWarps][ST];
  __shared__ long long s_line[3 * kWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = blockIdx.x * kWarps + warp;  // the piece
  uint8_t* ring = smem + warp * C::kWarp;
  uint8_t* sq = ring + C::kRing;
  float* s_p = reinterpret_cast<float*>(kQRegs ? sq : sq + C::kQ);  // [kRows][kKeys]
  const uint32_t ring_a = smem_u32(ring), sq_a = smem_u32(sq);
  const Space ws = space<DP>(a.workspace, gridDim.x * kWarps);

  // the join's blocks may start as soon as every block of this grid runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what came before on the stream

  // The line is cut as it comes, or (with X) each of few row tiles for itself: parts of it, else 0.
  int parts = 0;
  Piece pc;
  if (!X || !cut_tiles(a, me, gridDim.x * kWarps, &pc, &parts))
    pc = cut_line<kWarps, kWarps>(a.b.B, kLeast, s_line, [&](int b) { return tiles_of<X>(a, sequence<X>(a, b, false)).all; });
  if (lane == 0) ws.open[me].parts = 0;
  int b = pc.b;
  long long at = pc.at;
  const T* kbase = (const T*)a.c.k;
  const T* vbase = (const T*)a.c.v;

  for (long long line = pc.beg; line < pc.end;) {
    Seq s = sequence<X>(a, b, false);
    Tiles tl = tiles_of<X>(a, s);
    while (at >= tl.all) {  // the next sequence with a tile
      at -= tl.all;
      s = sequence<X>(a, ++b, false);
      tl = tiles_of<X>(a, s);
    }
    // the run: key tiles [kt0, kt1) of one row tile and head
    const int seg = (int)quotient(at, tl.key_tiles), kt0 = (int)(at - (long long)seg * tl.key_tiles);
    const int kt1 = (int)min((long long)tl.key_tiles, kt0 + (pc.end - line));
    // heads of a row tile side by side, row tiles behind them
    const int rt = seg / a.c.heads, h = seg - rt * a.c.heads;
    const int row0 = rt * kRows, cnt = min(kRows, s.n * a.group - row0);
    const bool few = cnt <= kRows / 2;  // then the tile's upper rows take the lower parts of the weights (Weights)

    // the keys that this thread's two rows see, and those that any row does
    const int r_a = lane >> 2, r_b = r_a + 8;
    int lo_a = 0, hi_a = 0, lo_b = 0, hi_b = 0, lo = 0, hi = s.len;
    // rows of one token, or of tokens that see the same keys, see all that is fetched: they need no mask of their own
    bool mixed = false;
    // with X: lane r's row sees `mine`; some row of the tile [0, c) and [lo, hi), all of them [0, c_all) and [lo_all,
    // hi_all); key tiles of the first keys, and how many are skipped behind them
    Sight mine{0, 0, 0};
    int c = 0, c_all = 0, lo_all = 0, hi_all = 0, first_tiles = 0, skip = 0;
    int w0, w1;
    if constexpr (X) {
      const int row = row0 + min(lane, cnt - 1), ahead = row0 / a.group;
      mine = sight(a, s, row / a.group);
      mixed = ahead != (row0 + cnt - 1) / a.group;
      c = c_all = mine.c;
      lo = lo_all = mine.lo;
      hi = hi_all = mine.hi;
      if (mixed) {
        c = __reduce_max_sync(0xffffffffu, c), c_all = __reduce_min_sync(0xffffffffu, c_all);
        lo = __reduce_min_sync(0xffffffffu, lo), lo_all = __reduce_max_sync(0xffffffffu, lo_all);
        hi = __reduce_max_sync(0xffffffffu, hi), hi_all = __reduce_min_sync(0xffffffffu, hi_all);
      }
      if (a.mask == kMaskTree) {  // all drafts are fetched, whoever sees them: even a single row has a mask
        hi = s.len;
        mixed = true;
      }
      if (lo <= c) c = lo = 0;
      first_tiles = (c + kKeys - 1) / kKeys;
      const int from = max(lo / kKeys, first_tiles);
      skip = from - first_tiles;
      w0 = kt0, w1 = min(kt1, (hi + kKeys - 1) / kKeys - skip);
    } else {
      if (!a.ranges) {
        if (r_a < cnt) hi_a = hi;
        if (r_b < cnt) hi_b = hi;
      } else {
        int f = 0, e = 0;  // lane r holds row r's
        if (lane < cnt) seen_range(a, s.r0 + (row0 + lane) / a.group, s.len, &f, &e);
        lo_a = __shfl_sync(0xffffffffu, f, r_a), hi_a = __shfl_sync(0xffffffffu, e, r_a);
        lo_b = __shfl_sync(0xffffffffu, f, r_b), hi_b = __shfl_sync(0xffffffffu, e, r_b);
        lo = __reduce_min_sync(0xffffffffu, f < e ? f : 0x7fffffff);
        hi = __reduce_max_sync(0xffffffffu, e);
      }
      const bool differ = (r_a < cnt && (lo_a != lo || hi_a != hi)) || (r_b < cnt && (lo_b != lo || hi_b != hi));
      mixed = __any_sync(0xffffffffu, differ);
      w0 = hi > 0 ? max(kt0, lo / kKeys) : kt1, w1 = min(kt1, (hi + kKeys - 1) / kKeys);
    }
    // first key of key tile kt, and whether some row sees a key
    auto key_of = [&](int kt) { return (X && kt >= first_tiles ? kt + skip : kt) * kKeys; };
    auto in_sight = [&](int key) { return (key >= lo && key < hi) || (X && key < c); };
    uint64_t drafts = 0;  // of the drafts from this one on, those that the lane's row sees
    int drafts_from = -64;
    Family kin = {};
    if constexpr (X) {
      if (a.mask == kMaskTree && key_of(w1) > s.len - s.n) kin = family(a, s);
    }

    const int* table = a.b.pages + b * a.b.page_stride;

    // The page of this lane's key in tile kt (lane & 15), asked for a tile ahead of
    // the loads that need it; -1 if no row sees the key.
    auto lookup = [&](int kt) {
      const int key = key_of(kt) + (lane & 15);
      return kt < w1 && in_sight(key) ? table[key / a.c.page_size] : -1;
    };
    auto issue = [&](int kt, int page) {
      const int st = kt % ST;
      const int key = key_of(kt) + (lane & 15);
      const uint32_t dk = ring_a + st * 2 * C::kHalf, dv = dk + C::kHalf;
      const bool take = page >= 0 && page < a.c.pages;
      if (!take && in_sight(key) && a.b.status) atomicCAS(a.b.status, 0, (int)kDevBadPage);
      long long ko = 0, vo = 0;
      if (take) {
        const int off = key % a.c.page_size;
        ko = page * a.c.k_page + h * a.c.k_head + off * a.c.k_row;
        vo = page * a.c.v_page + h * a.c.v_head + off * a.c.v_row;
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, take) & 0xffffu;
      if (lane == 0) s_seen[warp][st] = seen;
      constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;  // rows per instruction
#pragma unroll
      for (int i = 0; i < kKeys / RPI; ++i) {
        const int r = i * RPI + lane / CH, c = lane % CH;
        const long long kr = __shfl_sync(0xffffffffu, ko, r), vr = __shfl_sync(0xffffffffu, vo, r);
        const bool ok = ((seen >> r) & 1) && c * 8 < a.c.D;
        const uint32_t d = r * DP * 2 + ((c ^ (r & 7)) << 4);
        cp_async16(dk + d, kbase + (ok ? kr + c * 8 : 0), ok);
        cp_async16(dv + d, vbase + (ok ? vr + c * 8 : 0), ok);
      }
    };

    // everything that only waits for memory first: the first pages' numbers and q, then the first tiles
    int page[ST];
#pragma unroll
    for (int i = 0; i < ST; ++i) page[i] = lookup(w0 + i);
    constexpr int NQ = kRows * CH / 32;
    uint4 qv[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int r = (i * 32 + lane) / CH, c = lane % CH;
      qv[i] = make_uint4(0, 0, 0, 0);  // past the rows and channels
      if (r < cnt && c * 8 < a.c.D) {
        const int t = (row0 + r) / a.group, g = row0 + r - t * a.group;
        const T* src = (const T*)a.q + (long long)(s.r0 + t) * a.q_t + (long long)(h * a.group + g) * a.q_h + c * 8;
        if (((uintptr_t)src & 15) == 0) {
          qv[i] = *reinterpret_cast<const uint4*>(src);
        } else {
          uint32_t w[4];
          const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = (uint32_t)e[2 * j] | ((uint32_t)e[2 * j + 1] << 16);
          qv[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      if (w0 + i < w1) issue(w0 + i, page[i]);
      cp_commit();
    }
    int ahead = page[ST - 1];  // of tile kt + ST - 1
    // q by way of shared memory: 16-byte chunk c of row r at chunk c ^ (r & 7)
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int r = (i * 32 + lane) / CH, c = lane % CH;
      *reinterpret_cast<uint4*>(sq + r * DP * 2 + ((c ^ (r & 7)) << 4)) = qv[i];
    }
    __syncwarp();
    uint32_t qf[kQRegs ? NK : 1][4];
    const uint32_t q_row = sq_a + (lane & 15) * DP * 2;
    if (kQRegs) {
#pragma unroll
      for (int k = 0; k < NK; ++k) ldsm4(q_row + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4), qf[kQRegs ? k : 0]);
      __syncwarp();
    }

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;

    for (int kt = w0; kt < w1; ++kt) {
      cp_wait<ST - 2>();
      __syncwarp();
      const int st = kt % ST;
      const uint32_t sk = ring_a + st * 2 * C::kHalf, sv = sk + C::kHalf;
      const uint32_t seen = s_seen[warp][st];
      if (seen) {
        const int key0 = key_of(kt);
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
        uint32_t vis_a = seen, vis_b = seen;
        if constexpr (X) {
          if (!(key0 + kKeys <= c_all || (key0 >= lo_all && key0 + kKeys <= hi_all))) {
            part = true;
            uint32_t vis = sight_bits(mine, key0);
            const int d0 = key0 - (s.len - s.n);
            if (a.mask == kMaskTree && d0 + kKeys > 0) {
              if (d0 + kKeys > drafts_from + 64) {
                drafts_from = max(d0, 0);
                drafts = ancestors(a, s, kin, (row0 + min(lane, cnt - 1)) / a.group, drafts_from);
              }
              vis |= (uint32_t)(d0 >= drafts_from ? drafts >> (d0 - drafts_from) : drafts << (drafts_from - d0));
            }
            if (lane >= cnt) vis = 0;  // the tile has no such row; its place holds the lower parts of another's products
            vis_a &= __shfl_sync(0xffffffffu, vis, r_a);
            vis_b &= __shfl_sync(0xffffffffu, vis, r_b);
          }
        } else if (mixed) {
          part = part || __any_sync(0xffffffffu, (r_a < cnt && (key0 < lo_a || key0 + kKeys > hi_a)) ||
                                                     (r_b < cnt && (key0 < lo_b || key0 + kKeys > hi_b)));
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[n][i] *= a.scale_log2;
            if (part) {
              const int kk = n * 8 + (lane & 3) * 2 + (i & 1);
              bool hidden;
              if constexpr (X) {
                hidden = !(((i < 2 ? vis_a : vis_b) >> kk) & 1);
              } else {
                const int key = key0 + kk, f = i < 2 ? lo_a : lo_b, e = i < 2 ? hi_a : hi_b;
                hidden = !((seen >> kk) & 1) || key < f || key >= e;
              }
              if (hidden) sc[n][i] = -INFINITY;
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
          const float c_o = few ? c_a : c_b;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            o[i][0] *= c_a;
            o[i][1] *= c_a;
            o[i][2] *= c_o;
            o[i][3] *= c_o;
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
        if (few) hi4[1] = lo4[0], hi4[3] = lo4[2];
        // A value that some rows see and others do not must not reach the
        // others: 0 times an infinity or a NaN is a NaN.  Such values are
        // taken out of the tile and added to the rows that see them.
        bool odd = false;
        if (mixed && part) {
          for (int i = lane; i < kKeys * CH; i += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(ring + (sv - ring_a) + i * 16);
            odd |= odd32<T>(v.x) || odd32<T>(v.y) || odd32<T>(v.z) || odd32<T>(v.w);
          }
          odd = __any_sync(0xffffffffu, odd);
          if (odd) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s_p[(i < 2 ? r_a : r_b) * kKeys + n * 8 + (lane & 3) * 2 + (i & 1)] = sc[n][i] == -INFINITY ? -1.f : p[n][i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int c = i * 8 + (lane & 3) * 2 + (j & 1);
                for (int k = 0; k < kKeys; ++k) {
                  const float w = s_p[(j < 2 ? r_a : r_b) * kKeys + k];
                  const uint8_t* e = ring + (sv - ring_a) + k * DP * 2 + ((((c >> 3) ^ (k & 7)) << 4) | ((c & 7) * 2));
                  const T v = *reinterpret_cast<const T*>(e);
                  if (w >= 0.f && odd16<T>(*reinterpret_cast<const uint16_t*>(e))) o[i][j] += w * val<T>(v);
                }
              }
            __syncwarp();
            for (int i = lane; i < kKeys * DP; i += 32) {
              uint16_t* e = reinterpret_cast<uint16_t*>(ring + (sv - ring_a)) + i;
              if (odd16<T>(*e)) *e = 0;
            }
            __syncwarp();
          }
        }
        const uint32_t vrow = sv + (lane & 15) * DP * 2;
        if (few) {
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) {
            uint32_t bv[4];
            ldsm4t(vrow + (((2 * n + (lane >> 4)) ^ (lane & 7)) << 4), bv);
            mma16816<T>(o[2 * n], hi4, bv[0], bv[1]);
            mma16816<T>(o[2 * n + 1], hi4, bv[2], bv[3]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) {
            uint32_t bv[4];
            ldsm4t(vrow + (((2 * n + (lane >> 4)) ^ (lane & 7)) << 4), bv);
            mma16816<T>(o[2 * n], hi4, bv[0], bv[1]);
            mma16816<T>(o[2 * n + 1], hi4, bv[2], bv[3]);
            mma16816<T>(o[2 * n], lo4, bv[0], bv[1]);
            mma16816<T>(o[2 * n + 1], lo4, bv[2], bv[3]);
          }
        }
      }
      __syncwarp();
      if (kt + ST - 1 < w1) issue(kt + ST - 1, ahead);
      cp_commit();
      ahead = lookup(kt + ST);
    }
    cp_wait<0>();

    // ------------------------------------------------------- out, or a part of it
    const float unbias = Weights<T>::kBias != 0.f ? exp2f(-Weights<T>::kBias) : 1.f;
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l_a += __shfl_xor_sync(0xffffffffu, l_a, d);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, d);
    }
    l_a *= unbias;
    l_b *= unbias;
    if (few) {
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        o[i][0] += o[i][2];
        o[i][1] += o[i][3];
      }
    }
    const bool whole = kt0 == 0 && kt1 == tl.key_tiles;
    const long long slot = 2LL * me + (kt0 == 0 ? 1 : 0);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int r = w ? r_b : r_a;
      const float m = w ? m_b : m_a, l = w ? l_b : l_a;
      if (r >= cnt) continue;
      if (whole) {
        const float rl = l == 0.f ? 0.f : unbias / l;
        T* dst = out_row<T>(a, s, h, row0 + r);
        const bool even = ((uintptr_t)dst & 3) == 0;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          const int c = i * 8 + (lane & 3) * 2;
          if (c >= a.c.D) continue;
          // a row that saw nothing: zeros, whatever else its products hold
          const float x = l == 0.f ? 0.f : o[i][2 * w] * rl, y = l == 0.f ? 0.f : o[i][2 * w + 1] * rl;
          const T e[2] = {round_to<T>(x), round_to<T>(y)};
          if (even) {
            *reinterpret_cast<uint32_t*>(dst + c) = *reinterpret_cast<const uint32_t*>(e);
          } else {
            dst[c] = e[0];
            dst[c + 1] = e[1];
          }
        }
        if ((lane & 3) == 0) put_lse(a, s, h, row0 + r, m, l);
      } else {
        float* dst = ws.o + (slot * kRows + r) * DP;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
          *reinterpret_cast<float2*>(dst + i * 8 + (lane & 3) * 2) = make_float2(o[i][2 * w] * unbias, o[i][2 * w + 1] * unbias);
        if ((lane & 3) == 0) ws.ml[slot * kRows + r] = make_float2(m, l);
      }
    }
    if (!whole && kt0 == 0 && lane == 0) {
      const long long last = line + tl.key_tiles - 1;  // the row tile's last tile: its piece is the last part's
      ws.open[me] = Open{parts ? parts - 1 : pc.holder(last) - me, h, row0, cnt, s, 0};
    }
    __syncwarp();
    at += kt1 - kt0;
    line += kt1 - kt0;
  }
}

// Joins the parts of the row tiles that the pieces of block `blockIdx.x` left open,
// row `blockIdx.y` of each, in the order of the keys.  Eight warps share the open
// pieces (a task each, or several to a task): lane i forms the weight of the i-th
// part of its warp, all lanes add up the parts' channels, eight parts asked for
// together, and the warps of a task meet in shared memory.  Rows of sequences
// without a key get their zeros here.
constexpr int kJoinWarps = 8;
template <typename T, int DP>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int N = DP / 32;  // channels per lane
  __shared__ float s_v[kJoinWarps][DP];
  __shared__ float2 s_ml[kJoinWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  const Space ws = space<DP>(a.workspace, gridDim.x * kWarps);
  const Open* open = ws.open + blockIdx.x * kWarps;
  // lane w: piece w
  const Open mine = lane < kWarps ? open[lane] : Open{0, 0, 0, 0, {0, 0, 0}, 0};
  uint32_t todo = __ballot_sync(0xffffffffu, mine.parts > 0 && r < mine.cnt);
  const int tasks = __popc(todo);
  if (tasks > 0) {
    const int per = tasks > 2 ? 2 : tasks == 2 ? 4 : 8;  // warps per task (four tasks at most)
    const int sub = warp % per, nth = warp / per;
    for (int i = 0; i < nth; ++i) todo &= todo - 1;
    const bool any = todo != 0;
    const int w0 = any ? __ffs(todo) - 1 : 0, me = blockIdx.x * kWarps + w0;
    Open o;
    o.parts = __shfl_sync(0xffffffffu, mine.parts, w0);
    o.h = __shfl_sync(0xffffffffu, mine.h, w0);
    o.row0 = __shfl_sync(0xffffffffu, mine.row0, w0);
    o.s.r0 = __shfl_sync(0xffffffffu, mine.s.r0, w0);
    const int n = any ? o.parts + 1 : 0;
    float m = -INFINITY, l = 0.f, v[N] = {};
    for (int i0 = sub; i0 < n; i0 += 32 * per) {
      const int k = min(32, (n - i0 + per - 1) / per);  // parts i0, i0 + per, ..
      float2 ml = make_float2(-INFINITY, 0.f);
      const int i = i0 + lane * per;
      if (lane < k) ml = ws.ml[(2LL * (me + i) + (i == 0 ? 1 : 0)) * kRows + r];
      float top = 0.f, w = 0.f, f = 0.f;
      for (int q0 = 0; q0 < k; q0 += 8) {
        float2 x[8][N / 2];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int p = i0 + min(q0 + q, k - 1) * per;
          const float2* src =
              reinterpret_cast<const float2*>(ws.o + ((2LL * (me + p) + (p == 0 ? 1 : 0)) * kRows + r) * DP + lane * N);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) x[q][e] = src[e];
        }
        if (q0 == 0) {  // the weights, while the first channels are on their way
          top = ml.x;
#pragma unroll
          for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          top = fmaxf(top, m);
          w = lane < k ? weight(ml.x, top) : 0.f;
          f = weight(m, top);
          float part = lane < k ? ml.y * w : 0.f;
#pragma unroll
          for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
          l = l * f + part;
          m = top;
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] *= f;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float wi = __shfl_sync(0xffffffffu, w, (q0 + q) & 31);
          if (q0 + q < k) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
              v[2 * e] = fmaf(x[q][e].x, wi, v[2 * e]);
              v[2 * e + 1] = fmaf(x[q][e].y, wi, v[2 * e + 1]);
            }
          }
        }
      }
    }
    if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < N; ++e) s_v[warp][lane * N + e] = v[e];
    __syncthreads();
    if (sub == 0 && any) {
      float top = -INFINITY;
      for (int w = 0; w < per; ++w) top = fmaxf(top, s_ml[warp + w].x);
      l = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = 0.f;
      for (int w = 0; w < per; ++w) {
        const float2 ml = s_ml[warp + w];
        const float f = weight(ml.x, top);
        l += ml.y * f;
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = fmaf(s_v[warp + w][lane * N + e], f, v[e]);
      }
      const float rl = l == 0.f ? 0.f : 1.f / l;
      T* dst = out_row<T>(a, o.s, o.h, o.row0 + r);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (lane * N + e < a.c.D) dst[lane * N + e] = round_to<T>(l == 0.f ? 0.f : v[e] * rl);
      if (lane == 0) put_lse(a, o.s, o.h, o.row0 + r, top, l);
    }
  }
  if (r == 0) put_empty<T>(a, blockIdx.x, gridDim.x);
}

template <typename T, int DP, bool X>
cudaError_t go_split(const AttnArgs& a, int sms, cudaStream_t s) {
  using C = Cfg<DP>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem((const void*)kv_split_kernel<T, DP, X>, C::kSmem, &allowed);
  if (e != cudaSuccess) return e;
  const int G = sms * C::kCtas;
  // each may start as the kernel before it drains, and waits for its end
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(G);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  e = cudaLaunchKernelEx(&cfg, kv_split_kernel<T, DP, X>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(G, a.b.cu ? kRows : std::min(kRows, a.group));  // rows that a tile can have
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<T, DP>, a);
}

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

template <typename T, bool X>
cudaError_t by_dim(const AttnArgs& a, int sms, cudaStream_t s) {
  switch (padded(a.c.D)) {
    case 64: return go_split<T, 64, X>(a, sms, s);
    case 128: return go_split<T, 128, X>(a, sms, s);
    default: return go_split<T, 256, X>(a, sms, s);
  }
}
template <typename T>
cudaError_t by_mask(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.mask == kMaskRanges ? by_dim<T, false>(a, sms, s) : by_dim<T, true>(a, sms, s);
}

}  // namespace

long long kv_attention_workspace(const AttnArgs& a, int sms) {
  const int DP = padded(a.c.D);
  return space_bytes(DP, sms * kWarps * (DP == 256 ? Cfg<256>::kCtas : Cfg<128>::kCtas));
}

cudaError_t launch_kv_attention(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.c.elem == 1 ? by_mask<__nv_bfloat16>(a, sms, s) : by_mask<__half>(a, sms, s);
}

}  // namespace wan
