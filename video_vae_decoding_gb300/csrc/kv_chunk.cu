// Attention of many new tokens over a paged key-value cache: a flash kernel on
// the fifth-generation tensor cores.
//
// For 256 rows (row r of a sequence and key head h: token r / group, query head
// h * group + r % group) in two halves of 128, per block of up to 128 keys j:
//   S = Q_t K_j^T            (t = 0, 1: the halves; M = 128, N = 128)
//   P_t = 2^(scale S - m)    one thread per row: running maximum m, moved only
//                            when a block exceeds it by 8 (O is then rescaled)
//   O_t += P_t V_j           P_t read from tensor memory
// and O_t / l at the end.  A softmax reads S into registers at once, so that the
// tensor cores form the next S while it works.  TMEM has 512 columns: S takes 128,
// which the halves, half a period apart, take in turn; a P 64 and an O_t DP.
//  D <= 64    two P for each half: its P V has a block's time more.  (An S for each
//             half instead: 154 us below instead of 134.)
//  D <= 128   one P for each half
//  D <= 256   one half of 128 rows
// What else was tried at D = 128, cycles per block of 128 keys and 256 rows (2048 of
// them products):
//   S_t for each half with P_t in its place    3100, and P V has to be waited for
//                                               before the next Q K
//   64 keys, two S buffers a half              4300: with N = 64 the first operand's
//                                               way from shared memory, 64 cycles
//                                               an instruction, bounds Q K
//   one S, 16 softmax warps                    4000: they starve the issuing warps
//   weights kept until P's room is free        2900: they do not fit the registers
//   this                                       2600
// A tile of at most 128 rows puts its rows in both halves, which take the key
// blocks in turn, and adds the halves up at the end.
//
// Bound: the tensor cores, 4 D operations per row and key; K and V come through
// a ring each and serve both halves, so a block of 128 keys asks 64 KB (D = 128) for
// 33.6 MFLOP.  880 tokens of 16 heads of 128 against 27,280 keys take 174 us, 1.13
// PFLOP/s (59% of a large library product's); with heads of 64 135 us, where the
// softmax bounds, and with 8 heads of 256 246 us: 128 KB a block for 16.8 MFLOP is 8
// TB/s from the L2.
// V is taken as it lies in the cache, [key][channel]: the MMA's second operand
// with its N dimension contiguous, so nothing is transposed on the way.
//
// Pages: a block is as many whole pages as fit 128 keys (each one TMA box of
// its rows, rounded up to 8), or a part of a longer page.  Rows past a page's
// end, a page that the cache does not have and pages past the sequence read as
// zeros (the TMA's fill).
//
// The line of (sequence, row tile, head, key block) is cut into equal pieces,
// one per SM, as in the split kernel (weighed by what a block costs in a larger
// and in a smaller tile); the join adds up what a cut divides.
//
// The second form (X) is for rows that see by their place (a window with first keys,
// a tree of drafts): blocks are made of the pages that some row of the tile sees.
// A window of 9 latent frames and the first one, 880 tokens of 16 heads of 128, takes
// 86 us (0.73 PFLOP/s: runs of 30 blocks, of which start and end are a quarter), 64
// drafts of 24 sequences of up to 9000 keys, 32 heads on 8, 133 us, ragged windows of
// 1000 keys at heads of 64 84 us.
#include <type_traits>

#include "kv_common.cuh"
#include "kv_chunk.h"

namespace wan {

namespace {

// Warps 0 loads K, 1 issues Q K, 2 issues P V, 3 loads V (and owns TMEM); 4-7 softmax of half 0, 8-11 of
// half 1: a thread per row (TMEM lane).
constexpr int kThreads = 384;
constexpr int kHalfRows = 128;
constexpr int kBlock = 128;       // key columns of a block
constexpr int kBoxBytes = 16384;  // 128 rows x 64 channels
constexpr int kLeast = 5;         // units of a piece: a block's (with ten blocks' calls of 100 tokens take 42 us instead of 21)
constexpr float kSlack = 8.f;    // log2 units that the reference maximum may lag behind

// Rows of a row tile: at a head dim above 128 O takes half of TMEM, which leaves room for one half.
__host__ __device__ inline constexpr int tile_rows(int D) { return D > 128 ? kHalfRows : 2 * kHalfRows; }

template <int DP>
struct Cfg {
  static constexpr bool kOne = DP > 128;  // one half (warps 8-11 have nothing to do)
  static constexpr int kRows = tile_rows(DP);
  static constexpr int ND = DP / 64;
  // K or V of a block fill a slot; above 128 channels a slot holds 64 of K's or 128 of V's (a product with fewer
  // columns of V takes no less time)
  static constexpr int kKeyBoxes = kOne ? 1 : ND, kValBoxes = kOne ? 2 : ND;  // 64-channel boxes of a slot
  static constexpr int kKeySlot = kKeyBoxes * kBoxBytes, kValSlot = kValBoxes * kBoxBytes;
  // K and V have a ring each: a barrier is then waited for by one warp, phase by phase, and a parity never stands for
  // another lap of the ring than the next
  static constexpr int kKeySlots = DP == 64 ? 5 : DP == 128 ? 2 : 4, kValSlots = DP == 64 ? 5 : 3;
  static constexpr int kQ = (kOne ? 1 : 2) * ND * kBoxBytes;
  static constexpr int kSmem = kQ + kKeySlots * kKeySlot + kValSlots * kValSlot + 1024 + 1024;
};

// Weights 2^(x - m) are rounded once to the operands' type: a second part would add
// half to the products, which bound this kernel, and TMEM has no room for it at 128
// channels.  880 tokens against 27,280 keys in bfloat16 are then off by 2.3e-3 (1.7e-3
// is the result's rounding alone), ragged chunks in float16 by 2.9e-4 (2.1e-4).
// Weights reach 2^kSlack; in float16 they are taken 2^7 times larger (65504 is the
// end), so that keys down to 2^-31 of the largest still count.
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

// Waits for the phase of `parity` to complete; false, and `code` in the status word if
// there is one, if it has not after 2^18 tries.  A try that fails sleeps for 3.7 us (the
// self test measures a second for all of them); what is waited for takes microseconds.
// Tries are counted, not timed as in mbar_wait_bounded: a clock read in the loop, behind
// however many tries, costs 2 to 10% of a call at 64 channels and 1 to 5% at 128.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* err, int code) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 262144;\n"
      "WAIT_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra WAIT_%=;\n"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (__builtin_expect(!done, 0)) {
    if (err) atomicCAS(err, 0, code);
    return false;
  }
  return true;
}

// One try.  It takes 100 cycles or more to answer, even if the phase is complete:
// asked ahead of need, the answer costs nothing.
__device__ __forceinline__ uint32_t ask_phase(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done;
}

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
// One thread of the calling warp (converged; the same one at each call, but not lane 0 by any rule).
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

// q is in shared memory, and what all rows of a half see is known: the softmax's warps and warp 1 (named barrier 2).
template <int THREADS>
__device__ __forceinline__ void q_sync() { asm volatile("bar.sync 2, %0;" ::"n"(THREADS) : "memory"); }
// The 256 softmax threads (named barrier 1).
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

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

// A row tile: up to tile_rows rows of a sequence, and the blocks [k0, k1) that some of
// them see (one block if they see none: it leaves their zeros).
struct RowTile {
  int b, rt;  // b < 0: none
  int k0, k1;
};
// With X (rows see by their place) its rows see the first keys and a window.  What holds them is taken together: units (pages,
// or the blocks of a longer page) 0 .. firsts - 1, and `skip` units further on the rest of `units`; a block takes as many
// units as it has pages.  (With blocks of the window alone and of the first keys alone, ragged prompts with windows of 1000 keys
// and pages of 32 took 11 us more, of 103.)
struct SightTile : RowTile {
  int firsts, skip, units, pad;
};
template <bool X>
using Tile = std::conditional_t<X, SightTile, RowTile>;
// Room for the row tiles of T tokens in B sequences; those of a sequence that starts at row r0 stand from r0 * group /
// tile_rows + b on, so that sequences never meet.
__host__ __device__ inline long long row_tiles(const AttnArgs& a) {
  return (long long)a.b.T * a.group / tile_rows(a.c.D) + a.b.B;
}

// What a row tile with a head takes of the line: kRunUnits (start, end and the blocks at a mask's edge), and for each
// block kPairUnits, or kSingleUnits in a tile of at most 128 rows.  They stand for what these cost.  us with 30, 45, 60, 80 for
// a run: two chunks of 1300 causal tokens of 48 heads 123, 120, 127, 124; 64 drafts of 24 sequences 146, 140, 133, 136; ragged
// causal chunks at heads of 64 93, 92, 91, 94; 880 tokens against 27,280 keys 173, 170, 175, 182.  (A smaller tile does
// half the arithmetic, but asks for K and V as fast as a larger one would at twice the speed.)
constexpr int kPairUnits = 5, kSingleUnits = 4, kRunUnits = 60;
constexpr int kSightSingleUnits = 3;  // with X (trees of up to 47 drafts 40 us with 4, 38 with 3)
template <bool X>
__device__ __forceinline__ int tile_weight(const AttnArgs& a, const Seq& s, int rt) {
  const bool single = a.c.D <= 128 && s.n * a.group - rt * tile_rows(a.c.D) <= kHalfRows;
  return !single ? kPairUnits : X ? kSightSingleUnits : kSingleUnits;
}

constexpr int kFaultBytes = 16;
template <bool X>
struct Space {
  int* fault;  // a wait ran out: no row of the call is to be believed
  Tile<X>* tiles;
  Open* open;
  float2* ml;  // [2 G][rows of a tile]
  float4* o;   // [2 G][DP / 4][rows of a tile]: the rows side by side
};
template <int DP, bool X>
__host__ __device__ inline Space<X> space(const AttnArgs& a, int G) {
  Space<X> s;
  s.fault = (int*)a.workspace;
  s.tiles = (Tile<X>*)((char*)a.workspace + kFaultBytes);
  s.open = (Open*)(s.tiles + row_tiles(a));
  s.ml = (float2*)(s.open + G);
  s.o = (float4*)(s.ml + (size_t)2 * G * Cfg<DP>::kRows);
  return s;
}

// The row tiles of a call, a warp for each place.
constexpr int kPlanWarps = 4;
template <bool X>
__global__ void __launch_bounds__(32 * kPlanWarps)
    kv_chunk_plan_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ ChunkGeo geo) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, tile = tile_rows(a.c.D);
  const long long place = (long long)blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (place >= row_tiles(a)) return;
  Tile<X> t{};
  t.b = -1;
  for (int b0 = 0; b0 < a.b.B; b0 += 32) {
    Seq s{0, 0, 0};
    long long rt = 0;
    if (b0 + lane < a.b.B) {
      s = sequence<X>(a, b0 + lane, false);
      rt = place - ((long long)s.r0 * a.group / tile + b0 + lane);
    }
    const uint32_t mine = __ballot_sync(0xffffffffu, s.len > 0 && rt >= 0 && rt * tile < (long long)s.n * a.group);
    if (mine == 0) continue;
    const int from = __ffs(mine) - 1;
    t.b = b0 + from;
    t.rt = __shfl_sync(0xffffffffu, (int)rt, from);
    s.r0 = __shfl_sync(0xffffffffu, s.r0, from);
    s.n = __shfl_sync(0xffffffffu, s.n, from);
    s.len = __shfl_sync(0xffffffffu, s.len, from);
    t.k1 = blocks_of(geo, a.c.page_size, s.len);
    if constexpr (X) {
      // a window moves on with its tokens: the first one's begins, the last one's ends first keys and window of the tile
      const int row0 = t.rt * tile;
      const Sight from = sight(a, s, row0 / a.group), to = sight(a, s, (min(row0 + tile, s.n * a.group) - 1) / a.group);
      int c = to.c, lo = from.lo;
      const int hi = a.mask == kMaskTree ? s.len : to.hi;
      if (lo <= c) c = lo = 0;
      const bool pages = geo.parts == 1;
      auto unit = [&](int key) { return pages ? key / a.c.page_size : block_of_key(geo, a.c.page_size, key); };
      t.firsts = c > 0 ? unit(c - 1) + 1 : 0;
      t.skip = max(unit(lo), t.firsts) - t.firsts;
      t.units = unit(hi - 1) + 1 - t.skip;
      t.k0 = 0;
      t.k1 = pages ? (t.units + geo.pages - 1) / geo.pages : t.units;
    } else if (a.ranges) {
      int lo = 0x7fffffff, hi = 0;
      const int row0 = t.rt * tile, last = (min(row0 + tile, s.n * a.group) - 1) / a.group;
      for (int i = row0 / a.group + lane; i <= last; i += 32) {
        int x, y;
        seen_range(a, s.r0 + i, s.len, &x, &y);
        if (x < y) lo = min(lo, x), hi = max(hi, y);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      t.k0 = hi > 0 ? block_of_key(geo, a.c.page_size, lo) : 0;
      t.k1 = hi > 0 ? block_of_key(geo, a.c.page_size, hi - 1) + 1 : 1;
    }
    break;
  }
  if (lane == 0) space<64, X>(a, 0).tiles[place] = t;
  if (place == 0 && lane == 0) *space<64, X>(a, 0).fault = 0;
}

// A run: blocks [k0, k1) of one row tile and head.
struct alignas(16) Run {
  Seq s;
  int b, h, row0, cnt;
  int k0, k1;
  int first, last;           // of the tile's blocks [first, last)
  int blocks;                // k1 - k0; 0: the piece has no more runs
  int all_lo[2], all_hi[2];  // per half: keys that every row sees
  int odd_lo, odd_hi;        // first and last block with odd values (below) of keys that the sequence has
  uint32_t odd_some;         // bit j % 32: block j may be one
  ChunkGeo geo;              // the call's, for what has no registers for them
  int page_size;
  int firsts, skip, units;   // with X: the tile's
  int all_c[2];              // and all rows of a half see [0, all_c) too
};

// Where thread 0 stands on the line (in shared memory: the softmax has no register to spare).
struct alignas(16) Cursor {
  Piece pc;
  long long line, at;  // the next unit of the line, and of row tile i
  int i;
};

// The keys of block j's columns: columns [0, at_c) hold those from base_c on, [at_c, rows) those from base on (both less the
// column).
struct Columns {
  int base_c, base, at_c, rows;
  __device__ __forceinline__ int key(int column) const { return (column < at_c ? base_c : base) + column; }
};
template <bool X>
__device__ __forceinline__ Columns columns_of(const ChunkGeo& geo, int page_size, const Run* run, int j) {
  Columns k{0, 0, 0, 0};
  if (X && geo.parts == 1) {
    k.rows = geo.pages * page_size;
    k.base_c = j * k.rows;
    k.base = k.base_c + run->skip * page_size;
    k.at_c = min(max((run->firsts - j * geo.pages) * page_size, 0), k.rows);
  } else {
    block_keys(geo, page_size, j, &k.base, &k.rows);
  }
  return k;
}

// Keys that some row of a tile does not see: an infinity or a NaN (an odd value) among
// their values must not meet a weight of zero.  Such values leave the block here (V in
// `count` slots from the ring's number `at` on, read by a half's 128 threads), and
// the rows that see them get them at the end (what stands behind the end of the sequence
// is nobody's).  Where both halves' products read the
// slot, half 0 does this for both, ahead of its arrival and so of either product: no
// product reads a value while it changes.  Not inline but for windows and trees at
// heads of 64: the softmax's loop needs the registers (two chunks of 1300 causal
// tokens of 48 heads 127 us, 134 inline; ragged windows at heads of 64 89 and 85).
template <int DP, bool X>
constexpr bool kCleanInline = X && DP == 64;
template <typename T>
__device__ __forceinline__ uint32_t even32(uint32_t v) {
  return (odd16<T>(v) ? 0u : v & 0xffffu) | (odd16<T>(v >> 16) ? 0u : v & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ bool odd128(const uint4& v) {
  return odd32<T>(v.x) || odd32<T>(v.y) || odd32<T>(v.z) || odd32<T>(v.w);
}
// The rest of clean_values, where there are such values: they leave the block, and the run learns of those of the sequence.
template <typename T, int DP, bool X>
__device__ __forceinline__ void drop_values(uint8_t* ring, int at, int count, int thread, int block, Run* run) {
  using C = Cfg<DP>;
  const Columns k = columns_of<X>(run->geo, run->page_size, run, block);
  bool held = false;
  for (int u = at; u < at + count; ++u) {
    uint4* v = reinterpret_cast<uint4*>(ring + u % C::kValSlots * C::kValSlot);
    for (int e = thread; e < C::kValSlot / 16; e += kHalfRows) {
      const uint4 w = v[e];
      if (!odd128<T>(w)) continue;
      const int column = (e >> 3) & (kBlock - 1);  // 128 bytes a row of a box
      held |= column < k.rows && k.key(column) < run->s.len;
      v[e] = make_uint4(even32<T>(w.x), even32<T>(w.y), even32<T>(w.z), even32<T>(w.w));
    }
  }
  if (!held) return;
  atomicMin(&run->odd_lo, block);
  atomicMax(&run->odd_hi, block);
  atomicOr(&run->odd_some, 1u << (block & 31));
  __threadfence_block();
}
template <typename T, int DP, bool X>
__device__ __noinline__ void drop_values_apart(uint8_t* ring, int at, int count, int thread, int block, Run* run) {
  drop_values<T, DP, X>(ring, at, count, thread, block, run);
}
template <typename T, int DP, bool X>
__device__ __forceinline__ bool clean_values(uint8_t* ring, uint64_t* full, int at, int count, int thread, int block, Run* run,
                                             int* err) {
  using C = Cfg<DP>;
  constexpr int SV = C::kValSlots;
  bool odd = false;
  for (int u = at; u < at + count; ++u) {
    if (!wait_phase(&full[u % SV], (u / SV) & 1, err, kDevTimeoutFull)) return false;
    const uint4* v = reinterpret_cast<const uint4*>(ring + u % SV * C::kValSlot);
#pragma unroll 8
    for (int e = thread; e < C::kValSlot / 16; e += kHalfRows) odd |= odd128<T>(v[e]);
  }
  if (odd) {
    if constexpr (kCleanInline<DP, X>) drop_values_apart<T, DP, X>(ring, at, count, thread, block, run);
    else drop_values<T, DP, X>(ring, at, count, thread, block, run);
  }
  fence_proxy_async_smem();
  return true;
}
template <typename T, int DP, bool X>
__device__ __noinline__ bool clean_values_apart(uint8_t* ring, uint64_t* full, int at, int count, int thread, int block, Run* run,
                                                int* err) {
  return clean_values<T, DP, X>(ring, full, at, count, thread, block, run, err);
}

// Windows and trees: adds the odd values of a run's blocks to the rows that see them, to row `row` of the tile, which the
// thread has written as output, or as a part in `o`.  Called where the run is over: the softmax's loop needs the registers.
// What a row sees of 64 columns is found once for all channels, and a lane looks whether one of 32 keys has such a value (a
// chain of 1024 drafts with an infinity in the first and in the last takes 218 us, as without; with a walk up the tree for each
// key and 16 channels it took 5800.  24 trees of 64 drafts with NaN behind the sequences' ends 136, where those were walked for
// too 3100).  With ranges the softmax's threads do it, key by key, as they put out 16 channels: a range is soon looked up,
// and that loop loses 10 to 27% by how it is then compiled if they do not.
template <typename T, int DP>
__device__ __noinline__ void give_back(const AttnArgs& a, const Run* run, int row, float4* o, int me) {
  const Seq s = run->s;
  const ChunkGeo& geo = run->geo;
  const bool real = row < run->cnt;
  const int lane = threadIdx.x & 31, page_size = a.c.page_size, mine = real ? (run->row0 + row) / a.group : -1;
  const bool whole = run->k0 == run->first && run->k1 == run->last;
  T* const dst = real ? out_row<T>(a, s, run->h, run->row0 + row) : nullptr;
  float4* const part = o + ((2LL * me + (run->k0 == run->first ? 1 : 0)) * (DP / 4)) * Cfg<DP>::kRows + row;
  Sight v{0, 0, 0};
  if (real) v = sight(a, s, mine);
  const int* table = a.b.pages + run->b * a.b.page_stride;
  __syncwarp();
  Family kin = {};
  if (a.mask == kMaskTree) kin = family(a, s);
  const int odd_lo = run->odd_lo, odd_hi = run->odd_hi;
  for (int j = odd_lo; j <= odd_hi; ++j) {
    if (geo.parts > 1 && j == run->firsts) j += run->skip;  // (what lies between first keys and window is in no block)
    if (j > odd_hi || !((run->odd_some >> (j & 31)) & 1)) continue;
    const Columns k = columns_of<true>(geo, page_size, run, j);
    for (int c0 = 0; c0 < k.rows; c0 += 64) {
      uint32_t sees[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int col = c0 + 32 * w;
        const uint32_t firsts = low_bits(k.at_c - col);
        sees[w] = (sight_bits(v, k.base_c + col) & firsts) | (sight_bits(v, k.base + col) & ~firsts);
      }
      const int d0 = k.base + c0 - (s.len - s.n);
      if (a.mask == kMaskTree && d0 > -64) {
        uint64_t up = ancestors(a, s, kin, mine, max(d0, 0));
        if (d0 < 0) up <<= -d0;
        sees[0] |= (uint32_t)up, sees[1] |= (uint32_t)(up >> 32);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int col = c0 + 32 * w;
        if (!real) sees[w] = 0;
        sees[w] &= low_bits(k.rows - col);
        const uint32_t any = __reduce_or_sync(0xffffffffu, sees[w]);
        unsigned long long src = 0;
        bool odd = false;
        if ((any >> lane) & 1) {
          const int key = k.key(col + lane), page = kv_page(table, key, page_size, a.c.pages);
          if (page >= 0) {
            const T* p = (const T*)a.c.v + page * a.c.v_page + run->h * a.c.v_head + (key % page_size) * a.c.v_row;
            src = (unsigned long long)p;
            for (int c = 0; c < a.c.D; c += 8) odd |= odd128<T>(*reinterpret_cast<const uint4*>(p + c));
          }
        }
        const uint32_t odds = __ballot_sync(0xffffffffu, odd);
        for (int c = 0; c < a.c.D && odds; c += 8) {
          float sum[8] = {};
          bool some = false;
          for (uint32_t left = odds; left; left &= left - 1) {
            const int l = __ffs(left) - 1;
            const uint4 x = *reinterpret_cast<const uint4*>((const T*)__shfl_sync(0xffffffffu, src, l) + c);
            if (!((sees[w] >> l) & 1) || !odd128<T>(x)) continue;
            some = true;
            const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint16_t bits = (uint16_t)(words[e / 2] >> (16 * (e & 1)));
              if (odd16<T>(bits)) sum[e] += val<T>(*reinterpret_cast<const T*>(&bits));
            }
          }
          if (some) {
            for (int e = 0; e < 8; ++e) {
              if (sum[e] == 0.f) continue;
              if (!whole) (&part[(size_t)((c + e) / 4) * Cfg<DP>::kRows].x)[(c + e) & 3] += sum[e];
              else dst[c + e] = round_to<T>(val<T>(dst[c + e]) + sum[e]);
            }
          }
          __syncwarp();
        }
      }
    }
  }
}

template <typename T, int DP, bool X>
__global__ void __launch_bounds__(kThreads, 1)
    kv_chunk_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                    const __grid_constant__ AttnArgs a, const __grid_constant__ ChunkGeo geo) {
  using C = Cfg<DP>;
  constexpr int SK = C::kKeySlots, SV = C::kValSlots, S = SK + SV, ND = C::ND, kRows = C::kRows;
  constexpr bool kOne = C::kOne;
  constexpr int kSoftEnd = kOne ? 8 : 12;  // softmax warps are 4 up to this one
  // the only shared memory of the kernel, so it starts on a 1024-byte boundary, as the swizzled boxes must
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(2 * sizeof(Run) + sizeof(Cursor) + 8 * (2 * S + 15) + 8 + 128 + 16 <= 1024, "barriers and the run's description");
  uint8_t* sQ = smem;  // [half][64-channel box][128 rows]
  uint8_t *sK = sQ + C::kQ, *sV = sK + SK * C::kKeySlot;  // SK slots of K, SV of V; their barriers in this order
  uint64_t* full = reinterpret_cast<uint64_t*>(sV + SV * C::kValSlot);
  uint64_t* empty = full + S;
  uint64_t* s_full = empty + S;   // [2] a block's S of half t in TMEM
  uint64_t* s_free = s_full + 2;  // [2] 128 arrivals: it has been read
  uint64_t* p_full = s_free + 2;  // [half][P buffer] 128 arrivals: P_t in TMEM (and O_t rescaled)
  uint64_t* o_done = p_full + 4;  // [half][P buffer] O_t += P_t V_j complete
  uint64_t* done = o_done + 4;    // [2] all products issued by warp 1, and by warp 2, complete
  uint64_t* told = done + 2;      // the next run is described
  if (smem_u32(smem) & 1023) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) *space<DP, X>(a, gridDim.x).fault = 1;
    if (a.b.status) atomicCAS(a.b.status, 0, (int)kDevTimeoutFull);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(told + 1);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* hole = tmem_slot + 2;  // [32]: bit i of hole[c % 32]: page i of the c-th block is none of the cache's
  Run* runs = reinterpret_cast<Run*>((reinterpret_cast<uintptr_t>(hole + 32) + 15) & ~uintptr_t(15));  // [2]
  Cursor* cursor = reinterpret_cast<Cursor*>(runs + 2);
  float* half_ml = reinterpret_cast<float*>(cursor + 1);  // [2][128] reference and sum of half 1, handed to half 0

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = gridDim.x, me = blockIdx.x;
  const Space<X> ws = space<DP, X>(a, G);
  const int page_size = a.c.page_size;
  int* const err = a.b.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&s_free[t]), 128);
      mbar_init(smem_u32(&done[t]), 1);
    }
    for (int t = 0; t < 4; ++t) {
      mbar_init(smem_u32(&p_full[t]), 128);
      mbar_init(smem_u32(&o_done[t]), 1);
    }
    mbar_init(smem_u32(told), 1);
    *stop = 0;
    fence_mbar_init();
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
  }
  // rows of a slot that no box fills stay zero: their weights are zero, and 0 times a stray NaN would not be
  if (geo.pages * geo.box_rows < kBlock) {
    for (int i = threadIdx.x; i < (SK * C::kKeySlot + SV * C::kValSlot) / 16; i += kThreads)
      reinterpret_cast<uint4*>(sK)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan
  auto units = [&](const RowTile& t, int w) { return (long long)(kRunUnits + w * (t.k1 - t.k0)); };
  const Piece cut = cut_line<kThreads / 32, 1>((int)row_tiles(a), kLeast, reinterpret_cast<long long*>(half_ml), [&](int i) {
    const Tile<X> t = ws.tiles[i];
    return t.b < 0 ? 0 : a.c.heads * units(t, tile_weight<X>(a, sequence<X>(a, t.b, false), t.rt));
  });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // S at tS; half t's block number c (of all its blocks so far): P at p_at(t, c), its barriers number bar_of(t, c), phase
  // phase_of(c); O at tO + DP t.  With two P buffers a half's P V has a block's time more.
  constexpr int kTwoP = DP == 64 ? 1 : 0;
  const uint32_t tS = tmem, tO = tmem + (kTwoP ? 384 : 256);
  auto p_at = [&](int t, int c) { return tmem + 128 + (kTwoP ? 128 * t + 64 * (c & 1) : 64 * t); };
  auto bar_of = [&](int t, int c) { return 2 * t + (kTwoP ? c & 1 : 0); };
  auto phase_of = [&](int c) { return (kTwoP ? c >> 1 : c) & 1; };

  int it = 0;                 // blocks so far (all roles count alike)
  int ns[2] = {0, 0};         // blocks of each half so far

  // The piece's next run (thread 0).
  auto describe = [&](Run* run) {
    const Piece& pc = cursor->pc;
    long long line = cursor->line, at = cursor->at;
    int i = cursor->i;
    run->blocks = 0;
    while (line < pc.end && run->blocks == 0) {
      Tile<X> t = ws.tiles[i];
      Seq s{0, 0, 0};
      long long n = 0;  // units of a head
      int w = 0;
      for (;;) {
        if (t.b >= 0) {
          s = sequence<X>(a, t.b, false);
          w = tile_weight<X>(a, s, t.rt);
          n = units(t, w);
          if (at < a.c.heads * n) break;
          at -= a.c.heads * n;
        }
        if (++i >= row_tiles(a)) return;  // (the tables changed under the call)
        t = ws.tiles[i];
      }
      const int h = (int)quotient(at, n), u0 = (int)(at - h * n), u1 = (int)min(n, u0 + (pc.end - line));
      run->s = s;
      run->b = t.b;
      run->h = h;
      run->row0 = t.rt * kRows;
      run->cnt = min(kRows, s.n * a.group - run->row0);
      run->first = t.k0;
      run->last = t.k1;
      // a block belongs to the piece that holds its last unit
      run->k0 = t.k0 + max(0, u0 - kRunUnits) / w;
      run->k1 = t.k0 + max(0, u1 - kRunUnits) / w;
      run->blocks = run->k1 - run->k0;
      for (int t = 0; t < 2; ++t) {
        run->all_lo[t] = 0;
        run->all_hi[t] = 0x7fffffff;
      }
      run->odd_lo = 0x7fffffff;
      run->odd_hi = -1;
      run->odd_some = 0;
      run->geo = geo;
      run->page_size = page_size;
      if constexpr (X) {
        run->all_c[0] = run->all_c[1] = 0x7fffffff;
        run->firsts = t.firsts;
        run->skip = t.skip;
        run->units = t.units;
      }
      if (run->k0 == t.k0 && run->k1 > t.k0 && run->k1 < t.k1)
        ws.open[me] = Open{pc.holder(line + n - u0 - 1) - me, h, run->row0, run->cnt, s, 0};
      at += u1 - u0;
      line += u1 - u0;
    }
    cursor->line = line;
    cursor->at = at;
    cursor->i = i;
  };
  if (threadIdx.x == 0) {
    ws.open[me].parts = 0;
    cursor->pc = cut;
    cursor->line = cut.beg;
    cursor->at = cut.at;
    cursor->i = cut.b;
    describe(&runs[0]);
  }
  __syncthreads();

  // The first V of the next run, and q, come while this one ends: q in its room from the last Q K on (by warp 1), where the
  // halves do not need that for their sums and its rows can be copied as they are.  880 tokens against 27,280 keys take 175 us
  // with q ahead, 202 without; with X a window of 9 latent frames 92 and 87; at heads of 64 ragged causal chunks 107 and 92
  // (too little time to fill).
  constexpr bool kValuesAhead = DP > 64, kAheadOfRun = DP > 64 && !X;
  const bool q_plain = a.scale_log2 > 0.f && ((uintptr_t)a.q & 15) == 0 && (a.q_t & 7) == 0 && (a.q_h & 7) == 0;
  bool q_came = false;
  // where row `row` of a run has its q (-1: the tile has no such row)
  constexpr int CH = DP / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows that a warp fetches in a step
  auto q_of = [&](const Run* run, int row) {
    if (row >= run->cnt) return -1LL;
    const int t = (run->row0 + row) / a.group, g = run->row0 + row - t * a.group;
    return (long long)(run->s.r0 + t) * a.q_t + (long long)(run->h * a.group + g) * a.q_h;
  };

  for (int r = 0; runs[r & 1].blocks > 0; ++r) {
    Run* const run = &runs[r & 1];
    const int h = run->h, row0 = run->row0, cnt = run->cnt, k0 = run->k0, k1 = run->k1;
    const Seq s = run->s;
    const bool split = !kOne && cnt <= kHalfRows;  // both halves hold the same rows and take the blocks in turn
    const int half = (warp - 4) >> 2;     // softmax warps
    // softmax threads: the row (TMEM lane) in their half, and the keys that it sees
    const int hrow = 32 * (warp & 3) + lane;
    const int row = (split ? 0 : half * kHalfRows) + hrow;
    const bool softmax = warp >= 4 && warp < kSoftEnd, real = softmax && row < cnt;
    int lo = 0, hi = 0x40000000;  // rows past the tile's see everything: they need no mask
    int first_keys = 0;           // with X: [0, first_keys) too, and drafts
    if (softmax) {
      if (real) {
        if constexpr (X) {
          const Sight v = sight(a, s, (row0 + row) / a.group);
          first_keys = v.c, lo = v.lo, hi = v.hi;
          atomicMin(&run->all_c[half], first_keys);
        } else {
          seen_range(a, s.r0 + (row0 + row) / a.group, s.len, &lo, &hi);
        }
        if (lo > 0) atomicMax(&run->all_lo[half], lo);
        atomicMin(&run->all_hi[half], hi);
      }
    }
    if (softmax && !q_came) {
      // q is negated for a negative scale (the maximum is then that of q . k) and cleared for a scale of zero
      // (whose product with a hidden key's -inf is none).  A warp fetches its 32 rows whole, side by side, and stores
      // them when all are on their way: lane i knows where row i is.
      const bool flip = a.scale_log2 < 0.f;
      const long long at = q_of(run, row);
      const int c = lane % CH;
      uint8_t* const q = sQ + (half * ND + (c >> 3)) * kBoxBytes;
      const bool whole16 = ((uintptr_t)a.q & 15) == 0 && (a.q_t & 7) == 0 && (a.q_h & 7) == 0;
      constexpr int kBatch = CH < 16 ? CH : 16;  // steps whose loads are all on their way before the first is stored
#pragma unroll 1
      for (int i0 = 0; i0 < CH; i0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const long long from = __shfl_sync(0xffffffffu, at, (i0 + i) * RPI + lane / CH);
          v[i] = make_uint4(0, 0, 0, 0);
          if (from >= 0 && c * 8 < a.c.D && a.scale_log2 != 0.f) {
            const T* src = (const T*)a.q + from + c * 8;
            if (whole16) {
              v[i] = *reinterpret_cast<const uint4*>(src);
            } else {
              const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
              v[i] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                                e[6] | (uint32_t)e[7] << 16);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int to = 32 * (warp & 3) + (i0 + i) * RPI + lane / CH;
          const uint32_t sign = flip ? 0x80008000u : 0u;
          *reinterpret_cast<uint4*>(q + to * 128 + (((c & 7) ^ (to & 7)) << 4)) =
              make_uint4(v[i].x ^ sign, v[i].y ^ sign, v[i].z ^ sign, v[i].w ^ sign);
        }
      }
      fence_proxy_async_smem();
    }
    if (warp == 1 && q_came) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
    }
    if (softmax || warp == 1) q_sync<kOne ? 160 : 288>();
    q_came = kAheadOfRun && q_plain && !split;  // (of the next run)
    const int j0 = k0, nb = k1 - k0;
    // blocks of each half
    const int nh[2] = {split ? (nb + 1) / 2 : nb, kOne ? 0 : split ? nb / 2 : nb};
    const int boxes = (a.c.D + 63) / 64;                                       // of a page's rows
    const int pk = kOne ? boxes : 1, pv = kOne ? (boxes + 1) / 2 : 1;  // slots of a block
    bool ok = true;

    // -------------------------------------------------- loads: K, and V
    // blocks [n0, n1) of a run whose first block is the it-th
    auto loads = [&](auto which, const Run* run, int it, int n0, int n1) {
      constexpr bool ofK = decltype(which)::value;
      const int h = run->h, o0 = run->k0 + n0, j0 = X && geo.parts > 1 && o0 >= run->firsts ? o0 + run->skip : o0;
      const CUtensorMap* map = ofK ? &mapK : &mapV;
      const int* table = a.b.pages + run->b * a.b.page_stride;
      const int held = (run->s.len + page_size - 1) / page_size;  // pages of the sequence
      const int box = geo.parts == 1 ? geo.pages * geo.box_rows * 128 : kBoxBytes;  // bytes
      constexpr int per = ofK ? C::kKeyBoxes : C::kValBoxes, slot_bytes = ofK ? C::kKeySlot : C::kValSlot;
      const int pb = ofK ? pk : pv;
      uint8_t* const ring = ofK ? sK : sV;
      // All counted along: a division here would queue behind the softmax's exponentials.  The lane's page of block
      // j: its place `idx` in the table and the rows `off` of it that come first; asked for two blocks ahead.
      int idx = geo.parts == 1 ? j0 * geo.pages + lane : j0 / geo.parts, part = geo.parts == 1 ? 0 : j0 - idx * geo.parts;
      int idx2 = idx, part2 = part;
      const int wide = lane < geo.pages ? held : 0;
      // With X the lane's page is a unit: its place in the table comes from it.  Of a longer page: blocks to the one behind
      // the first keys, and where that one is.
      int left = 0, left2 = 0, idx_to = 0, part_to = 0;
      const int firsts = X ? run->firsts : 0, skip = X ? run->skip : 0, limit = X && geo.parts == 1 ? (wide ? run->units : 0) : wide;
      if constexpr (X) {
        left = left2 = firsts - o0;
        if (geo.parts > 1 && left > 0) {
          idx_to = (firsts + skip) / geo.parts;
          part_to = firsts + skip - idx_to * geo.parts;
        }
      }
      auto advance = [&](int& i, int& p, int& left) {
        if (geo.parts == 1) i += geo.pages;
        else if (X && --left == 0) i = idx_to, p = part_to;
        else if (++p == geo.parts) p = 0, ++i;
      };
      auto place = [&](int i) { return X && geo.parts == 1 && i >= firsts ? i + skip : i; };
      auto entry = [&](int n) {
        const int e = n < n1 && idx2 < limit ? table[place(idx2)] : (int)a.c.pages;  // past the cache, which reads as zeros
        advance(idx2, part2, left2);
        return e;
      };
      int page = entry(n0), next = entry(n0 + 1);
      constexpr int slots = ofK ? SK : SV, first = ofK ? 0 : SK;
      int slot = (it + n0) * pb % slots, lap = (it + n0) * pb / slots;
      for (int n = n0; n < n1 && ok; ++n) {
        const int after = entry(n + 2);
        const int off = part * kBlock;
        const bool none = idx < limit && (page < 0 || page >= a.c.pages);
        advance(idx, part, left);
        if (none) {
          page = (int)a.c.pages;
          if (err) atomicCAS(err, 0, (int)kDevBadPage);
        }
        if (ofK) {
          const uint32_t nones = __ballot_sync(0xffffffffu, none);
          if (lane == 0) hole[(it + n) & 31] = nones;
        }
        const bool withheld = ofK && it + n + 1 == a.stall_at1;  // (the failure self test)
        for (int u = 0; u < pb && ok; ++u) {
          const int count = kOne ? min(per, boxes - u * per) : per;  // (each has a channel: D > DP - 64)
          int good = 1;
          if (lane == 0) {
            if (lap > 0) good = wait_phase(&empty[first + slot], (lap - 1) & 1, err, kDevTimeoutEmpty);
            if (*stop) good = 0;
            if (good && !withheld) mbar_arrive_expect_tx(smem_u32(&full[first + slot]), count * box);
          }
          ok = __shfl_sync(0xffffffffu, good, 0);
          if (!ok) break;
          if (lane < geo.pages && !withheld) {  // one box per lane, of the page that the lane holds
            int c[3];
            c[geo.dim_row] = off;
            c[geo.dim_head] = h;
            c[geo.dim_page] = page;
            const uint32_t d = smem_u32(ring + slot * slot_bytes) + lane * geo.box_rows * 128;
#pragma unroll
            for (int v = 0; v < per; ++v)
              if (v < count)
                tma_load_4d(d + v * kBoxBytes, map, smem_u32(&full[first + slot]), 64 * (u * per + v), c[0], c[1], c[2]);
          }
          if (++slot == slots) slot = 0, ++lap;
        }
        page = next;
        next = after;
      }
      if (!ok) *stop = 1;
    };
    if (warp == 0) {
      // K of the first blocks of the next run is asked for before this one ends (as many as surely find room: their
      // slots held blocks of this run or an earlier one, whose products wait for nothing of this warp)
      const int kAhead = SK / pk;
      loads(std::true_type(), run, it, r > 0 ? min(nb, kAhead) : 0, nb);
      Run* const next = &runs[(r + 1) & 1];
      if (lane == 0) {
        describe(next);
        mbar_arrive(smem_u32(told));
      }
      __syncwarp();
      if (ok && next->blocks > 0) loads(std::true_type(), next, it + nb, 0, min(next->blocks, kAhead));
    } else if (warp == 3) {
      // as with K: the slots that V of the next run's first blocks takes held blocks whose products need nothing of this warp
      const int kAhead = kValuesAhead ? SV / pv : 0;
      loads(std::false_type(), run, it, r > 0 ? min(nb, kAhead) : 0, nb);
      const Run* const next = &runs[(r + 1) & 1];
      if (kValuesAhead && ok && !__all_sync(0xffffffffu, wait_phase(told, r & 1, err, kDevTimeoutFull))) {
        ok = false;
        *stop = 1;
      }
      if (kValuesAhead && ok && next->blocks > 0) loads(std::false_type(), next, it + nb, 0, min(next->blocks, kAhead));
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------- products: Q K, and P V
      // A whole warp walks the steps (what it computes stays in uniform
      // registers, which the instructions take their operands from); one thread
      // issues.  The steps alternate between the halves: step g is half g % 2's
      // block number g / 2.  The two kinds of product touch nothing in common, so
      // each warp goes by its own barriers.
      const int dn = (a.c.D + 15) / 16;  // k steps of S, N / 16 of O
      const bool one = elect();
      const bool turns = !split && !kOne;  // both halves take every block
      const int steps = turns ? 2 * nb : nb;
      if (warp == 1) {
        const uint32_t idS = idesc(Pack<T>::kFormat, false, kBlock);
        const uint32_t q0 = desc_k(smem_u32(sQ)), kd0 = desc_k(smem_u32(sK));
        int slot = it * pk % SK, phase = (it * pk / SK) & 1;
        uint32_t there = 0;  // the block's K (its first slot) is known to be there (asked a step ahead)
        for (int g = 0; g < steps; ++g) {
          const int t = kOne ? 0 : g & 1;
          const bool starts = !turns || t == 0, ends = !turns || t == 1;  // the block's first and last step
          if (starts && !__all_sync(0xffffffffu, there)) ok = wait_phase(&full[slot], phase, err, kDevTimeoutFull);
          // the S buffer, once the step that used it last (the half's own, or the other's) has been read
          if (kOne) {
            if (g > 0 && ok) ok = wait_phase(&s_free[0], (ns[0] + g - 1) & 1, err, kDevTimeoutAccum);
          } else {
            if (g > 0 && ok) ok = wait_phase(&s_free[t ^ 1], (ns[t ^ 1] + ((g - 1) >> 1)) & 1, err, kDevTimeoutAccum);
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t q = q0 + t * (ND * kBoxBytes >> 4), s_at = tS;
          for (int u = 0; u < pk; ++u) {
            if (kOne && u > 0) {
              ok = wait_phase(&full[slot], phase, err, kDevTimeoutFull);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t k = kd0 + slot * (C::kKeySlot >> 4), qu = q + u * (kBoxBytes >> 4);
            if (one) {
#pragma unroll
              for (int e = 0; e < 4 * C::kKeyBoxes; ++e)
                if (4 * u + e < dn)
                  umma_ss(s_at, qu + (e >> 2) * (kBoxBytes >> 4) + 2 * (e & 3), k + (e >> 2) * (kBoxBytes >> 4) + 2 * (e & 3),
                          idS, u > 0 || e > 0);
              if (u == pk - 1) umma_commit(smem_u32(&s_full[t]));
              if (ends) umma_commit(smem_u32(&empty[slot]));
            }
            if (ends && ++slot == SK) slot = 0, phase ^= 1;
          }
          if (!ok) break;
          if (ends) there = g + 1 < steps && ask_phase(&full[slot], phase);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (kAheadOfRun && ok && q_came) {
          const int t = turns ? 1 : kOne ? 0 : (steps - 1) & 1;  // the last step's half
          ok = wait_phase(told, r & 1, err, kDevTimeoutFull);
          if (ok) ok = wait_phase(&s_full[t], (ns[t] + nh[t] - 1) & 1, err, kDevTimeoutAccum);
          ok = __all_sync(0xffffffffu, ok);
          const Run* const next = &runs[(r + 1) & 1];
          if (ok && next->blocks > 0) {
            // the products that read q are complete
            const bool twice = !kOne && next->cnt <= kHalfRows;  // the same rows for both halves
            const int c = lane % CH;
#pragma unroll 1
            for (int w = 0; w < kRows / 32; ++w) {
              const long long at = q_of(next, 32 * (twice ? w & 3 : w) + lane);
              const uint32_t q = smem_u32(sQ) + ((w >> 2) * ND + (c >> 3)) * kBoxBytes;
#pragma unroll 4
              for (int i = 0; i < CH; ++i) {
                const int from_row = i * RPI + lane / CH, to = 32 * (w & 3) + from_row;
                const long long from = __shfl_sync(0xffffffffu, at, from_row);
                const bool take = from >= 0 && c * 8 < a.c.D;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q + to * 128 + (((c & 7) ^ (to & 7)) << 4)),
                             "l"((const T*)a.q + (take ? from + c * 8 : 0)), "r"(take ? 16 : 0)
                             : "memory");
              }
            }
          }
        }
      } else {
        const uint32_t vd0 = desc_v(smem_u32(sV)), id0 = idesc(Pack<T>::kFormat, true, 16 * min(4 * C::kValBoxes, dn));
        int slot = it * pv % SV, phase = (it * pv / SV) & 1;
        uint32_t there = 0;
        for (int g = 0; g < steps; ++g) {
          const int t = kOne ? 0 : g & 1, i = kOne ? g : g >> 1;
          const bool starts = !turns || t == 0, ends = !turns || t == 1;
          if (starts && !__all_sync(0xffffffffu, there)) ok = wait_phase(&full[SK + slot], phase, err, kDevTimeoutFull);
          const int c = ns[t] + i;
          if (ok) ok = wait_phase(&p_full[bar_of(t, c)], phase_of(c), err, kDevTimeoutAccum);
          if (!ok) break;
          tc_fence_after();
          for (int u = 0; u < pv; ++u) {
            if (kOne && u > 0) {
              ok = wait_phase(&full[SK + slot], phase, err, kDevTimeoutFull);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t v = vd0 + slot * (C::kValSlot >> 4), p = p_at(t, c);
            const uint32_t idO = u == 0 ? id0 : idesc(Pack<T>::kFormat, true, 16 * (dn - 4 * C::kValBoxes));
            if (one) {
#pragma unroll
              for (int e = 0; e < kBlock / 16; ++e) umma_ts(tO + DP * t + 64 * C::kValBoxes * u, p + 8 * e, v + 128 * e, idO, i > 0 || e > 0);
              if (u == pv - 1) umma_commit(smem_u32(&o_done[bar_of(t, c)]));
              if (ends) umma_commit(smem_u32(&empty[SK + slot]));
            }
            if (ends && ++slot == SV) slot = 0, phase ^= 1;
          }
          if (!ok) break;
          if (ends) there = g + 1 < steps && ask_phase(&full[SK + slot], phase);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) *stop = 1;
    } else if (softmax) {
      // -------------------------------------------------------- softmax, output
      const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t myS = tS + lane_off, myO = tO + DP * half + lane_off;
      const float sc = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
      const int n0 = ns[half], mine = nh[half], step = split ? 2 : 1;
      const int all_lo = run->all_lo[half], all_hi = run->all_hi[half];
      float m = -INFINITY, l = 0.f;
      float ref = -Pack<T>::kBias;  // what the weights are relative to: m, or 0 while it is -inf
      // Blocks [plain_lo, plain_hi) hold keys that all rows of this half see in all
      // their columns, but for the last part of a long page: `behind` parts come
      // after the block in its page.
      int plain_lo = 0x7fffffff, plain_hi = 0, behind = 1;
      int plain_first = 0;  // with X blocks [0, plain_first) do too
      const bool tails = geo.parts > 1 ? page_size % kBlock != 0 : geo.pages * page_size != kBlock;
      // Where both halves take every block, half 0, whose product comes first, cleans a block's values (below) for both:
      // its blocks are plain if all rows of the tile see them.
      const bool turns = !split && !kOne, cleans = !turns || half == 0;
      if (mine > 0 && !(geo.parts == 1 && tails)) {
        const int p_lo = turns && cleans ? max(all_lo, run->all_lo[1]) : all_lo;
        const int p_hi = turns && cleans ? min(all_hi, run->all_hi[1]) : all_hi;
        if (X && geo.parts == 1) {
          const int c = min(turns && cleans ? min(run->all_c[0], run->all_c[1]) : run->all_c[half], s.len);
          plain_lo = max((p_lo + page_size - 1) / page_size - run->skip, run->firsts);
          plain_lo = (plain_lo + geo.pages - 1) / geo.pages;
          plain_hi = max(min(p_hi, s.len) / page_size - run->skip, 0) / geo.pages;
          plain_first = c / page_size / geo.pages;
        } else {
          plain_lo = p_lo > 0 ? block_of_key(geo, page_size, p_lo - 1) + 1 : 0;
          plain_hi = block_of_key(geo, page_size, min(p_hi, s.len));
          if constexpr (X) {
            const int c = turns && cleans ? min(run->all_c[0], run->all_c[1]) : run->all_c[half];
            plain_first = block_of_key(geo, page_size, min(c, s.len));
          }
        }
      }
      // with X, the block at hand: the tile's number j0 (+ 1) of it, in a longer page its own, and the first number behind the gap
      // if that is still ahead
      int at = j0 + (split ? half : 0), gap = 0x7fffffff;
      if (X && geo.parts > 1) {
        if (at >= run->firsts) at += run->skip;
        else gap = run->firsts;
      }
      if (tails) behind = geo.parts - 1 - at % geo.parts;
      // A block's values are cleaned behind its weights, when S has left the registers, and ahead of the barrier that the products
      // wait for; with ranges and heads of 64 ahead of the weights (880 tokens against 27,280 keys 135 us, 139 behind them).
      constexpr bool kCleanFirst = !X && DP == 64;
      uint32_t s_there = 0;  // S of block i is known to be there
      for (int i = 0; i < mine; ++i) {
        const int o = j0 + (split ? 2 * i + half : i), j = X ? at : o;
        const bool inside = (j >= plain_lo && j < plain_hi) || (X && j < plain_first), plain = inside && behind != 0;
        if (tails && geo.parts > 1) behind = behind >= step ? behind - step : behind - step + geo.parts;
        if constexpr (X) {
          at += step;
          if (at >= gap) {  // (once: the gap is behind it then)
            at += run->skip;
            gap = 0x7fffffff;
            if (tails) behind = geo.parts - 1 - at % geo.parts;
          }
        }
        const int c = n0 + i;
        // with X, in a block that is not plain: the columns that the row sees (found ahead of S, which fills the registers)
        uint32_t vis[X ? 4 : 1];
        bool hidden = false;  // some row does not see some key of the block, whose values this half cleans
        if constexpr (X) {
          if (__builtin_expect(!plain, 0)) {
            // columns [0, at_c) are keys from base_c on, those behind them from base on (both less the column)
            int base_c = 0, base = 0, at_c = 0, rows = page_size - (geo.parts - 1) * kBlock;  // inside: the last part of a page
            if (!inside) {
              if (geo.parts == 1) {
                rows = geo.pages * page_size;
                base_c = j * rows;
                base = base_c + run->skip * page_size;
                at_c = min(max((run->firsts - j * geo.pages) * page_size, 0), rows);
              } else {
                block_keys(geo, page_size, j, &base, &rows);
              }
              const int c_all = min(run->all_c[0], run->all_c[1]), lo_all = max(run->all_lo[0], run->all_lo[1]),
                        hi_all = min(run->all_hi[0], run->all_hi[1]);
              auto all_see = [&](int k0, int k1) { return k0 >= k1 || k1 <= c_all || (k0 >= lo_all && k1 <= hi_all); };
              hidden = cleans && !(all_see(base_c, base_c + at_c) && all_see(base + at_c, base + rows));
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t firsts = low_bits(at_c - 32 * w);
              const Sight v{first_keys, lo, hi};
              vis[w] = inside ? ~0u : (sight_bits(v, base_c + 32 * w) & firsts) | (sight_bits(v, base + 32 * w) & ~firsts);
            }
            const int d0 = base - (s.len - s.n);
            if (a.mask == kMaskTree && !inside && d0 + kBlock > 0) {
              const Family kin = family(a, s);
#pragma unroll 1
              for (int v = 0; v < 2; ++v) {
                const int from = d0 + 64 * v;
                if (from <= -64) continue;
                uint64_t bits = ancestors(a, s, kin, real ? (row0 + row) / a.group : -1, max(from, 0));
                if (from < 0) bits <<= -from;
                if (v == 0) vis[0] |= (uint32_t)bits, vis[1] |= (uint32_t)(bits >> 32);
                else vis[2] |= (uint32_t)bits, vis[3] |= (uint32_t)(bits >> 32);
              }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) vis[w] &= low_bits(rows - 32 * w);
          }
        }
        // Cleans the block's values.  The lap of the ring before this block's has to be known to be there: the P V before the last
        // one of this half is, which is enough where both halves take all blocks and a block one slot.
        auto clean = [&] {
          if (ok && i > 0 && (split || kOne)) ok = wait_phase(&o_done[bar_of(half, c - 1)], phase_of(c - 1), err, kDevTimeoutAccum);
          if constexpr (kCleanInline<DP, X>) ok = ok && clean_values<T, DP, X>(sV, full + SK, (it + o - j0) * pv, pv, hrow, j, run, err);
          else ok = ok && clean_values_apart<T, DP, X>(sV, full + SK, (it + o - j0) * pv, pv, hrow, j, run, err);
          return ok = __all_sync(0xffffffffu, ok);
        };
        if (!__all_sync(0xffffffffu, s_there)) ok = wait_phase(&s_full[half], (n0 + i) & 1, err, kDevTimeoutAccum);
        __syncwarp();
        tc_fence_after();
        const uint32_t nones = hole[(it + o - j0) & 31];
        float x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(myS + 32 * c, x[c]);
        // P's room is free once its last P V is complete (as is O then, with one P)
        const int held = c - 1 - kTwoP;
        const uint32_t o_there = i > kTwoP ? ask_phase(&o_done[bar_of(half, held)], phase_of(held)) : 1u;
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&s_free[half]));
        if (__builtin_expect(!plain || nones != 0, 0)) {
          if constexpr (X) {
            if (plain) vis[0] = vis[1] = vis[2] = vis[3] = ~0u;
            const int per = geo.parts == 1 ? page_size : kBlock;
            for (uint32_t left = nones; left; left &= left - 1) {  // pages that the cache does not have
              const int p0 = (__ffs(left) - 1) * per;
#pragma unroll
              for (int w = 0; w < 4; ++w) vis[w] &= ~(low_bits(p0 + per - 32 * w) & ~low_bits(p0 - 32 * w));
            }
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (!__all_sync(0xffffffffu, vis[w] == ~0u)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((vis[w] >> e) & 1)) x[w][e] = -INFINITY;
              }
          } else {
            // columns [d0, d1) are keys of this row, [u0, u1) of all rows of this half; in the last part of a page that all
            // see, the page's rows (without block_keys' division)
            int d0 = 0, d1 = plain ? kBlock : page_size - (geo.parts - 1) * kBlock, u0 = d0, u1 = d1;
            if (!inside) {
              int base, rows;
              block_keys(geo, page_size, j, &base, &rows);
              d0 = lo - base, d1 = min(rows, hi - base);
              u0 = all_lo - base, u1 = min(rows, all_hi - base);
              if (cleans) hidden = base < max(run->all_lo[0], run->all_lo[1]) || base + rows > min(run->all_hi[0], run->all_hi[1]);
            }
            // by groups of 16 columns, if some row does not see them all
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (u0 > 16 * q || u1 < 16 * q + 16) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (16 * q + e < d0 || 16 * q + e >= d1) x[q >> 1][16 * (q & 1) + e] = -INFINITY;
              }
            const int per = geo.parts == 1 ? page_size : kBlock;
            for (uint32_t left = nones; left; left &= left - 1) {
              const int p0 = (__ffs(left) - 1) * per;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (32 * c + e >= p0 && 32 * c + e < p0 + per) x[c][e] = -INFINITY;
            }
            if (kCleanFirst && hidden && !clean()) break;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = x[c][0];
#pragma unroll
          for (int e = 1; e < 31; e += 2) mx[c] = max3(mx[c], x[c][e], x[c][e + 1]);
          mx[c] = fmaxf(mx[c], x[c][31]);
        }
        const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        if (__builtin_expect(__any_sync(0xffffffffu, mb > m + kSlack || !o_there || !ok), 0)) {
          if (ok && i > 0) ok = wait_phase(&o_done[bar_of(half, c - 1)], phase_of(c - 1), err, kDevTimeoutAccum);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          float alpha = 1.f;
          if (mb > m + kSlack) {
            alpha = weight(m, mb);
            m = mb;
            ref = m - Pack<T>::kBias;
          }
          l *= alpha;
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < DP / 16; ++c) {
              uint32_t r[16];
              tmem_ld16(myO + 16 * c, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st16(myO + 16 * c, r);
            }
            tmem_st_wait();
          }
        }
        // the P V that read P's room last was seen complete (asked ahead, or awaited above): its reads come before the stores
        tc_fence_after();
        const float2 sc2 = make_float2(sc, sc), nr2 = make_float2(-ref, -ref);
        const uint32_t myP = p_at(half, c) + lane_off;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 e = fma2(make_float2(x[q][2 * k], x[q][2 * k + 1]), sc2, nr2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[k & 1] = add2(sum[k & 1], e);
            p[k] = Pack<T>::two(e.x, e.y);
          }
          tmem_st16(myP + 16 * q, p);
        }
        tmem_st_wait();
        if (!kCleanFirst && __builtin_expect(hidden, 0) && !clean()) break;
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[bar_of(half, c)]));
        s_there = ask_phase(&s_full[half], (n0 + i + 1) & 1);
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      }
      if (ok && mine > 0)
        ok = __all_sync(0xffffffffu,
                        wait_phase(&o_done[bar_of(half, n0 + mine - 1)], phase_of(n0 + mine - 1), err, kDevTimeoutAccum));
      if (!ok) *stop = 1;
      tc_fence_after();
      const bool whole = k0 == run->first && k1 == run->last;
      const long long part = 2LL * me + (k0 == run->first ? 1 : 0);
      // Both halves' rows are the same: half 1 hands its sums to half 0, through
      // the room of q (which no MMA needs any more).
      float4* const other = reinterpret_cast<float4*>(sQ);  // [DP / 4][128 rows]
      float f0 = 1.f, f1 = 0.f;                             // weights of the halves' sums
      if (split) {
        softmax_sync();
        if (half == 1) {
          half_ml[hrow] = ref;
          half_ml[kHalfRows + hrow] = l;
#pragma unroll 1
          for (int c = 0; c < DP / 16 && mine > 0; ++c) {
            uint32_t r[16];
            tmem_ld16(myO + 16 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              other[(4 * c + e) * kHalfRows + hrow] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                                                 __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
          }
        }
        softmax_sync();
        if (half == 0 && nh[1] > 0 && half_ml[kHalfRows + hrow] != 0.f) {
          const float r1 = half_ml[hrow], l1 = half_ml[kHalfRows + hrow];
          if (l == 0.f) {
            f0 = 0.f;
            f1 = 1.f;
            ref = r1;
            l = l1;
          } else {
            const float to = fmaxf(ref, r1);
            f0 = weight(ref, to);
            f1 = weight(r1, to);
            l = l * f0 + l1 * f1;
            ref = to;
          }
        }
      }
      if (!split || half == 0) {
        const float rl = l == 0.f ? 0.f : 1.f / l;
        const int odd_lo = max(run->odd_lo, j0), odd_hi = min(run->odd_hi, k1 - 1);
        T* dst = real ? out_row<T>(a, s, h, row0 + row) : nullptr;
#pragma unroll 1
        for (int c = 0; c < DP / 16; ++c) {
          uint32_t r[16];
          __syncwarp();
          tmem_ld16(myO + 16 * c, r);
          tmem_ld_wait();
          float v[16];
          // (what TMEM holds for a row that saw nothing, or a channel past D, is nobody's)
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = mine > 0 && l != 0.f && 16 * c < a.c.D && f0 != 0.f ? __uint_as_float(r[e]) * f0 : 0.f;
          if (f1 != 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 o = other[(4 * c + e) * kHalfRows + hrow];
              if (16 * c < a.c.D) {
                v[4 * e] += o.x * f1;
                v[4 * e + 1] += o.y * f1;
                v[4 * e + 2] += o.z * f1;
                v[4 * e + 3] += o.w * f1;
              }
            }
          }
          if (!X && __builtin_expect(odd_lo <= odd_hi && real, 0)) {
            const int* table = a.b.pages + run->b * a.b.page_stride;
            int k_lo, k_hi, kr;
            block_keys(geo, page_size, odd_lo, &k_lo, &kr);
            block_keys(geo, page_size, odd_hi, &k_hi, &kr);
            k_hi += kr;
            for (int k = max(lo, k_lo); k < min(hi, k_hi); ++k) {
              const int page = kv_page(table, k, page_size, a.c.pages);
              if (page < 0) continue;
              const T* src = (const T*)a.c.v + page * a.c.v_page + h * a.c.v_head + (k % page_size) * a.c.v_row;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (16 * c + e < a.c.D && odd16<T>(reinterpret_cast<const uint16_t*>(src)[16 * c + e]))
                  v[e] += val<T>(src[16 * c + e]);
            }
          }
          if (real && !whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              ws.o[(part * (DP / 4) + 4 * c + e) * kRows + row] =
                  make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          } else if (real) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = Pack<T>::two(v[2 * e] * rl, v[2 * e + 1] * rl);
            const int left = a.c.D - 16 * c;
            if (((uintptr_t)dst & 15) == 0) {
              if (left >= 8) *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
              if (left >= 16) *reinterpret_cast<uint4*>(dst + 16 * c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (e < left) reinterpret_cast<uint16_t*>(dst)[16 * c + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            }
          }
        }
        if (real) {
          if (whole) put_lse(a, s, h, row0 + row, ref, l);
          else ws.ml[part * kRows + row] = make_float2(ref, l);
        }
      }
    }
    it += nb;
    ns[0] += nh[0];
    ns[1] += nh[1];
    // TMEM reads of this run come before the next run's MMAs
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*stop) break;
    if constexpr (X) {
      if (__builtin_expect(run->odd_lo <= run->odd_hi, 0)) {
        if (warp >= 4 && warp < kSoftEnd) give_back<T, DP>(a, run, threadIdx.x - 128, ws.o, me);
        __syncthreads();  // before the run's room is another's
      }
    }
  }

  if (warp == 1) asm volatile("cp.async.wait_all;" ::: "memory");
  // after a wait that ran out: the loads in flight arrive, and the MMAs complete, before the memory is given back
  if (*stop && warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_wait_bounded(smem_u32(&full[s]), 0, err, kDevTimeoutFull, 20000000);
      mbar_wait_bounded(smem_u32(&full[s]), 1, err, kDevTimeoutFull, 20000000);
    }
  }
  if ((warp == 1 || warp == 2) && elect()) {  // the thread that issued them: a commit speaks of its own thread's products
    umma_commit(smem_u32(&done[warp - 1]));
    mbar_wait_bounded(smem_u32(&done[warp - 1]), 0, err, kDevTimeoutAccum);
  }
  tc_fence_before();
  __syncthreads();
  if (*stop && threadIdx.x == 0) *ws.fault = 1;  // for the join, which tells the caller
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the row tile that block `blockIdx.x` left open, in the
// order of the keys.  A warp takes 8 rows x 16 channels: 128-byte reads of the
// parts, 32-byte writes of the rows.
constexpr int kJoinThreads = 256;
template <typename T, int DP, bool X>
__global__ void __launch_bounds__(kJoinThreads) kv_chunk_join_kernel(const __grid_constant__ AttnArgs a, const int G) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kRows = Cfg<DP>::kRows;
  const int me = blockIdx.x;
  const Space<X> ws = space<DP, X>(a, G);
  const Open op = ws.open[me];
  // Rows of sequences without a key get their zeros here.  Where a wait ran out the other rows, written or not, become
  // NaN: the call may have no status word to tell it.
  const bool fault = *ws.fault != 0;
  if (blockIdx.y == 0) put_empty<T>(a, me, G, fault);
  if (op.parts == 0 || fault) return;
  const int row0 = op.row0, cnt = op.cnt;
  const int lane = threadIdx.x & 31;
  for (int w = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); w < kRows / 8 * (DP / 16);
       w += gridDim.y * (kJoinThreads / 32)) {
    const int r = w / (DP / 16) * 8 + (lane & 7), c = w % (DP / 16) * 4 + (lane >> 3);  // row, four channels
    if (r >= cnt) continue;
    float m = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 4;  // loads of as many parts are in flight together
    for (int i0 = 0; i0 <= op.parts; i0 += kAhead) {
      float2 ml[kAhead];
      float4 x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = min(i0 + u, op.parts);
        const long long part = 2LL * (me + i) + (i == 0 ? 1 : 0);
        ml[u] = ws.ml[part * kRows + r];
        x[u] = ws.o[(part * (DP / 4) + c) * kRows + r];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (i0 + u > op.parts || ml[u].y == 0.f) continue;  // none, or nothing seen there
        const float n = fmaxf(m, ml[u].x);
        const float f = weight(m, n), g = weight(ml[u].x, n);
        l = l * f + ml[u].y * g;
        v.x = v.x * f + x[u].x * g;
        v.y = v.y * f + x[u].y * g;
        v.z = v.z * f + x[u].z * g;
        v.w = v.w * f + x[u].w * g;
        m = n;
      }
    }
    const float rl = l == 0.f ? 0.f : 1.f / l;
    if (4 * c < a.c.D) {
      T* dst = out_row<T>(a, op.s, op.h, row0 + r) + 4 * c;
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
    if (c == 0) put_lse(a, op.s, op.h, row0 + r, m, l);
  }
}

template <typename T, int DP, bool X>
cudaError_t go(const ChunkLaunch& L, int sms, cudaStream_t s) {
  using C = Cfg<DP>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem((const void*)kv_chunk_kernel<T, DP, X>, C::kSmem, &allowed);
  if (e != cudaSuccess) return e;
  // each may start as the kernel before it drains, and waits for its end
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3((unsigned)((row_tiles(L.a) + kPlanWarps - 1) / kPlanWarps));
  cfg.blockDim = dim3(32 * kPlanWarps);
  e = cudaLaunchKernelEx(&cfg, kv_chunk_plan_kernel<X>, L.a, L.geo);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  e = cudaLaunchKernelEx(&cfg, kv_chunk_kernel<T, DP, X>, L.k, L.v, L.a, L.geo);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(sms, 16);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_chunk_join_kernel<T, DP, X>, L.a, sms);
}

}  // namespace

bool kv_chunk_geometry(const AttnArgs& a, ChunkGeo* g) {
  const int ps = a.c.page_size;
  g->box_rows = ps >= kBlock ? kBlock : (ps + 7) / 8 * 8;
  g->parts = ps > kBlock ? (ps + kBlock - 1) / kBlock : 1;
  g->pages = g->parts > 1 ? 1 : kBlock / g->box_rows;
  // pages whose rows are no multiple of 8 leave gaps between them in a block: one such page to a block, or none
  return ps % 8 == 0 || g->pages == 1;
}

long long kv_chunk_workspace(const AttnArgs& a, int sms) {
  const int DP = a.c.D <= 64 ? 64 : a.c.D <= 128 ? 128 : 256;
  return kFaultBytes + row_tiles(a) * (long long)(a.mask == kMaskRanges ? sizeof(Tile<false>) : sizeof(Tile<true>)) + (long long)sms * (sizeof(Open) + 2 * tile_rows(DP) * (sizeof(float2) + (size_t)DP * sizeof(float)));
}

namespace {

template <bool X>
cudaError_t by_kind(const ChunkLaunch& L, int sms, cudaStream_t s) {
  const bool bf16 = L.a.c.elem == 1;
  if (L.a.c.D <= 64) return bf16 ? go<__nv_bfloat16, 64, X>(L, sms, s) : go<__half, 64, X>(L, sms, s);
  if (L.a.c.D <= 128) return bf16 ? go<__nv_bfloat16, 128, X>(L, sms, s) : go<__half, 128, X>(L, sms, s);
  return bf16 ? go<__nv_bfloat16, 256, X>(L, sms, s) : go<__half, 256, X>(L, sms, s);
}

}  // namespace

cudaError_t launch_kv_chunk(const ChunkLaunch& L, int sms, cudaStream_t s) {
  return L.a.mask == kMaskRanges ? by_kind<false>(L, sms, s) : by_kind<true>(L, sms, s);
}

}  // namespace wan
