// Moves inside a paged key-value cache: copies of whole sequences (forks), and
// the compaction of a sequence's kept keys.
//
// Bound: memory.  Rows of a head (2 D bytes) move as 16-byte pieces; a warp
// takes as many rows at a time as its lanes hold, so what a row needs (page,
// place) is the same for its lanes or is looked up by one and passed on.
#include <algorithm>

#include "ptx.cuh"
#include "token_ops.h"

namespace wan {

namespace {

__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((unsigned long long)a | (unsigned long long)b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ void tell(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// ------------------------------------------------------------------- forks
// Forks of one source are copied together: a row is read once and written to
// each copy (three copies of a cache of 223 MB: 894 MB instead of 1341, 157 us, 5.7
// TB/s; one copy of 819 MB 6.2 TB/s, as far as its reads and writes are as many).
//
// The work of a call is one line of row groups (source, page, K or V, head,
// rows), laid out from the lengths on the device: one long sequence is spread over
// the whole card, and a captured graph follows its lengths.
// (A clip's three copies in us: 157 so, 159 with four blocks an SM, 171 with two, 164 with turns of 64.)
constexpr int kForkWarps = 8, kForkCtas = 3;
constexpr int kAhead = 4;  // row groups that a warp has in flight
constexpr int kTurn = 8;   // and that it takes at a time, if there are as many for each

struct ForkPlan {  // per fork, in shared memory
  int source, target;
  int next;         // the next fork of the same source (-1: none); forks that are left out are in no chain
  int len;          // keys of the source; -1: the fork is left out
  long long begin;  // of the line (only the first fork of a source has groups on it)
};

__global__ void __launch_bounds__(32 * kForkWarps, kForkCtas) kv_fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  ForkPlan* plan = reinterpret_cast<ForkPlan*>(smem);
  __shared__ long long s_warp[kForkWarps];
  constexpr int kThreads = 32 * kForkWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int CH = a.c.D / 8, RPW = 32 / CH;  // 16-byte pieces of a row, rows of a group
  const int size = a.c.page_size;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    const int p = a.sources[i], t = a.targets[i];
    plan[i].source = p;
    plan[i].target = t;
    int len = -1;
    if (p >= 0 && p < a.B && t >= 0 && t < a.B && kv_length(a.lengths[p], a.max_pages, size, &len)) {
      const int copied = a.share ? (len % size ? 1 : 0) : (len + size - 1) / size;
      if (copied > a.fresh_pages) len = -1;
    } else {
      len = -1;
    }
    plan[i].len = len;
  }
  __syncthreads();
  // A fork whose target is a source, or the target of an earlier one, would race with it.
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    const int t = plan[i].target;
    bool left_out = plan[i].len < 0;
#pragma unroll 8
    for (int k = 0; k < a.N; ++k) left_out = left_out || plan[k].source == t || (k < i && plan[k].target == t);
    if (left_out) tell(a.status, kDevBadLength);
    plan[i].next = left_out;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.N; i += kThreads)
    if (plan[i].next) plan[i].len = -1;
  __syncthreads();
  // chains of forks of one source, and the groups of each chain's first
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    const int len = plan[i].len, p = plan[i].source;
    int next = a.N;
    bool first = len > 0;
#pragma unroll 8
    for (int k = 0; k < a.N; ++k) {
      const bool same = plan[k].len >= 0 && plan[k].source == p;
      first = first && !(same && k < i);
      if (same && k > i) next = min(next, k);
    }
    long long groups = 0;
    if (first) {
      const long long whole = a.share ? 0 : len / size;
      groups = 2LL * a.c.heads * (whole * ((size + RPW - 1) / RPW) + (len % size + RPW - 1) / RPW);
    }
    plan[i].next = len > 0 && next < a.N ? next : -1;
    plan[i].begin = groups;
  }
  __syncthreads();
  // where each begins: forks side by side in a thread, in rounds
  long long total = 0;
  for (int i0 = 0; i0 < a.N; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const long long mine = i < a.N ? plan[i].begin : 0;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    long long before = total + incl - mine;
#pragma unroll
    for (int w = 0; w < kForkWarps; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    if (i < a.N) plan[i].begin = before;
    __syncthreads();
  }

  // the tables: rows that are written are read by no fork
  for (int i = blockIdx.x; i < a.N; i += gridDim.x) {
    const ForkPlan f = plan[i];
    if (f.len < 0) continue;
    const int whole = a.share ? f.len / size : 0, held = (f.len + size - 1) / size;
    const int* from = a.pages + f.source * a.page_stride;
    int* to = a.pages + f.target * a.page_stride;
    for (int j = threadIdx.x; j < held; j += kThreads) to[j] = j < whole ? from[j] : a.fresh[i * a.fresh_stride + j - whole];
    if (threadIdx.x == 0) a.lengths[f.target] = f.len;
  }

  // The line goes round the warps, a few groups at a time: what is copied at one time lies together in memory.
  const long long W = (long long)gridDim.x * kForkWarps, each = min((long long)kTurn, quotient(total + W - 1, W));
  const int sub = lane / CH, ch = lane - sub * CH, full = (size + RPW - 1) / RPW;
  int i = 0;  // the last fork that begins at or before the turn (forks without groups begin with the next one)
  for (long long turn = (long long)blockIdx.x * kForkWarps + warp; turn * each < total; turn += W) {
    long long at = turn * each;
    const long long end = min(total, at + each);
    while (at < end) {
      // group g of a plane (page j of fork i's, K or V, head), and how many of the plane's there are from it on
      while (i + 1 < a.N && plan[i + 1].begin <= at) ++i;
      const int len = plan[i].len, whole = len / size;  // full pages
      const long long off = at - plan[i].begin, page_groups = 2LL * a.c.heads * full, in_full = a.share ? 0 : whole * page_groups;
      const int j = a.share ? whole : (int)(off < in_full ? quotient(off, page_groups) : whole);
      const long long r = off < in_full ? off - j * page_groups : off - in_full;
      const int rows = j < whole ? size : len - whole * size, per = (rows + RPW - 1) / RPW;
      const int plane = (int)quotient(r, per), g = (int)(r - (long long)plane * per);
      const int n = (int)min((long long)(per - g), end - at);
      at += n;
      const bool ofv = plane >= a.c.heads;
      const long long s_page = ofv ? a.c.v_page : a.c.k_page, s_row = ofv ? a.c.v_row : a.c.k_row;
      const long long first = (ofv ? (plane - a.c.heads) * a.c.v_head : plane * a.c.k_head) + (g * RPW + sub) * s_row + ch * 8;
      uint16_t* const base = (uint16_t*)(ofv ? a.c.v : a.c.k) + first;
      const int page = a.pages[plan[i].source * a.page_stride + j], left = sub < RPW ? rows - g * RPW - sub : 0;
      if (page < 0 || page >= a.c.pages) {
        tell(a.status, kDevBadPage);
        continue;
      }
      for (int b = 0; b < n; b += kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (b + u < n && (b + u) * RPW < left) v[u] = *reinterpret_cast<const uint4*>(base + page * s_page + (b + u) * RPW * s_row);
        for (int m = i; m >= 0; m = plan[m].next) {
          const int to = a.fresh[m * a.fresh_stride + (a.share ? 0 : j)];
          if (to < 0 || to >= a.c.pages) {
            tell(a.status, kDevBadPage);
            continue;
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
            if (b + u < n && (b + u) * RPW < left) *reinterpret_cast<uint4*>(base + to * s_page + (b + u) * RPW * s_row) = v[u];
        }
      }
    }
  }
}

// -------------------------------------------------------------- compaction
// Key keep[j] of a sequence moves to place first + j, in place; keep ascends.
// Blocks share a sequence, head and K or V in one of two ways:
//  - where no key's old place is a new one (keep[0] >= first + n, as when a window
//    rolls on by more than its length), each takes its part of the keys, in any
//    order;
//  - otherwise each takes a slice of channels of all keys and goes through them in
//    steps of many rows.  Since keep[j] >= first + j, what a later step reads lies
//    behind all places that earlier ones write: the rows of step c + 1 are asked
//    for, a barrier says that those of step c are all read, and they are stored.
// 11,440 keys of 16 heads of 128 in the first way (187 MB read and written) take 34
// us, 5.4 TB/s; 13 sequences of up to 1900 scattered keys, 8 heads of 96, 24 us.  For
// the second way's steps a call of few planes has blocks of up to 32 warps: 16,368
// scattered keys of 27,280, 16 heads of 128 (268 MB), 59 us.
constexpr int kMoveLanes = 32;  // warps of the blocks that share an SM
constexpr int kMoveAhead = 4;  // row groups of a warp in a step

// Of the row that this lane looks up:
struct Ask {
  int from, to, pf, pt;  // places (to < 0: nothing moves) and the numbers of their pages
};
struct Move {
  long long from, to;  // in elements; from < 0: none
};

template <int kMoveWarps>
__global__ void __launch_bounds__(32 * kMoveWarps, kMoveLanes / kMoveWarps)
    kv_compact_kernel(const __grid_constant__ CompactArgs a, const int blocks, const int ordered) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.y % blocks, plane = blockIdx.y / blocks;
  const bool ofv = plane >= a.c.heads;
  const int h = ofv ? plane - a.c.heads : plane, size = a.c.page_size;
  const long long s_page = ofv ? a.c.v_page : a.c.k_page, s_row = ofv ? a.c.v_row : a.c.k_row;

  int k0, n, first;
  const long long room = (long long)a.b.max_pages * size;
  bool good = kv_rows(a.b.cu, a.b.T, b, &k0, &n);
  good = kv_length(a.b.lengths[b], a.b.max_pages, size, &first) && good;
  if (first + (long long)n > room) good = false;
  if (!good) n = 0;
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    if (!good) tell(a.b.status, kDevBadLength);
    a.lengths[b] = first + n;
  }
  if (n == 0) return;
  const int* table = a.b.pages + b * a.b.page_stride;
  const int* keep = a.keep + k0;

  const bool apart = blocks > 1 && keep[0] >= first && keep[0] - first >= n;
  if (!apart && part >= ordered) return;
  const int CH = a.c.D / 8;                                              // 16-byte pieces of a row
  const int slice = apart ? CH : (CH + ordered - 1) / ordered, c0 = apart ? 0 : part * slice;  // this block's
  if (c0 >= CH) return;
  uint16_t* const base = (uint16_t*)(ofv ? a.c.v : a.c.k) + h * (ofv ? a.c.v_head : a.c.k_head) + c0 * 8;
  const int RPW = min(8, 32 / slice);        // rows of a group
  const int look = kMoveAhead * RPW;         // rows that a warp looks up for a step, one a lane
  const int step = kMoveWarps * look;
  const int sub = lane / slice, ch = lane - sub * slice;
  const bool busy = sub < RPW && c0 + ch < CH;
  // What a step needs is asked for ahead of it: which keys three steps, their pages two, the keys themselves one.
  auto key = [&](int c) {  // of the lane's row, -1 for one that is left out
    const uint32_t j = (uint32_t)c * step + warp * look + lane;
    if (lane >= look || j >= (uint32_t)n) return -1;
    const int from = keep[j], before = j > 0 ? keep[j - 1] : -1;
    return from > before && from >= first + (apart ? n : (int)j) && from < room ? from : -1;
  };
  auto pages = [&](int c, int from) {
    const uint32_t j = (uint32_t)c * step + warp * look + lane;
    Ask q{from, -1, 0, 0};
    if (lane < look && j < (uint32_t)n) {
      q.to = first + (int)j;
      if (from < 0) {
        tell(a.b.status, kDevBadLength);
        q.to = -1;
      } else if (from == q.to) {
        q.to = -1;
      } else {
        q.pf = table[from / size];
        q.pt = table[q.to / size];
      }
    }
    return q;
  };
  auto rows = [&](const Ask& q) {
    Move m{-1, 0};
    if (q.to >= 0) {
      if (q.pf < 0 || q.pf >= a.c.pages || q.pt < 0 || q.pt >= a.c.pages) {
        tell(a.b.status, kDevBadPage);
      } else {
        m.from = q.pf * s_page + q.from % size * s_row;
        m.to = q.pt * s_page + q.to % size * s_row;
      }
    }
    return m;
  };
  auto load = [&](const Move& m, uint4 (&v)[kMoveAhead]) {
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const long long o = __shfl_sync(0xffffffffu, m.from, min(31, u * RPW + sub));
      if (busy && o >= 0) v[u] = *reinterpret_cast<const uint4*>(base + o + ch * 8);
    }
  };
  auto store = [&](const Move& m, const uint4 (&v)[kMoveAhead]) {
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const long long f = __shfl_sync(0xffffffffu, m.from, min(31, u * RPW + sub));
      const long long o = __shfl_sync(0xffffffffu, m.to, min(31, u * RPW + sub));
      if (busy && f >= 0) *reinterpret_cast<uint4*>(base + o + ch * 8) = v[u];
    }
  };
  const int steps = (n + step - 1) / step;
  // this block's: every `blocks`-th, or all
  const int beg = apart ? part : 0, by = apart ? blocks : 1;
  if (beg >= steps) return;
  uint4 v0[kMoveAhead], v1[kMoveAhead];
  Move m0 = rows(pages(beg, key(beg))), m1;
  load(m0, v0);
  Ask next = pages(beg + by, key(beg + by));
  int then = key(beg + 2 * by);
  // stores step c, whose rows are on their way, and asks for those of step c + by
  auto turn = [&](int c, const Move& mine, const uint4 (&v)[kMoveAhead], Move& other, uint4 (&w)[kMoveAhead]) {
    other = rows(next);
    load(other, w);
    next = pages(c + 2 * by, then);
    then = key(c + 3 * by);
    if (!apart) __syncthreads();
    store(mine, v);
  };
  for (int c = beg; c < steps; c += 2 * by) {
    turn(c, m0, v0, m1, v1);
    if (c + by >= steps) break;
    turn(c + by, m1, v1, m0, v0);
  }
}

}  // namespace

cudaError_t launch_kv_fork(const ForkArgs& a, int sms, cudaStream_t s) {
  static_assert(kMaxForks * sizeof(ForkPlan) <= 48 * 1024, "more shared memory has to be asked for");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(sms * kForkCtas);
  cfg.blockDim = dim3(32 * kForkWarps);
  cfg.dynamicSmemBytes = a.N * sizeof(ForkPlan);
  return cudaLaunchKernelEx(&cfg, kv_fork_kernel, a);
}

template <int W>
static cudaError_t go_compact(const CompactArgs& a, long long planes, int slices, int sms, cudaStream_t s) {
  // Three times as many small blocks as are resident, so that ragged sequences even out (13 of 500 to 1900 kept keys take 24.6
  // us, 27.8 with one time); of large ones as many, whose starts would come one after the other (a clip's roll 39 us with
  // three times); fewer for a call of few keys.
  const long long step = W * kMoveAhead * std::max(1, 32 / (a.c.D / 8)), steps = std::max(1LL, a.b.T / (a.b.B * step));
  const long long resident = (long long)(kMoveLanes / W) * sms;
  const long long want = W <= 8 ? (3 * resident + planes - 1) / planes : std::max((long long)slices, resident / planes);
  const int blocks = (int)std::max(1LL, std::min(steps, want));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(a.b.B, a.planes * blocks);
  cfg.blockDim = dim3(32 * W);
  return cudaLaunchKernelEx(&cfg, kv_compact_kernel<W>, a, blocks, std::min(blocks, slices));
}

cudaError_t launch_kv_compact(const CompactArgs& a, int sms, cudaStream_t s) {
  // In steps, planes in slices of 64 bytes or more have to keep the card busy: the fewer, the more warps each.  us for
  // 16,368 of 27,280 keys of 16 heads of 128 (32 planes, 268 MB) in blocks of 4, 8, 16, 32 warps: 166, 106, 77, 59; for 8
  // sequences of 8000 and 8 heads (128 planes, 367 MB) 86, 66, 71, 80; for the first way's 11,440 keys 32, 32, 33, 34.
  const int slices = std::max(1, a.c.D / 32);
  const long long planes = (long long)a.planes * a.b.B, most = (long long)kMoveLanes * sms / (planes * slices);
  if (a.b.T < 64LL * a.b.B || most < 8) return go_compact<4>(a, planes, slices, sms, s);
  if (most < 16) return go_compact<8>(a, planes, slices, sms, s);
  if (most < 32) return go_compact<16>(a, planes, slices, sms, s);
  return go_compact<32>(a, planes, slices, sms, s);
}

}  // namespace wan
