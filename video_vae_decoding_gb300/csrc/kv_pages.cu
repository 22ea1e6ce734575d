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

__device__ __forceinline__ void tell(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// ------------------------------------------------------------------- forks
// Forks of one source are copied together: a row is read once and written to
// each copy (three copies of a cache of 223 MB: 894 MB instead of 1341).
//
// The work of a call is one line of row groups (source, page, K or V, head,
// rows) that is cut into equal pieces, one per warp, from the lengths on the
// device: one long sequence is spread over the whole card, and a captured
// graph follows its lengths.
constexpr int kForkWarps = 8, kForkCtas = 4;
constexpr int kAhead = 4;  // row groups that a warp has in flight

struct ForkPlan {  // per fork, in shared memory
  int source, target;
  int next;         // the next fork of the same source (-1: none); forks that are left out are in no chain
  int len;          // keys of the source; -1: the fork is left out
  long long begin;  // of the line (only the first fork of a source has groups on it)
};

__global__ void __launch_bounds__(32 * kForkWarps, kForkCtas) kv_fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  ForkPlan* plan = reinterpret_cast<ForkPlan*>(smem);
  __shared__ long long s_warp[kForkWarps + 1];
  constexpr int kThreads = 32 * kForkWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int CH = a.c.D / 8, RPW = 32 / CH;  // 16-byte pieces of a row, rows of a group
  const int size = a.c.page_size;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    plan[i].source = a.sources[i];
    plan[i].target = a.targets[i];
  }
  __syncthreads();
  // A fork whose target is a source, or the target of an earlier one, would race with it.
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    const int p = plan[i].source, t = plan[i].target;
    int len = 0, code = 0;
    if (p < 0 || p >= a.B || t < 0 || t >= a.B) {
      code = kDevBadLength;
    } else {
      for (int k = 0; k < a.N; ++k)
        if (plan[k].source == t || (k < i && plan[k].target == t)) code = kDevBadLength;
      if (!kv_length(a.lengths[p], a.max_pages, size, &len)) code = kDevBadLength;
      const int copied = a.share ? (len % size ? 1 : 0) : (len + size - 1) / size;
      if (copied > a.fresh_pages) code = kDevBadLength;
    }
    if (code) tell(a.status, code);
    plan[i].len = code ? -1 : len;
  }
  __syncthreads();
  // chains of forks of one source, and the groups of each chain's first
  constexpr int kEach = kMaxForks / kThreads;  // forks of a thread, side by side
  long long groups[kEach], mine = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x * kEach + e;
    groups[e] = 0;
    if (i >= a.N) continue;
    int next = -1;
    const int len = plan[i].len;
    if (len > 0) {
      bool first = true;
      for (int k = 0; k < i; ++k) first = first && !(plan[k].len >= 0 && plan[k].source == plan[i].source);
      for (int k = a.N - 1; k > i; --k)
        if (plan[k].len >= 0 && plan[k].source == plan[i].source) next = k;
      if (first) {
        const long long whole = a.share ? 0 : len / size;
        groups[e] = 2LL * a.c.heads * (whole * ((size + RPW - 1) / RPW) + (len % size + RPW - 1) / RPW);
      }
    }
    plan[i].next = next;
    mine += groups[e];
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kForkWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x * kEach + e;
    if (i < a.N) plan[i].begin = before;
    before += groups[e];
  }
  __syncthreads();

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

  // this warp's piece of the line
  const long long W = (long long)gridDim.x * kForkWarps, me = (long long)blockIdx.x * kForkWarps + warp;
  const long long each = total / W, more = total - each * W;
  long long at = me * each + min(me, more);
  const long long end = at + each + (me < more ? 1 : 0);
  if (at >= end) return;
  int i = 0;  // the last fork that begins at or before `at` (forks without groups begin with the next one)
  {
    int lo = 0, hi = a.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (plan[mid].begin <= at) lo = mid; else hi = mid;
    }
    i = lo;
  }
  // place in fork i's groups: page j of those that are copied, plane (K or V, head), group g
  int len, whole, j, plane, g, rows, per;
  auto enter = [&](long long off) {
    len = plan[i].len;
    whole = len / size;  // full pages
    const int full = (size + RPW - 1) / RPW;
    const long long page_groups = 2LL * a.c.heads * full, in_full = a.share ? 0 : whole * page_groups;
    j = a.share ? whole : (int)(off < in_full ? off / page_groups : whole);
    const long long r = off < in_full ? off - j * page_groups : off - in_full;
    rows = j < whole ? size : len - whole * size;
    per = (rows + RPW - 1) / RPW;
    plane = (int)(r / per);
    g = (int)(r - (long long)plane * per);
  };
  enter(at - plan[i].begin);
  const int sub = lane / CH, ch = lane - sub * CH;
  const bool busy = sub < RPW;
  while (at < end) {
    // up to kAhead groups of fork i's chain
    uint4 v[kAhead];
    int jj[kAhead], hd[kAhead], row[kAhead];
    bool ofv[kAhead], live[kAhead];
    const int chain = i;
    int n = 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      live[u] = false;
      if (at >= end || i != chain) continue;
      n = u + 1;
      jj[u] = j;
      ofv[u] = plane >= a.c.heads;
      hd[u] = ofv[u] ? plane - a.c.heads : plane;
      row[u] = g * RPW + sub;
      const int page = a.pages[plan[i].source * a.page_stride + j];
      const bool there = page >= 0 && page < a.c.pages;
      if (!there) tell(a.status, kDevBadPage);
      live[u] = there && busy && row[u] < rows;
      if (live[u]) {
        const long long o = ofv[u] ? page * a.c.v_page + hd[u] * a.c.v_head + row[u] * a.c.v_row
                                   : page * a.c.k_page + hd[u] * a.c.k_head + row[u] * a.c.k_row;
        v[u] = *reinterpret_cast<const uint4*>((const uint16_t*)(ofv[u] ? a.c.v : a.c.k) + o + ch * 8);
      }
      // the next group
      ++at;
      if (++g == per) {
        g = 0;
        if (++plane == 2 * a.c.heads) {
          plane = 0;
          ++j;
          if (j == whole && len > whole * size) {
            rows = len - whole * size;
            per = (rows + RPW - 1) / RPW;
          } else if (j >= whole && at < end) {  // the next fork with groups
            do ++i; while (i + 1 < a.N && plan[i + 1].begin <= at);
            enter(at - plan[i].begin);
          }
        }
      }
    }
    for (int m = chain; m >= 0; m = plan[m].next) {
      const int skip = a.share ? plan[m].len / size : 0;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (u >= n) continue;
        const int page = a.fresh[m * a.fresh_stride + jj[u] - skip];
        const bool there = page >= 0 && page < a.c.pages;
        if (!there) tell(a.status, kDevBadPage);
        if (there && live[u]) {
          const long long o = ofv[u] ? page * a.c.v_page + hd[u] * a.c.v_head + row[u] * a.c.v_row
                                     : page * a.c.k_page + hd[u] * a.c.k_head + row[u] * a.c.k_row;
          *reinterpret_cast<uint4*>((uint16_t*)(ofv[u] ? a.c.v : a.c.k) + o + ch * 8) = v[u];
        }
      }
    }
  }
}

// -------------------------------------------------------------- compaction
// Key keep[j] of a sequence moves to place first + j, in place: since keep[j] >=
// first + j, a row is read before, or in the same step as, any row whose place
// it is.  A block moves a slice of channels of one sequence, head and K or V, in
// steps of many rows: the rows of step c + 1 are asked for, a barrier says that
// those of step c are all in registers, and they are stored.  What a later step
// reads lies behind all places that earlier ones write.
constexpr int kMoveWarps = 16;
constexpr int kMoveAhead = 4;  // row groups of a warp in a step

struct Move {  // of the row that this lane looks up
  long long from, to;  // in elements; from < 0: none
};

__global__ void __launch_bounds__(32 * kMoveWarps) kv_compact_kernel(const __grid_constant__ CompactArgs a, const int slice) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int CH = a.c.D / 8, slices = (CH + slice - 1) / slice;
  const int part = blockIdx.y % slices, plane = blockIdx.y / slices;
  const bool ofv = plane >= a.c.heads;
  const int h = ofv ? plane - a.c.heads : plane, size = a.c.page_size;
  const long long s_page = ofv ? a.c.v_page : a.c.k_page, s_row = ofv ? a.c.v_row : a.c.k_row;
  uint16_t* const base = (uint16_t*)(ofv ? a.c.v : a.c.k) + h * (ofv ? a.c.v_head : a.c.k_head) + part * slice * 8;

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

  const int RPW = min(8, 32 / slice);        // rows of a group
  const int look = kMoveAhead * RPW;         // rows that a warp looks up for a step, one a lane
  const int step = kMoveWarps * look;
  const int sub = lane / slice, ch = lane - sub * slice;
  const bool busy = sub < RPW && part * slice + ch < CH;
  auto lookup = [&](int c) {
    const uint32_t j = (uint32_t)c * step + warp * look + lane;
    Move m{-1, 0};
    if (lane < look && j < (uint32_t)n) {
      const int from = keep[j], to = first + (int)j;
      if (from < to || from >= room) {
        tell(a.b.status, kDevBadLength);
      } else if (from != to) {
        const int pf = kv_page(table, from, size, a.c.pages), pt = kv_page(table, to, size, a.c.pages);
        if (pf < 0 || pt < 0) {
          tell(a.b.status, kDevBadPage);
        } else {
          m.from = pf * s_page + from % size * s_row;
          m.to = pt * s_page + to % size * s_row;
        }
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
  uint4 v0[kMoveAhead], v1[kMoveAhead];
  Move m0 = lookup(0), m1;
  load(m0, v0);
  for (int c = 0; c < steps; c += 2) {
    m1 = lookup(c + 1);
    load(m1, v1);
    __syncthreads();
    store(m0, v0);
    if (c + 1 >= steps) break;
    m0 = lookup(c + 2);
    load(m0, v0);
    __syncthreads();
    store(m1, v1);
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

cudaError_t launch_kv_compact(const CompactArgs& a, int sms, cudaStream_t s) {
  // Slices of 64 bytes or more, two blocks for each SM if there are as many.
  const int CH = a.c.D / 8;
  int slice = CH;
  while (slice > 4 && (long long)a.b.B * 2 * a.c.heads * ((CH + slice - 1) / slice) < 2 * sms) slice = (slice + 1) / 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(a.b.B, 2 * a.c.heads * ((CH + slice - 1) / slice));
  cfg.blockDim = dim3(32 * kMoveWarps);
  return cudaLaunchKernelEx(&cfg, kv_compact_kernel, a, slice);
}

}  // namespace wan
