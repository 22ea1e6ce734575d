// Launch descriptors of the token operators (rotary positions, the paged
// key-value cache and the attention that reads it), shared by the C ABI
// (token_api.cu) and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace wan {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxRotaryPairs = kMaxHeadDim / 2;
constexpr int kMaxRotaryAxes = 4;

// Codes of a batch's status word, besides the bounded waits' (ptx.cuh).
enum TokenError : int {
  kDevBadPage = 4,    // a page number outside the cache
  kDevBadLength = 5,  // a length, token range or position outside what the batch describes
  kDevBadParent = 6,  // a drafted token's parent is none of the drafts before it
};

// Pair j turns by position[axis[j]] * turn[j], in units of 2^-64 of a full
// turn: the 64-bit product wraps exactly as the angle does, without any 64-bit
// floating point and without a table.  What a far position loses is the
// frequency's own rounding (2^-52 of itself, and 2^-64 of a turn) times it.
struct RotaryPlan {
  uint64_t turn[kMaxRotaryPairs];
  uint8_t axis[kMaxRotaryPairs];
  int pairs, axes;
  int interleaved;  // pair j is channels (2j, 2j + 1); otherwise (j, j + pairs)
  int inverse;      // opposite angles
};

struct RotaryArgs {
  RotaryPlan plan;
  const void* x;
  void* out;
  long long xb, xs, xh, ob, os, oh;  // strides in elements (batch, token, head)
  const void* pos;                   // [B or 1][S][axes], int32 or int64
  int pos64;
  long long pos_b;  // positions' batch stride (values)
  int B, S, H, D;
  int elem;   // 0 fp32, 1 bf16, 2 fp16
  int width;  // elements per access that pointers and strides allow (a power of two, 16 bytes at most)
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s);

// A cache of pages: element (page, head, row, channel) of k at
//   k + page*k_page + head*k_head + row*k_row + channel, and likewise v.
struct KvCache {
  void *k, *v;
  int elem;  // 1 bf16, 2 fp16
  int heads, page_size, D;
  long long pages;
  long long k_page, k_head, k_row, v_page, v_head, v_row;
};
// The sequences of a call: sequence b holds lengths[b] keys, key i in row
// i % page_size of page pages[b*page_stride + i / page_size]; its new tokens
// are rows cu[b] .. cu[b+1]-1 of the token tensors (cu null: row b).
struct KvBatch {
  const int* pages;
  long long page_stride;
  int max_pages, B;
  const int* lengths;
  const int* cu;
  int T;  // rows of the token tensors
  int* status;
};

struct AppendArgs {
  RotaryPlan plan;  // pairs 0: nothing is turned
  KvCache c;
  KvBatch b;
  const void *k, *v, *q;
  void* qo;
  long long k_t, k_h, v_t, v_h, q_t, q_h, qo_t, qo_h;
  int q_heads;
  const void* pos;  // [T][axes]
  int pos64;
  int width;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s);

// What a row sees.  Beside a range of its own (or every key), its place in the
// sequence can tell: new tokens are then the sequence's last keys.
enum AttnMask : int {
  kMaskRanges = 0,
  kMaskWindow = 1,  // the first `sinks` keys and a window of frames
  kMaskTree = 2,    // what comes before the new tokens, its ancestors among them and itself
};
// New tokens that a sequence of a tree call may have: a row finds its ancestors by a walk, whose length this bounds.
constexpr int kMaxDrafts = 1024;

struct AttnArgs {
  KvCache c;
  KvBatch b;
  const void* q;
  void* out;
  float* lse;        // [T][q_heads], optional
  const int* ranges; // [T][2]: first and one past the last key a row sees, optional
  long long q_t, q_h, o_t, o_h;
  int q_heads, group;
  float scale_log2;  // scale * log2(e)
  void* workspace;
  int stall_at1;  // failure self test: 1-based block of keys that is never loaded (0: none)
  int mask;       // AttnMask
  // window: the token at place p sees [0, sinks) and the keys of [e - span, e), e the end of its frame
  uint32_t frame, span;  // span: whole frames
  int sinks;
  const int* parents;    // tree: [T] place of each draft's parent among its sequence's, -1 for none
};
// Bytes of workspace of a call (a bound from host-side sizes alone).
long long kv_attention_workspace(const AttnArgs& a, int sms);
cudaError_t launch_kv_attention(const AttnArgs& a, int sms, cudaStream_t s);

// Sequences targets[i] become copies of sources[i].
constexpr int kMaxForks = 1024;
struct ForkArgs {
  KvCache c;
  int *pages, *lengths;  // the call's tables, [B][max_pages] and [B]
  long long page_stride;
  int max_pages, B;
  const int *sources, *targets;  // [N]
  const int* fresh;              // [N][fresh_pages]: pages for what is copied
  long long fresh_stride;
  int fresh_pages, N;
  int share;  // whole pages are shared, and only the last, partly filled one is copied
  int* status;
};
cudaError_t launch_kv_fork(const ForkArgs& a, int sms, cudaStream_t s);

// Key keep[cu[b] + j] of sequence b moves to place first + j (b.lengths: first; b.cu, b.T: ranges of keep).
struct CompactArgs {
  KvCache c;
  KvBatch b;
  const int* keep;
  int* lengths;  // [B]: keys that are left
  int planes;    // heads of K and of V, or of K alone (k and v are one tensor, whose rows move once)
};
cudaError_t launch_kv_compact(const CompactArgs& a, int sms, cudaStream_t s);

// Raises a kernel's dynamic shared memory limit once per device: `done` holds a
// bit per device that has it (a call costs 0.5 us on the launch path).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// ---------------------------------------------------- shared index arithmetic
// Range of a batch's rows that sequence b owns; false if cu does not describe
// a range of the T rows, or one that starts before the previous sequence's.
__host__ __device__ inline bool kv_rows(const int* cu, int T, int b, int* r0, int* n) {
  if (!cu) {
    *r0 = b;
    *n = b < T ? 1 : 0;
    return b < T;
  }
  const int lo = cu[b], hi = cu[b + 1];
  *r0 = lo;
  *n = hi - lo;
  if (lo >= 0 && hi >= lo && hi <= T && (b == 0 || cu[b - 1] <= lo)) return true;
  *r0 = 0;
  *n = 0;
  return false;
}
// Keys of sequence b that its page table can hold; false if the length is not
// among them.
__host__ __device__ inline bool kv_length(int len, int max_pages, int page_size, int* out) {
  const long long most = (long long)max_pages * page_size;
  if (len >= 0 && len <= most) {
    *out = len;
    return true;
  }
  *out = 0;
  return false;
}
// The page of key i, or -1 if the table names none of the cache's pages.
__host__ __device__ inline int kv_page(const int* row, int i, int page_size, long long pages) {
  const int p = row[i / page_size];
  return p >= 0 && p < pages ? p : -1;
}

}  // namespace wan
