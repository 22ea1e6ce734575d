// C ABI of the token operators (include/wan_vae.h): argument checks and
// launches.
#include <algorithm>
#include <cmath>
#include <map>
#include <set>
#include <utility>
#include <vector>

#include "host.h"
#include "kv_chunk.h"
#include "ptx.cuh"
#include "token_ops.h"

namespace wan {

namespace {

// freq / (2 pi) turns per position, as a fraction of one turn in 2^-64.
uint64_t turns(double freq) {
  double t = freq / 6.283185307179586476925286766559;
  t -= std::floor(t);
  // t < 1, but rounding may have reached it: one turn is none
  return t >= 1.0 ? 0 : (uint64_t)std::ldexp(t, 64);
}

wan_status plan_of(const wan_rotation* r, int head_dim, RotaryPlan* p) {
  if (r->pairs < 1 || r->pairs > kMaxRotaryPairs || 2 * r->pairs > head_dim)
    return fail(WAN_ERR_INVALID_ARG, "%d rotated pairs do not fit a head dim of %d", r->pairs, head_dim);
  if (r->axes < 1 || r->axes > kMaxRotaryAxes) return fail(WAN_ERR_INVALID_ARG, "%d axes (1 to 4)", r->axes);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(WAN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!r->freq || !r->axis) return fail(WAN_ERR_INVALID_ARG, "null frequencies or axes");
  for (int j = 0; j < r->pairs; ++j) {
    if (!std::isfinite(r->freq[j])) return fail(WAN_ERR_INVALID_ARG, "frequency %d is not finite", j);
    if (r->axis[j] < 0 || r->axis[j] >= r->axes) return fail(WAN_ERR_INVALID_ARG, "pair %d: axis %d", j, r->axis[j]);
    p->turn[j] = turns(r->freq[j]);
    p->axis[j] = (uint8_t)r->axis[j];
  }
  p->pairs = r->pairs;
  p->axes = r->axes;
  p->interleaved = r->interleaved;
  p->inverse = 0;
  return WAN_OK;
}

// Elements per access: the largest power of two (up to 16 bytes) that the
// address and every stride along a dimension longer than one are multiples of.
int access_width(int size, int width, const void* p, std::initializer_list<std::pair<int64_t, int64_t>> dims) {
  uint64_t bits = (uint64_t)(uintptr_t)p;
  for (const auto& d : dims)
    if (d.first > 1) bits |= (uint64_t)(d.second * size);
  while (width > 1 && bits % (uint64_t)(width * size)) width /= 2;
  return width;
}

int elem_size(int dtype) { return dtype == WAN_F32 ? 4 : 2; }

wan_status check_cache(const wan_kv_cache* c, KvCache* o) {
  if (!c || !c->k || !c->v) return fail(WAN_ERR_INVALID_ARG, "null cache");
  if (c->dtype != WAN_BF16 && c->dtype != WAN_F16)
    return fail(WAN_ERR_DTYPE, "the cache's dtype must be WAN_BF16 or WAN_F16, not %d", c->dtype);
  if (c->heads < 1 || c->page_size < 1 || c->pages < 1 || c->pages > 0x7fffffffLL)
    return fail(WAN_ERR_INVALID_ARG, "cache of %lld pages of %d rows, %d heads", (long long)c->pages, c->page_size,
                c->heads);
  if (c->head_dim < 8 || c->head_dim % 8)
    return fail(WAN_ERR_INVALID_ARG, "the cache's head dim must be a multiple of 8, not %d", c->head_dim);
  if (c->head_dim > kMaxHeadDim) return fail(WAN_ERR_UNSUPPORTED, "head dim %d (at most 256)", c->head_dim);
  if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return fail(WAN_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  const int64_t st[6] = {c->k_page, c->k_head, c->k_row, c->v_page, c->v_head, c->v_row};
  for (int64_t s : st)
    if (s < 0 || s % 8) return fail(WAN_ERR_INVALID_ARG, "cache strides must be multiples of 8, not %lld", (long long)s);
  *o = KvCache{c->k, c->v, c->dtype, c->heads, c->page_size, c->head_dim, c->pages,
               c->k_page, c->k_head, c->k_row, c->v_page, c->v_head, c->v_row};
  return WAN_OK;
}

wan_status check_batch(const wan_kv_batch* b, int page_size, KvBatch* o) {
  if (!b || !b->lengths || !b->pages) return fail(WAN_ERR_INVALID_ARG, "null batch, page table or lengths");
  if (b->batch < 1 || b->max_pages < 1) return fail(WAN_ERR_INVALID_ARG, "%d sequences of %d pages", b->batch, b->max_pages);
  if (b->page_stride < 0 || (b->page_stride < b->max_pages && b->batch > 1 && b->page_stride != 0))
    return fail(WAN_ERR_INVALID_ARG, "page_stride %lld for rows of %d", (long long)b->page_stride, b->max_pages);
  if (b->tokens < 0) return fail(WAN_ERR_INVALID_ARG, "%d tokens", b->tokens);
  if (!b->cu_tokens && b->tokens < b->batch)
    return fail(WAN_ERR_SHAPE, "%d token rows for %d sequences of one token each", b->tokens, b->batch);
  if ((int64_t)b->max_pages * page_size > 0x7fffffffLL - 1024)
    return fail(WAN_ERR_UNSUPPORTED, "a page table of %d pages of %d keys (2^31 keys at most)", b->max_pages, page_size);
  *o = KvBatch{b->pages, b->page_stride, b->max_pages, b->batch, b->lengths, b->cu_tokens, b->tokens, b->status};
  return WAN_OK;
}

// One row of the cache per (page, head, row).
wan_status check_written(const KvCache& c) {
  const int64_t need[6] = {c.pages, c.heads, c.page_size, c.pages, c.heads, c.page_size};
  const int64_t have[6] = {c.k_page, c.k_head, c.k_row, c.v_page, c.v_head, c.v_row};
  for (int i = 0; i < 6; ++i)
    if (need[i] > 1 && have[i] == 0) return fail(WAN_ERR_INVALID_ARG, "a cache that is written to must not be broadcast");
  return WAN_OK;
}

// Whether k and v are one tensor, and whether a row of k has memory in common with one of v.
bool same_rows(const KvCache& c) {
  return c.k == c.v && (c.pages == 1 || c.k_page == c.v_page) && (c.heads == 1 || c.k_head == c.v_head) &&
         (c.page_size == 1 || c.k_row == c.v_row);
}
// Rows meet if some sum of steps along the pages, heads and rows of k and of v makes up for their distance, but for less than
// a row.  Steps are taken from the longest stride on, those alone from which the shorter ones can still reach; where
// strides are so entangled that there are more than 4096 of them to look at, they count as meeting.
bool rows_meet(const KvCache& c) {
  using wide = __int128;  // a stride times a count may pass 64 bits
  struct Step {
    wide stride, lo, hi;  // times that it can be taken
  };
  Step steps[6];
  int count = 0;
  const int64_t n[3] = {c.pages, c.heads, c.page_size}, ks[3] = {c.k_page, c.k_head, c.k_row}, vs[3] = {c.v_page, c.v_head, c.v_row};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (ks[i] == vs[i]) {
      steps[count++] = {ks[i], 1 - n[i], n[i] - 1};
    } else {
      steps[count++] = {ks[i], 0, n[i] - 1};
      steps[count++] = {vs[i], 1 - n[i], 0};
    }
  }
  std::sort(steps, steps + count, [](const Step& x, const Step& y) { return x.stride > y.stride; });
  wide least[7] = {}, most[7] = {};  // what the steps from one on can add
  for (int i = count; i-- > 0;) {
    least[i] = least[i + 1] + steps[i].lo * steps[i].stride;
    most[i] = most[i + 1] + steps[i].hi * steps[i].stride;
  }
  const wide apart = ((wide)(intptr_t)c.k - (wide)(intptr_t)c.v) / 2;
  if (apart + most[0] <= -c.D || apart + least[0] >= c.D) return false;  // (two allocations: no division)
  const auto floor_div = [](wide x, wide y) { return x / y - (x % y < 0); };  // y > 0
  int budget = 4096;
  const auto found = [&](const auto& self, int i, wide at) -> bool {
    if (i == count) return at > -c.D && at < c.D;
    const Step& s = steps[i];  // -D < at + times * stride + (what the rest adds) < D
    const wide lo = std::max(s.lo, floor_div(-c.D - most[i + 1] - at, s.stride) + 1);
    const wide hi = std::min(s.hi, -floor_div(-(c.D - least[i + 1] - at), s.stride) - 1);
    for (wide t = lo; t <= hi; ++t)
      if (--budget < 0 || self(self, i + 1, at + t * s.stride)) return true;
    return false;
  };
  return found(found, 0, apart);
}

// Whether two arrays of numbers have memory in common.
bool meet(const int32_t* x, int64_t n, const int32_t* y, int64_t m) {
  const uintptr_t a = (uintptr_t)x, b = (uintptr_t)y;
  return n > 0 && m > 0 && a < b + 4 * (uintptr_t)m && b < a + 4 * (uintptr_t)n;
}
// Whether two tables whose ranges meet are different columns of one: rows as far apart, and none of one's columns the other's.
bool columns_apart(const int32_t* x, int64_t x_stride, int64_t x_columns, int64_t x_rows, const int32_t* y, int64_t y_stride,
                   int64_t y_columns, int64_t y_rows) {
  if (x_rows > 1 && y_rows > 1 && x_stride != y_stride) return false;
  const int64_t stride = x_rows > 1 ? x_stride : y_stride;  // (two single rows that meet are not apart)
  if (stride <= 0 || (x_rows <= 1 && y_rows <= 1)) return false;
  int64_t col = (((intptr_t)x - (intptr_t)y) / 4) % stride;  // of x's first column among y's
  if (col < 0) col += stride;
  return col >= y_columns && col + x_columns <= stride;
}

wan_status sm_count(int* n) {
  int dev;
  CUDA_TRY(cudaGetDevice(&dev));
  CUDA_TRY(cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev));
  return WAN_OK;
}

// Where the kernel for many tokens takes over from the split kernel: from kChunkRows rows of a sequence (tokens x query
// heads of a key head) on average, unless the call is so small that its longer start counts: fewer than kChunkWork
// products of a row with a key, by the keys that the tables have room for.  us with split / many tokens: 34 tokens of 4
// heads a key head (136 rows) against 1300 keys of 16 heads 49 / 37, 170 tokens against 600 keys of 4 heads 17 / 21,
// 13 tokens of 2 rows against 1500 keys 17 / 26.
constexpr int kChunkRows = 64;
constexpr double kChunkWork = 6e5;

// Rows that see by their place: from 20 rows on, and by the keys that a window leaves.  us with split / many tokens: a tree of
// 5 drafts of 4 heads a key head against 4000 keys, 8 sequences of 8 heads, 62 / 51; of 16 drafts of one head against 3000
// keys, 32 sequences, 94 / 100, of 32 drafts 152 / 101; one of 26 drafts of 16 heads against 2000 keys 21 / 24, of 48
// 25 / 25, of 64 30 / 25; 100 tokens of 4 sequences with a window of 1000 keys 46 / 29.
constexpr int kMaskedRows = 20;
constexpr double kMaskedWork = 1.3e6;

bool chunk_rows(const AttnArgs& a, ChunkGeo* g) {
  double keys = (double)a.b.max_pages * a.c.page_size;
  if (a.mask == kMaskWindow) keys = std::min(keys, (double)a.span + a.sinks);
  return (int64_t)a.b.T * a.group >= (int64_t)(a.mask == kMaskRanges ? kChunkRows : kMaskedRows) * a.b.B &&
         (double)a.b.T * a.q_heads * keys >= (a.mask == kMaskRanges ? kChunkWork : kMaskedWork) && kv_chunk_geometry(a, g);
}
int64_t workspace_of(const AttnArgs& a, bool chunk, int sms) {
  const int64_t split = kv_attention_workspace(a, sms);
  return chunk ? std::max<int64_t>(split, kv_chunk_workspace(a, sms)) : split;
}

// Tensor map over a cache: channels, then rows, heads and pages in the order of
// their strides.  False if the strides cannot be described.
bool cache_map(const KvCache& c, const void* base, long long page, long long head, long long row, ChunkGeo* g,
               CUtensorMap* m) {
  struct Dim {
    uint64_t n;
    long long stride;
    int* place;
    uint32_t box;
  };
  Dim d[3] = {{(uint64_t)c.page_size, row, &g->dim_row, (uint32_t)g->box_rows},
              {(uint64_t)c.heads, head, &g->dim_head, 1},
              {(uint64_t)c.pages, page, &g->dim_page, 1}};
  // a dimension of one is never stepped along: it goes last, with any stride that fits
  std::stable_sort(d, d + 3, [](const Dim& x, const Dim& y) {
    return (x.n > 1) != (y.n > 1) ? x.n > 1 : x.n > 1 && x.stride < y.stride;
  });
  uint64_t dims[4] = {(uint64_t)c.D}, strides[3];
  uint32_t box[4] = {64};
  const uint32_t step[4] = {1, 1, 1, 1};
  uint64_t last = (uint64_t)c.D * 2;
  for (int i = 0; i < 3; ++i) {
    if (d[i].n > 1 && d[i].stride <= 0) return false;
    *d[i].place = i;
    dims[i + 1] = d[i].n;
    strides[i] = d[i].n > 1 ? (uint64_t)d[i].stride * 2 : last;
    last = strides[i] * d[i].n;
    box[i + 1] = d[i].box;
    if (strides[i] >= 1ull << 40) return false;
  }
  const auto encode = tensor_map_encoder();
  return encode && encode(m, c.elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                          const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor maps of a call by the kernel for many tokens; false if there is none, or if k and v order their dimensions
// differently.
bool chunk_maps(const AttnArgs& a, ChunkLaunch* L) {
  ChunkGeo gk = L->geo;
  return cache_map(a.c, a.c.k, a.c.k_page, a.c.k_head, a.c.k_row, &gk, &L->k) &&
         cache_map(a.c, a.c.v, a.c.v_page, a.c.v_head, a.c.v_row, &L->geo, &L->v) && gk.dim_row == L->geo.dim_row &&
         gk.dim_head == L->geo.dim_head && gk.dim_page == L->geo.dim_page;
}

wan_status check_heads(const KvCache& c, int q_heads) {
  if (q_heads < 1 || q_heads % c.heads)
    return fail(WAN_ERR_SHAPE, "%d query heads are no multiple of the cache's %d", q_heads, c.heads);
  return WAN_OK;
}

}  // namespace

}  // namespace wan

using namespace wan;

extern "C" {

wan_status wan_rotary(const void* x, const int64_t x_strides[3], void* out, const int64_t out_strides[3],
                      int32_t dtype, int32_t B, int32_t T, int32_t heads, int32_t head_dim, const void* positions,
                      int32_t positions_64, int64_t positions_batch, const wan_rotation* rotation, int32_t inverse,
                      wan_cuda_stream stream) {
  API_GUARD({
    if (dtype != WAN_F32 && dtype != WAN_BF16 && dtype != WAN_F16) return fail(WAN_ERR_DTYPE, "dtype %d", dtype);
    if (B < 0 || T < 0 || heads < 1) return fail(WAN_ERR_INVALID_ARG, "%d x %d tokens of %d heads", B, T, heads);
    if (head_dim < 2 || head_dim % 2) return fail(WAN_ERR_INVALID_ARG, "head dim %d must be even", head_dim);
    if (head_dim > kMaxHeadDim) return fail(WAN_ERR_UNSUPPORTED, "head dim %d (at most 256)", head_dim);
    if (!rotation || !x_strides || !out_strides) return fail(WAN_ERR_INVALID_ARG, "null argument");
    if ((int64_t)B * T > 0x7fffffffLL || heads > 65535)
      return fail(WAN_ERR_UNSUPPORTED, "%lld tokens of %d heads", (long long)B * T, heads);
    RotaryArgs a;
    WAN_TRY(plan_of(rotation, head_dim, &a.plan));
    if (B == 0 || T == 0) return WAN_OK;
    if (!x || !out || !positions) return fail(WAN_ERR_INVALID_ARG, "null argument");
    const int size = elem_size(dtype);
    if (((uintptr_t)x | (uintptr_t)out) % size || (uintptr_t)positions % (positions_64 ? 8 : 4))
      return fail(WAN_ERR_INVALID_ARG, "x, out or positions not aligned to their elements");
    const int64_t dims[3] = {B, T, heads};
    for (int i = 0; i < 3; ++i)
      if (dims[i] > 1 && out_strides[i] == 0) return fail(WAN_ERR_INVALID_ARG, "out must not be broadcast");
    if (positions_batch < 0) return fail(WAN_ERR_INVALID_ARG, "positions_batch %lld", (long long)positions_batch);
    a.plan.inverse = inverse != 0;
    a.x = x;
    a.out = out;
    a.xb = x_strides[0], a.xs = x_strides[1], a.xh = x_strides[2];
    a.ob = out_strides[0], a.os = out_strides[1], a.oh = out_strides[2];
    a.pos = positions;
    a.pos64 = positions_64 != 0;
    a.pos_b = positions_batch;
    a.B = B, a.S = T, a.H = heads, a.D = head_dim;
    a.elem = dtype;
    a.width = access_width(size, 16 / size, x, {{B, a.xb}, {T, a.xs}, {heads, a.xh}});
    a.width = access_width(size, a.width, out, {{B, a.ob}, {T, a.os}, {heads, a.oh}});
    CUDA_TRY(launch_rotary(a, (cudaStream_t)stream));
    return WAN_OK;
  })
}

wan_status wan_kv_check(const wan_kv_batch* batch, int32_t page_size, int64_t pages, int32_t append) {
  API_GUARD({
    if (page_size < 1 || pages < 1) return fail(WAN_ERR_INVALID_ARG, "%lld pages of %d rows", (long long)pages, page_size);
    KvBatch b;
    WAN_TRY(check_batch(batch, page_size, &b));
    std::set<std::pair<int, int>> rows;  // (page, row) of every new token
    int next = 0;
    for (int i = 0; i < b.B; ++i) {
      int r0, n, len;
      if (!kv_rows(b.cu, b.T, i, &r0, &n) || (b.cu && r0 != next))
        return fail(WAN_ERR_INVALID_ARG, "sequence %d: its token range is none of the %d rows, or not the next one", i, b.T);
      next = r0 + n;
      if (!kv_length(b.lengths[i], b.max_pages, page_size, &len))
        return fail(WAN_ERR_INVALID_ARG, "sequence %d: length %d in a table of %d pages of %d keys", i, b.lengths[i],
                    b.max_pages, page_size);
      const int* row = b.pages + i * b.page_stride;
      for (int64_t k = 0; k < len; k += page_size)
        if (kv_page(row, (int)k, page_size, pages) < 0)
          return fail(WAN_ERR_INVALID_ARG, "sequence %d: page %d is number %d of a cache of %lld", i, (int)(k / page_size),
                      row[k / page_size], (long long)pages);
      if (!append) continue;
      if (n > len) return fail(WAN_ERR_INVALID_ARG, "sequence %d: %d new tokens among %d keys", i, n, len);
      for (int k = len - n; k < len; ++k)
        if (!rows.insert({row[k / page_size], k % page_size}).second)
          return fail(WAN_ERR_INVALID_ARG, "sequence %d: key %d shares its row with another new token", i, k);
    }
    return WAN_OK;
  })
}

wan_status wan_kv_check_compact(const wan_kv_batch* batch, const int32_t* held, const int32_t* keep, int32_t page_size,
                                int64_t pages) {
  API_GUARD({
    if (page_size < 1 || pages < 1) return fail(WAN_ERR_INVALID_ARG, "%lld pages of %d rows", (long long)pages, page_size);
    KvBatch b;
    WAN_TRY(check_batch(batch, page_size, &b));
    if (!b.cu || !held || (!keep && b.T > 0)) return fail(WAN_ERR_INVALID_ARG, "null ranges, lengths or keys");
    struct Place {
      int sequence, key;
    };
    std::map<std::pair<int, int>, Place> written;  // by page and row
    std::set<int> pages_written;
    for (int i = 0; i < b.B; ++i) {
      int r0, n, first, len;
      if (!kv_rows(b.cu, b.T, i, &r0, &n)) return fail(WAN_ERR_INVALID_ARG, "sequence %d: its range is none of the %d keys", i, b.T);
      if (!kv_length(held[i], b.max_pages, page_size, &len))
        return fail(WAN_ERR_INVALID_ARG, "sequence %d: length %d in a table of %d pages of %d keys", i, held[i], b.max_pages, page_size);
      if (!kv_length(b.lengths[i], b.max_pages, page_size, &first) || first > len)
        return fail(WAN_ERR_INVALID_ARG, "sequence %d: %d first keys of %d", i, b.lengths[i], len);
      const int* row = b.pages + i * b.page_stride;
      for (int j = 0; j < n; ++j) {
        const int from = keep[r0 + j], to = first + j;
        if (from < to || from >= len || (j > 0 && from <= keep[r0 + j - 1]))
          return fail(WAN_ERR_INVALID_ARG, "sequence %d: key %d of %d cannot move to place %d behind key %d", i, from, len, to,
                      j > 0 ? keep[r0 + j - 1] : -1);
        if (from == to) continue;
        for (const int k : {from, to})
          if (kv_page(row, k, page_size, pages) < 0)
            return fail(WAN_ERR_INVALID_ARG, "sequence %d: page %d is number %d of a cache of %lld", i, k / page_size,
                        row[k / page_size], (long long)pages);
        const auto put = written.insert({{row[to / page_size], to % page_size}, Place{i, to}});
        if (!put.second)
          return fail(WAN_ERR_INVALID_ARG, "sequence %d: place %d shares its row with place %d of sequence %d", i, to,
                      put.first->second.key, put.first->second.sequence);
        pages_written.insert(row[to / page_size]);
      }
    }
    // nothing that moves may land in a row that stands for another key
    for (int i = 0; i < b.B; ++i) {
      const int* row = b.pages + i * b.page_stride;
      for (int64_t k0 = 0; k0 < held[i]; k0 += page_size) {
        const int page = row[k0 / page_size];
        if (!pages_written.count(page)) continue;
        for (int r = 0; r < page_size && k0 + r < held[i]; ++r) {
          const auto w = written.find({page, r});
          if (w != written.end() && (w->second.sequence != i || w->second.key != k0 + r))
            return fail(WAN_ERR_INVALID_ARG, "sequence %d: key %d has its row in page %d, which place %d of sequence %d would be written to",
                        i, (int)(k0 + r), page, w->second.key, w->second.sequence);
        }
      }
    }
    return WAN_OK;
  })
}

wan_status wan_kv_status(int32_t* status, wan_cuda_stream stream) {
  API_GUARD({
    if (!status) return fail(WAN_ERR_INVALID_ARG, "null status word");
    int code = 0;
    CUDA_TRY(cudaMemcpyAsync(&code, status, sizeof(int), cudaMemcpyDeviceToHost, (cudaStream_t)stream));
    CUDA_TRY(cudaStreamSynchronize((cudaStream_t)stream));
    if (code == 0) return WAN_OK;
    CUDA_TRY(cudaMemsetAsync(status, 0, sizeof(int), (cudaStream_t)stream));
    if (code == kDevBadPage) return fail(WAN_ERR_INTERNAL, "a page table named a page outside the cache (code %d)", code);
    if (code == kDevBadParent)
      return fail(WAN_ERR_INTERNAL, "a drafted token's parent is none of the drafts before it (code %d)", code);
    if (code == kDevBadLength)
      return fail(WAN_ERR_INTERNAL, "a sequence's length or token range does not fit its batch (code %d)", code);
    return fail(WAN_ERR_INTERNAL, "a token kernel reported error %d (a bounded wait expired)", code);
  })
}

wan_status wan_kv_append(const wan_kv_cache* cache, const wan_kv_batch* batch, const void* k, int64_t k_token,
                         int64_t k_head, const void* v, int64_t v_token, int64_t v_head, const void* q,
                         int32_t q_heads, int64_t q_token, int64_t q_head, void* q_out, int64_t q_out_token,
                         int64_t q_out_head, const wan_rotation* rotation, const void* positions,
                         int32_t positions_64, wan_cuda_stream stream) {
  API_GUARD({
    AppendArgs a;
    WAN_TRY(check_cache(cache, &a.c));
    WAN_TRY(check_batch(batch, a.c.page_size, &a.b));
    if (rotation) {
      WAN_TRY(plan_of(rotation, a.c.D, &a.plan));
    } else {
      a.plan.pairs = 0;
      a.plan.axes = 0;
      a.plan.interleaved = 1;
      a.plan.inverse = 0;
    }
    if ((q != nullptr) != (q_out != nullptr)) return fail(WAN_ERR_INVALID_ARG, "q and q_out go together");
    if (q && q_heads < 1) return fail(WAN_ERR_INVALID_ARG, "%d query heads", q_heads);
    const int64_t strides[8] = {k_token, k_head, v_token, v_head, q ? q_token : 0, q ? q_head : 0, 1, 1};
    for (int64_t s : strides)
      if (s < 0) return fail(WAN_ERR_INVALID_ARG, "negative stride");
    const int T = a.b.T;
    if (q && ((T > 1 && q_out_token <= 0) || (q_heads > 1 && q_out_head <= 0)))
      return fail(WAN_ERR_INVALID_ARG, "q_out must not be broadcast");
    // one row of the cache per (page, head, row)
    const int64_t need[6] = {a.c.pages, a.c.heads, a.c.page_size, a.c.pages, a.c.heads, a.c.page_size};
    const int64_t have[6] = {a.c.k_page, a.c.k_head, a.c.k_row, a.c.v_page, a.c.v_head, a.c.v_row};
    for (int i = 0; i < 6; ++i)
      if (need[i] > 1 && have[i] == 0) return fail(WAN_ERR_INVALID_ARG, "a cache that is appended to must not be broadcast");
    if ((q ? q_heads : 0) + 2LL * a.c.heads > 60000) return fail(WAN_ERR_UNSUPPORTED, "%d heads", a.c.heads);
    if (T == 0) return WAN_OK;
    if (!k || !v || (rotation && !positions)) return fail(WAN_ERR_INVALID_ARG, "null keys, values or positions");
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)q | (uintptr_t)q_out) & 1 ||
        (uintptr_t)positions % (positions_64 ? 8 : 4))
      return fail(WAN_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    a.k = k, a.v = v, a.q = q, a.qo = q_out;
    a.k_t = k_token, a.k_h = k_head, a.v_t = v_token, a.v_h = v_head;
    a.q_t = q_token, a.q_h = q_head, a.qo_t = q_out_token, a.qo_h = q_out_head;
    a.q_heads = q ? q_heads : 0;
    a.pos = positions;
    a.pos64 = positions_64 != 0;
    a.width = access_width(2, 8, k, {{T, k_token}, {a.c.heads, k_head}});
    a.width = access_width(2, a.width, v, {{T, v_token}, {a.c.heads, v_head}});
    if (q) {
      a.width = access_width(2, a.width, q, {{T, q_token}, {q_heads, q_head}});
      a.width = access_width(2, a.width, q_out, {{T, q_out_token}, {q_heads, q_out_head}});
    }
    CUDA_TRY(launch_kv_append(a, (cudaStream_t)stream));
    return WAN_OK;
  })
}

static wan_status attention_args(const wan_kv_cache* cache, const wan_kv_batch* batch, int32_t q_heads, AttnArgs* a) {
  WAN_TRY(check_cache(cache, &a->c));
  WAN_TRY(check_batch(batch, a->c.page_size, &a->b));
  WAN_TRY(check_heads(a->c, q_heads));
  if ((int64_t)a->b.T * q_heads > 0x7fffffffLL) return fail(WAN_ERR_UNSUPPORTED, "%d tokens of %d heads", a->b.T, q_heads);
  a->q_heads = q_heads;
  a->group = q_heads / a->c.heads;
  a->stall_at1 = 0;
  a->mask = kMaskRanges;
  a->ranges = a->parents = nullptr;
  a->frame = a->span = 1;
  a->sinks = 0;
  return WAN_OK;
}

// An attention call whose sizes and mask are in `a`; its tensors and launch.
static wan_status attend(AttnArgs& a, const void* q, int64_t q_token, int64_t q_head, double scale, void* out,
                         int64_t out_token, int64_t out_head, float* lse, void* workspace, int64_t workspace_bytes,
                         wan_cuda_stream stream) {
  a.scale_log2 = (float)(scale * 1.4426950408889634);  // log2(e)
  if (!std::isfinite(a.scale_log2)) return fail(WAN_ERR_INVALID_ARG, "the scale is not finite, or too large");
  const int T = a.b.T;
  if (q_token < 0 || q_head < 0) return fail(WAN_ERR_INVALID_ARG, "negative stride");
  if ((T > 1 && out_token <= 0) || (a.q_heads > 1 && out_head <= 0))
    return fail(WAN_ERR_INVALID_ARG, "out must not be broadcast");
  if (T == 0) return WAN_OK;
  if (!q || !out) return fail(WAN_ERR_INVALID_ARG, "null q or out");
  if (a.mask == kMaskTree && !a.parents) return fail(WAN_ERR_INVALID_ARG, "null parents");
  if (((uintptr_t)q | (uintptr_t)out) & 1 || ((uintptr_t)lse | (uintptr_t)a.ranges | (uintptr_t)a.parents) & 3)
    return fail(WAN_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  int sms = 0;
  WAN_TRY(sm_count(&sms));
  ChunkLaunch L;
  bool chunk = chunk_rows(a, &L.geo);
  const int64_t bytes = workspace_of(a, chunk, sms);
  if (!workspace || ((uintptr_t)workspace & 15) || workspace_bytes < bytes)
    return fail(WAN_ERR_INVALID_ARG, "workspace of %lld bytes, 16-byte aligned, needed (%lld given)", (long long)bytes,
                (long long)workspace_bytes);
  a.q = q, a.out = out, a.lse = lse;
  a.q_t = q_token, a.q_h = q_head, a.o_t = out_token, a.o_h = out_head;
  a.workspace = workspace;
  if (chunk) {
    chunk = chunk_maps(a, &L);  // without them the split kernel runs (there is room for either)
    L.a = a;
  }
  CUDA_TRY(chunk ? launch_kv_chunk(L, sms, (cudaStream_t)stream) : launch_kv_attention(a, sms, (cudaStream_t)stream));
  return WAN_OK;
}

wan_status wan_kv_attention(const wan_kv_cache* cache, const wan_kv_batch* batch, const void* q, int32_t q_heads,
                            int64_t q_token, int64_t q_head, const int32_t* ranges, float scale, void* out,
                            int64_t out_token, int64_t out_head, float* lse, void* workspace,
                            int64_t workspace_bytes, wan_cuda_stream stream) {
  API_GUARD({
    AttnArgs a;
    WAN_TRY(attention_args(cache, batch, q_heads, &a));
    a.ranges = ranges;
    return attend(a, q, q_token, q_head, scale, out, out_token, out_head, lse, workspace, workspace_bytes, stream);
  })
}

wan_status wan_kv_window_attention(const wan_kv_cache* cache, const wan_kv_batch* batch, const void* q, int32_t q_heads,
                                   int64_t q_token, int64_t q_head, int32_t window, int32_t sinks, int32_t frame,
                                   float scale, void* out, int64_t out_token, int64_t out_head, float* lse,
                                   void* workspace, int64_t workspace_bytes, wan_cuda_stream stream) {
  API_GUARD({
    AttnArgs a;
    WAN_TRY(attention_args(cache, batch, q_heads, &a));
    if (window < 1 || frame < 1 || sinks < 0)
      return fail(WAN_ERR_INVALID_ARG, "a window of %d frames of %d keys, and %d first keys", window, frame, sinks);
    a.mask = kMaskWindow;
    a.frame = (uint32_t)frame;
    // (a frame's end is below 2^32, and 2^31 - 1 keys behind it may be short of the window)
    a.span = (uint32_t)std::min<int64_t>((int64_t)window * frame, 0xffffffffLL);
    a.sinks = sinks;
    return attend(a, q, q_token, q_head, scale, out, out_token, out_head, lse, workspace, workspace_bytes, stream);
  })
}

wan_status wan_kv_tree_attention(const wan_kv_cache* cache, const wan_kv_batch* batch, const void* q, int32_t q_heads,
                                 int64_t q_token, int64_t q_head, const int32_t* parents, float scale, void* out,
                                 int64_t out_token, int64_t out_head, float* lse, void* workspace,
                                 int64_t workspace_bytes, wan_cuda_stream stream) {
  API_GUARD({
    AttnArgs a;
    WAN_TRY(attention_args(cache, batch, q_heads, &a));
    a.mask = kMaskTree;
    a.parents = parents;
    return attend(a, q, q_token, q_head, scale, out, out_token, out_head, lse, workspace, workspace_bytes, stream);
  })
}

wan_status wan_kv_fork(const wan_kv_cache* cache, int32_t* pages, int64_t page_stride, int32_t max_pages,
                       int32_t sequences, int32_t* lengths, const int32_t* sources, const int32_t* targets,
                       const int32_t* fresh, int64_t fresh_stride, int32_t fresh_pages, int32_t forks, int32_t share,
                       int32_t* status, wan_cuda_stream stream) {
  API_GUARD({
    ForkArgs a;
    WAN_TRY(check_cache(cache, &a.c));
    WAN_TRY(check_written(a.c));
    const wan_kv_batch batch{pages, page_stride, max_pages, sequences, lengths, lengths, 0, status};
    KvBatch b;
    WAN_TRY(check_batch(&batch, a.c.page_size, &b));
    if (sequences > 1 && page_stride < max_pages)
      return fail(WAN_ERR_INVALID_ARG, "a page table that is written to must not be broadcast");
    if (forks < 0 || fresh_pages < 0) return fail(WAN_ERR_INVALID_ARG, "%d forks with %d pages each", forks, fresh_pages);
    if (forks > kMaxForks) return fail(WAN_ERR_UNSUPPORTED, "%d forks (at most %d a call)", forks, kMaxForks);
    if (fresh_stride < 0 || (fresh_stride < fresh_pages && forks > 1))
      return fail(WAN_ERR_INVALID_ARG, "fresh_stride %lld for rows of %d", (long long)fresh_stride, fresh_pages);
    if (share != 0 && share != 1) return fail(WAN_ERR_INVALID_ARG, "share must be 0 or 1");
    if (forks == 0) return WAN_OK;
    if (!sources || !targets || (!fresh && fresh_pages > 0)) return fail(WAN_ERR_INVALID_ARG, "null argument");
    if (((uintptr_t)pages | (uintptr_t)lengths | (uintptr_t)sources | (uintptr_t)targets | (uintptr_t)fresh |
         (uintptr_t)status) & 3)
      return fail(WAN_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    const int64_t table = (int64_t)(sequences - 1) * page_stride + max_pages, rest = (int64_t)(forks - 1) * fresh_stride + fresh_pages;
    const bool beside = fresh_pages > 0 && meet(fresh, rest, pages, table) && !columns_apart(fresh, fresh_stride, fresh_pages, forks, pages, page_stride, max_pages, sequences);
    if (beside || (fresh_pages > 0 && meet(fresh, rest, lengths, sequences)) || meet(sources, forks, pages, table) ||
        meet(targets, forks, pages, table) || meet(sources, forks, lengths, sequences) || meet(targets, forks, lengths, sequences) ||
        meet(lengths, sequences, pages, table))
      return fail(WAN_ERR_INVALID_ARG, "sources, targets, fresh, lengths and the page table must not share memory");
    a.pages = pages, a.lengths = lengths;
    a.page_stride = page_stride, a.max_pages = max_pages, a.B = sequences;
    a.sources = sources, a.targets = targets, a.fresh = fresh;
    a.fresh_stride = fresh_stride, a.fresh_pages = fresh_pages, a.N = forks;
    a.share = share;
    a.status = status;
    int sms = 0;
    WAN_TRY(sm_count(&sms));
    CUDA_TRY(launch_kv_fork(a, sms, (cudaStream_t)stream));
    return WAN_OK;
  })
}

wan_status wan_kv_compact(const wan_kv_cache* cache, const wan_kv_batch* batch, const int32_t* keep, int32_t* lengths,
                          wan_cuda_stream stream) {
  API_GUARD({
    CompactArgs a;
    WAN_TRY(check_cache(cache, &a.c));
    WAN_TRY(check_written(a.c));
    WAN_TRY(check_batch(batch, a.c.page_size, &a.b));
    if (!a.b.cu || !lengths || (!keep && a.b.T > 0)) return fail(WAN_ERR_INVALID_ARG, "null ranges, keys or lengths");
    if (((uintptr_t)a.b.pages | (uintptr_t)a.b.lengths | (uintptr_t)a.b.cu | (uintptr_t)keep | (uintptr_t)lengths |
         (uintptr_t)a.b.status) & 3)
      return fail(WAN_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    if (meet(lengths, a.b.B, a.b.lengths, a.b.B) || meet(lengths, a.b.B, a.b.cu, a.b.B + 1LL) || meet(lengths, a.b.B, keep, a.b.T) ||
        meet(lengths, a.b.B, a.b.pages, (a.b.B - 1) * a.b.page_stride + a.b.max_pages))
      return fail(WAN_ERR_INVALID_ARG, "lengths must not share memory with what the call reads");
    if (a.c.heads > 1000) return fail(WAN_ERR_UNSUPPORTED, "%d heads (at most 1000)", a.c.heads);
    const bool one = same_rows(a.c);
    if (!one && rows_meet(a.c))
      return fail(WAN_ERR_INVALID_ARG, "k and v must be one tensor or have no memory in common: their rows move in place");
    a.planes = (one ? 1 : 2) * a.c.heads;
    a.keep = keep;
    a.lengths = lengths;
    int sms = 0;
    WAN_TRY(sm_count(&sms));
    CUDA_TRY(launch_kv_compact(a, sms, (cudaStream_t)stream));
    return WAN_OK;
  })
}

int64_t wan_kv_attention_workspace(const wan_kv_cache* cache, const wan_kv_batch* batch, int32_t q_heads) {
  try {
    AttnArgs a;
    int sms = 0;
    if (attention_args(cache, batch, q_heads, &a) != WAN_OK || sm_count(&sms) != WAN_OK) return -1;
    ChunkGeo g;
    return workspace_of(a, chunk_rows(a, &g), sms);
  } catch (...) {
    fail(WAN_ERR_INTERNAL, "unexpected C++ exception");
    return -1;
  }
}

int64_t wan_kv_masked_attention_workspace(const wan_kv_cache* cache, const wan_kv_batch* batch, int32_t q_heads) {
  try {
    AttnArgs a;
    int sms = 0;
    if (attention_args(cache, batch, q_heads, &a) != WAN_OK || sm_count(&sms) != WAN_OK) return -1;
    a.mask = kMaskTree;
    ChunkGeo g;
    return workspace_of(a, chunk_rows(a, &g), sms);
  } catch (...) {
    fail(WAN_ERR_INTERNAL, "unexpected C++ exception");
    return -1;
  }
}

wan_status wan_selftest_kv_attention_timeout(int32_t head_dim, int32_t* device_code, wan_cuda_stream stream) {
  API_GUARD({
    if (device_code) *device_code = 0;
    if (head_dim < 8 || head_dim % 8 || head_dim > kMaxHeadDim)
      return fail(WAN_ERR_INVALID_ARG, "head dim %d (a multiple of 8 up to 256)", head_dim);
    cudaStream_t s = (cudaStream_t)stream;
    // 290 tokens of 4 query heads against 500 keys of 2 heads, 10 tokens without a key, and 10 rows behind them
    constexpr int kHeads = 2, kQHeads = 4, kPage = 64, kPages = 8, kSeqs = 2, kNew = 290, kOwned = 300, kRows = 310;
    const int32_t tables[2 * kPages + kSeqs + kSeqs + 1] = {0, 1, 2, 3, 4, 5, 6, 7, 0, 0, 0, 0, 0, 0, 0, 0,
                                                            500, 0, 0, kNew, kOwned};
    const int64_t plane = (int64_t)kPage * head_dim, cache_bytes = kPages * kHeads * plane * 2;
    const int64_t row = (int64_t)kQHeads * head_dim, out_n = kRows * row, lse_n = (int64_t)kRows * kQHeads;
    wan_kv_cache c{(void*)16, (void*)16, WAN_BF16, kHeads, kPage, head_dim, kPages, kHeads * plane, plane, head_dim,
                   kHeads * plane, plane, head_dim};
    wan_kv_batch b{(int32_t*)16, kPages, kPages, kSeqs, (int32_t*)16, (int32_t*)16, kRows, nullptr};
    AttnArgs a;
    int sms = 0;
    WAN_TRY(attention_args(&c, &b, kQHeads, &a));
    WAN_TRY(sm_count(&sms));
    ChunkLaunch L;
    if (!kv_chunk_geometry(a, &L.geo)) return fail(WAN_ERR_INTERNAL, "the kernel for many tokens does not take the case");
    // one allocation: K, V, q | out | lse | tables | status word | workspace, each on a 256-byte boundary
    const int64_t sizes[6] = {2 * cache_bytes + out_n * 2, out_n * 2, lse_n * 4, (int64_t)sizeof(tables), 4,
                              kv_chunk_workspace(a, sms)};
    int64_t at[7] = {0};
    for (int i = 0; i < 6; ++i) at[i + 1] = (at[i] + sizes[i] + 255) / 256 * 256;
    std::vector<uint16_t> out(out_n);
    std::vector<float> lse(lse_n);
    struct Mem {
      char* p = nullptr;
      cudaStream_t s;
      ~Mem() {
        if (p) cudaFreeAsync(p, s);
      }
    } mem;
    mem.s = s;
    CUDA_TRY(cudaMallocAsync((void**)&mem.p, at[6], s));
    a.c.k = mem.p;
    a.c.v = mem.p + cache_bytes;
    a.q = mem.p + 2 * cache_bytes;
    a.out = mem.p + at[1];
    a.lse = (float*)(mem.p + at[2]);
    int* table = (int*)(mem.p + at[3]);
    a.b.pages = table;
    a.b.lengths = table + 2 * kPages;
    a.b.cu = table + 2 * kPages + kSeqs;
    int* word = (int*)(mem.p + at[4]);
    a.workspace = mem.p + at[5];
    a.ranges = nullptr;
    a.q_t = a.o_t = row;
    a.q_h = a.o_h = head_dim;
    a.scale_log2 = 1.f;
    a.stall_at1 = 1;  // each SM's first block of keys is never loaded
    if (!chunk_maps(a, &L)) return fail(WAN_ERR_INTERNAL, "no tensor map of the case");
    int code = 0;
    for (int told = 1; told >= 0; --told) {  // with a status word, and without
      a.b.status = told ? word : nullptr;
      L.a = a;
      CUDA_TRY(cudaMemsetAsync(mem.p, 0, at[1], s));
      CUDA_TRY(cudaMemsetAsync(mem.p + at[1], 0x11, at[6] - at[1], s));
      CUDA_TRY(cudaMemsetAsync(word, 0, 4, s));
      CUDA_TRY(cudaMemcpyAsync(table, tables, sizeof(tables), cudaMemcpyHostToDevice, s));
      CUDA_TRY(launch_kv_chunk(L, sms, s));
      if (told) CUDA_TRY(cudaMemcpyAsync(&code, word, 4, cudaMemcpyDeviceToHost, s));
      CUDA_TRY(cudaMemcpyAsync(out.data(), a.out, out_n * 2, cudaMemcpyDeviceToHost, s));
      CUDA_TRY(cudaMemcpyAsync(lse.data(), a.lse, lse_n * 4, cudaMemcpyDeviceToHost, s));
      CUDA_TRY(cudaStreamSynchronize(s));
      for (int64_t i = 0; i < out_n; ++i) {
        const int64_t r = i / row;
        const uint16_t e = out[i];
        if (r < kNew ? (e & 0x7fff) <= 0x7f80 : e != (r < kOwned ? 0 : 0x1111))
          return fail(WAN_ERR_INTERNAL, "row %lld holds %#x after a wait that ran out", (long long)r, e);
      }
      for (int64_t i = 0; i < kNew * kQHeads; ++i)
        if (!std::isnan(lse[i])) return fail(WAN_ERR_INTERNAL, "lse %lld is a number after a wait that ran out", (long long)i);
    }
    if (device_code) *device_code = code;
    if (code) return fail(WAN_ERR_INTERNAL, "a token kernel reported error %d (a bounded wait expired)", code);
    return WAN_OK;
  })
}

}  // extern "C"
