// Launch descriptor of the attention of many new tokens (kv_chunk.cu).
#pragma once

#include <cuda.h>

#include "token_ops.h"

namespace wan {

// How pages fill the blocks of 128 key columns, and how the tensor maps order
// their dimensions (channels first, then rows, heads and pages by stride).
struct ChunkGeo {
  int box_rows;  // rows of a TMA box: the page's rows rounded up to 8, at most 128
  int pages;     // pages per block (parts == 1), else 1
  int parts;     // blocks per page (pages longer than a block), else 1
  int dim_row, dim_head, dim_page;  // positions among the map's dimensions 1..3 (0-based)
};
struct ChunkLaunch {
  CUtensorMap k, v;  // box 64 channels x box_rows rows
  AttnArgs a;
  ChunkGeo geo;
};
// False if the kernel does not take the cache's page size or head dim.
bool kv_chunk_geometry(const AttnArgs& a, ChunkGeo* g);
long long kv_chunk_workspace(const AttnArgs& a, int sms);
cudaError_t launch_kv_chunk(const ChunkLaunch& L, int sms, cudaStream_t s);

}  // namespace wan
