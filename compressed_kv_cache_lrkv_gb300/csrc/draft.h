// draft.h -- argument blocks and launchers of the calls around drafted tokens: rotary positions and page operations
// (rope.cu, pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lrkv.h"

namespace lrkv {

struct RopeArgs {
    lrkv_rope_plan plan;
    const void* x;
    void* y;
    const int32_t *x_index, *y_index, *positions;
    long long x_rows, y_rows, x_row, x_head, y_row, y_head;  // rows that exist, strides in elements
    uint32_t* status;
    int n, heads, width, begin;
    int transpose, in_place;
};
cudaError_t launch_rope(const RopeArgs& a, bool fp32, int sms, cudaStream_t stream);

// Pools as 16-byte units: a token row of pool p is u[p] units.
struct PoolArgs {
    uint4* base[LRKV_MAX_POOLS];
    long long layer[LRKV_MAX_POOLS];  // units between layers
    int u[LRKV_MAX_POOLS];
    int pools, layers, num_blocks;
    int units;  // of a token row over all pools
};
struct PageArgs {
    int32_t *refs, *table, *lens;
    const int32_t *a, *b;  // reserve: -, new_tokens; fork: parents, children; free: seqs, keep_lens (or null)
    uint32_t* status;
    int num_blocks, max_pages, batch, n;
};
struct CompactArgs {
    PoolArgs p;
    const int32_t *table, *path, *path_lens;
    int32_t *lens, *new_lens;
    uint32_t* status;
    int max_pages, batch, max_path;
};
cudaError_t launch_pages_reserve(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_pages_fork(const PoolArgs& p, const PageArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_pages_free(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_pages_copy(const PoolArgs& src, const PoolArgs& dst, const int32_t* src_pages,
                              const int32_t* dst_pages, int n, int sms, uint32_t* status, cudaStream_t stream);
cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream);

}  // namespace lrkv
