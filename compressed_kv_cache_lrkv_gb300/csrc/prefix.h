// prefix.h -- decode of a batch whose sequences share a prefix: argument block and launchers.
#pragma once

#include "kernels.h"

namespace lrkv {

struct PrefixArgs {
    // Queries, q~, factors, output (or partials out) and, where the sequences have tokens of their
    // own, their lengths and the workspace their scan leaves its partials in.
    DecodeArgs d;
    const uint16_t *sK, *sV, *zK, *zV;  // pools that hold the prefix's pages
    const int32_t* blocks;              // [max_blocks] pages of the prefix
    const int32_t* len;                 // [1] tokens of the prefix
    int max_blocks;
    int suffix;                         // 1: the sequences' own partials are in d's workspace
    int nsplit;                         // pieces the prefix is cut into
    float* ml;                          // [B][H][nsplit][2] running max (log2 domain) and sum
    float* acc;                         // [B][H][nsplit][D_H + R]
};

// Pieces a prefix of up to max_blocks pages is cut into, and the workspace of its partials.
int prefix_splits(int H, int R, int B, int max_blocks, int sms);
size_t prefix_workspace_bytes(int H, int D_H, int R, int B, int nsplit);
void prefix_carve_workspace(PrefixArgs* a, void* ws, int D_H, int R);

cudaError_t launch_prefix_scan(const PrefixArgs& a, int D_H, int R, int D_R, cudaStream_t stream);
// Log-sum-exp merge of the prefix's partials with the sequences' own; B^V and the bf16 output, or
// merged partials where d.part_out is set.
cudaError_t launch_prefix_combine(const PrefixArgs& a, int D_H, int R, cudaStream_t stream);

}  // namespace lrkv
