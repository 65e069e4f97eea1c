// prefix.h -- decode of a batch whose sequences share a prefix: argument block and launchers.
#pragma once

#include "kernels.h"

namespace lrkv {

struct PrefixArgs {
    // Queries, q~, factors, output (or partials out) and, where the sequences have tokens of their
    // own, their lengths and the workspace their scan leaves its partials in.
    DecodeArgs d;
    const uint16_t *sK, *zK;            // the pools that the tensor maps show (logits formed again, prefix.cu)
    const int32_t* blocks;              // [max_blocks] pages of the prefix
    const int32_t* len;                 // [1] tokens of the prefix
    int max_blocks;
    int suffix;                         // 1: the sequences' own partials are in d's workspace
    int nsplit, zw, hb, ns, htiles;     // the plan below
    float* ml;                          // [B][H][nsplit][2] running max (log2 domain) and sum
    float* acc;                         // [B][H][nsplit][D_H + R]
};

// How the scan cuts the work.  A CTA's 128 query rows are hb heads x ns sequences with hb r = zw
// columns of latents (zw 64 or 128); tiles = ceil(H / hb) ceil(B / ns), each cut into nsplit pieces
// of the prefix; own_sms SMs are left to the scan of the sequences' own tokens (0: it runs after).
struct PrefixPlan {
    int zw, hb, ns, htiles, stiles, nsplit, own_sms;
};
// own_bytes: cache bytes the sequences' own tokens may have (0: none are scanned).
PrefixPlan prefix_plan(int H, int D_H, int R, int D_R, int B, int max_blocks, double own_bytes, int sms);
// Pieces at most of any plan for these sizes (prefix_plan never takes more than two waves of pieces).
int prefix_most_splits(int H, int D_H, int R, int D_R, int B, int max_blocks, int sms);
size_t prefix_workspace_bytes(int H, int D_H, int R, int B, int nsplit);
void prefix_carve_workspace(PrefixArgs* a, void* ws, int D_H, int R);

// Maps over the pools, boxes of 64 tokens x 64 columns, 128-byte swizzle: s^K ([s^K | k^R]), s^V as
// [num_blocks * 64][d_h (+ d_rope)], z^K, z^V as [num_blocks * 64][H r].
struct PrefixMaps {
    CUtensorMap sK, sV, zK, zV;
};
cudaError_t launch_prefix_scan(const PrefixMaps& maps, const PrefixArgs& a, int D_H, int R, int D_R,
                               cudaStream_t stream);
// Log-sum-exp merge of the prefix's partials with the sequences' own; B^V and the bf16 output, or
// merged partials where d.part_out is set.
cudaError_t launch_prefix_combine(const PrefixArgs& a, int D_H, int R, int sms, cudaStream_t stream);

}  // namespace lrkv
