// tree.h -- attention of drafted tokens over the cache (tree.cu): argument block and launcher.
#pragma once

#include "kernels.h"

namespace lrkv {

struct TreeArgs {
    // Queries ([batch * T][H][..], B = batch * T: the absorb takes every drafted token as a query), factors, block
    // table, lengths, q~, status, limits.
    DecodeArgs d;
    const uint16_t *sK, *zK, *sV, *zV;  // the pools that the tensor maps show
    const unsigned long long* mask;     // [batch][T], or null: a chain
    const int32_t* tree_lens;           // [batch], or null: T
    int batch, T;
    int zw, hb, ns, htiles, tmax;  // the tile (below); tmax: tiles of a sequence with T drafted tokens
    int gang, gangs, gmax;         // CTAs that take neighbouring tiles together, gangs, groups of a sequence's tiles
    int tn, rs;                    // drafted tokens of a tile at most (T or ns), rows kept of a tile (hb tn and up to 31)
    int2* seg_table;               // [batch * tmax] first partial and their number
    float2* ml;                    // [slot][rs] running max (log2 domain) and sum
    float4* acc;                   // [slot][(D_H + R) / 4][rs]
};

// A CTA's 128 query rows are hb heads x ns drafted tokens of one sequence, with hb r = zw columns of latents.
struct TreePlan {
    int zw, hb, ns, htiles, stiles;
};
TreePlan tree_plan(int H, int D_H, int R, int D_R, int T);
size_t tree_workspace_bytes(int H, int D_H, int R, int D_R, int batch, int T, int sms);
void tree_carve_workspace(TreeArgs* a, void* ws, int D_H, int R, int D_R, int sms);

// Maps over the pools: [s^K | k^R], s^V as [num_blocks * 64][d_h (+ d_rope)], box 64 columns x 64 tokens, 128-byte
// swizzle; z^K, z^V as [num_blocks * 64][H r], the same box.  For zw = 32 s^V, z^K and z^V have boxes of 32 columns x 64
// tokens with 64-byte swizzle.
struct TreeMaps {
    CUtensorMap sK, sV, zK, zV;
};
cudaError_t launch_tree(const TreeMaps& maps, const TreeArgs& a, int D_H, int R, int D_R, cudaStream_t stream);

}  // namespace lrkv
