// tree.h -- attention of drafted tokens over the cache (tree.cu): argument block and launcher.
#pragma once

#include "kernels.h"

namespace lrkv {

struct TreeArgs {
    DecodeArgs d;  // queries ([batch * T][H][..], B = batch * T), factors, block table, lengths, q~
    const uint16_t *sK, *sV, *zK, *zV;
    const unsigned long long* mask;  // [batch][T], or null: a chain
    const int32_t* tree_lens;        // [batch], or null: T
    int batch, T;
};
size_t tree_workspace_bytes(int H, int D_H, int R, int D_R, int batch, int T, int sms);
cudaError_t launch_tree(TreeArgs a, int D_H, int R, int D_R, void* ws, int sms, cudaStream_t stream);

}  // namespace lrkv
