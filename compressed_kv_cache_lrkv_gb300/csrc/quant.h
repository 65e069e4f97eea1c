// quant.h -- the 8-bit rows of a quantised cache, and the launchers that write, read and
// attend over them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace lrkv {

// Values per scale.  One power-of-two scale per 32 values: 1/32 of overhead, and 32 covers one
// head's latents at r = 32, two at r = 16, four at r = 8, so a head never has two scales.
constexpr int kQuantBlock = 32;

// Byte layout of a token's row (see lrkv_cache_quantize in lrkv.h):
//   [s^K (d_h + d_rope) | s^V (d_h) | z^K (H r, padded to 16) | z^V (ditto) | scale bytes | pad]
// The row is an odd number of 16-byte units long: consecutive tokens' rows then start 16 bytes
// (mod 128) times an odd number apart, so the same 16-byte chunk of eight consecutive tokens lies
// in eight different groups of shared-memory banks, and rows copied as they are can be read by
// token without bank conflicts.
struct QuantLayout {
    int d_k, d_h, HR;                 // widths of s^K, s^V, z^K (= z^V)
    int off_sV, off_zK, off_zV;       // byte offsets (s^K is at 0)
    int off_sc;                       // scale bytes: s^K's blocks, s^V's, z^K's, z^V's
    int nb_sK, nb_sV, nb_z;           // blocks of each part
    int row_bytes;
};

__host__ __device__ inline QuantLayout quant_layout(int d_h, int d_rope, int H, int r) {
    QuantLayout q{};
    q.d_k = d_h + d_rope;
    q.d_h = d_h;
    q.HR = H * r;
    q.off_sV = q.d_k;
    q.off_zK = q.off_sV + d_h;
    const int zpad = (q.HR + 15) & ~15;
    q.off_zV = q.off_zK + zpad;
    q.off_sc = q.off_zV + zpad;
    q.nb_sK = q.d_k / kQuantBlock;
    q.nb_sV = d_h / kQuantBlock;
    q.nb_z = (q.HR + kQuantBlock - 1) / kQuantBlock;
    const int units = (q.off_sc + q.nb_sK + q.nb_sV + 2 * q.nb_z + 15) / 16;
    q.row_bytes = 16 * (units | 1);
    return q;
}

struct QuantStoreArgs {
    uint16_t *sK, *sV, *zK, *zV;  // bf16 pools (read by quantize, written by dequantize)
    uint8_t* rows;                // quantised rows
    const int32_t* bf_slots;      // [n] token slots in the bf16 pools
    const int32_t* q_slots;       // [n] token slots in the quantised rows
    uint32_t* status;
    int n;
    long long bf_nslots, q_nslots;
    QuantLayout q;
};
cudaError_t launch_cache_quantize(const QuantStoreArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_cache_dequantize(const QuantStoreArgs& a, int sms, cudaStream_t stream);

// Decode over quantised rows.  `d` carries queries, factors, outputs, workspace and the work plan
// as for the bf16 decode (its pools are unused); one layer, one head group.
struct QuantDecodeArgs {
    DecodeArgs d;
    const uint8_t* rows;  // [num_blocks * 64][q.row_bytes]
    QuantLayout q;
};
size_t quant_decode_workspace_bytes(int H, int D_H, int R, int B, int nranges);
cudaError_t launch_quant_decode(QuantDecodeArgs a, void* ws, int D_H, int R, int D_R, int sms, int smem_limit,
                                cudaStream_t stream);

}  // namespace lrkv
