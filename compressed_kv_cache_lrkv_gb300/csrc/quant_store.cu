// quant_store.cu -- a cache quantised as it is written, and read back.
//
// Each block of 32 values x_i of a token's row has one scale 2^k:
//     k = exponent(max |x_i|) - 6,   q_i = min(127, max(-127, rint(x_i / 2^k)))
// so the largest magnitude lands in [64, 128).  bf16 has 8 significant bits, so the division (a
// power of two) is exact, the largest quotient is 127.5, and every value is stored to within half
// a step: |x_i - q_i 2^k| <= 2^(k-1) <= max|x| 2^-7.  q_i 2^k has 7 significant bits and is
// exact in bf16, so reading back rounds nothing.
// Both directions move each value once and do a handful of operations on it: bound by memory (by
// the launch for a decode step's few rows).  A warp takes one token's row, a lane eight
// consecutive values (16 bytes of bf16, 8 of the row); the four lanes of a block agree on its
// scale with two shuffles.
#include "lrkv_internal.cuh"
#include "quant.h"

namespace lrkv {

namespace {

constexpr int kStoreWarps = 8;

// Where the eight values of lane-chunk c of a row lie.  Chunks are counted part after part, each
// part padded to whole blocks (four chunks).
struct Chunk {
    int part;   // 0..3: s^K, s^V, z^K, z^V
    int first;  // first value within the part; >= its width where the chunk is padding
    int width;
    int off;    // byte offset of the part in the row
    int sc;     // byte offset of the part's scales
};
__device__ __forceinline__ Chunk chunk_at(const QuantLayout& q, int c) {
    const int c1 = q.nb_sK * 4, c2 = c1 + q.nb_sV * 4, c3 = c2 + q.nb_z * 4;
    if (c < c1) return {0, c * 8, q.d_k, 0, q.off_sc};
    if (c < c2) return {1, (c - c1) * 8, q.d_h, q.off_sV, q.off_sc + q.nb_sK};
    if (c < c3) return {2, (c - c2) * 8, q.HR, q.off_zK, q.off_sc + q.nb_sK + q.nb_sV};
    return {3, (c - c3) * 8, q.HR, q.off_zV, q.off_sc + q.nb_sK + q.nb_sV + q.nb_z};
}
__device__ __forceinline__ int total_chunks(const QuantLayout& q) { return (q.nb_sK + q.nb_sV + 2 * q.nb_z) * 4; }

// The pair of token slots of row i, or false where a slot is negative (the row is skipped) or
// out of range (reported and skipped).
__device__ __forceinline__ bool row_slots(const QuantStoreArgs& a, int i, int lane, long long* bf, long long* qs) {
    *bf = a.bf_slots[i];
    *qs = a.q_slots[i];
    if (*bf < 0 || *qs < 0) return false;
    if (*bf >= a.bf_nslots || *qs >= a.q_nslots) {
        if (lane == 0) set_status(a.status, LRKV_DEV_BAD_SLOT);
        return false;
    }
    return true;
}

__device__ __forceinline__ uint16_t* part_row(const QuantStoreArgs& a, const Chunk& ch, long long slot) {
    uint16_t* base = ch.part == 0 ? a.sK : ch.part == 1 ? a.sV : ch.part == 2 ? a.zK : a.zV;
    return base + slot * ch.width + ch.first;
}

__global__ void __launch_bounds__(kStoreWarps * 32) quantize_kernel(const QuantStoreArgs a) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * kStoreWarps + (threadIdx.x >> 5);
    long long bf, qs;
    if (i >= a.n || !row_slots(a, i, lane, &bf, &qs)) return;
    uint8_t* row = a.rows + qs * a.q.row_bytes;
    const int nc = total_chunks(a.q);
    for (int c0 = 0; c0 < nc; c0 += 32) {
        const int c = c0 + lane;
        const Chunk ch = chunk_at(a.q, min(c, nc - 1));
        const bool live = c < nc && ch.first < ch.width;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = *reinterpret_cast<const uint4*>(part_row(a, ch, bf));
        // the largest magnitude of the block as bf16 bits (their order is that of the values; a NaN
        // or infinity ends with exponent 255)
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = (int)(mx >> 7);
        // scale byte e: scale 2^(e - 127); at least 1 (2^-126: smaller values are flushed towards
        // zero in steps of it), 255 for a block with a NaN or infinity
        const int e = ex == 255 ? 255 : max(ex - 6, 1);
        // 2^-(e - 127): e is in [1, 248] for a finite block, so its exponent field 254 - e is in [6, 253]
        const float inv = __uint_as_float((uint32_t)(254 - min(e, 253)) << 23);
        if (live) {
            uint32_t out[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float lo = ex == 255 ? 0.f : fminf(fmaxf(rintf(bf16lo(w[k]) * inv), -127.f), 127.f);
                const float hi = ex == 255 ? 0.f : fminf(fmaxf(rintf(bf16hi(w[k]) * inv), -127.f), 127.f);
                const uint32_t b = (uint32_t)((int)lo + 128) | ((uint32_t)((int)hi + 128) << 8);
                out[k >> 1] |= b << (16 * (k & 1));
            }
            *reinterpret_cast<uint2*>(row + ch.off + ch.first) = make_uint2(out[0], out[1]);
            if ((c & 3) == 0) row[ch.sc + (ch.first >> 5)] = (uint8_t)e;
        }
    }
}

__global__ void __launch_bounds__(kStoreWarps * 32) dequantize_kernel(const QuantStoreArgs a) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * kStoreWarps + (threadIdx.x >> 5);
    long long bf, qs;
    if (i >= a.n || !row_slots(a, i, lane, &bf, &qs)) return;
    const uint8_t* row = a.rows + qs * a.q.row_bytes;
    const int nc = total_chunks(a.q);
    for (int c = lane; c < nc; c += 32) {
        const Chunk ch = chunk_at(a.q, c);
        if (ch.first >= ch.width) continue;
        const uint2 v = *reinterpret_cast<const uint2*>(row + ch.off + ch.first);
        const uint32_t e = row[ch.sc + (ch.first >> 5)];
        // scale 2^(e - 127); byte 255 stands for NaN, byte 0 (a row never written) for zero
        const float s = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
        const uint32_t w[2] = {v.x, v.y};
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int lo = (int)((w[k >> 1] >> (16 * (k & 1))) & 0xff) - 128;
            const int hi = (int)((w[k >> 1] >> (16 * (k & 1) + 8)) & 0xff) - 128;
            out[k] = pack_bf16x2((float)lo * s, (float)hi * s);
        }
        *reinterpret_cast<uint4*>(part_row(a, ch, bf)) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

}  // namespace

cudaError_t launch_cache_quantize(const QuantStoreArgs& a, cudaStream_t stream) {
    quantize_kernel<<<(a.n + kStoreWarps - 1) / kStoreWarps, kStoreWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_dequantize(const QuantStoreArgs& a, cudaStream_t stream) {
    dequantize_kernel<<<(a.n + kStoreWarps - 1) / kStoreWarps, kStoreWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace lrkv
