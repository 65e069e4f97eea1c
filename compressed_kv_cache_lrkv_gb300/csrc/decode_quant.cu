// decode_quant.cu -- factored decode over a cache of 8-bit rows (quant.h).
//
// Per sequence b and head h, with q~_h = q_h B_h^K and the rows' values s, z read as q_i 2^k:
//     score_t = (q_h . s^K_t + q~_h . z^K_{h,t}) * scale,   out_h = sum p s^V + B_h^V (sum p z^V)
// A block per (split, head, sequence); a warp takes every eighth token of the split with an online
// softmax of its own, the warps' states are merged at the end into one partial.
#include "lrkv_internal.cuh"
#include "quant.h"

namespace lrkv {

namespace {

constexpr int kSplits = 16;
constexpr int kWarps = 8;

// Value of byte u of block scale byte e.
__device__ __forceinline__ float quant_scale(uint32_t e) {
    return e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
}

template <int D_H, int R, int D_R>
__global__ void __launch_bounds__(kWarps * 32) quant_scan_kernel(const QuantDecodeArgs a) {
    constexpr int D_K = D_H + D_R, W = D_H + R;
    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DecodeArgs& d = a.d;
    const int slot = b * kSplits + split;
    if (split == 0 && h == 0 && threadIdx.x == 0) d.seg_table[b] = make_int2(b * kSplits, kSplits);
    float* pml = d.part_ml + ((size_t)h * d.pmax + slot) * 2;
    float* pacc = d.part_acc + ((size_t)h * d.pmax + slot) * W;
    const int L = d.seq_lens[b];
    const bool good = L >= 1 && L <= d.max_pages * kBlockSize;
    const int per = good ? (L + kSplits - 1) / kSplits : 0;
    const int t0 = split * per, t1 = good ? min(L, t0 + per) : 0;

    const uint16_t* q = d.q + ((size_t)b * d.H + h) * D_K;
    float qr[D_K / 32], o[D_H / 32];
#pragma unroll
    for (int i = 0; i < D_K / 32; ++i) qr[i] = __uint_as_float((uint32_t)q[i * 32 + lane] << 16);
#pragma unroll
    for (int i = 0; i < D_H / 32; ++i) o[i] = 0.f;
    const float qt = lane < R ? d.qt[((size_t)b * d.H + h) * R + lane] : 0.f;
    float oz = 0.f, m = -INFINITY, l = 0.f;
    for (int t = t0 + warp; t < t1; t += kWarps) {
        const int blk = d.block_table[(size_t)b * d.max_pages + t / kBlockSize];
        if (blk < 0 || blk >= d.num_blocks) {
            if (lane == 0) set_status(d.status, LRKV_DEV_BAD_BLOCK);
            continue;
        }
        const uint8_t* row = a.rows + ((size_t)blk * kBlockSize + t % kBlockSize) * a.q.row_bytes;
        const uint8_t* sc = row + a.q.off_sc;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < D_K / 32; ++i) s = fmaf(qr[i], ((int)row[i * 32 + lane] - 128) * quant_scale(sc[i]), s);
        const int zi = h * R + lane;
        if (lane < R)
            s = fmaf(qt, ((int)row[a.q.off_zK + zi] - 128) * quant_scale(sc[a.q.nb_sK + a.q.nb_sV + (zi >> 5)]), s);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= d.scale_log2;
        const float mn = fmaxf(m, s);
        const float al = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * al + p;
#pragma unroll
        for (int i = 0; i < D_H / 32; ++i)
            o[i] = fmaf(p, ((int)row[a.q.off_sV + i * 32 + lane] - 128) * quant_scale(sc[a.q.nb_sK + i]), o[i] * al);
        if (lane < R)
            oz = fmaf(p,
                      ((int)row[a.q.off_zV + zi] - 128) *
                          quant_scale(sc[a.q.nb_sK + a.q.nb_sV + a.q.nb_z + (zi >> 5)]),
                      oz * al);
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][W];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < D_H / 32; ++i) so[warp][i * 32 + lane] = o[i];
    if (lane < R) so[warp][D_H + lane] = oz;
    __syncthreads();
    float M = -INFINITY;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    float ls = 0.f, v = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        const float x = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M);
        ls = fmaf(x, sl[w], ls);
        if (threadIdx.x < W) v = fmaf(x, so[w][threadIdx.x], v);
    }
    if (threadIdx.x < W) pacc[threadIdx.x] = v;
    if (threadIdx.x == 0) {
        pml[0] = M;
        pml[1] = ls;
    }
}

template <int D_H, int R, int D_R>
cudaError_t launch_t(const QuantDecodeArgs& a, int sms, cudaStream_t stream) {
    quant_scan_kernel<D_H, R, D_R><<<dim3(kSplits, a.d.H, a.d.B), kWarps * 32, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_decode_combine(a.d, D_H, R, sms, stream);
}

}  // namespace

size_t quant_decode_workspace_bytes(int H, int D_H, int R, int B, int nranges) {
    (void)nranges;
    return decode_workspace_bytes(H, D_H, R, B, B * kSplits);
}

cudaError_t launch_quant_decode(QuantDecodeArgs a, void* ws, int D_H, int R, int D_R, int sms, int smem_limit,
                                cudaStream_t stream) {
    (void)smem_limit;
    decode_carve_workspace(&a.d, ws, a.d.H, D_H, R, a.d.B, a.d.B * kSplits);
    const cudaError_t e = launch_decode_absorb(a.d, D_H, R, D_R, stream);
    if (e != cudaSuccess) return e;
#define LRKV_QD(DH, RR)                                                                             \
    if (D_H == DH && R == RR)                                                                       \
        return D_R == 0 ? launch_t<DH, RR, 0>(a, sms, stream) : launch_t<DH, RR, 64>(a, sms, stream);
    LRKV_QD(64, 8) LRKV_QD(64, 16) LRKV_QD(64, 32) LRKV_QD(128, 8) LRKV_QD(128, 16) LRKV_QD(128, 32)
#undef LRKV_QD
    return cudaErrorInvalidValue;
}

}  // namespace lrkv
