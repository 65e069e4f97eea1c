// prefix.cu -- one decode step of a batch whose sequences share a prefix.
//
// Softmax attention over the prefix's tokens and a sequence's own is the log-sum-exp merge of the
// two parts' states (m, l, acc), so the prefix is scanned once for the whole batch:
//     per (sequence b, head h):  s_t = (q_bh . s^K_t + q~_bh . z^K_{h,t}) * scale * log2 e
//     m = max s_t,  l = sum 2^(s_t - m),  acc = sum 2^(s_t - m) [s^V_t | z^V_{h,t}]
// and the combine merges its pieces with the partials of the sequences' own scan.
// A block per (piece, head, sequence); a warp takes every eighth token with an online softmax of
// its own, the warps' states are merged at the end.
#include "lrkv_internal.cuh"
#include "prefix.h"

namespace lrkv {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float bf(const uint16_t* p, size_t i) { return __uint_as_float((uint32_t)p[i] << 16); }

__device__ __forceinline__ bool prefix_good(const PrefixArgs& a, int P) {
    return P >= 0 && P <= a.max_blocks * kBlockSize;
}

template <int D_H, int R, int D_R>
__global__ void __launch_bounds__(kWarps * 32) prefix_scan_kernel(const PrefixArgs a) {
    constexpr int D_K = D_H + D_R, W = D_H + R;
    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DecodeArgs& d = a.d;
    const int P = prefix_good(a, a.len[0]) ? a.len[0] : 0;
    const int per = (P + a.nsplit - 1) / a.nsplit;
    const int t0 = split * per, t1 = min(P, t0 + per);
    float qr[D_K / 32], o[D_H / 32];
    const uint16_t* q = d.q + ((size_t)b * d.H + h) * D_K;
#pragma unroll
    for (int i = 0; i < D_K / 32; ++i) qr[i] = bf(q, i * 32 + lane);
#pragma unroll
    for (int i = 0; i < D_H / 32; ++i) o[i] = 0.f;
    const float qt = lane < R ? d.qt[((size_t)b * d.H + h) * R + lane] : 0.f;
    float oz = 0.f, m = -INFINITY, l = 0.f;
    for (int t = t0 + warp; t < t1; t += kWarps) {
        const int blk = a.blocks[t / kBlockSize];
        if (blk < 0 || blk >= d.num_blocks) {
            if (lane == 0) set_status(d.status, LRKV_DEV_BAD_BLOCK);
            continue;
        }
        const size_t row = (size_t)blk * kBlockSize + t % kBlockSize;
        const size_t zrow = (row * d.H + h) * R + lane;
        float s = lane < R ? qt * bf(a.zK, zrow) : 0.f;
#pragma unroll
        for (int i = 0; i < D_K / 32; ++i) s = fmaf(qr[i], bf(a.sK, row * D_K + i * 32 + lane), s);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= d.scale_log2;
        const float mn = fmaxf(m, s);
        const float al = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * al + p;
#pragma unroll
        for (int i = 0; i < D_H / 32; ++i) o[i] = fmaf(p, bf(a.sV, row * D_H + i * 32 + lane), o[i] * al);
        if (lane < R) oz = fmaf(p, bf(a.zV, zrow), oz * al);
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
    const size_t at = ((size_t)b * d.H + h) * a.nsplit + split;
    if (threadIdx.x < W) a.acc[at * W + threadIdx.x] = v;
    if (threadIdx.x == 0) {
        a.ml[at * 2] = M;
        a.ml[at * 2 + 1] = ls;
    }
}

// grid (H, B), a thread per column of the accumulator.
template <int D_H, int R>
__global__ void __launch_bounds__(192) prefix_combine_kernel(const PrefixArgs a) {
    constexpr int W = D_H + R;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const DecodeArgs& d = a.d;
    const int P = a.len[0], L = a.suffix ? d.seq_lens[b] : 0;
    const bool bad = !prefix_good(a, P) || L < 0 || L > d.max_pages * kBlockSize || (!d.part_out && P + L == 0);
    float* pdst = d.part_out ? d.part_out + ((size_t)b * d.H + h) * (W + 2) : nullptr;
    uint16_t* dst = d.out + ((size_t)b * d.H + h) * D_H;
    if (bad) {
        if (tid == 0 && h == 0) set_status(d.status, LRKV_DEV_BAD_SEQLEN);
        if (pdst) {
            for (int i = tid; i < W + 2; i += blockDim.x) pdst[i] = i == W ? -INFINITY : 0.f;
        } else {
            for (int i = tid; i < D_H; i += blockDim.x) dst[i] = 0;
        }
        return;
    }
    const size_t at = ((size_t)b * d.H + h) * a.nsplit;
    const float* ml0 = a.ml + at * 2;
    const float* ac0 = a.acc + at * W;
    int np = 0;
    const float *ml1 = nullptr, *ac1 = nullptr;
    if (L > 0) {
        const int2 fe = d.seg_table[b * d.nhg + h / (d.H / d.nhg)];
        np = fe.y;
        ml1 = d.part_ml + ((size_t)h * d.pmax + fe.x) * 2;
        ac1 = d.part_acc + ((size_t)h * d.pmax + fe.x) * W;
    }
    const int n0 = P > 0 ? a.nsplit : 0;
    float M = -INFINITY;
    for (int i = 0; i < n0; ++i) M = fmaxf(M, ml0[2 * i]);
    for (int i = 0; i < np; ++i) M = fmaxf(M, ml1[2 * i]);
    float l = 0.f, v = 0.f;
    for (int i = 0; i < n0; ++i) {
        const float w = ml0[2 * i] == -INFINITY ? 0.f : exp2f(ml0[2 * i] - M);
        l = fmaf(w, ml0[2 * i + 1], l);
        if (tid < W && w != 0.f) v = fmaf(w, ac0[(size_t)i * W + tid], v);
    }
    for (int i = 0; i < np; ++i) {
        const float w = ml1[2 * i] == -INFINITY ? 0.f : exp2f(ml1[2 * i] - M);
        l = fmaf(w, ml1[2 * i + 1], l);
        if (tid < W && w != 0.f) v = fmaf(w, ac1[(size_t)i * W + tid], v);
    }
    if (pdst) {
        if (tid < W) pdst[tid] = v;
        if (tid == 0) {
            pdst[W] = M;
            pdst[W + 1] = l;
        }
        return;
    }
    __shared__ float sv[W];
    if (tid < W) sv[tid] = v;
    __syncthreads();
    if (tid < D_H) {
        float x = sv[tid];
        const uint16_t* bv = d.BV + ((size_t)h * D_H + tid) * R;
#pragma unroll
        for (int j = 0; j < R; ++j) x = fmaf(bf(bv, j), sv[D_H + j], x);
        const __nv_bfloat16 ob = __float2bfloat16_rn(l > 0.f ? x / l : 0.f);
        dst[tid] = *reinterpret_cast<const uint16_t*>(&ob);
    }
}

}  // namespace

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int prefix_splits(int H, int R, int B, int max_blocks, int sms) {
    (void)H, (void)R, (void)B, (void)sms;
    return max_blocks < 16 ? max_blocks : 16;
}

size_t prefix_workspace_bytes(int H, int D_H, int R, int B, int nsplit) {
    const size_t n = (size_t)B * H * nsplit;
    return align256(n * 2 * sizeof(float)) + align256(n * (D_H + R) * sizeof(float));
}

void prefix_carve_workspace(PrefixArgs* a, void* ws, int D_H, int R) {
    (void)D_H, (void)R;
    a->ml = static_cast<float*>(ws);
    a->acc = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                      align256((size_t)a->d.B * a->d.H * a->nsplit * 2 * sizeof(float)));
}

cudaError_t launch_prefix_scan(const PrefixArgs& a, int D_H, int R, int D_R, cudaStream_t stream) {
    const dim3 grid(a.nsplit, a.d.H, a.d.B);
#define LRKV_PS(DH, RR)                                                                           \
    if (D_H == DH && R == RR) {                                                                   \
        if (D_R == 0)                                                                             \
            prefix_scan_kernel<DH, RR, 0><<<grid, kWarps * 32, 0, stream>>>(a);                   \
        else                                                                                      \
            prefix_scan_kernel<DH, RR, 64><<<grid, kWarps * 32, 0, stream>>>(a);                  \
        return cudaGetLastError();                                                                \
    }
    LRKV_PS(64, 8) LRKV_PS(64, 16) LRKV_PS(64, 32) LRKV_PS(128, 8) LRKV_PS(128, 16) LRKV_PS(128, 32)
#undef LRKV_PS
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_combine(const PrefixArgs& a, int D_H, int R, cudaStream_t stream) {
#define LRKV_PC(DH, RR)                                                               \
    if (D_H == DH && R == RR) {                                                       \
        prefix_combine_kernel<DH, RR><<<dim3(a.d.H, a.d.B), 192, 0, stream>>>(a);     \
        return cudaGetLastError();                                                    \
    }
    LRKV_PC(64, 8) LRKV_PC(64, 16) LRKV_PC(64, 32) LRKV_PC(128, 8) LRKV_PC(128, 16) LRKV_PC(128, 32)
#undef LRKV_PC
    return cudaErrorInvalidValue;
}

}  // namespace lrkv
