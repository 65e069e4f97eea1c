// tree.cu -- attention of the drafted tokens of a batch over the cache: token i of sequence b sees the sequence's
// tokens and the drafted ones of its mask.
//     s_t = ([q | q^R] . [s^K_t | k^R_t] + (q B_h^K) . z^K_{h,t}) scale,  p = softmax over what is seen,
//     out = sum p_t s^V_t + B_h^V sum p_t z^V_{h,t}
#include "lrkv_internal.cuh"
#include "tree.h"

namespace lrkv {

namespace {

// One block per (head, query), four warps that take every fourth token, a lane's share of the features each.
__global__ void __launch_bounds__(128) tree_kernel(const TreeArgs a, const int D_H, const int R, const int D_R) {
    const DecodeArgs& d = a.d;
    const int h = blockIdx.x, b = blockIdx.y / a.T, i = blockIdx.y - b * a.T;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D_K = D_H + D_R, W = D_H + R;
    __shared__ float q[192], qt[32], sm[4], sl[4], acc_s[4][160], o[160];
    const int L = d.seq_lens[b], n = a.tree_lens ? a.tree_lens[b] : a.T;
    const size_t row = ((size_t)b * a.T + i) * d.H + h;
    uint16_t* out = d.out + row * D_H;
    if (L < 0 || n < 0 || n > a.T || (long long)L + n > (long long)d.max_pages * kBlockSize) {
        if (threadIdx.x == 0) set_status(d.status, LRKV_DEV_BAD_SEQLEN);
        for (int c = threadIdx.x; c < D_H; c += 128) out[c] = 0;
        return;
    }
    if (i >= n) return;
    for (int c = threadIdx.x; c < D_K; c += 128) q[c] = __uint_as_float((uint32_t)d.q[row * D_K + c] << 16);
    __syncthreads();
    if (threadIdx.x < R) {
        float s = 0.f;
        for (int c = 0; c < D_H; ++c)
            s = fmaf(q[c], __uint_as_float((uint32_t)d.BK[((size_t)h * D_H + c) * R + threadIdx.x] << 16), s);
        qt[threadIdx.x] = s;
    }
    __syncthreads();
    const unsigned long long mask = a.mask ? a.mask[(size_t)b * a.T + i] : ~0ull >> (63 - i);
    float m = -INFINITY, l = 0.f, acc[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    for (int t = warp; t < L + n; t += 4) {
        if (t >= L && !(mask >> (t - L) & 1)) continue;
        const int page = d.block_table[(size_t)b * d.max_pages + t / kBlockSize];
        if (page < 0 || page >= d.num_blocks) {
            if (lane == 0) set_status(d.status, LRKV_DEV_BAD_BLOCK);
            continue;
        }
        const size_t slot = (size_t)page * kBlockSize + t % kBlockSize;
        auto val = [](uint16_t x) { return __uint_as_float((uint32_t)x << 16); };
        float s = 0.f;
        for (int c = lane; c < D_K; c += 32) s = fmaf(q[c], val(a.sK[slot * D_K + c]), s);
        if (lane < R) s = fmaf(qt[lane], val(a.zK[(slot * d.H + h) * R + lane]), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= d.scale_log2;
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
        for (int e = 0; e < 5; ++e) {
            const int c = e * 32 + lane;
            if (c >= W) break;
            const float v = val(c < D_H ? a.sV[slot * D_H + c] : a.zV[(slot * d.H + h) * R + c - D_H]);
            acc[e] = fmaf(p, v, acc[e] * f);
        }
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    for (int e = 0; e < 5; ++e)
        if (e * 32 + lane < W) acc_s[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float ls = 0.f, w[4];
    for (int k = 0; k < 4; ++k) {
        w[k] = sm[k] == -INFINITY ? 0.f : exp2f(sm[k] - M);
        ls = fmaf(w[k], sl[k], ls);
    }
    for (int c = threadIdx.x; c < W; c += 128) {
        float x = 0.f;
        for (int k = 0; k < 4; ++k) x += w[k] == 0.f ? 0.f : w[k] * acc_s[k][c];
        o[c] = ls == 0.f ? 0.f : x / ls;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D_H; c += 128) {
        float x = o[c];
        for (int k = 0; k < R; ++k)
            x = fmaf(o[D_H + k], __uint_as_float((uint32_t)d.BV[((size_t)h * D_H + c) * R + k] << 16), x);
        const __nv_bfloat16 y = __float2bfloat16_rn(x);
        out[c] = *reinterpret_cast<const uint16_t*>(&y);
    }
}

}  // namespace

size_t tree_workspace_bytes(int, int, int, int, int, int, int) { return 256; }

cudaError_t launch_tree(TreeArgs a, int D_H, int R, int D_R, void*, int, cudaStream_t stream) {
    tree_kernel<<<dim3(a.d.H, a.batch * a.T), 128, 0, stream>>>(a, D_H, R, D_R);
    return cudaGetLastError();
}

}  // namespace lrkv
