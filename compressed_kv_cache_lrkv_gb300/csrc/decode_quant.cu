// decode_quant.cu -- factored decode over a cache of 8-bit rows (quant.h).
//
// Per sequence b and head h, with q~_h = q_h B_h^K and the rows' values read as q_i 2^k:
//     score_t = (q_h . s^K_t + q~_h . z^K_{h,t}) * scale,   out_h = sum p s^V + B_h^V (sum p z^V)
// Absorb and combine are the bf16 decode's; the scan between them is here.
//
// A row is half as many bytes as in bf16, so a scan at the memory's pace has half the time per
// value, and each value must first be widened.  All products are therefore fed to the tensor
// cores (mma.sync m16n8k16), the latents' too, straight from the row bytes:
//   - a byte u = q + 128 becomes fp16 by one byte permute (two values 1024 + u at a time, exact);
//     the offset 1152 = 1024 + 128 leaves the sums again as -1152 sum q~ (in the K sums' start) and
//     -1152 sum w (one product with a constant A per tile);
//   - tokens are the M of the logits' product (A = 16 tokens x 16 features, B = features x 8
//     heads) and the K of the values' (A = features x 16 tokens, B = 16 tokens x 8 heads), so both
//     leave a thread the same two heads and the probabilities pass from one to the other by a
//     transpose within the warp (movmatrix);
//   - a head's latents meet that head's q~ (or weights) only: B holds the head's column and zeros
//     elsewhere, and the eight heads of a tile accumulate into the same registers;
//   - scales: one per (token, head's block) multiplies the K sums in fp32; the V weights are
//     w_t = 2^(s_t + k_t - mz) in fp16 with a running maximum mz of their own, so tokens whose
//     scales differ by any power of two lose nothing but what is small beside the largest;
//   - the shared rows s^K, s^V (used by all heads) are widened to bf16 once per 16 tokens by
//     converter warps (q_i 2^k is exact in bf16).
// Warps of a CTA: consumers (NT x 8 heads each, NG groups taking 16-token tiles in turn), one
// producer (bulk copies of whole rows, which lie contiguous within a page, into a ring of
// stages), three or four converters; connected by mbarriers only, so they drift freely.  One CTA per
// SM; the work is cut as in the bf16 decode (decode_work.cuh).
#include <cuda_fp16.h>

#include "decode_work.cuh"
#include "lrkv_internal.cuh"
#include "quant.h"

namespace lrkv {

namespace {

#ifndef MOST1
#define MOST1 8
#endif
constexpr int kConsumers1 = MOST1, kConverters1 = 3;  // one tile of 8 heads per consumer warp
constexpr int kConsumers2 = 8, kConverters2 = 3;  // two
constexpr int kThreads1 = (kConsumers1 + 1 + kConverters1) * 32;
constexpr int kThreads2 = (kConsumers2 + 1 + kConverters2) * 32;
constexpr int kMaxWalkers = 16;   // warps of a CTA at most
constexpr float kLazy = 8.0f;     // maxima are raised when exceeded by this much (log2 units)

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_16816_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two bytes of x, chosen by sel (0x4140: bytes 0, 1; 0x4342: 2, 3; 0x4240: 0, 2; 0x4341: 1, 3), as
// fp16 values 1024 + byte: the fp16 with high byte 0x64 and low byte u.
__device__ __forceinline__ uint32_t bytes_f16(uint32_t x, uint32_t sel) {
    uint32_t v;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(x), "r"(0x64646464u), "r"(sel));
    return v;
}
constexpr float kByteOffset = 1152.0f;          // 1024 + u = q + 1152
constexpr uint32_t kMinusOffset2 = 0xe480e480u;  // fp16 (-1152, -1152)
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
// Values q_i 2^k of two bytes (b0, b1 of [b0, 0, b1, 0]) as bf16, s2 = (2^k, 2^k): with the low seven
// bits in its mantissa bf16 holds 128 + u mod 128, from which 256 or, where the byte's top bit is
// set, 128 is taken; both steps and the product are exact.
__device__ __forceinline__ uint32_t bytes_bf16(uint32_t v, __nv_bfloat162 s2) {
    const uint32_t lo = (v & 0x007f007fu) | 0x43004300u, hi = (v & 0x00800080u) ^ 0x43804380u;
    const __nv_bfloat162 r = __hmul2(
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi)), s2);
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Scale of a block: 2^(e - 127); NaN for byte 255, zero for 0 (a cleared row).
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e == 255 ? 0x7fc00000u : e << 23); }

// try_wait that may sleep in hardware for some microseconds before it reports failure: a waiting warp
// then takes few issue slots from the others.
__device__ __forceinline__ bool mbar_try_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

// Bounded wait of a whole warp; false (with the abort flag set) once it, or any other, gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                          uint64_t limit_ns) {
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (__all_sync(0xffffffffu, mbar_try_sleep(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_sleep(bar, parity))) return true;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) {
            set_status(status, LRKV_DEV_TIMEOUT);
            *abort_flag = 1;
            return false;
        }
    }
}

struct QuantPlan {
    int nt;                      // tiles of 8 heads per consumer warp
    int nwh, ng;                 // consumer warps over the heads, groups
    int ncv;                     // converter warps
    int st;                      // tiles (of TOK tokens) per stage
    int nslot, ncb;              // stages of the ring, widened tiles
    int stage_bytes, cb_bytes;
    int threads, smem_bytes;
};

struct QuantScanArgs {
    QuantDecodeArgs a;
    QuantPlan p;
};

// One warp's walk over the CTA's segments.
struct alignas(16) Walker {
    SegWalk walk;
    int valid, vb, g0, g1, slot;
    template <class W>
    __device__ __forceinline__ void advance(const W& w) {
        valid = walk.next(w, &vb, &g0, &g1, &slot);
    }
};
static_assert(sizeof(Walker) == 48, "walkers are an array in shared memory with the work plan behind it");

// Row stride (floats) of a head in the staging of the group merge: 4 mod 16, so that the four head
// pairs and eight columns of a warp's store fall on different banks.
__host__ __device__ constexpr int merge_stride(int W) { return W % 16 == 0 ? W + 4 : W + 12; }

// Row stride (bytes) of a widened tile [s^K | s^V] in bf16: an odd number of 16-byte units.
__host__ __device__ constexpr int cb_stride(int D_K, int D_H) { return (D_K + D_H) * 2 + 16; }

template <int D_H, int R, int D_R, int NT, int TOK>
__global__ void __launch_bounds__(NT == 1 ? kThreads1 : kThreads2, 1) quant_scan_kernel(const QuantScanArgs args) {
    constexpr int D_K = D_H + D_R, W = D_H + R, WS = merge_stride(W);
    constexpr int SB = cb_stride(D_K, D_H);
    constexpr int NKK = D_K / 16;
    constexpr int NZC = R > 16 ? R / 16 : 1;       // 16-byte chunks of a head's latents (r = 8: of two heads')
    constexpr int NCH = 8 * R / 16;                // chunks of a tile of 8 heads
    constexpr int TPP = kBlockSize / TOK;          // tiles per page
    using WorkQ = WorkT<TOK>;
    static_assert(sizeof(WorkQ) <= 96 && alignof(WorkQ) <= 16, "room for the plan in shared memory");
    static_assert(kThreads1 <= 32 * kMaxWalkers && kThreads2 <= 32 * kMaxWalkers, "walkers");
    const DecodeArgs& a = args.a.d;
    const QuantLayout& ql = args.a.q;
    const QuantPlan& p = args.p;
    const int RB = ql.row_bytes;
    const int H = a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NCW = p.nwh * p.ng;
    const int nslot = p.nslot, ncb = p.ncb, ST = p.st;

    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    const uint32_t ring = smem_u32(smem);
    const uint32_t cbuf = ring + nslot * p.stage_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + nslot * p.stage_bytes + ncb * p.cb_bytes);
    uint64_t* full = bars;
    uint64_t* empty = full + nslot;
    uint64_t* cfull = empty + nslot;
    uint64_t* cempty = cfull + ncb;
    uint64_t* merged = cempty + ncb;
    int* meta = reinterpret_cast<int*>(merged + 2);
    volatile int* abort_flag = meta + nslot;
    int* slc = meta + ((nslot + 1 + 3) & ~3);
    Walker* walkers = reinterpret_cast<Walker*>(slc + kSeqCache);
    WorkQ* work = reinterpret_cast<WorkQ*>(walkers + kMaxWalkers);

    if (threadIdx.x == 0) {
        for (int i = 0; i < nslot; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), NCW + p.ncv);
        }
        for (int i = 0; i < ncb; ++i) {
            mbar_init(smem_u32(cfull + i), p.ncv);
            mbar_init(smem_u32(cempty + i), p.nwh);
        }
        mbar_init(smem_u32(merged), NCW);
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int b = threadIdx.x; b < a.B && b < kSeqCache; b += blockDim.x) slc[b] = a.seq_lens[b];
    __syncthreads();
    if (warp == 0) {
        WorkQ w{a.seq_lens, slc, a.B, 1, a.max_pages * kBlockSize, a.nranges, 0, 0, 1, 0};
        w.lgh = 0;
        w.template plan<32>(a.bubble, lane);
        if (lane == 0) *work = w;
    }
    __syncthreads();
    Walker& wk = walkers[warp];
    if (lane == 0) {
        wk.walk.start(blockIdx.x);
        wk.advance(*work);
    }
    __syncwarp();

    // Tile indices below count the CTA's tiles from its first (u) and its stages (k), alike in all
    // warps.  Every consumer and converter waits for and releases every stage in turn (not only those
    // with a tile of its own), and a widened tile's slot always belongs to the same group and converter
    // (ncb is a multiple of both counts), so nobody can miss a round of a barrier or take one for another.
    if (warp == NCW) {
        // ---------------------------------------------------------------- producer
        const uint64_t pol = policy_evict_first();
        int k = 0, segs = 0, issued = 0;
        while (wk.valid) {
            const int b = wk.vb, g0 = wk.g0, g1 = wk.g1;
            if (lane == 0 && g0 == 0) {
                // a sequence's first segment records where the combine finds its partials
                const int gr = work->gran(b);
                const int np = work->pieces ? work->npieces(b, work->chunk)
                                            : work->range_of(wk.walk.seg_start + gr - 1) - (wk.slot - b) + 1;
                a.seg_table[b] = make_int2(wk.slot, np);
            }
            // the ring's memory serves the group merge at the end of a segment
            bool ok = segs == 0 || p.ng == 1 ||
                      warp_wait(smem_u32(merged), (segs - 1) & 1, abort_flag, a.status, a.wait_ns);
            const int32_t* bt = a.block_table + (size_t)b * a.max_pages;
            const int last_page = (g1 - 1) / TPP;
            int page0 = g0 / TPP, ids = page0 + lane <= last_page ? bt[page0 + lane] : -1;
            for (int s = g0 / ST; s <= (g1 - 1) / ST; ++s, ++k) {
                const int slot = k % nslot;
                const int f = max(g0, s * ST), e = min(g1, (s + 1) * ST);
                const int page = f / TPP;
                if (page - page0 >= 32) {
                    page0 = page;
                    ids = page0 + lane <= last_page ? bt[page0 + lane] : -1;
                }
                const int blk = __shfl_sync(0xffffffffu, ids, page - page0);
                if (ok && k >= nslot)
                    ok = warp_wait(smem_u32(empty + slot), (k / nslot - 1) & 1, abort_flag, a.status, a.wait_ns);
                ok = ok && !__any_sync(0xffffffffu, *abort_flag != 0);
                if (ok && lane == 0) {
                    if (blk < 0 || blk >= a.num_blocks) {
                        set_status(a.status, LRKV_DEV_BAD_BLOCK);
                        meta[slot] = 0;
                        mbar_arrive(smem_u32(full + slot));
                    } else {
                        meta[slot] = 1;
                        const uint32_t bytes = (uint32_t)(e - f) * TOK * RB;
                        mbar_arrive_expect_tx(smem_u32(full + slot), bytes);
                        bulk_load_hint(ring + slot * p.stage_bytes + (f - s * ST) * TOK * RB,
                                       args.a.rows + ((size_t)blk * kBlockSize + (f % TPP) * TOK) * RB, bytes,
                                       smem_u32(full + slot), pol);
                    }
                }
                if (ok) issued = k + 1;
                __syncwarp();
            }
            ++segs;
            if (lane == 0) wk.advance(*work);
            __syncwarp();
        }
        // After an expired wait, let the copies in flight land before the CTA exits.
        if (*abort_flag)
            for (int i = max(0, issued - nslot); i < issued; ++i)
                mbar_wait(smem_u32(full + i % nslot), (i / nslot) & 1, a.status);
    } else if (warp > NCW) {
        // ---------------------------------------------------------------- converters
        const int cv = warp - NCW - 1;
        constexpr int U = (D_K + D_H) / 8;  // 8-value units of a row
        int k = 0, u = 0;
        while (wk.valid) {
            const int b = wk.vb, g0 = wk.g0, g1 = wk.g1;
            const int L = b < kSeqCache ? slc[b] : a.seq_lens[b];
            for (int s = g0 / ST; s <= (g1 - 1) / ST; ++s, ++k) {
                const int slot = k % nslot;
                bool ok = warp_wait(smem_u32(full + slot), (k / nslot) & 1, abort_flag, a.status, a.wait_ns);
                const int f = max(g0, s * ST), e = min(g1, (s + 1) * ST);
                for (int t = f; t < e; ++t, ++u) {
                    const int cb = u % ncb;
                    if (ok && u >= ncb)
                        ok = warp_wait(smem_u32(cempty + cb), (u / ncb - 1) & 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) continue;
                    if (meta[slot]) {
                        const int nvalid = min(TOK, L - t * TOK);
                        const uint32_t src = ring + slot * p.stage_bytes + (t - s * ST) * TOK * RB;
                        const uint32_t dst = cbuf + cb * p.cb_bytes;
#pragma unroll 4
                        for (int i = cv * 32 + lane; i < TOK * U; i += p.ncv * 32) {
                            const int row = i / U, c = i - row * U;
                            const uint32_t ra = src + row * RB;
                            uint32_t x[2], o[4];
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(ra + c * 8));
                            const uint32_t sb = lds8(ra + ql.off_sc + (c >> 2));
                            // the scale twice in bf16 (NaN for byte 255); zero for tokens behind the end (their
                            // probabilities are 0, and 0 x NaN is not)
                            uint32_t s2 = sb == 255 ? 0x7fc07fc0u : sb * 0x00800080u;
                            s2 = row < nvalid ? s2 : 0u;
                            const __nv_bfloat162 sc = *reinterpret_cast<const __nv_bfloat162*>(&s2);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[j] = bytes_bf16(__byte_perm(x[j >> 1], 0u, j & 1 ? 0x4342 : 0x4140), sc);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + row * SB + c * 16),
                                         "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                         : "memory");
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(cfull + cb));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(empty + slot));
            }
            __syncwarp();
            if (lane == 0) wk.advance(*work);
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- consumers
        const int grp = warp / p.nwh, wh = warp - grp * p.nwh;
        const int h0 = wh * NT * 8;                  // first head of this warp
        const int g = lane >> 2, tq = lane & 3;
        const int nct = NCW * 32;
        const int g8 = TOK == 16 ? g + 8 : g;        // rows 8..15 of a tile of 8 tokens: masked copies of 0..7
        const int zc0 = h0 * R / 16;                 // this warp's first 16-byte chunk of a row's latents
        pdl_wait();  // q~ written by the absorb kernel
        int k = 0, u = 0;
        while (wk.valid) {
            const int b = wk.vb, g0 = wk.g0, g1 = wk.g1, pslot = wk.slot;
            const int L = b < kSeqCache ? slc[b] : a.seq_lens[b];
            // Queries as B fragments (features x heads, head h0 + 8 nt + g in this lane's column)
            uint32_t qb[NKK][NT][2];
            uint32_t qz[NZC][NT][2];
            float ci[NT][2];  // start of the latent logits' sums
            float fz[NT][2];  // power of two that q~ was divided by, for heads 2 tq, 2 tq + 1 of each tile
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = h0 + nt * 8 + g;
                const bool live = h < H;
                const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + ((size_t)b * H + (live ? h : 0)) * D_K);
#pragma unroll
                for (int kk = 0; kk < NKK; ++kk) {
                    qb[kk][nt][0] = live ? q[kk * 8 + tq] : 0u;
                    qb[kk][nt][1] = live ? q[kk * 8 + 4 + tq] : 0u;
                }
                // q~: this lane holds features 4 tq .. 4 tq + 3 of each chunk (the A fragments' order), scaled
                // by the power of two that brings the head's largest magnitude into [1, 2)
                const float* qt = a.qt + ((size_t)b * H + (live ? h : 0)) * R;
                float v[NZC][4], mx = 0.f;
#pragma unroll
                for (int c = 0; c < NZC; ++c) {
                    const int f0 = R == 8 ? (tq * 4) & 7 : c * 16 + tq * 4;
                    const float4 x = *reinterpret_cast<const float4*>(qt + f0);
                    const bool mine = live && (R != 8 || (tq >> 1) == (g & 1));
                    v[c][0] = mine ? x.x : 0.f;
                    v[c][1] = mine ? x.y : 0.f;
                    v[c][2] = mine ? x.z : 0.f;
                    v[c][3] = mine ? x.w : 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(v[c][i]));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const uint32_t ex = min(max(__float_as_uint(mx) >> 23, 1u), 253u);
                const float inv = __uint_as_float((254u - ex) << 23);
                const float fac = __uint_as_float(ex << 23);
#pragma unroll
                for (int c = 0; c < NZC; ++c) {
                    qz[c][nt][0] = pack_f16x2(v[c][0] * inv, v[c][1] * inv);
                    qz[c][nt][1] = pack_f16x2(v[c][2] * inv, v[c][3] * inv);
                }
                fz[nt][0] = __shfl_sync(0xffffffffu, fac, 8 * tq);
                fz[nt][1] = __shfl_sync(0xffffffffu, fac, 8 * tq + 4);
                // the products take 1152 + q for q: the sums start from -1152 sum q~ (as rounded).  (Against
                // a typical sum the offset is some 160 times as large, so fp32 keeps 16 bits of it, more than
                // q~ has.)
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < NZC; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&qz[c][nt][i]));
                        sum += x.x + x.y;
                    }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                ci[nt][0] = -kByteOffset * __shfl_sync(0xffffffffu, sum, 8 * tq);
                ci[nt][1] = -kByteOffset * __shfl_sync(0xffffffffu, sum, 8 * tq + 4);
            }
            float o[D_H / 16][NT][4], oz[NZC][NT][4];
            float m[NT][2], mz[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < D_H / 16; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
#pragma unroll
                for (int i = 0; i < NZC; ++i) oz[i][nt][0] = oz[i][nt][1] = oz[i][nt][2] = oz[i][nt][3] = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nt][e] = mz[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                }
            }
            for (int s = g0 / ST; s <= (g1 - 1) / ST; ++s, ++k) {
                const int slot = k % nslot;
                bool ok = warp_wait(smem_u32(full + slot), (k / nslot) & 1, abort_flag, a.status, a.wait_ns);
                const int f = max(g0, s * ST), e1 = min(g1, (s + 1) * ST);
                const int have = meta[slot];
#pragma unroll 1
                for (int t = f; t < e1; ++t, ++u) {
                    if (u % p.ng != grp) continue;
                    const int cb = u % ncb;
                    if (ok) ok = warp_wait(smem_u32(cfull + cb), (u / ncb) & 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) continue;
                    if (have) {
                        const int nvalid = min(TOK, L - t * TOK);
                        const uint32_t row0 = ring + slot * p.stage_bytes + (t - s * ST) * TOK * RB;
                        const uint32_t cv = cbuf + cb * p.cb_bytes;
                        const bool in0 = g < nvalid, in1 = TOK == 16 && g + 8 < nvalid;

                        // --- shared logits [q | q^R] . [s^K | k^R]: 16 tokens x 8 heads
                        float c[NT][4], cz[NT][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) c[nt][i] = cz[nt][i] = 0.f;  // (every cz is set below)
                        {
                            const int r16 = TOK == 16 ? lane & 15 : lane & 7;
                            const uint32_t ad = cv + r16 * SB + (lane >> 4) * 16;
#pragma unroll
                            for (int kk = 0; kk < NKK; ++kk) {
                                uint32_t af[4];
                                ldmatrix_x4(ad + kk * 32, af[0], af[1], af[2], af[3]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_16816(c[nt], af, qb[kk][nt][0], qb[kk][nt][1]);
                            }
                        }
                        // --- latent logits q~ . z^K, chunk by chunk of 16 bytes: of a product with all eight
                        // heads' q~ only the columns of the chunk's own head (r = 8: two heads) are kept.  (Heads
                        // past the last read whatever follows in shared memory: finite, and never stored.)
                        {
                            const uint32_t z0 = row0 + g * RB + ql.off_zK + zc0 * 16 + tq * 4;
                            const uint32_t z1 = row0 + g8 * RB + ql.off_zK + zc0 * 16 + tq * 4;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < NCH / NZC; ++j) {
                                    float d[4] = {ci[nt][0], ci[nt][1], ci[nt][0], ci[nt][1]};
#pragma unroll
                                    for (int zc = 0; zc < NZC; ++zc) {
                                        const int at = (nt * NCH + j * NZC + zc) * 16;
                                        const uint32_t x0 = lds32(z0 + at), x1 = lds32(z1 + at);
                                        mma_16816_f16(d, bytes_f16(x0, 0x4140), bytes_f16(x1, 0x4140),
                                                      bytes_f16(x0, 0x4342), bytes_f16(x1, 0x4342), qz[zc][nt][0],
                                                      qz[zc][nt][1]);
                                    }
                                    if (tq == (R == 8 ? j : j >> 1)) {
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            if (R == 8 || (i & 1) == (j & 1)) cz[nt][i] = d[i];
                                    }
                                }
                        }
                        // --- logits s (log2 units) and s + k of the z^V scales; element i: token g (+ 8 for
                        // i >= 2), head 2 tq + (i & 1)
                        float sv[NT][4], sw[NT][4];
                        bool raise = false;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = i & 1;
                                const int blk = min(((h0 + nt * 8 + 2 * tq + e) * R) / kQuantBlock, ql.nb_z - 1);
                                const uint32_t sa = row0 + (i < 2 ? g : g8) * RB + ql.off_sc + ql.nb_sK + ql.nb_sV + blk;
                                const uint32_t bk = lds8(sa), bv = lds8(sa + ql.nb_z);
                                const float s =
                                    fmaf(cz[nt][i] * fz[nt][e], scale_of(bk), c[nt][i]) * a.scale_log2;
                                // exponent of the scale: a NaN block's is NaN, a cleared row's -infinity
                                const float ke = bv == 255 ? __uint_as_float(0x7fc00000u)
                                                           : bv == 0 ? -INFINITY : (float)((int)bv - 127);
                                const bool in = i < 2 ? in0 : in1;
                                sv[nt][i] = in ? s : -INFINITY;
                                sw[nt][i] = in ? s + ke : -INFINITY;
                                raise |= sv[nt][i] > m[nt][e] + kLazy || sw[nt][i] > mz[nt][e] + kLazy;
                            }
                        // maxima are the same in the eight lanes that share two heads, and raised together
                        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float x = fmaxf(sv[nt][e], sv[nt][2 + e]), y = fmaxf(sw[nt][e], sw[nt][2 + e]);
#pragma unroll
                                    for (int d = 4; d < 32; d <<= 1) {
                                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                                    }
                                    x = fmaxf(x, m[nt][e]);
                                    y = fmaxf(y, mz[nt][e]);
                                    const float al = m[nt][e] == -INFINITY ? 0.f : ex2_approx(m[nt][e] - x);
                                    const float az = mz[nt][e] == -INFINITY ? 0.f : ex2_approx(mz[nt][e] - y);
                                    m[nt][e] = x;
                                    mz[nt][e] = y;
                                    l[nt][e] *= al;
#pragma unroll
                                    for (int i = 0; i < D_H / 16; ++i) {
                                        o[i][nt][e] *= al;
                                        o[i][nt][2 + e] *= al;
                                    }
#pragma unroll
                                    for (int i = 0; i < NZC; ++i) {
                                        oz[i][nt][e] *= az;
                                        oz[i][nt][2 + e] *= az;
                                    }
                                }
                        }
                        // --- p = 2^(s - m) and w = 2^(s + k - mz), transposed into B fragments
                        uint32_t pb[NT][2], wb[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float pp[4], ww[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = i & 1;
                                const bool in = i < 2 ? in0 : in1;
                                pp[i] = in ? ex2_approx(sv[nt][i] - m[nt][e]) : 0.f;
                                // (mz is -infinity as long as every block of the head was all zeros)
                                ww[i] = in && sw[nt][i] != -INFINITY ? ex2_approx(sw[nt][i] - mz[nt][e]) : 0.f;
                            }
                            l[nt][0] += pp[0] + pp[2];
                            l[nt][1] += pp[1] + pp[3];
                            pb[nt][0] = movmatrix_trans(pack_bf16x2(pp[0], pp[1]));
                            pb[nt][1] = movmatrix_trans(pack_bf16x2(pp[2], pp[3]));
                            wb[nt][0] = movmatrix_trans(pack_f16x2(ww[0], ww[1]));
                            wb[nt][1] = movmatrix_trans(pack_f16x2(ww[2], ww[3]));
                        }
                        // --- shared values: O^T (d x heads) += s^V^T . P
                        {
                            const int r16 = TOK == 16 ? (lane & 7) + ((lane >> 4) << 3) : lane & 7;
                            const uint32_t ad = cv + r16 * SB + D_K * 2 + ((lane >> 3) & 1) * 16;
#pragma unroll
                            for (int i = 0; i < D_H / 16; ++i) {
                                uint32_t af[4];
                                ldmatrix_x4_trans(ad + i * 32, af[0], af[1], af[2], af[3]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_16816(o[i][nt], af, pb[nt][0], pb[nt][1]);
                            }
                        }
                        // --- latent values, two 16-byte chunks at a time: rows of the transposed 16-bit
                        // elements are pairs of features, row g of A takes the even one, row g + 8 the odd one
                        {
                            const int r16 = TOK == 16 ? lane & 15 : lane & 7;
                            const uint32_t zr = row0 + r16 * RB + ql.off_zV + (zc0 + (lane >> 4)) * 16;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                // the offset 1152 of the bytes' products, taken off tile by tile (so that the
                                // sums never grow with it)
#pragma unroll
                                for (int zc = 0; zc < NZC; ++zc)
                                    mma_16816_f16(oz[zc][nt], kMinusOffset2, kMinusOffset2, kMinusOffset2, kMinusOffset2,
                                                  wb[nt][0], wb[nt][1]);
#pragma unroll
                                for (int c2 = 0; c2 < NCH; c2 += 2) {
                                    uint32_t x[4];
                                    ldmatrix_x4_trans(zr + (nt * NCH + c2) * 16, x[0], x[1], x[2], x[3]);
#pragma unroll
                                    for (int w = 0; w < 2; ++w) {
                                        const int ch = c2 + w;
                                        const bool mine = R == 8 ? (g >> 1) == ch : g == (R == 32 ? ch >> 1 : ch);
                                        const int zc = R == 32 ? ch & 1 : 0;
                                        mma_16816_f16(oz[zc][nt], bytes_f16(x[2 * w], 0x4240),
                                                      bytes_f16(x[2 * w], 0x4341), bytes_f16(x[2 * w + 1], 0x4240),
                                                      bytes_f16(x[2 * w + 1], 0x4341), mine ? wb[nt][0] : 0u,
                                                      mine ? wb[nt][1] : 0u);
                                    }
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(cempty + cb));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(empty + slot));
            }
            // --- this group's state over the segment
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                    // the latents' sums brought to the probabilities' maximum
                    const float fac = mz[nt][e] == -INFINITY ? 0.f : ex2_approx(mz[nt][e] - m[nt][e]);
#pragma unroll
                    for (int i = 0; i < NZC; ++i) {
                        oz[i][nt][e] *= fac;
                        oz[i][nt][2 + e] *= fac;
                    }
                    // a NaN sum is handed on as NaN values with a weight, not as an empty part
                    if (l[nt][e] != l[nt][e]) {
                        l[nt][e] = 1.f;
                        if (!(fabsf(m[nt][e]) < INFINITY)) m[nt][e] = 0.f;
#pragma unroll
                        for (int i = 0; i < D_H / 16; ++i)
                            o[i][nt][e] = o[i][nt][2 + e] = __uint_as_float(0x7fc00000u);
                    }
                }
            const bool direct = p.ng == 1;
            float* const sml = reinterpret_cast<float*>(smem);
            float* const sacc = sml + ((p.ng * H * 2 + 3) & ~3);
            float* swt = sacc + (size_t)p.ng * H * WS;  // [group][head] weights
            const size_t hs_ml = direct ? (size_t)a.pmax * 2 : 2, hs_acc = direct ? (size_t)a.pmax * W : WS;
            float* gml = direct ? a.part_ml + (size_t)pslot * 2 : sml + (size_t)grp * H * 2;
            float* gacc = direct ? a.part_acc + (size_t)pslot * W : sacc + (size_t)grp * H * WS;
            if (!direct) named_bar(1, nct);  // every tile of the segment consumed: the ring is idle
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = h0 + nt * 8 + 2 * tq + e;
                    if (h >= H) continue;
                    if (g == 0) {
                        gml[h * hs_ml] = m[nt][e];
                        gml[h * hs_ml + 1] = l[nt][e];
                    }
                    float* dst = gacc + h * hs_acc;
#pragma unroll
                    for (int i = 0; i < D_H / 16; ++i) {
                        dst[i * 16 + g] = o[i][nt][e];
                        dst[i * 16 + 8 + g] = o[i][nt][2 + e];
                    }
                    if (R == 8) {
                        if ((g >> 2) == e)
                            *reinterpret_cast<float2*>(dst + D_H + (g & 3) * 2) = make_float2(oz[0][nt][e], oz[0][nt][2 + e]);
                    } else {
#pragma unroll
                        for (int i = 0; i < NZC; ++i)
                            *reinterpret_cast<float2*>(dst + D_H + i * 16 + g * 2) =
                                make_float2(oz[i][nt][e], oz[i][nt][2 + e]);
                    }
                }
            if (!direct) {
                named_bar(1, nct);
                const int ng = p.ng;
                float* pml = a.part_ml + (size_t)pslot * 2;
                float* pacc = a.part_acc + (size_t)pslot * W;
                for (int h = threadIdx.x; h < H; h += nct) {
                    float M = -INFINITY, Ls = 0.f;
                    for (int i = 0; i < ng; ++i) M = fmaxf(M, sml[(i * H + h) * 2]);
                    for (int i = 0; i < ng; ++i) {
                        const float mi = sml[(i * H + h) * 2];
                        const float w = mi == -INFINITY ? 0.f : ex2_approx(mi - M);
                        swt[i * H + h] = w;
                        Ls = fmaf(w, sml[(i * H + h) * 2 + 1], Ls);
                    }
                    *reinterpret_cast<float2*>(pml + (size_t)h * a.pmax * 2) = make_float2(M, Ls);
                }
                named_bar(1, nct);
                constexpr int W4 = W / 4;
                for (int i4 = threadIdx.x; i4 < H * W4; i4 += nct) {
                    const int h = i4 / W4, c4 = i4 - h * W4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i = 0; i < ng; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(sacc + ((size_t)i * H + h) * WS + c4 * 4);
                        const float w = swt[i * H + h];
                        v.x = fmaf(w, x.x, v.x);
                        v.y = fmaf(w, x.y, v.y);
                        v.z = fmaf(w, x.z, v.z);
                        v.w = fmaf(w, x.w, v.w);
                    }
                    *reinterpret_cast<float4*>(pacc + (size_t)h * a.pmax * W + c4 * 4) = v;
                }
                fence_proxy_async_smem();  // generic accesses of the ring before the next segment's copies
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(merged));
            }
            __syncwarp();
            if (lane == 0) wk.advance(*work);
            __syncwarp();
        }
    }
    pdl_trigger();  // the combine waits for this grid's end
}

// Tokens of a tile.
int tile_tokens(int H, int R) { return R == 32 && H > 96 ? 8 : 16; }

template <int D_H, int R, int D_R>
bool make_plan(QuantPlan* p, const QuantLayout& q, int H, int smem_limit) {
    p->nt = H > 8 * kConsumers1 ? 2 : 1;
    // a row of more than 96 heads of r = 32 is so long that two stages of 16 tokens do not fit
    const int tok = tile_tokens(H, R);
    const int most = p->nt == 2 ? kConsumers2 : kConsumers1;
    p->ncv = p->nt == 2 ? kConverters2 : kConverters1;
    p->nwh = (H + 8 * p->nt - 1) / (8 * p->nt);
    const int ng_most = most / p->nwh > 1 ? most / p->nwh : 1;
    p->cb_bytes = tok * cb_stride(D_H + D_R, D_H);
    const int WS = merge_stride(D_H + R);
    const int tile = tok * q.row_bytes;
    // tiles per stage: a copy instruction costs its thread some 60 to 80 ns, so short rows are brought a page
    // (or half) at a time, as long as six stages fit in the ring
    p->st = 1;
    while (p->st * tok < kBlockSize && p->st * tile * 2 <= 28 << 10) p->st *= 2;
    p->stage_bytes = p->st * tile;
    auto fixed = [&](int nslot, int ncb) {
        return (2 * nslot + 2 * ncb + 2) * 8 + ((nslot + 1 + 3) & ~3) * 4 + kSeqCache * 4 + kMaxWalkers * (int)sizeof(Walker) +
               96 + 128;
    };
    for (int want = 3; want >= 2; --want)          // stages at least
        for (int ng = ng_most; ng >= 1; --ng)
            for (int mul = 2; mul >= 1; --mul) {   // widened tiles per group
                const int ncb = ng * mul;
                int nslot = 16;
                while (nslot > 1 && nslot * p->stage_bytes + ncb * p->cb_bytes + fixed(nslot, ncb) > smem_limit) --nslot;
                if (nslot < want) continue;
                if (ng > 1 && ((size_t)ng * H * (WS + 3) + 3) * 4 > (size_t)nslot * p->stage_bytes) continue;
                p->ng = ng;
                p->ncb = ncb;
                p->nslot = nslot;
                p->threads = (p->nwh * ng + 1 + p->ncv) * 32;
                p->smem_bytes = nslot * p->stage_bytes + ncb * p->cb_bytes + fixed(nslot, ncb);
                return true;
            }
    return false;
}

template <int D_H, int R, int D_R>
cudaError_t launch_t(QuantScanArgs& x, int sms, int smem_limit, cudaStream_t stream) {
    if (!make_plan<D_H, R, D_R>(&x.p, x.a.q, x.a.d.H, smem_limit)) return cudaErrorInvalidConfiguration;
    const int tok = tile_tokens(x.a.d.H, R);
    auto kern = x.p.nt == 1 ? quant_scan_kernel<D_H, R, D_R, 1, 16> : quant_scan_kernel<D_H, R, D_R, 2, 16>;
    if constexpr (R == 32) {
        if (tok == 8) kern = quant_scan_kernel<D_H, R, D_R, 2, 8>;
    }
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, x.p.smem_bytes);
    if (e != cudaSuccess) return e;
    // a pipeline drain and refill at a sequence boundary costs about as long as streaming 128 KB through
    // one SM (in granules of the plan)
    const int gran = tok * x.a.q.row_bytes;
    x.a.d.bubble = ((128 << 10) + gran - 1) / gran;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(x.a.d.nranges < sms ? x.a.d.nranges : sms);
    cfg.blockDim = dim3(x.p.threads);
    cfg.dynamicSmemBytes = x.p.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, static_cast<const QuantScanArgs>(x));
    return e != cudaSuccess ? e : launch_decode_combine(x.a.d, D_H, R, sms, stream);
}

}  // namespace

// The workspace is the bf16 decode's (its layout has room for head groups, which this scan has not).
size_t quant_decode_workspace_bytes(int H, int D_H, int R, int B, int nranges) {
    return decode_workspace_bytes(H, D_H, R, B, nranges);
}

cudaError_t launch_quant_decode(QuantDecodeArgs a, void* ws, int D_H, int R, int D_R, int sms, int smem_limit,
                                cudaStream_t stream) {
    decode_carve_workspace(&a.d, ws, a.d.H, D_H, R, a.d.B, a.d.nranges);
    const cudaError_t e = launch_decode_absorb(a.d, D_H, R, D_R, stream);
    if (e != cudaSuccess) return e;
    QuantScanArgs x{a, {}};
#define LRKV_QD(DH, RR)                                                                                         \
    if (D_H == DH && R == RR)                                                                                   \
        return D_R == 0 ? launch_t<DH, RR, 0>(x, sms, smem_limit, stream)                                       \
                        : launch_t<DH, RR, 64>(x, sms, smem_limit, stream);
    LRKV_QD(64, 8) LRKV_QD(64, 16) LRKV_QD(64, 32) LRKV_QD(128, 8) LRKV_QD(128, 16) LRKV_QD(128, 32)
#undef LRKV_QD
    return cudaErrorInvalidValue;
}

}  // namespace lrkv
