// prefix.cu -- one decode step of a batch whose sequences share a prefix.
//
// Softmax attention over the prefix's tokens and a sequence's own is the log-sum-exp merge of the
// two parts' states (m, l, acc), so the prefix is scanned once for the whole batch:
//     per (sequence b, head h):  s_t = (q_bh . s^K_t + q~_bh . z^K_{h,t}) * scale * log2 e
//     m = max s_t,  l = sum 2^(s_t - m),  acc = sum 2^(s_t - m) [s^V_t | z^V_{h,t}]
// and the combine merges its pieces with the partials of the sequences' own scan.
//
// The scan is bound by the tensor cores or the memory, depending on the batch: per cached token and
// head it does 4 B (d_h + r) flops on 4 (d_h / H + r) bytes.  A CTA has 128 query rows, hb heads x
// ns sequences, and treats them as one attention problem of width d_h + zw, zw = hb r:
//     S = [Q | diag(Q~)] . [s^K | z^K of the hb heads]^T,   O += P . [s^V | z^V of the hb heads]
// where a row of diag(Q~) holds q~ in its own head's r columns and zeros elsewhere, and of a row's zw
// latent sums only its own head's r are used.  That is hb times the latents' products needed, on
// tensor cores that would otherwise wait: with a head per tile (no waste) the shared rows would be
// read hb times as often, and the prefix's rows of a batch of 16 would fill an eighth of a tile.
// zw = 128 for few sequences, 64 for more (prefix_tile).
// Per 64-token page: S by tcgen05.mma (M = 128, N = 64, K = d_k + 2 zw), P = 2^(S scale log2 e - m) in bf16
// into one of two TMEM buffers, O by tcgen05.mma with A = P from TMEM (N = d_h + zw).  Warp roles and the lazily
// raised maximum as in the prefill (prefill_tc.cu): warp 0 key producer, 6 value producer (TMA, 128-byte swizzle),
// 1 issues S, 7 issues P V; 2..5 and 8..11 take the first and the second 32 tokens of a page for one query row
// per thread (one warp per scheduler spent some 1000 cycles on a page's 64, twice what the MMAs need).
// Measured, the call as a whole: 32 heads of r = 16 x 16 sequences behind 8,192 tokens 25 us, 32 heads of r = 32 x
// 32 sequences behind 32,768 56 us, 128 heads of r = 16 with the positional key x 48 behind 4,001 65 us.  A page
// takes a CTA some 1,900 cycles, of which its products need 1,280 (d_h = zw = 128); the rest is the chain S, softmax,
// P V of one tile, and a piece's start and end some 6 us.
#include <type_traits>
#include <utility>

#include "lrkv_internal.cuh"
#include "prefix.h"
#include "tile_attn.cuh"

namespace lrkv {

namespace {

constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

__device__ __forceinline__ bool prefix_good(const PrefixArgs& a, int P) {
    return P >= 0 && P <= a.max_blocks * kBlockSize;
}

// [Q | diag(Q~)] is the A operand of S, diag(Q~) as two matrices: q~ rounded to bf16, and what that rounding
// left, rounded to bf16 (each a product with the same z^K).  With the first alone the output's relative error was
// 0.0031, of which the output's own rounding is 0.0016; with both it is 0.0024.
// As many of its 64-column blocks as fit sit in TMEM (an MMA of N = 64 would read twice as many bytes of
// A from shared memory as of B, and shared memory is what bounds it: 32 heads of r = 32 x 32 sequences, 32 K tokens,
// 33 us instead of 38), the rest (zw = 128 with d_h = 128) in shared memory.  Shared memory: those blocks (16 KB
// each), a ring of key stages [64 tokens][D_K + ZW] and one of value stages [64][D_H + ZW] (64-column
// blocks of 8 KB), barriers.  As many stages as fit.
template <int D_H, int D_R, int ZW>
struct PxLayout {
    static constexpr int D_K = D_H + D_R;
    static constexpr int NBK = (D_K + ZW) / 64, NBV = (D_H + ZW) / 64;  // 64-column blocks of a key / value row
    static constexpr int NBQ = NBK + ZW / 64, QROOM = (384 - D_H - ZW) / 32;  // blocks of Q, and room in TMEM
    static constexpr int QBT = NBQ < QROOM ? NBQ : QROOM, QBS = NBQ - QBT;  // in TMEM, in shared memory
    static constexpr uint32_t Q_BYTES = QBS * 16384, K_BYTES = NBK * 8192, V_BYTES = NBV * 8192;
    static constexpr uint32_t ROOM = 232448 - 1024 - 1536 - Q_BYTES;
    static constexpr int BOTH = ROOM / (K_BYTES + V_BYTES);
    static constexpr int VST = BOTH > 4 ? 4 : BOTH;
    static constexpr int KST = VST < 4 && ROOM - VST * (K_BYTES + V_BYTES) >= K_BYTES ? VST + 1 : VST;
    static constexpr uint32_t OFF_K = Q_BYTES, OFF_V = OFF_K + KST * K_BYTES, OFF_BAR = OFF_V + VST * V_BYTES;
    static constexpr uint32_t OFF_MX = OFF_BAR + 512, SMEM = OFF_MX + 1024 + 1024;
    static_assert(VST >= 2 && SMEM <= 232448, "stages");
    // TMEM columns: S, two P buffers, O, Q (two bf16 a column in P and Q).  The rows take S into registers
    // at once, so the next page's S is computed while they work on this one's.  (With two S buffers and P written
    // over S, S_{j+1} had to wait for P_{j-1} V_{j-1}: 1700 cycles a page instead of 1200.)
    static constexpr uint32_t TM_S = 0, TM_P = 64, TM_O = 128, TM_Q = TM_O + D_H + ZW;
    static_assert(TM_Q + QBT * 32 <= 512, "TMEM");
};

constexpr int lcm2(int n) { return n % 2 ? 2 * n : n; }

// f(j, U) for the tiles j0 + U < nt, U = 0, 1, .., stopping at the first failure: tile loops unrolled
// over the ring's stages and the S buffers, so that every operand of every MMA is loop-invariant.
template <class F, int... U>
__device__ __forceinline__ bool tiles(F&& f, int j0, int nt, std::integer_sequence<int, U...>) {
    return ((j0 + U < nt ? f(j0 + U, std::integral_constant<int, U>{}) : true) && ...);
}

template <int D_H, int D_R, int ZW>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_scan_kernel(const __grid_constant__ PrefixMaps m, const PrefixArgs a, const int R) {
    using Lay = PxLayout<D_H, D_R, ZW>;
    constexpr int D_K = Lay::D_K, NBK = Lay::NBK, NBQ = Lay::NBQ, NBV = Lay::NBV, KST = Lay::KST, VST = Lay::VST;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
    const uint32_t S0 = smem_u32(smem);
    const DecodeArgs& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = d.H, W = D_H + R;
    const int ht = blockIdx.x % a.htiles, stile = blockIdx.x / a.htiles, split = blockIdx.y;
    const int h0 = ht * a.hb, b0 = stile * a.ns;
    const int P = prefix_good(a, a.len[0]) ? a.len[0] : 0;
    // this piece: pages [pg0, pg0 + nt)
    const int np = (P + kBlockSize - 1) / kBlockSize;
    const int pg0 = (int)((long long)np * split / a.nsplit);
    const int nt = (int)((long long)np * (split + 1) / a.nsplit) - pg0;

    // this thread's query row (softmax warps): TMEM lane = row = head x ns + sequence; and its half of a page
    const int qq = warp & 3, half = warp >> 3;
    const int row = qq * 32 + lane;
    const int hl = row / a.ns, rb = b0 + row - hl * a.ns, rh = h0 + hl;
    const bool live = rh < H && rb < d.B;
    const size_t at = ((size_t)rb * H + rh) * a.nsplit + split;
    if (nt == 0) {  // an empty piece: its sums are not read
        pdl_wait();  // (this grid's end stands for that of the launches before it)
        if (warp >= 8 && live) {
            a.ml[at * 2] = -INFINITY;
            a.ml[at * 2 + 1] = 0.f;
        }
        return;
    }

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
    uint64_t* q_ready = bars + 0;
    uint64_t* s_full = bars + 1;    // S_j computed
    uint64_t* s_read = bars + 2;    // and taken by all rows
    // p_full[j % 2]: P_j written.  Two, because S_{j+1} may be there before P_j: with one barrier the rows
    // could write P_{j+1}, a softmax of some 0.5 us later, before warp 7 has looked at the phase of P_j.  P_{j+2}
    // needs P_j V_j.
    uint64_t* p_full = bars + 4;    // [2]
    uint64_t* o_done = bars + 6;    // [2] o_done[j % 2]: P_j V_j complete, P buffer j % 2 free
    uint64_t* s_drain = bars + 8;   // all S MMAs of the CTA complete
    uint64_t* pv_drain = bars + 9;
    uint64_t* k_full = bars + 10;   // [4]
    uint64_t* k_empty = bars + 14;
    uint64_t* v_full = bars + 18;
    uint64_t* v_empty = bars + 22;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
    volatile int* abort_flag = reinterpret_cast<int*>(bars + 27);
    auto B = [&](uint64_t* p) { return smem_u32(p); };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };

    if (threadIdx.x == 0) {
        mbar_init(B(q_ready), 256);
        mbar_init(B(s_full), 1);
        mbar_init(B(s_read), 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(B(p_full + i), 256);
            mbar_init(B(o_done + i), 1);
        }
        mbar_init(B(s_drain), 1);
        mbar_init(B(pv_drain), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(B(k_full + i), 1);
            mbar_init(B(k_empty + i), 1);
            mbar_init(B(v_full + i), 1);
            mbar_init(B(v_empty + i), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const bool keys = warp == 0;  // (of the two producers)
    int issued = 0;               // stages a producer has filled
    if (warp == 0 || warp == 6) {
        // ---------------------------------------------------------------- TMA producers
        const int oob_row = d.num_blocks * kBlockSize;  // whole box out of bounds: zeros
        auto fetch = [&](int batch) {
            const int i = batch * 32 + lane;
            int r = oob_row;
            if (i < nt) {
                const int blk = a.blocks[pg0 + i];
                if (blk >= 0 && blk < d.num_blocks)
                    r = blk * kBlockSize;
                else
                    set_status(d.status, LRKV_DEV_BAD_BLOCK);
            }
            return r;
        };
        const int depth = keys ? KST : VST;
        const uint32_t stage_bytes = keys ? Lay::K_BYTES : Lay::V_BYTES;
        const int nblk = keys ? D_K / 64 : D_H / 64;
        uint64_t* full = keys ? k_full : v_full;
        uint64_t* empty = keys ? k_empty : v_empty;
        const CUtensorMap* ms = keys ? &m.sK : &m.sV;
        const CUtensorMap* mz = keys ? &m.zK : &m.zV;
        const uint32_t ring = S0 + (keys ? Lay::OFF_K : Lay::OFF_V);
        int cur = fetch(0), nxt = fetch(1);
        int st = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            if (j > 0 && (j & 31) == 0) {
                cur = nxt;
                nxt = fetch((j >> 5) + 1);
            }
            const int prow = __shfl_sync(0xffffffffu, cur, j & 31);
            if ((j >= depth && !wait_role(B(empty + st), phase, d)) || aborted()) {
                ok = false;
                break;
            }
            if (lane == 0) {
                uint32_t dst = ring + st * stage_bytes;
                const uint32_t bar = B(full + st);
                mbar_arrive_expect_tx(bar, stage_bytes);
                for (int bk = 0; bk < nblk; ++bk, dst += 8192) tma_load_2d(dst, ms, 64 * bk, prow, bar);
                for (int bk = 0; bk < ZW / 64; ++bk, dst += 8192) tma_load_2d(dst, mz, h0 * R + 64 * bk, prow, bar);
            }
            __syncwarp();
            issued = j + 1;
            if (++st == depth) {
                st = 0;
                phase ^= 1;
            }
        }
        if (!ok) *abort_flag = 1;
    } else if (warp == 1) {
        // ---------------------------------------------------------------- score MMAs
        constexpr uint32_t id_S = idesc_bf16_f32(128, 64);
        const uint64_t dQ = kdesc128(S0), dK = kdesc128(S0 + Lay::OFF_K);
        auto s_tile = [&](int j, auto UU) -> bool {
            constexpr int st = decltype(UU)::value % KST;
            if (aborted() || !wait_role(B(k_full + st), (j / KST) & 1, d) ||
                (j >= 1 && !wait_role(B(s_read), (j - 1) & 1, d)))
                return false;
            tc_fence_after();
            constexpr uint64_t so = st * (Lay::K_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < NBQ * 4; ++kk) {
                const int kb = kk >> 2 < NBK ? kk >> 2 : (kk >> 2) - ZW / 64;  // z^K's blocks twice
                const uint64_t bd = dK + so + ((kb * 8192 + (kk & 3) * 32) >> 4);
                if (elect_one_sync()) {
                    if (kk < Lay::QBT * 4)
                        tc_mma_bf16_ts(tmem + Lay::TM_S, tmem + Lay::TM_Q + kk * 8, bd, id_S, kk > 0);
                    else
                        tc_mma_bf16(tmem + Lay::TM_S, dQ + ((((kk >> 2) - Lay::QBT) * 16384 + (kk & 3) * 32) >> 4), bd,
                                    id_S, 1);
                }
            }
            if (elect_one_sync()) {
                tc_commit(B(s_full));
                tc_commit(B(k_empty + st));
            }
            __syncwarp();
            return true;
        };
        bool ok = wait_role(B(q_ready), 0, d);
        tc_fence_after();
        for (int j = 0; j < nt && ok; j += KST) ok = tiles(s_tile, j, nt, std::make_integer_sequence<int, KST>{});
        if (!ok) *abort_flag = 1;
        // every MMA this warp issued has finished before the CTA tears TMEM down
        if (elect_one_sync()) tc_commit(B(s_drain));
        __syncwarp();
        drain(B(s_drain), 0, d.status);
    } else if (warp == 7) {
        // ---------------------------------------------------------------- P V MMAs
        constexpr uint32_t id_PV = idesc_bf16_f32(128, D_H + ZW) | (1u << 16);  // B is MN-major
        const uint64_t dV = mndesc128(S0 + Lay::OFF_V);
        auto pv_tile = [&](int j, auto UU) -> bool {
            constexpr int U = decltype(UU)::value, st = U % VST, sb = U & 1;
            if (aborted() || !wait_role(B(p_full + sb), (j >> 1) & 1, d) ||
                !wait_role(B(v_full + st), (j / VST) & 1, d))
                return false;
            tc_fence_after();
            constexpr uint64_t so = st * (Lay::V_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < kBlockSize / 16; ++kk)
                if (elect_one_sync())
                    tc_mma_bf16_ts(tmem + Lay::TM_O, tmem + Lay::TM_P + sb * 32 + kk * 8, dV + so + (kk * 2048 >> 4),
                                   id_PV, (j | kk) != 0);
            if (elect_one_sync()) {
                tc_commit(B(o_done + sb));
                tc_commit(B(v_empty + st));
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        for (int j = 0; j < nt && ok; j += lcm2(VST))
            ok = tiles(pv_tile, j, nt, std::make_integer_sequence<int, lcm2(VST)>{});
        if (!ok) *abort_flag = 1;
        if (elect_one_sync()) tc_commit(B(pv_drain));
        __syncwarp();
        drain(B(pv_drain), 0, d.status);
    } else {
        // ---------------------------------------------------------------- query rows: softmax, partials
        const uint32_t tl = (uint32_t)(qq * 32) << 16;
        {
            // [Q | diag(Q~)] row, block by block of 64 columns: into TMEM (two columns a register), or K-major with
            // 128-byte swizzle (16-byte chunk c at c ^ (row mod 8)).  The two halves' threads of a row take every
            // other block.
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const size_t qr = (size_t)(live ? rb : 0) * H + (live ? rh : 0);
            const uint4* q = reinterpret_cast<const uint4*>(d.q + qr * D_K);
            const float* qt = d.qt + qr * R;
            bool waited = false;
#pragma unroll
            for (int bk = 0; bk < NBQ; ++bk) {
                if ((bk & 1) != half) continue;
                if (bk >= D_K / 64 && !waited) {
                    pdl_wait();     // q~
                    pdl_trigger();  // the scan of the sequences' own tokens may fill the SMs that this grid leaves
                    waited = true;
                }
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint4 x = zero;
                    if (bk < D_K / 64) {
                        if (live) x = q[bk * 8 + c];
                    } else {
                        const int col = (bk - (bk < NBK ? D_K / 64 : NBK)) * 64 + c * 8 - hl * R;
                        if (live && col >= 0 && col < R) {
                            const float4 y = *reinterpret_cast<const float4*>(qt + col);
                            const float4 z = *reinterpret_cast<const float4*>(qt + col + 4);
                            x = make_uint4(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w), pack_bf16x2(z.x, z.y),
                                           pack_bf16x2(z.z, z.w));
                            if (bk >= NBK)  // what the rounding left
                                x = make_uint4(pack_bf16x2(y.x - bf16lo(x.x), y.y - bf16hi(x.x)),
                                               pack_bf16x2(y.z - bf16lo(x.y), y.w - bf16hi(x.y)),
                                               pack_bf16x2(z.x - bf16lo(x.z), z.y - bf16hi(x.z)),
                                               pack_bf16x2(z.z - bf16lo(x.w), z.w - bf16hi(x.w)));
                        }
                    }
                    v[4 * c] = x.x;
                    v[4 * c + 1] = x.y;
                    v[4 * c + 2] = x.z;
                    v[4 * c + 3] = x.w;
                }
                if (bk < Lay::QBT) {
                    tmem_st_32x32b_x32(tmem + tl + Lay::TM_Q + bk * 32, v);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(smem + (bk - Lay::QBT) * 16384 + row * 128 +
                                                  ((c ^ (row & 7)) << 4)) =
                            make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                }
            }
            // (a half without a block of q~ waits too: this grid's end stands for that of the launches before it, and
            // the next launch must find q~ there)
            if (!waited) {
                pdl_wait();
                pdl_trigger();
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(B(q_ready));
        }
        bool ok = true;
        float mref = -INFINITY, l = 0.f;
        int vst = 0;
        uint32_t vphase = 0;
        // [row][page parity][half], later [row][half] sums: eight bytes that only the row's two threads touch
        uint16_t* const mxs = reinterpret_cast<uint16_t*>(smem + Lay::OFF_MX) + row * 4;
        // After an expired wait the loop goes on without work, so that the two halves still meet at their barrier.
        for (int j = 0; j < nt; ++j) {
            // visible tokens of this page: none of a page with a bad id
            const int blk = a.blocks[pg0 + j];
            const int lim = blk >= 0 && blk < d.num_blocks ? P - (pg0 + j) * kBlockSize : 0;
            ok = ok && !aborted() && wait_role(B(s_full), j & 1, d);
            uint32_t sv[32];
            float mx = -INFINITY;
            if (ok) {
                tc_fence_after();
                tmem_ld_32x32b_x32(tmem + tl + Lay::TM_S + half * 32, sv);
                tc_fence_before();
                mbar_arrive(B(s_read));
                if (lim < kBlockSize) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) sv[e] = half * 32 + e < lim ? sv[e] : 0xff800000u;
                    // rows of s^V, z^V behind the end may hold any bits: cleared before P V reads them
                    ok = wait_role(B(v_full + vst), vphase, d);
                    const int vr = row & 63;
                    if (ok && vr >= lim) {
                        const uint4 z = make_uint4(0, 0, 0, 0);
                        for (int bk = (row >> 6) + 2 * half; bk < NBV; bk += 4) {
                            uint4* r0 =
                                reinterpret_cast<uint4*>(smem + Lay::OFF_V + vst * Lay::V_BYTES + bk * 8192 + vr * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) r0[i] = z;
                        }
                    }
                }
                float m4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = max_nan(__uint_as_float(sv[i]), __uint_as_float(sv[4 + i]));
#pragma unroll
                for (int e = 8; e < 32; ++e) m4[e & 3] = max_nan(m4[e & 3], __uint_as_float(sv[e]));
                mx = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
                // diag(Q~)'s zeros times another head's NaN or infinity are NaN (and so is what rounding an infinite
                // product left): such logits are formed again from the row's own head alone.  (The look for
                // them, in the maximum's own instructions and a vote, costs 1%: 55.2 us -> 56.0 for 32,768 tokens;
                // a page with one such token takes 5 us more, one full of them 150.)
                if (__any_sync(0xffffffffu, mx != mx)) {
                    uint32_t nans = 0;
#pragma unroll
                    for (int e = 0; e < 32; ++e) nans |= (__uint_as_float(sv[e]) != __uint_as_float(sv[e])) << e;
                    const size_t qr = (size_t)rb * H + rh;
                    for (uint32_t todo = live ? nans : 0u; todo != 0; todo &= todo - 1) {
                        const int e = __ffs(todo) - 1;
                        const size_t t = (size_t)blk * kBlockSize + half * 32 + e;
                        const float x = dot8(d.q + qr * D_K, a.sK + t * D_K, D_K) +
                                        dot8(d.qt + qr * R, a.zK + (t * H + rh) * R, R);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sv[i] = i == e ? __float_as_uint(x) : sv[i];
                    }
                    __syncwarp();
                    mx = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(sv[e]));
                }
                mx *= d.scale_log2;
            }
            if (++vst == VST) {
                vst = 0;
                vphase ^= 1;
            }
            // The row's maximum over both halves, exchanged in bf16 rounded up (a truncated one hides up to 1/128 of a
            // positive maximum, from 2^14 on more than the log2 units that make p overflow).  (The next write to this
            // parity's slot comes after the next page's barrier.)
            mxs[(j & 1) * 2 + half] = (uint16_t)((__float_as_uint(mx) + (mx > 0.f ? 0xffffu : 0u)) >> 16);
            named_bar(1 + qq, 64);
            const uint32_t both = *reinterpret_cast<const uint32_t*>(mxs + (j & 1) * 2);
            bool raise = fmaxf(bf16lo(both), bf16hi(both)) > mref + kRescaleThreshold;  // or the row's first token
            float alpha = 1.f;
            // Where it may have to be raised, the exact maxima decide, and become the reference, so that the heaviest
            // token's probability, 1, is not rounded (pieces of a page or two: the output's error 0.0018 instead of
            // 0.0027).  Every thread follows the exchange, after an expired wait too: the halves' references, and so
            // their barriers, stay the same.
            if (__any_sync(0xffffffffu, raise)) {
                float* const fx = reinterpret_cast<float*>(mxs);  // [half], over both parities' slots
                named_bar(1 + qq, 64);
                fx[half] = mx;
                named_bar(1 + qq, 64);
                const float mnew = fmaxf(fx[0], fx[1]);
                named_bar(1 + qq, 64);
                raise = mnew > mref + kRescaleThreshold;
                if (raise) {
                    alpha = mref == -INFINITY ? 0.f : ex2_approx(mref - mnew);
                    mref = mnew;
                }
            }
            if (!ok) continue;
            // p = 2^(s scale log2 e - m), 0 everywhere as long as the row has seen no token
            const float nm = mref == -INFINITY ? -INFINITY : -mref;
            float r4[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float p0 = ex2_approx(fmaf(__uint_as_float(sv[e]), d.scale_log2, nm));
                const float p1 = ex2_approx(fmaf(__uint_as_float(sv[e + 1]), d.scale_log2, nm));
                r4[(e >> 1) & 3] += p0 + p1;
                pk[e / 2] = pack_bf16x2(p0, p1);
            }
            if (j >= 2) {  // P_{j-2} V_{j-2} has read this P buffer
                ok = wait_role(B(o_done + (j & 1)), ((j - 2) >> 1) & 1, d);
                if (!ok) continue;
                tc_fence_after();
            }
            tmem_st_32x32b_x16(tmem + tl + Lay::TM_P + (j & 1) * 32 + half * 16, pk);
            l = l * alpha + ((r4[0] + r4[1]) + (r4[2] + r4[3]));
            // O may only be rescaled once P_{j-1} V_{j-1} has finished accumulating into it
            if (j > 0 && __any_sync(0xffffffffu, raise)) {
                ok = wait_role(B(o_done + ((j - 1) & 1)), ((j - 1) >> 1) & 1, d);
                if (!ok) continue;
                tc_fence_after();
                uint32_t v[32];
#pragma unroll 1
                for (int c = half; c < (D_H + ZW) / 32; c += 2) {
                    tmem_ld_32x32b_x32(tmem + tl + Lay::TM_O + c * 32, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                    tmem_st_32x32b_x32(tmem + tl + Lay::TM_O + c * 32, v);
                }
            }
            tmem_wait_st();
            fence_proxy_async_smem();  // cleared value rows (if any) before the tensor cores read them
            tc_fence_before();
            mbar_arrive(B(p_full + (j & 1)));
        }
        tmem_wait_st();  // (a wait that ran out may have left stores to TMEM behind)
        // the row's sum over both halves
        named_bar(1 + qq, 64);  // (the maxima have been read)
        float* const ls = reinterpret_cast<float*>(smem + Lay::OFF_MX) + row * 2;
        ls[half] = l;
        named_bar(1 + qq, 64);
        l += ls[half ^ 1];
        // ---- partials, unnormalised
        const uint32_t rs = 16u * ((W / 4) | 1);  // row stride of their staging
        if (ok) ok = wait_role(B(o_done + ((nt - 1) & 1)), ((nt - 1) >> 1) & 1, d);
        if (ok) {
            tc_fence_after();
            const bool nan = l != l;  // handed on as NaN values with a weight, not as an empty part
            if (nan) {
                l = 1.f;
                if (!(fabsf(mref) < INFINITY)) mref = 0.f;
            }
            if (live && half == 0) {
                a.ml[at * 2] = mref;
                a.ml[at * 2 + 1] = l;
            }
            // The row goes through shared memory (the rings are idle: every copy has landed and every MMA that reads
            // them is done) and leaves in one bulk copy: stored straight from registers, a warp's 16-byte pieces of 32
            // rows took 4 to 5 us.  Rows start an odd number of 16-byte units apart.
            uint8_t* const srow = smem + row * rs;
            const uint4 nan4 = make_uint4(0x7fc00000u, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u);
#pragma unroll 1
            for (int c = half; c < D_H / 32; c += 2) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + tl + Lay::TM_O + c * 32, v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(srow + c * 128 + i * 16) =
                        nan ? nan4 : make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            // latent sums: 32 columns at a time, each row keeps its own head's
#pragma unroll 1
            for (int c = half; c < ZW / 32; c += 2) {
                // (a warp's rows span heads hl of its first to its last lane)
                const int first = (qq * 32) / a.ns * R, last = (qq * 32 + 31) / a.ns * R + R;
                if (c * 32 + 32 <= first || c * 32 >= last) continue;
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + tl + Lay::TM_O + D_H + c * 32, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int col = c * 32 + i * 4 - hl * R;
                    if (col >= 0 && col < R)
                        *reinterpret_cast<uint4*>(srow + (D_H + col) * 4) =
                            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
            fence_proxy_async_smem();
        } else {
            *abort_flag = 1;
        }
        named_bar(1 + qq, 64);  // both halves of the rows are written
        if (ok && half == 0) {
            if (live) {
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a.acc + at * W),
                             "r"(S0 + row * rs), "r"(W * 4)
                             : "memory");
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    // Whichever wait ran out, and however late: the copies in flight land before the block gives up its shared memory.
    if ((warp == 0 || warp == 6) && *abort_flag) {
        const int depth = keys ? KST : VST;
        for (int k = max(0, issued - depth); k < issued; ++k)
            drain(B((keys ? k_full : v_full) + k % depth), (k / depth) & 1, d.status);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merge of the prefix's pieces and the sequences' own partials: grid (H, ceil(B / blockDim.z)), block
// (W / 4 column quads, slices, sequences).  A slice merges every blockDim.y-th partial of its sequence, PPS
// loads in flight; the slices are merged in shared memory; then B_h^V, copied there meanwhile for all
// sequences of the block.  The host takes as many slices as fill the GPU about once: each block is one chain of
// dependent loads of some 5 us, so a second wave costs as much as the first.  (One thread per column walking
// all partials: 27 us for 32 heads x 32 sequences x 20 partials; eight slices for every block: 10 us there, but 18
// for 128 heads x 48 sequences x 5.)
template <int D_H, int R>
__global__ void __launch_bounds__(512) prefix_combine_kernel(const PrefixArgs a) {
    constexpr int W = D_H + R, W4 = W / 4, ROWS_MAX = 512 / W4, PPS = 6;
    const DecodeArgs& d = a.d;
    const int c4 = threadIdx.x, sl = threadIdx.y, nsl = blockDim.y;
    const int h = blockIdx.x, b = blockIdx.y * blockDim.z + threadIdx.z;
    const int tid = (threadIdx.z * nsl + sl) * W4 + c4, nthreads = W4 * nsl * blockDim.z;
    __shared__ float sm_m[ROWS_MAX], sm_l[ROWS_MAX];
    __shared__ __align__(16) float sm_acc[ROWS_MAX][W];
    __shared__ __align__(16) uint16_t sm_bv[D_H * R];
    const bool have = b < d.B;
    const int P = a.len[0], L = a.suffix && have ? d.seq_lens[b] : 0;
    const bool bad = !prefix_good(a, P) || L < 0 || L > d.max_pages * kBlockSize || (!d.part_out && P + L == 0);
    if (!d.part_out) {
        const uint16_t* bv = d.BV + (size_t)h * D_H * R;
        for (int i = tid; i < D_H * R / 8; i += nthreads)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(sm_bv + i * 8)), "l"(bv + i * 8)
                         : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    pdl_wait();  // the scans
    const int row0 = threadIdx.z * nsl;  // the sequence's rows of sm_acc
    float m = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (have && !bad) {
        const size_t at = ((size_t)b * d.H + h) * a.nsplit;
        const float2* ml0 = reinterpret_cast<const float2*>(a.ml) + at;
        const float4* ac0 = reinterpret_cast<const float4*>(a.acc + at * W);
        const int n0 = P > 0 ? a.nsplit : 0;
        int n = n0;
        const float2* ml1 = ml0;
        const float4* ac1 = ac0;
        if (L > 0) {
            const int2 fe = d.seg_table[b * d.nhg + h / (d.H / d.nhg)];
            n += fe.y;
            ml1 = reinterpret_cast<const float2*>(d.part_ml) + (size_t)h * d.pmax + fe.x - n0;
            ac1 = reinterpret_cast<const float4*>(d.part_acc + ((size_t)h * d.pmax + fe.x) * W) - (ptrdiff_t)n0 * W4;
        }
        for (int p0 = sl; p0 < n; p0 += nsl * PPS) {
            float2 ml[PPS];
            float4 x[PPS];
#pragma unroll
            for (int u = 0; u < PPS; ++u) {
                const int p = p0 + u * nsl;
                ml[u] = p < n ? (p < n0 ? ml0 : ml1)[p] : make_float2(-INFINITY, 0.f);
                x[u] = p < n ? (p < n0 ? ac0 : ac1)[(size_t)p * W4 + c4] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < PPS; ++u) mn = fmaxf(mn, ml[u].x);
            if (mn == -INFINITY) continue;
            const float sc = m == -INFINITY ? 0.f : exp2f(m - mn);
            l *= sc;
            v.x *= sc;
            v.y *= sc;
            v.z *= sc;
            v.w *= sc;
#pragma unroll
            for (int u = 0; u < PPS; ++u) {
                if (ml[u].x == -INFINITY) continue;  // an empty piece: its sums were not written
                const float w = exp2f(ml[u].x - mn);
                l = fmaf(w, ml[u].y, l);
                v.x = fmaf(w, x[u].x, v.x);
                v.y = fmaf(w, x[u].y, v.y);
                v.z = fmaf(w, x[u].z, v.z);
                v.w = fmaf(w, x[u].w, v.w);
            }
            m = mn;
        }
    }
    *reinterpret_cast<float4*>(&sm_acc[row0 + sl][c4 * 4]) = v;
    if (c4 == 0) {
        sm_m[row0 + sl] = m;
        sm_l[row0 + sl] = l;
    }
    __syncthreads();
    float* pdst = d.part_out ? d.part_out + ((size_t)b * d.H + h) * (W + 2) : nullptr;
    if (sl == 0) {
        float M = -INFINITY;
        for (int i = 0; i < nsl; ++i) M = fmaxf(M, sm_m[row0 + i]);
        float ls = 0.f;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < nsl; ++i) {
            const float w = sm_m[row0 + i] == -INFINITY ? 0.f : exp2f(sm_m[row0 + i] - M);
            const float4 x = *reinterpret_cast<const float4*>(&sm_acc[row0 + i][c4 * 4]);
            ls = fmaf(w, sm_l[row0 + i], ls);
            t.x = fmaf(w, x.x, t.x);
            t.y = fmaf(w, x.y, t.y);
            t.z = fmaf(w, x.z, t.z);
            t.w = fmaf(w, x.w, t.w);
        }
        if (have && bad && h == 0 && c4 == 0) set_status(d.status, LRKV_DEV_BAD_SEQLEN);
        if (have && pdst) {  // unnormalised (a bad length: the empty state)
            pdst[c4 * 4] = t.x;
            pdst[c4 * 4 + 1] = t.y;
            pdst[c4 * 4 + 2] = t.z;
            pdst[c4 * 4 + 3] = t.w;
            if (c4 == 0) {
                pdst[W] = M;
                pdst[W + 1] = ls;
            }
        }
        // (the sum is 0 for a bad length, and where every page of the tokens was a bad one: zeros)
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        *reinterpret_cast<float4*>(&sm_acc[row0][c4 * 4]) = make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv);
    }
    if (pdst) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!have) return;
    for (int i = sl * W4 + c4; i < D_H; i += nsl * W4) {
        float x = sm_acc[row0][i];
        const uint4* bvr = reinterpret_cast<const uint4*>(sm_bv + i * R);
        const float* z = &sm_acc[row0][D_H];
#pragma unroll
        for (int k = 0; k < R / 8; ++k) {
            const uint4 w = bvr[k];
            x = fmaf(bf16lo(w.x), z[k * 8 + 0], x);
            x = fmaf(bf16hi(w.x), z[k * 8 + 1], x);
            x = fmaf(bf16lo(w.y), z[k * 8 + 2], x);
            x = fmaf(bf16hi(w.y), z[k * 8 + 3], x);
            x = fmaf(bf16lo(w.z), z[k * 8 + 4], x);
            x = fmaf(bf16hi(w.z), z[k * 8 + 5], x);
            x = fmaf(bf16lo(w.w), z[k * 8 + 6], x);
            x = fmaf(bf16hi(w.w), z[k * 8 + 7], x);
        }
        const __nv_bfloat16 ob = __float2bfloat16_rn(x);
        d.out[((size_t)b * d.H + h) * D_H + i] = *reinterpret_cast<const uint16_t*>(&ob);
    }
}

}  // namespace

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Which tile: the fewest columns to take, tiles x (d_k + d_h + 2 zw) (one of 64 columns covers twice the
// sequences of one of 128 with half the heads).  128 heads of r = 16 x 48 sequences, positional key: 48 tiles of
// 128 columns, 64 us; 64 of 64, 84 us.  (The second product with z^K does not count: the tensor cores wait for the
// softmax, and 32 heads of r = 32 x 32 sequences take 55 us with it and 57 without.)
static PrefixPlan prefix_tile(int H, int D_H, int R, int D_R, int B) {
    PrefixPlan best{};
    long long best_cost = -1;
    for (int zw = 128; zw >= 64; zw /= 2) {
        PrefixPlan p{};
        p.zw = zw;
        p.hb = zw / R;
        p.ns = 128 / p.hb;
        p.htiles = (H + p.hb - 1) / p.hb;
        p.stiles = (B + p.ns - 1) / p.ns;
        const long long cost = (long long)p.htiles * p.stiles * (2 * D_H + D_R + 2 * zw);
        if (best_cost < 0 || cost < best_cost) {
            best = p;
            best_cost = cost;
        }
    }
    return best;
}

int prefix_most_splits(int H, int D_H, int R, int D_R, int B, int max_blocks, int sms) {
    const PrefixPlan t = prefix_tile(H, D_H, R, D_R, B);
    const long long n = 2LL * sms / ((long long)t.htiles * t.stiles);
    return (int)(n < 1 ? 1 : n < max_blocks ? n : max_blocks);
}

// How many pieces, and whether some SMs are kept for the scan of the sequences' own tokens, by a model of
// the two launches in us: a piece costs 6 (queries, pipeline fill, partials) and 0.8 a page of 512 columns,
// the pieces of all tiles run in waves of one CTA per SM; the other scan costs 6, as much again for each
// sequence that a CTA meets, and streams 28 bytes a ns on one SM.  Of the own tables' capacity half is
// taken to be in use.  Measured: 32 heads x 16 sequences behind 8 K tokens 33 us one after the other, 25 side by
// side; 128 x 48 behind 4 K 76 and 66.  The lengths are on the device, so the plan knows the tables' widths alone: the
// first case with own tables of 8 and 16 pages a sequence 25 us, of 32 and more (planned one after the other) 33; with
// 128, 256, 512 and 2,048 pages listed for the prefix's 128 25, 25, 28 and 47.  The search takes the host 0.3 to 3 us
// for short prefixes or many tiles, some 10 for one tile of 512 pages.
PrefixPlan prefix_plan(int H, int D_H, int R, int D_R, int B, int max_blocks, double own_bytes, int sms) {
    PrefixPlan best = prefix_tile(H, D_H, R, D_R, B);
    const long long ntiles = (long long)best.htiles * best.stiles;
    const double page = 0.8 * (2 * D_H + D_R + 2 * best.zw) / 512;
    double least = -1;
    for (int own = 0; own <= sms / 2; own += 8) {
        const int n = sms - own, m = own ? own : sms;
        const double t_own = own_bytes > 0 ? 6 + 6 * (1 + (double)B / m) + own_bytes / 2 / 28e3 / m : 0;
        for (int s = 1; s <= max_blocks && (s == 1 || ntiles * s <= 2LL * n); ++s) {
            const long long waves = (ntiles * s + n - 1) / n;
            const double t_prefix = waves * (page * ((max_blocks + s - 1) / s) + 6);
            const double hi = t_own > t_prefix ? t_own : t_prefix, lo = t_own + t_prefix - hi;
            const double t = own ? hi + 0.1 * lo : t_own + t_prefix;
            if (least < 0 || t < least) {
                least = t;
                best.nsplit = s;
                best.own_sms = own;
            }
        }
        if (own_bytes <= 0) break;
    }
    return best;
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

template <int D_H, int D_R, int ZW>
static cudaError_t launch_scan_t(const PrefixMaps& maps, const PrefixArgs& a, int R, cudaStream_t stream) {
    constexpr uint32_t smem = PxLayout<D_H, D_R, ZW>::SMEM;
    auto kern = prefix_scan_kernel<D_H, D_R, ZW>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int stiles = (a.d.B + a.ns - 1) / a.ns;
    return launch_dependent(kern, dim3(a.htiles * stiles, a.nsplit), dim3(kThreads), smem, stream, maps, a, R);
}

cudaError_t launch_prefix_scan(const PrefixMaps& maps, const PrefixArgs& a, int D_H, int R, int D_R,
                               cudaStream_t stream) {
#define LRKV_PS(DH, DR)                                                               \
    if (D_H == DH && D_R == DR)                                                       \
        return a.zw == 128 ? launch_scan_t<DH, DR, 128>(maps, a, R, stream)           \
                           : launch_scan_t<DH, DR, 64>(maps, a, R, stream);
    LRKV_PS(64, 0) LRKV_PS(64, 64) LRKV_PS(128, 0) LRKV_PS(128, 64)
#undef LRKV_PS
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_combine(const PrefixArgs& a, int D_H, int R, int sms, cudaStream_t stream) {
#define LRKV_PC(DH, RR)                                                               \
    if (D_H == DH && R == RR) {                                                       \
        constexpr int W4 = (DH + RR) / 4;                                             \
        int nsl = 1;                                                                  \
        while (nsl < 8 && (long long)a.d.H * a.d.B * W4 * nsl * 2 <= sms * 1536LL && W4 * nsl * 2 <= 512) nsl *= 2;   \
        int nseq = 1;                                                                 \
        while (nseq < a.d.B && W4 * nsl * nseq * 2 <= 256) nseq *= 2;                 \
        return launch_dependent(prefix_combine_kernel<DH, RR>, dim3(a.d.H, (a.d.B + nseq - 1) / nseq), \
                                dim3(W4, nsl, nseq), 0, stream, a);                   \
    }
    LRKV_PC(64, 8) LRKV_PC(64, 16) LRKV_PC(64, 32) LRKV_PC(128, 8) LRKV_PC(128, 16) LRKV_PC(128, 32)
#undef LRKV_PC
    return cudaErrorInvalidValue;
}

}  // namespace lrkv
