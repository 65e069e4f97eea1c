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
//     the offset 1152 = 1024 + 128 leaves the sums again as -1152 sum q~ (in the latents' K sums'
//     start; s^K's likewise or by a product with a constant A) and -1152 sum w (one such product per tile);
//   - tokens are the M of the logits' product (A = 16 tokens x 16 features, B = features x 8
//     heads) and the K of the values' (A = features x 16 tokens, B = 16 tokens x 8 heads), so both
//     leave a thread the same two heads and the probabilities pass from one to the other by a
//     transpose within the warp (movmatrix);
//   - a head's latents meet that head's q~ (or weights) only: B holds the head's column and zeros
//     elsewhere, and the eight heads of a tile accumulate into the same registers;
//   - scales: one per (token, head's block) multiplies the K sums in fp32; the V weights are
//     w_t = 2^(s_t + k_t - mz) in fp16 with a running maximum mz of their own, so tokens whose
//     scales differ by any power of two lose nothing but what is small beside the largest;
//   - s^K enters the logits in the same way, 32 features (a block) at a time; s^V, whose sums over
//     tokens cannot be scaled afterwards, is widened to bf16 (q_i 2^k is exact) once per 16 tokens
//     by converter warps.
// Warps of a CTA: consumers (8 heads each, ng groups taking 16-token tiles in turn), one
// producer (bulk copies of whole rows, which lie contiguous within a page, into a ring of
// stages), one or three converters; connected by mbarriers only, so they drift freely.  One CTA per
// SM; the work is cut as in the bf16 decode (decode_work.cuh).
//
// Measured: 24 sequences of 1 to 8,191 tokens, 32 heads of r = 16 and a positional key 46 us (the rows alone 18
// at the memory's pace); 4 of 16 to 32 K, 32 heads of r = 32, 50 (36); 8 of 8,192, 128 heads of r = 16, 86 (44);
// 16 of 2,048, 8 heads, 16 (2).  Bound by the consumers' instructions: a tile of 16 tokens x 8 heads takes a
// warp some 500, a quarter of them byte permutes, and up to 2,900 cycles with the rows already there; with twice as
// many warps each takes twice as long.  A third to a half of the issue slots are used; the waits are for the
// half-rate integer pipe, the tensor cores' results, and instructions (unrolled less, 128 heads gain and 32 lose).
// A call's start (plan, first copies: some 5 us) and end (groups merged, combine: 5 us) make up most of the short
// cases.
#include <cuda_fp16.h>

#include <type_traits>

#include "decode_work.cuh"
#include "lrkv_internal.cuh"
#include "quant.cuh"
#include "quant.h"

namespace lrkv {

namespace {

// Consumer warps at most: 8 (12 warps with the converters and the producer, so that a thread may hold
// 168 registers) for up to 64 heads, 16 (18 warps, 96 registers) for more.  Measured for 128 heads of
// r = 16: two tiles of 8 heads per warp in 12 warps 107 us, one with 16 consumers 97 at that time; for 32 heads
// more consumers are slower: with 8, 12 and 16 the ragged batch takes 45, 48 and 56 us, the long context 50, 60
// and 78 (every tile in work holds a stage of the ring as well).  Whole groups of warps take the tiles, so a head count
// that leaves warps over costs about as much as the next one that does not; 8 x 8,192 tokens of r = 16: 8 heads 23 us,
// 16 25, 24 and 32 30, 40 to 64 44 to 46, 72 71, 96 75, 112 80, 128 86.
// Warps that widen s^V: a tile takes one some 0.7 us.  With 8 consumers a tile is due every 0.75 us or less (one
// converter 54 us for the ragged batch, two 47, three 45), with 16 every 3 us, and the registers are worth more.
__host__ __device__ constexpr int converters(int cw) { return cw == 8 ? 3 : 1; }
constexpr int kMaxWalkers = 18;   // warps of a CTA at most
constexpr float kLazy = 8.0f;     // maxima are raised when exceeded by this much (log2 units)

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_16816_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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
// Plain loads from shared memory (the compiler may batch them, but not move them over a wait).
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    return *static_cast<const uint32_t*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    return *static_cast<const uint8_t*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Scale of a block: 2^(e - 127); NaN for byte 255, zero for 0 (a cleared row).
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e == 255 ? 0x7fc00000u : e << 23); }

// Byte i of x as a scale, NaN blocks apart.
__device__ __forceinline__ float byte_scale(uint32_t x, int i) {
    return __uint_as_float(__byte_perm(x, 0u, 0x0444 | (i << 12)) >> 1);
}

// try_wait that may sleep in hardware for some microseconds before it reports failure: a waiting warp then takes few
// issue slots from the others.
__device__ __forceinline__ bool mbar_try_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded wait of a whole warp; false (with the abort flag set) once it, or any other, gave up.  One look, then
// tries that sleep, unless the limit is a shortened one.  (Sleeping tries alone: 128 heads 87 us instead of 86, the
// ragged batch 46.6 instead of 45.7.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                          uint64_t limit_ns) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    const bool sleep = limit_ns == kWaitLimitNs;
    if (sleep && __all_sync(0xffffffffu, mbar_try_sleep(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        if (__all_sync(0xffffffffu, sleep ? mbar_try_sleep(bar, parity) : mbar_test(bar, parity))) return true;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) {
            set_status(status, LRKV_DEV_TIMEOUT);
            *abort_flag = 1;
            return false;
        }
    }
}

struct QuantPlan {
    int cw;                      // consumer warps the kernel is built for
    int nwh, ng;                 // consumer warps over the heads (8 each), groups
    int st;                      // tiles (of TOK tokens) per stage
    int own_stages;              // 1: a stage is one tile, and a slot of the ring always the same group's
    int nslot, ncb;              // stages of the ring, widened tiles (one to three per group)
    int stage_bytes, cb_bytes;
    int threads, smem_bytes;
};

struct QuantScanArgs {
    QuantDecodeArgs a;
    QuantPlan p;
};

// One warp's walk over the CTA's segments, as SegWalk's (decode_work.cuh, one layer), but stepped by the whole
// warp: the search for the sequence that a piece or range begins in takes 32 sequences at a time.  (One lane
// searching took up to 4 us of a CTA's start with 24 sequences.)
struct alignas(16) Walker {
    int item, gcur, gend, vstart, seg_start;
    int valid, vb, g0, g1, slot;

    // The first sequence b whose running total (of n(b), from `total` at b = 0 on) exceeds x, and the total before it.
    template <class W, class F>
    __device__ __forceinline__ static void search(const W& w, int x, int lane, F n, int* b_out, int* before) {
        int total = 0;
        for (int b0 = 0;; b0 += 32) {
            const int b = b0 + lane;
            const int mine = b < w.B ? n(b) : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += t;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, total + sum > x);
            if (hit || b0 + 32 >= w.B) {
                // (without a hit x lies behind the last sequence, which a plan never asks for: its last lane is taken)
                const int l = hit ? __ffs(hit) - 1 : min(31, w.B - 1 - b0);
                *b_out = b0 + l;
                *before = total + __shfl_sync(0xffffffffu, sum - mine, l);
                return;
            }
            total += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    __device__ __forceinline__ void start(int first_item) {
        item = first_item;
        gcur = gend = vstart = seg_start = vb = 0;
    }
    // Steps to the next segment (valid = 0: none left).  The whole warp calls it; lane 0 keeps the state.
    template <class W>
    __device__ __forceinline__ void advance(const W& w, int lane) {
        __syncwarp();
        Walker n = *this;
        n.valid = 1;
        if (w.pieces) {
            if (n.item >= w.work_items()) {
                n.valid = 0;
            } else {
                int b, base;
                search(w, n.item, lane, [&](int i) { return w.npieces(i, w.chunk); }, &b, &base);
                const unsigned gr = (unsigned)w.gran_b(b);
                const unsigned np = (gr + w.chunk - 1) / (unsigned)w.chunk, i = (unsigned)(n.item - base);
                const unsigned q = gr / np, r = gr - q * np;  // floor(i gr / np), i < np <= 2^16
                n.vb = b;
                n.g0 = (int)(i * q + (i * r) / np);
                n.g1 = (int)((i + 1) * q + ((i + 1) * r) / np);
                n.slot = n.item;
                n.item += gridDim.x;
            }
        } else {
            if (n.gcur >= n.gend) {
                if (n.gend > 0) n.item += gridDim.x;  // the current range is done
                if (n.item >= w.nranges) {
                    n.valid = 0;
                } else {
                    n.gcur = w.range_start(n.item);
                    n.gend = w.range_start(n.item + 1);
                    search(w, n.gcur, lane, [&](int i) { return w.gran_b(i); }, &n.vb, &n.vstart);
                }
            } else {
                // the range goes on in the next sequence that has tokens
                do {
                    ++n.vb;
                } while (n.vb < w.B && w.gran_b(n.vb) == 0);
            }
            if (n.valid) {
                const int gr = w.gran_b(n.vb), se = min(n.gend, n.vstart + gr);
                n.g0 = n.gcur - n.vstart;
                n.g1 = se - n.vstart;
                n.slot = n.vb + n.item;
                n.seg_start = n.gcur;
                n.gcur = se;
                if (se == n.vstart + gr) n.vstart = se;  // the next segment, if any, starts another sequence
            }
        }
        __syncwarp();
        if (lane == 0) *this = n;
        __syncwarp();
    }
};
static_assert(sizeof(Walker) == 48, "walkers are an array in shared memory with the work plan behind it");

// Row stride (floats) of a head in the staging of the group merge: 4 mod 16, so that the four head
// pairs and eight columns of a warp's store fall on different banks.
__host__ __device__ constexpr int merge_stride(int W) { return W % 16 == 0 ? W + 4 : W + 12; }

// Row stride (bytes) of a widened tile of s^V in bf16: an odd number of 16-byte units.
__host__ __device__ constexpr int cb_stride(int D_H) { return D_H * 2 + 16; }

template <int D_H, int R, int D_R, int CW, int TOK>
__global__ void __launch_bounds__((CW + 1 + converters(CW)) * 32, 1) quant_scan_kernel(const QuantScanArgs args) {
    constexpr int D_K = D_H + D_R, W = D_H + R, WS = merge_stride(W);
    constexpr int SB = cb_stride(D_H);
    constexpr int NKK = D_K / 16;
    constexpr int NZC = R > 16 ? R / 16 : 1;       // 16-byte chunks of a head's latents (r = 8: of two heads')
    constexpr int NCH = 8 * R / 16;                // chunks of a tile of 8 heads
    constexpr int TPP = kBlockSize / TOK;          // tiles per page
    constexpr int kConverters = converters(CW);
    constexpr int kUnroll = CW == 8 ? 8 : 2;       // of the loops over chunks (128 heads: 8 takes 104 us, 4 101, 2 90)
    // The bytes' offset leaves s^K's products by their sums' start instead of by products with a constant A, and
    // r <= 16 sums its values' products in two chains (ragged batch 47 -> 45 us).  With 16 consumers the shared
    // memory costs a stage, and the registers more than they bring (128 heads 90 -> 98).
    constexpr bool kSums = CW == 8;
    using WorkQ = WorkT<TOK>;
    static_assert(sizeof(WorkQ) <= 96 && alignof(WorkQ) <= 16, "room for the plan in shared memory");
    static_assert(CW + 1 + kConverters <= kMaxWalkers, "walkers");
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
    uint64_t* full = bars;               // a stage's rows have landed
    uint64_t* empty = full + nslot;      // every warp is done with the stage
    uint64_t* vfull = empty + nslot;     // a tile's s^V widened
    uint64_t* vempty = vfull + ncb;      // and read by its group
    uint64_t* merged = vempty + ncb;
    int* meta = reinterpret_cast<int*>(merged + 2);
    volatile int* abort_flag = meta + nslot;
    int* slc = meta + ((nslot + 1 + 3) & ~3);
    float* qsums = reinterpret_cast<float*>(slc + kSeqCache);  // [CW][D_K / 32][8]: -1152 x a block's sum of q
    Walker* walkers = reinterpret_cast<Walker*>(qsums + (kSums ? CW * (D_K / kQuantBlock) * 8 : 0));
    WorkQ* work = reinterpret_cast<WorkQ*>(walkers + kMaxWalkers);

    if (threadIdx.x == 0) {
        for (int i = 0; i < nslot; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), (p.own_stages ? p.nwh : NCW) + kConverters);
        }
        for (int i = 0; i < ncb; ++i) {
            mbar_init(smem_u32(vfull + i), 1);
            mbar_init(smem_u32(vempty + i), p.nwh);
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
    if (lane == 0) wk.start(blockIdx.x);
    wk.advance(*work, lane);

    // All roles walk the same tiles in the same order.  Tile u (counted over the CTA) belongs to group
    // u mod ng and is widened into buffer u mod ncb (ncb a multiple of ng), each buffer by one converter.
    // Every converter waits for and releases every stage in turn, also those without a tile of its own,
    // and so does every consumer unless each slot of the ring belongs to one group: nobody can then miss
    // a round of a barrier or take one for another.  Ring positions and phases are counted along (a
    // division by a run-time count costs as much as a chunk's product).
    // A role whose wait has run out (ok false) walks on to its end without waiting, copying or arriving again; every
    // other one then gives up at its next wait.
    int issued = 0;  // stages the producer has filled
    bool ok = true;
    if (warp == NCW) {
        // ---------------------------------------------------------------- producer
        const uint64_t pol = policy_evict_first();
        int slot = 0, segs = 0;
        uint32_t phase = 1;  // parity of the round before this one of a slot's `empty`
        while (wk.valid) {
            const int b = wk.vb, g0 = wk.g0, g1 = wk.g1;
            if (lane == 0 && g0 == 0) {
                // a sequence's first segment records where the combine finds its partials
                const int gr = work->gran(b);
                const int np = work->pieces ? work->npieces(b, work->chunk)
                                            : work->range_of(wk.seg_start + gr - 1) - (wk.slot - b) + 1;
                a.seg_table[b] = make_int2(wk.slot, np);
            }
            // the ring's memory serves the group merge at the end of a segment
            ok = ok && (segs == 0 || p.ng == 1 ||
                        warp_wait(smem_u32(merged), (segs - 1) & 1, abort_flag, a.status, a.wait_ns));
            const int32_t* bt = a.block_table + (size_t)b * a.max_pages;
            const int last_page = (g1 - 1) / TPP;
            int page0 = g0 / TPP, ids = page0 + lane <= last_page ? bt[page0 + lane] : -1;
            for (int f = g0; f < g1;) {
                const int e = min(g1, (f | (ST - 1)) + 1);  // stages are aligned in the sequence
                const int page = f / TPP;
                if (page - page0 >= 32) {
                    page0 = page;
                    ids = page0 + lane <= last_page ? bt[page0 + lane] : -1;
                }
                const int blk = __shfl_sync(0xffffffffu, ids, page - page0);
                if (ok && issued >= nslot)
                    ok = warp_wait(smem_u32(empty + slot), phase, abort_flag, a.status, a.wait_ns);
                ok = ok && !__any_sync(0xffffffffu, *abort_flag != 0);
                if (ok) {
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(full + slot);
                        if (blk < 0 || blk >= a.num_blocks) {
                            set_status(a.status, LRKV_DEV_BAD_BLOCK);
                            meta[slot] = 0;
                            mbar_arrive(bar);
                        } else {
                            meta[slot] = 1;
                            const uint32_t bytes = (uint32_t)(e - f) * TOK * RB;
                            mbar_arrive_expect_tx(bar, bytes);
                            bulk_load_hint(ring + slot * p.stage_bytes,
                                           args.a.rows + ((size_t)blk * kBlockSize + (f % TPP) * TOK) * RB, bytes, bar,
                                           pol);
                        }
                    }
                    ++issued;
                    if (++slot == nslot) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                __syncwarp();
                f = e;
            }
            ++segs;
            wk.advance(*work, lane);
        }
    } else if (warp > NCW) {
        // ---------------------------------------------------------------- converters
        const int cv = warp - NCW - 1;
        constexpr int U = D_H / 8;  // 8-value units of a row's s^V
        int slot = 0, cb = 0;
        bool first = true;          // the buffers' first round: nothing to wait for
        uint32_t phase = 0, cphase = 1;
        while (wk.valid) {
            const int b = wk.vb, g0 = wk.g0, g1 = wk.g1;
            const int L = b < kSeqCache ? slc[b] : a.seq_lens[b];
            for (int f = g0; f < g1;) {
                const int e = min(g1, (f | (ST - 1)) + 1);
                ok = ok && warp_wait(smem_u32(full + slot), phase, abort_flag, a.status, a.wait_ns);
                const int have = meta[slot];
                uint32_t src = ring + slot * p.stage_bytes;
                for (int t = f; t < e; ++t, src += TOK * RB) {
                    if (cb % kConverters == cv) {
                        const uint32_t dst = cbuf + cb * p.cb_bytes;
                        const int nvalid = L - t * TOK;
                        if (ok && !first) ok = warp_wait(smem_u32(vempty + cb), cphase, abort_flag, a.status, a.wait_ns);
                        if (ok && have) {
#pragma unroll 8
                            for (int i0 = 0; i0 < TOK * U; i0 += 32) {
                                const int i = i0 + lane;
                                const int row = i / U, c = i - row * U;
                                const uint32_t ra = src + row * RB;
                                uint32_t x[2], o[4];
                                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                             : "=r"(x[0]), "=r"(x[1])
                                             : "r"(ra + D_K + c * 8));
                                const uint32_t sb = lds8(ra + ql.off_sc + D_K / kQuantBlock + (c >> 2));
                                // zero for tokens behind the end (their probabilities are 0, and 0 x NaN is not)
                                const uint32_t s2 = row < nvalid ? scale_bf16x2(sb) : 0u;
                                const __nv_bfloat162 sc = *reinterpret_cast<const __nv_bfloat162*>(&s2);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    o[j] = bytes_bf16(__byte_perm(x[j >> 1], 0u, j & 1 ? 0x4342 : 0x4140), sc);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + row * SB + c * 16),
                                             "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]));
                            }
                        }
                        __syncwarp();
                        if (lane == 0 && ok) mbar_arrive(smem_u32(vfull + cb));
                    }
                    if (++cb == ncb) {
                        cb = 0;
                        cphase ^= 1;
                        first = false;
                    }
                }
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(smem_u32(empty + slot));
                if (++slot == nslot) {
                    slot = 0;
                    phase ^= 1;
                }
                f = e;
            }
            wk.advance(*work, lane);
        }
    } else {
        // ---------------------------------------------------------------- consumers
        const int grp = warp / p.nwh, wh = warp - grp * p.nwh;
        const int h0 = wh * 8;                  // first head of this warp
        const int g = lane >> 2, tq = lane & 3;
        const int nct = NCW * 32;
        const int g8 = TOK == 16 ? 8 * RB : 0;       // rows 8..15 of a tile of 8 tokens: masked copies of 0..7
        // Offsets of this lane's bytes in a tile of rows: latents of token g for the logits, of token
        // lane mod 16 for the values (transposed loads), scale bytes of heads 2 tq, 2 tq + 1.
        const int zk_off = g * RB + ql.off_zK + h0 * R + tq * 4;
        const int zv_off = (TOK == 16 ? lane & 15 : lane & 7) * RB + ql.off_zV + h0 * R + (lane >> 4) * 16;
        int sc_off[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            sc_off[e] = g * RB + ql.off_sc + ql.nb_sK + ql.nb_sV +
                        min(((h0 + 2 * tq + e) * R) / kQuantBlock, ql.nb_z - 1);
        constexpr int NSE = R == 32 ? 2 : 1;         // scales of the two heads (r <= 16: one block for both)
        const int sk_off = g * RB + tq * 4;          // s^K bytes of token g
        const int cv_off = (TOK == 16 ? (lane & 7) + ((lane >> 4) << 3) : lane & 7) * SB + ((lane >> 3) & 1) * 16;
        float* const qs = qsums + warp * (D_K / kQuantBlock) * 8;
        pdl_wait();  // q~ written by the absorb kernel
        int slot = 0, until = grp;  // until: tiles before this group's next
        int cb = grp;               // and its widened tile
        uint32_t phase = 0, cphase = 0;
        while (wk.valid) {
            const int b = wk.vb, g0 = wk.g0, g1 = wk.g1, pslot = wk.slot;
            const int L = b < kSeqCache ? slc[b] : a.seq_lens[b];
            // Queries and q~ as B fragments (features x heads, head h0 + g in this lane's column), fp16, each
            // divided by a power of two of its own that brings the head's largest magnitude into [1, 2): with one for
            // both the smaller, where it is below 2^-14 of the larger, would lose its bits.
            // This lane holds features 4 tq .. 4 tq + 3 of each chunk of 16 (the order of the A fragments).
            uint32_t qb[NKK][2];
            uint32_t qz[NZC][2];
            float ci[2];  // start of the latent logits' sums
            uint32_t pw = 0;  // exponents of the powers of q and q~, head 2 tq's and head 2 tq + 1's, a byte each
            const int h = h0 + g;
            const bool live = h < H;
            const uint16_t* q = a.q + ((size_t)b * H + (live ? h : 0)) * D_K + tq * 4;
            float mq = 0.f, mv = 0.f;
#pragma unroll
            for (int kk = 0; kk < NKK; ++kk) {
                const uint2 x = *reinterpret_cast<const uint2*>(q + kk * 16);
                qb[kk][0] = live ? x.x : 0u;
                qb[kk][1] = live ? x.y : 0u;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mq = fmaxf(mq, fmaxf(fabsf(bf16lo(qb[kk][i])), fabsf(bf16hi(qb[kk][i]))));
            }
            const float* qt = a.qt + ((size_t)b * H + (live ? h : 0)) * R;
            float v[NZC][4];
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
                for (int i = 0; i < 4; ++i) mv = fmaxf(mv, fabsf(v[c][i]));
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
                mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
            }
            const uint32_t exq = min(max(__float_as_uint(mq) >> 23, 1u), 253u);
            const uint32_t exv = min(max(__float_as_uint(mv) >> 23, 1u), 253u);
            const float invq = __uint_as_float((254u - exq) << 23), invv = __uint_as_float((254u - exv) << 23);
#pragma unroll
            for (int kk = 0; kk < NKK; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qb[kk][i] = pack_f16x2(bf16lo(qb[kk][i]) * invq, bf16hi(qb[kk][i]) * invq);
            // The products take 1152 + u for u: the sums start from -1152 sum q~, and -1152 sum q over each block
            // (as rounded).  (Against a typical sum the offset is some 160 times as large, so fp32 keeps 16 bits of
            // it, more than q and q~ have.  Taken off by products with a constant A, a block is a chain of four
            // products instead of two.)
#pragma unroll
            for (int bl = 0; bl < (kSums ? D_K / kQuantBlock : 0); ++bl) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&qb[2 * bl + (i >> 1)][i & 1]));
                    x += y.x + y.y;
                }
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (tq == 0) qs[bl * 8 + g] = -kByteOffset * x;
            }
            __syncwarp();
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < NZC; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    qz[c][i] = pack_f16x2(v[c][2 * i] * invv, v[c][2 * i + 1] * invv);
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&qz[c][i]));
                    sum += x.x + x.y;
                }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                pw |= __shfl_sync(0xffffffffu, exq | exv << 8, 8 * tq + 4 * e) << (16 * e);
                ci[e] = -kByteOffset * __shfl_sync(0xffffffffu, sum, 8 * tq + 4 * e);
            }
            float o[D_H / 16][4], oz[NZC][4];
            float m[2], mz[2], l[2];
#pragma unroll
            for (int i = 0; i < D_H / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
            for (int i = 0; i < NZC; ++i) oz[i][0] = oz[i][1] = oz[i][2] = oz[i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[e] = mz[e] = -INFINITY;
                l[e] = 0.f;
            }
            for (int f = g0; f < g1;) {
                const int e1 = min(g1, (f | (ST - 1)) + 1);
                if (p.own_stages && until > 0) {  // another group's stage
                    --until;
                    if (++slot == nslot) {
                        slot = 0;
                        phase ^= 1;
                    }
                    ++f;
                    continue;
                }
                ok = ok && warp_wait(smem_u32(full + slot), phase, abort_flag, a.status, a.wait_ns);
                const int have = meta[slot];
                const uint32_t stage = ring + slot * p.stage_bytes;
#pragma unroll 1
                for (; until < e1 - f; until += p.ng) {
                    const uint32_t row0 = stage + until * TOK * RB;
                    const int nvalid = L - (f + until) * TOK;
                    const bool in0 = g < nvalid, in1 = TOK == 16 && g + 8 < nvalid;
                    bool nan0 = false, nan1 = false;  // a block of s^K is a NaN block (tokens g, g + 8)
                    float c[4];
                    uint32_t kb[2][2], vb[2][2];  // scale bytes of z^K and z^V: token g (+ 8), head 2 tq (+ 1)
                    if (ok && have) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int e = 0; e < NSE; ++e) {
                                kb[hf][e] = lds8(row0 + sc_off[e] + hf * g8);
                                vb[hf][e] = lds8(row0 + sc_off[e] + hf * g8 + ql.nb_z);
                            }
                        // --- shared logits [q | q^R] . [s^K | k^R], block by block of 32 features: 16 tokens x 8
                        // heads
                        constexpr int NBK = D_K / kQuantBlock;
                        uint32_t sc0[2], sc1[2];  // scale bytes of the blocks
                        sc0[0] = lds32(row0 + g * RB + ql.off_sc);
                        sc1[0] = lds32(row0 + g * RB + g8 + ql.off_sc);
                        if (NBK > 4) {
                            sc0[1] = lds32(row0 + g * RB + ql.off_sc + 4);
                            sc1[1] = lds32(row0 + g * RB + g8 + ql.off_sc + 4);
                        }
#pragma unroll
                        for (int i = 0; i < (NBK + 3) / 4; ++i) {
                            constexpr uint32_t mask = NBK % 4 == 0 ? 0x80808080u : 0x00008080u;  // (64, 192: two blocks)
                            const uint32_t mk = i == NBK / 4 || NBK < 4 ? mask : 0x80808080u;
                            nan0 |= ((~sc0[i] - 0x01010101u) & sc0[i] & mk) != 0;  // a byte is 255
                            nan1 |= ((~sc1[i] - 0x01010101u) & sc1[i] & mk) != 0;
                        }
#pragma unroll
                        for (int bl = 0; bl < NBK; ++bl) {
                            float2 off = make_float2(0.f, 0.f);
                            if (kSums) off = *reinterpret_cast<const float2*>(qs + bl * 8 + 2 * tq);
                            float d[4] = {off.x, off.y, off.x, off.y};
#pragma unroll
                            for (int kk = 2 * bl; kk < 2 * bl + 2; ++kk) {
                                const uint32_t x0 = lds32(row0 + sk_off + kk * 16);
                                const uint32_t x1 = lds32(row0 + sk_off + g8 + kk * 16);
                                const uint32_t a0 = bytes_f16(x0, 0x4140), a1 = bytes_f16(x1, 0x4140),
                                               a2 = bytes_f16(x0, 0x4342), a3 = bytes_f16(x1, 0x4342);
                                if (!kSums)
                                    mma_16816_f16(d, kMinusOffset2, kMinusOffset2, kMinusOffset2, kMinusOffset2,
                                                  qb[kk][0], qb[kk][1]);
                                mma_16816_f16(d, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
                            }
                            const float f0 = byte_scale(sc0[bl >> 2], bl & 3), f1 = byte_scale(sc1[bl >> 2], bl & 3);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    c[i] = bl == 0 ? d[i] * (i < 2 ? f0 : f1) : fmaf(d[i], i < 2 ? f0 : f1, c[i]);
                        }
                    }
                    const uint32_t cvv = cbuf + cb * p.cb_bytes + cv_off;
                    if (ok && have) {
                        // --- latent logits q~ . z^K, chunk by chunk of 16 bytes: of a product with all eight
                        // heads' q~ only the columns of the chunk's own head (r = 8: two heads) are kept.
                        // (Heads past the last read whatever follows in shared memory: finite, never stored.)
                        float cz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll kUnroll
                        for (int j = 0; j < NCH / NZC; ++j) {
                            float d[4] = {ci[0], ci[1], ci[0], ci[1]};
#pragma unroll
                            for (int zc = 0; zc < NZC; ++zc) {
                                const uint32_t at = row0 + zk_off + (j * NZC + zc) * 16;
                                const uint32_t x0 = lds32(at), x1 = lds32(at + g8);
                                mma_16816_f16(d, bytes_f16(x0, 0x4140), bytes_f16(x1, 0x4140), bytes_f16(x0, 0x4342),
                                              bytes_f16(x1, 0x4342), qz[zc][0], qz[zc][1]);
                            }
                            const bool mine = tq == (R == 8 ? j : j >> 1);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (R == 8 || (i & 1) == (j & 1)) cz[i] = mine ? d[i] : cz[i];
                        }
                        // --- logits s (log2 units) and s + k, 2^k the scale of z^V; element i: token g (+ 8 for
                        // i >= 2), head 2 tq + (i & 1)
                        float sv[4], sw[4], ks[2][2], kv[2][2];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int e = 0; e < NSE; ++e) {
                                ks[hf][e] = scale_of((hf ? nan1 : nan0) ? 255u : kb[hf][e]);
                                // log2 of the scale: -infinity of a cleared row, +infinity of a NaN block, whose
                                // weight then becomes infinity - infinity
                                kv[hf][e] = lg2_approx(__uint_as_float(vb[hf][e] << 23));
                            }
                        // The powers times the softmax scale, formed tile by tile: 16 consumers have no registers for
                        // four floats, and the compiler must not form them before the loop (128 heads 91 us at that
                        // time, 98 where it may, 102 with floats).
                        if (!kSums) asm volatile("" : "+r"(pw));
                        float fq[2], fz[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            fq[e] = byte_scale(pw, 2 * e) * a.scale_log2;
                            fz[e] = byte_scale(pw, 2 * e + 1) * a.scale_log2;
                        }
                        float over = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i & 1, es = e & (NSE - 1), hf = i >> 1;
                            const float s = fmaf(cz[i], ks[hf][es] * fz[e], c[i] * fq[e]);
                            const bool in = hf ? in1 : in0;
                            sv[i] = in ? s : -INFINITY;
                            sw[i] = in ? s + kv[hf][es] : -INFINITY;
                            over = fmaxf(over, fmaxf(sv[i] - m[e], sw[i] - mz[e]));
                        }
                        // Maxima are the same in the eight lanes that share two heads, and raised together,
                        // by all heads of the tile, once some logit lies more than 2^8 above.  (At the start
                        // they are -infinity; -infinity - -infinity is a NaN, which fmaxf passes over.)
                        if (__any_sync(0xffffffffu, over > kLazy)) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = fmaxf(sv[e], sv[2 + e]), y = fmaxf(sw[e], sw[2 + e]);
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1) {
                                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                                }
                                x = fmaxf(x, m[e]);
                                y = fmaxf(y, mz[e]);
                                const float al = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - x);
                                const float az = mz[e] == -INFINITY ? 0.f : ex2_approx(mz[e] - y);
                                m[e] = x;
                                mz[e] = y;
                                l[e] *= al;
#pragma unroll
                                for (int i = 0; i < D_H / 16; ++i) {
                                    o[i][e] *= al;
                                    o[i][2 + e] *= al;
                                }
#pragma unroll
                                for (int i = 0; i < NZC; ++i) {
                                    oz[i][e] *= az;
                                    oz[i][2 + e] *= az;
                                }
                            }
                        }
                        // --- p = 2^(s - m) and w = 2^(s + k - mz), transposed into B fragments
                        float pp[4], ww[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i & 1;
                            const bool in = i < 2 ? in0 : in1;
                            pp[i] = in ? ex2_approx(sv[i] - m[e]) : 0.f;
                            // (mz is -infinity as long as every row of the block was a cleared one)
                            ww[i] = sw[i] == -INFINITY ? 0.f : ex2_approx(sw[i] - mz[e]);
                        }
                        l[0] += pp[0] + pp[2];
                        l[1] += pp[1] + pp[3];
                        const uint32_t pb0 = movmatrix_trans(pack_bf16x2(pp[0], pp[1]));
                        const uint32_t pb1 = movmatrix_trans(pack_bf16x2(pp[2], pp[3]));
                        const uint32_t wb0 = movmatrix_trans(pack_f16x2(ww[0], ww[1]));
                        const uint32_t wb1 = movmatrix_trans(pack_f16x2(ww[2], ww[3]));
                        // --- shared values: O^T (d x heads) += s^V^T . P
                        ok = warp_wait(smem_u32(vfull + cb), cphase, abort_flag, a.status, a.wait_ns);
#pragma unroll
                        for (int i = 0; i < D_H / 16; ++i) {
                            uint32_t af[4];
                            ldmatrix_x4_trans(cvv + i * 32, af[0], af[1], af[2], af[3]);
                            mma_16816(o[i], af, pb0, pb1);
                        }
                        // --- latent values, two 16-byte chunks at a time: rows of the transposed 16-bit
                        // elements are pairs of features, row g of A takes the even one, row g + 8 the odd
                        // one.  The offset 1152 of the bytes' products is taken off tile by tile (so that the
                        // sums never grow with it).
                        // (One accumulator would be a chain of all chunks' products; every other goes to a second one.)
                        float tz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int zc = 0; zc < NZC; ++zc)
                            mma_16816_f16(NZC == 1 && kSums ? tz : oz[zc], kMinusOffset2, kMinusOffset2, kMinusOffset2,
                                          kMinusOffset2, wb0, wb1);
#pragma unroll kUnroll
                        for (int c2 = 0; c2 < NCH; c2 += 2) {
                            uint32_t x[4];
                            ldmatrix_x4_trans(row0 + zv_off + c2 * 16, x[0], x[1], x[2], x[3]);
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                const int ch = c2 + w;
                                const bool mine = R == 8 ? (g >> 1) == ch : g == (R == 32 ? ch >> 1 : ch);
                                const int zc = R == 32 ? ch & 1 : 0;
                                mma_16816_f16(NZC == 1 && kSums && w ? tz : oz[zc], bytes_f16(x[2 * w], 0x4240),
                                              bytes_f16(x[2 * w], 0x4341), bytes_f16(x[2 * w + 1], 0x4240),
                                              bytes_f16(x[2 * w + 1], 0x4341),
                                              mine ? wb0 : 0u, mine ? wb1 : 0u);
                            }
                        }
                        if (NZC == 1 && kSums) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) oz[0][i] += tz[i];
                        }
                    }
                    if (ok && !have) ok = warp_wait(smem_u32(vfull + cb), cphase, abort_flag, a.status, a.wait_ns);
                    __syncwarp();
                    if (lane == 0 && ok) mbar_arrive(smem_u32(vempty + cb));
                    cb += p.ng;
                    if (cb >= ncb) {
                        cb = grp;
                        cphase ^= 1;
                    }
                }
                until -= e1 - f;
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(smem_u32(empty + slot));
                if (++slot == nslot) {
                    slot = 0;
                    phase ^= 1;
                }
                f = e1;
            }
            // --- this group's state over the segment
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
                    // the latents' sums brought to the probabilities' maximum
                    const float fac = mz[e] == -INFINITY ? 0.f : ex2_approx(mz[e] - m[e]);
#pragma unroll
                    for (int i = 0; i < NZC; ++i) {
                        oz[i][e] *= fac;
                        oz[i][2 + e] *= fac;
                    }
                    // a NaN sum is handed on as NaN values with a weight, not as an empty part
                    if (l[e] != l[e]) {
                        l[e] = 1.f;
                        if (!(fabsf(m[e]) < INFINITY)) m[e] = 0.f;
#pragma unroll
                        for (int i = 0; i < D_H / 16; ++i)
                            o[i][e] = o[i][2 + e] = __uint_as_float(0x7fc00000u);
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
                for (int e = 0; e < 2; ++e) {
                    const int h = h0 + 2 * tq + e;
                    if (h >= H) continue;
                    if (g == 0) {
                        gml[h * hs_ml] = m[e];
                        gml[h * hs_ml + 1] = l[e];
                    }
                    float* dst = gacc + h * hs_acc;
#pragma unroll
                    for (int i = 0; i < D_H / 16; ++i) {
                        dst[i * 16 + g] = o[i][e];
                        dst[i * 16 + 8 + g] = o[i][2 + e];
                    }
                    if (R == 8) {
                        if ((g >> 2) == e)
                            *reinterpret_cast<float2*>(dst + D_H + (g & 3) * 2) = make_float2(oz[0][e], oz[0][2 + e]);
                    } else {
#pragma unroll
                        for (int i = 0; i < NZC; ++i)
                            *reinterpret_cast<float2*>(dst + D_H + i * 16 + g * 2) =
                                make_float2(oz[i][e], oz[i][2 + e]);
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
            wk.advance(*work, lane);
        }
    }
    pdl_trigger();  // the combine waits for this grid's end
    // Whichever wait ran out, and however late: the copies in flight land (the full limit again) before the block
    // gives up its shared memory.
    __syncthreads();
    if (warp == NCW && *abort_flag)
        for (int i = max(0, issued - nslot); i < issued; ++i)
            mbar_wait(smem_u32(full + i % nslot), (i / nslot) & 1, a.status);
}

// Tokens of a tile.
int tile_tokens(int H, int R) { return R == 32 && H > 96 ? 8 : 16; }

template <int D_H, int R, int D_R>
bool make_plan(QuantPlan* p, const QuantLayout& q, int H, int smem_limit) {
    p->cw = H > 64 ? 16 : 8;
    // a row of more than 96 heads of r = 32 is so long that two stages of 16 tokens do not fit
    const int tok = tile_tokens(H, R);
    p->nwh = (H + 7) / 8;
    const int ng_most = p->cw / p->nwh;
    p->cb_bytes = tok * cb_stride(D_H);
    const int WS = merge_stride(D_H + R);
    const int tile = tok * q.row_bytes;
    // tiles per stage: a copy instruction costs its thread some 60 to 80 ns, so short rows are brought a page
    // (or half) at a time, as long as six stages fit in the ring
    p->st = 1;
    while (p->st * tok < kBlockSize && p->st * tile * 2 <= 28 << 10) p->st *= 2;
    p->stage_bytes = p->st * tile;
    auto fixed = [&](int nslot, int ncb) {
        return (2 * nslot + 2 * ncb + 2) * 8 + ((nslot + 1 + 3) & ~3) * 4 + kSeqCache * 4 +
               (p->cw == 8 ? p->cw * (D_H + D_R) : 0) + kMaxWalkers * (int)sizeof(Walker) + 96 + 128;
    };
    for (int want = 3; want >= 2; --want)          // stages at least
        for (int ng = ng_most; ng >= 1; --ng)
            for (int mul = 3; mul >= 1; --mul) {   // widened tiles per group
                const int ncb = ng * mul;
                int nslot = 16;
                while (nslot > 1 && nslot * p->stage_bytes + ncb * p->cb_bytes + fixed(nslot, ncb) > smem_limit) --nslot;
                if (nslot < want) continue;
                p->own_stages = p->st == 1 && nslot / ng * ng >= want;
                if (p->own_stages) nslot = nslot / ng * ng;
                if (ng > 1 && ((size_t)ng * H * (WS + 3) + 3) * 4 > (size_t)nslot * p->stage_bytes) continue;
                p->ng = ng;
                p->ncb = ncb;
                p->nslot = nslot;
                p->threads = (p->nwh * ng + 1 + converters(p->cw)) * 32;
                p->smem_bytes = nslot * p->stage_bytes + ncb * p->cb_bytes + fixed(nslot, ncb);
                return true;
            }
    return false;
}

template <int D_H, int R, int D_R>
cudaError_t launch_t(QuantScanArgs& x, int sms, int smem_limit, cudaStream_t stream) {
    if (!make_plan<D_H, R, D_R>(&x.p, x.a.q, x.a.d.H, smem_limit)) return cudaErrorInvalidConfiguration;
    const int tok = tile_tokens(x.a.d.H, R);
    auto kern = x.p.cw == 8 ? quant_scan_kernel<D_H, R, D_R, 8, 16> : quant_scan_kernel<D_H, R, D_R, 16, 16>;
    if constexpr (R == 32) {
        if (tok == 8) kern = quant_scan_kernel<D_H, R, D_R, 16, 8>;
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
