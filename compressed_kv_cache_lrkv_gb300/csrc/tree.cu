// tree.cu -- attention of the drafted tokens of a batch over the cache: token i of sequence b sees the sequence's
// tokens and the drafted ones of its mask.
//     s_t = ([q | q^R] . [s^K_t | k^R_t] + (q B_h^K) . z^K_{h,t}) scale,  p = softmax over what is seen,
//     out = sum p_t s^V_t + B_h^V sum p_t z^V_{h,t}
//
// The cached rows are the same for all heads and drafted tokens, so 128 query rows, hb heads x ns tokens of one
// sequence, are one attention tile of width d_h + zw, zw = hb r (as in prefix.cu, there over sequences):
//     S = [Q | diag(Q~)] . [s^K | z^K of the hb heads]^T,   O += P . [s^V | z^V of the hb heads]
// on tcgen05, M = 128, 64 tokens (a page) at a time.  zw is 32, 64 or 128 (tree_plan); 32 for up to 64 drafted tokens of
// r = 16, so that each latent is read by one tile.
//
// Three dependent launches: q~ (decode.cu's absorb, every drafted token a query), the scan, the merge.  The scan is
// persistent, one CTA an SM, with the tiles' pages divided evenly (Work).  Warps: 0 keys and 6 values (TMA), 1 issues
// all MMAs, 2 .. 5 and 8 .. 11 are two groups of 128 query rows that take the pages in turn.
//
// Measured (a call in a stream of others): 8 heads of 64, r = 16, 1 x 4 drafted behind 256 tokens 14 us; 16 x 16 behind
// 2,048 20 us; 32 heads of 128, r = 16, positional key, 24 x up to 26 behind 1 to 8,191 92 us; 32 heads, r = 32, 4 x 8
// behind 16 to 32 K 100 us (475 MB read, 70 us at the copy rate); 128 heads, r = 16, 8 x up to 64 behind 8,192 332 us, 316
// in bursts of a few ms (long context 95.6): a load of seconds runs at the power limit, with the SMs at 1.91 to 1.96 GHz.
// No single part bounds the scan.  In bursts, 128 heads and long context: as it is 317 and 95.7; without the softmax 309
// and 94.6; with a fraction of the score products and no maximum 284 and 90.6, of the value products 298 and 87.6, of
// both 282 and 85.8.  More warps of rows (two threads a row, or a third group) were slower.
#include "lrkv_internal.cuh"
#include "tile_attn.cuh"
#include "tree.h"

namespace lrkv {

namespace {

constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// What a piece's start and end cost, in pages: the work is cut as if every tile had that many more.  (In a graph, us, with
// 4 | 8 | 11 | 16: 24 sequences of 1 to 8,191 tokens 96.5 | 92.5 | 92.4 | 94.7, 16 x 16 tokens behind 2,048 19.7 | 19.4 |
// 18.8 | 19.4; 128 heads, the long context and short sequences within 2%.)
constexpr int kStartPages = 11;

__device__ __forceinline__ void named_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// [Q | diag(Q~)] is the A operand of S, diag(Q~) as two bf16 pieces (q~ rounded, and what that left). As many of
// its 64-column blocks as fit sit in TMEM, the rest in shared memory, beside rings of key stages
// [64 tokens][D_K + ZW] and value stages [64][D_H + ZW].
// TMEM columns: NSB S buffers of 64 columns (P, two bf16 a column, is written over the first half of its own S), O, Q.
// Three S buffers where Q fits beside them, so that a group of rows finds its next page computed when it is done with one.
template <int D_H, int D_R, int ZW>
struct TrLayout {
    static constexpr int D_K = D_H + D_R;
    static constexpr int ZBLK = ZW == 32 ? 1 : ZW / 64;                 // blocks of latents in a stage
    static constexpr uint32_t ZBLK_BYTES = ZW == 32 ? 4096 : 8192;
    static constexpr uint32_t K_BYTES = D_K / 64 * 8192 + ZBLK * ZBLK_BYTES, V_BYTES = D_H / 64 * 8192 + ZBLK * ZBLK_BYTES;
    static constexpr int NBQ = (D_K + 2 * ZW) / 64;
    static constexpr int NSB = (512 - 192 - D_H - ZW) / 32 >= NBQ ? 3 : 2, QROOM = (512 - 64 * NSB - D_H - ZW) / 32;
    static constexpr int QBT = NBQ < QROOM ? NBQ : QROOM, QBS = NBQ - QBT;  // blocks in TMEM, in shared memory
    static constexpr uint32_t Q_BYTES = QBS * 16384;
    static constexpr uint32_t ROOM = 232448 - 1024 - 5120 - Q_BYTES;
    static constexpr int BOTH = ROOM / (K_BYTES + V_BYTES);
    static constexpr int VST = BOTH > 6 ? 6 : BOTH;
    static constexpr int KST = VST < 6 && ROOM - VST * (K_BYTES + V_BYTES) >= K_BYTES ? VST + 1 : VST;
    static constexpr uint32_t OFF_K = Q_BYTES, OFF_V = OFF_K + KST * K_BYTES, OFF_BAR = OFF_V + VST * V_BYTES;
    static constexpr uint32_t OFF_ROW = OFF_BAR + 512;  // 128 references, then [piece's parity][group][128] (sum, reference)
    static constexpr uint32_t SMEM = OFF_ROW + 512 + 4096 + 1024;
    static_assert(VST >= 2 && KST >= NSB && SMEM <= 232448, "stages");
    static constexpr uint32_t TM_S = 0, TM_O = 64 * NSB, TM_Q = TM_O + D_H + ZW;
    static_assert(TM_Q + QBT * 32 <= 512, "TMEM");
};

// Lengths of sequence b: tokens before the drafted ones, drafted tokens, pages (0: nothing to do, or a bad length).
struct Seq {
    int L, n, pages;
    bool bad;
};
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b) {
    Seq s;
    s.L = a.d.seq_lens[b];
    s.n = a.tree_lens ? a.tree_lens[b] : a.T;
    s.bad = s.L < 0 || s.n < 0 || s.n > a.T || (long long)s.L + s.n > (long long)a.d.max_pages * kBlockSize;
    if (s.bad) s.L = s.n = 0;
    s.pages = s.n > 0 ? (s.L + s.n + kBlockSize - 1) / kBlockSize : 0;
    return s;
}
// Tiles of a sequence with n drafted tokens (tile t: token group t % st, head group t / st, st = ceil(n / ns)), taken
// `gang` at a time, and the sequence's units of work.
__device__ __forceinline__ int tiles_of(const TreeArgs& a, int n) { return (n + a.ns - 1) / a.ns * a.htiles; }
__device__ __forceinline__ int groups_of(const TreeArgs& a, int n) { return (tiles_of(a, n) + a.gang - 1) / a.gang; }
__device__ __forceinline__ long long units_of(const TreeArgs& a, const Seq& s) {
    return s.pages ? (long long)groups_of(a, s.n) * (s.pages + kStartPages) : 0;
}

// The work: groups of `gang` tiles, the groups of all sequences one after the other, a group's pages and then
// kStartPages empty units, cut into equal ranges, one for each gang of CTAs, of which each takes a tile of the group.
// So the CTAs that read one page's shared rows and the neighbouring latents of its tokens do it at about the same time:
// with a range of its own for each CTA, a call over 600 MB of cache read 1,520 MB.  A piece is what a range holds of a
// group's pages; piece (range, group) of member i leaves its partials at slot (range + group number) gang + i, which
// is different for all pieces, and `gang` apart for a tile's.
struct Work {
    long long total;
    int ranges;  // (no range is empty, so a tile's pieces are in consecutive ones)
    __device__ __forceinline__ Work(long long units, int gangs)
        : total(units), ranges(units < gangs ? (units > 0 ? (int)units : 1) : gangs) {}
    __device__ __forceinline__ long long start(int c) const { return c < ranges ? total * c / ranges : total; }
    __device__ __forceinline__ int range_of(long long u) const { return (int)(((u + 1) * ranges - 1) / total); }
};

// Walks a member's pieces of one range.
struct Walk {
    long long hi, u, seg;  // end of the range, the next unit to look at, first unit of group t
    int b, t, member;      // sequence, group of its tiles, which of them
    Seq s;
    // the piece: pages [p0, p0 + nt) of the sequence
    int p0, nt;

    __device__ __forceinline__ void begin(const TreeArgs& a, long long lo, long long hi_, int b0, long long base, int i) {
        hi = hi_;
        u = lo;
        b = b0;
        member = i;
        s = b < a.batch ? seq_of(a, b) : Seq{0, 0, 0, false};
        t = s.pages ? (int)((lo - base) / (s.pages + kStartPages)) : 0;
        seg = base + (long long)t * (s.pages + kStartPages);
    }
    __device__ __forceinline__ int tile(const TreeArgs& a) const { return t * a.gang + member; }
    __device__ __forceinline__ bool next(const TreeArgs& a) {
        while (u < hi && b < a.batch) {
            if (s.pages == 0 || t >= groups_of(a, s.n)) {
                if (++b < a.batch) s = seq_of(a, b);
                t = 0;
                continue;
            }
            const long long end = seg + s.pages + kStartPages;
            const int to = (int)((hi < end ? hi : end) - seg);
            p0 = (int)(u - seg);
            nt = (to < s.pages ? to : s.pages) - p0;
            if (nt > 0 && tile(a) < tiles_of(a, s.n)) return true;
            step();
        }
        return false;
    }
    __device__ __forceinline__ void step() {  // behind the group of the present piece
        seg += s.pages + kStartPages;
        u = seg;
        ++t;
    }
};

// The row's largest logit (log2 units), NaN where one is: of 64 in TMEM, of which those that are not seen become
// -infinity there.
__device__ __forceinline__ float look(uint32_t tS, bool all, unsigned long long seen, float scale_log2) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 64; c += 32, seen >>= 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tS + c, v);
        if (!all) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (uint32_t)seen >> e & 1 ? v[e] : 0xff800000u;
            tmem_st_32x32b_x32(tS + c, v);
            tmem_wait_st();
        }
        float m4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            m4[e] = max3_nan(__uint_as_float(v[e]), __uint_as_float(v[4 + e]), __uint_as_float(v[8 + e]));
#pragma unroll
        for (int e = 12; e < 28; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = max3_nan(m4[k], __uint_as_float(v[e + k]), __uint_as_float(v[e + 4 + k]));
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = max_nan(m4[k], __uint_as_float(v[28 + k]));
        mx = max3_nan(mx, max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
    }
    return mx * scale_log2;
}

// Those that are NaN, formed again from q, q~ and the pools; `slot`: of the first.
__device__ __noinline__ void form_again(uint32_t tS, bool live, size_t slot, const uint16_t* q, const float* qt,
                                        const uint16_t* sK, const uint16_t* zK, int D_K, int R, int H, int h) {
#pragma unroll 1
    for (int c = 0; c < 64; c += 8) {
        uint32_t v[8];
        tmem_ld_32x32b_x8(tS + c, v);
        uint32_t nans = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) nans |= (__uint_as_float(v[e]) != __uint_as_float(v[e]) ? 1u : 0u) << e;
        for (uint32_t todo = live ? nans : 0u; todo != 0; todo &= todo - 1) {
            const int e = __ffs(todo) - 1;
            const size_t t = slot + c + e;
            const uint32_t x = __float_as_uint(dot8(q, sK + t * D_K, D_K) + dot8(qt, zK + (t * H + h) * R, R));
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k == e ? x : v[k];
        }
        __syncwarp();
        tmem_st_32x32b_x8(tS + c, v);
    }
    tmem_wait_st();
}

// Half `part` of row vr of a value stage: cleared wholly, or its NaNs and infinities; whether there were any.
template <int D_H, int ZW>
__device__ __noinline__ bool clean_values(uint8_t* stage, int vr, int part, bool wholly) {
    constexpr int PB = ZW == 32 ? 64 : 128, PC = PB / 16;  // bytes of a row in a block, 16-byte pieces
    bool found = false;
#pragma unroll 1
    for (int bk = 0; bk < (D_H + ZW) * 2 / PB; ++bk) {
        // (rows are PB bytes apart: each begins with another of its pieces, and so in another bank)
        uint4* const r = reinterpret_cast<uint4*>(stage + bk * (PB * 64) + vr * PB);
        uint4 y[PC / 2];
#pragma unroll
        for (int i = 0; i < PC / 2; ++i) {
            uint4* const p = r + ((part * (PC / 2) + i + vr) & (PC - 1));
            if (wholly)
                *p = make_uint4(0, 0, 0, 0);
            else
                y[i] = *p;
        }
        if (wholly) continue;
#pragma unroll
        for (int i = 0; i < PC / 2; ++i) {
            uint32_t x[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool lo = (x[e] & 0x7f80u) == 0x7f80u, hi = (x[e] & 0x7f800000u) == 0x7f800000u;
                hit |= lo | hi;
                x[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
            }
            if (hit) r[(part * (PC / 2) + i + vr) & (PC - 1)] = make_uint4(x[0], x[1], x[2], x[3]);
            found |= hit;
        }
    }
    return found;
}

// A row's sums, as this thread has stored them (every second 32 columns of s^V and of the tile's latents), quads `rs`
// apart: what is not finite in the values of the drafted tokens `spoilt` is added.
__device__ __noinline__ void add_spoilt(float4* dst, int rs, unsigned long long spoilt, int part, int hl,
                                        const int32_t* pages, int L, const uint16_t* sV, const uint16_t* zV, int D_H,
                                        int R, int H, int h) {
    for (; spoilt != 0; spoilt &= spoilt - 1) {
        const int t = L + __ffsll(spoilt) - 1;
        const size_t at = (size_t)pages[t / kBlockSize] * kBlockSize + t % kBlockSize;
#pragma unroll 1
        for (int c = 0; c < D_H + R; c += 4) {
            if (((c < D_H ? c : hl * R + c - D_H) / 32 & 1) != part) continue;
            const uint2 y = *reinterpret_cast<const uint2*>(c < D_H ? sV + at * D_H + c : zV + (at * H + h) * R + c - D_H);
            float4 x = dst[(size_t)(c / 4) * rs];
            auto add = [](float& z, float e) { z += fabsf(e) < INFINITY ? 0.f : e; };
            add(x.x, bf16lo(y.x));
            add(x.y, bf16hi(y.x));
            add(x.z, bf16lo(y.y));
            add(x.w, bf16hi(y.y));
            dst[(size_t)(c / 4) * rs] = x;
        }
    }
}

template <int D_H, int D_R, int ZW>
__global__ void __launch_bounds__(kThreads, 1)
    tree_scan_kernel(const __grid_constant__ TreeMaps m, const __grid_constant__ TreeArgs a, const int R) {
    using Lay = TrLayout<D_H, D_R, ZW>;
    constexpr int D_K = Lay::D_K, NBQ = Lay::NBQ, NSB = Lay::NSB, KST = Lay::KST, VST = Lay::VST;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
    const uint32_t S0 = smem_u32(smem);
    const DecodeArgs& d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = d.H, W = D_H + R;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
    uint64_t* q_ready = bars + 0;   // Q of a piece written, O of the piece before it read
    uint64_t* p_full = bars + 1;    // [3] P_g written (g: pages of this CTA, counted through; buffer g % NSB)
    uint64_t* mma_drain = bars + 4;
    uint64_t* k_full = bars + 5;    // [6] keys of page g there (stage g % KST)
    uint64_t* s_done = bars + 11;   // S_g computed: the rows may read it, the stage is free
    uint64_t* v_full = bars + 17;   // values of page g there (stage g % VST)
    uint64_t* o_done = bars + 23;   // P_g V_g added to O, the stage is free
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 29);
    volatile int* abort_flag = reinterpret_cast<int*>(bars + 30);
    unsigned long long* poison = reinterpret_cast<unsigned long long*>(bars + 31);  // [2], by the piece's parity
    long long* plan = reinterpret_cast<long long*>(bars + 33);                      // total, first sequence, its base
    auto B = [&](uint64_t* p) { return smem_u32(p); };
    // (one arrival a warp: those of 32 lanes on one barrier take their turns)
    auto arrive = [&](uint64_t* p) {
        __syncwarp();
        if (lane == 0) mbar_arrive(B(p));
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };

    if (threadIdx.x == 32) {
        mbar_init(B(q_ready), 8);
        for (int i = 0; i < 3; ++i) mbar_init(B(p_full + i), 4);
        poison[0] = poison[1] = 0;
        mbar_init(B(mma_drain), 1);
        for (int i = 0; i < 6; ++i) {
            mbar_init(B(k_full + i), 1);
            mbar_init(B(s_done + i), 1);
            mbar_init(B(v_full + i), 1);
            mbar_init(B(o_done + i), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        // the units of all sequences, and the sequence that holds this range's first
        long long total = 0;
#pragma unroll 4
        for (int b = lane; b < a.batch; b += 32) total += units_of(a, seq_of(a, b));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const Work w(total, a.gangs);
        const long long lo = w.start(blockIdx.x / a.gang);
        long long base = 0;
        int first = a.batch;
        for (int b0 = 0; b0 < a.batch && first == a.batch; b0 += 32) {
            const long long v = b0 + lane < a.batch ? units_of(a, seq_of(a, b0 + lane)) : 0;
            long long incl = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const unsigned holds = __ballot_sync(0xffffffffu, base + incl > lo);
            if (holds) {
                const int l = __ffs(holds) - 1;
                first = b0 + l;
                base += __shfl_sync(0xffffffffu, incl - v, l);
            } else {
                base += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        if (lane == 0) {
            plan[0] = total;
            plan[1] = first;
            plan[2] = base;
        }
    }
    __syncwarp();
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Work work(plan[0], a.gangs);
    const int gang = blockIdx.x / a.gang, member = blockIdx.x - gang * a.gang;
    Walk w;
    w.begin(a, work.start(gang), work.start(gang + 1), (int)plan[1], plan[2], member);

    const bool keys = warp == 0;  // (of the two producers)
    int issued = 0;               // stages a producer has filled
    if (warp == 0 || warp == 6) {
        // ---------------------------------------------------------------- TMA producers
        const int oob_row = d.num_blocks * kBlockSize;  // whole box out of bounds: zeros
        const int depth = keys ? KST : VST;
        const uint32_t stage_bytes = keys ? Lay::K_BYTES : Lay::V_BYTES;
        // with zw = 32 the values come in blocks of 32 columns, 64-byte swizzle, s^V as z^V: one MMA takes them all
        const int cols = !keys && ZW == 32 ? 32 : 64, nblk = (keys ? D_K : D_H) / cols;
        uint64_t* full = keys ? k_full : v_full;
        uint64_t* empty = keys ? s_done : o_done;
        const CUtensorMap* ms = keys ? &m.sK : &m.sV;
        const CUtensorMap* mz = keys ? &m.zK : &m.zV;
        const uint32_t ring = S0 + (keys ? Lay::OFF_K : Lay::OFF_V);
        if (lane == 0) {
            prefetch_tmap(ms);
            prefetch_tmap(mz);
        }
        int st = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (; ok && w.next(a); w.step()) {
            const int32_t* pages = d.block_table + (size_t)w.b * d.max_pages + w.p0;
            const int x0 = w.tile(a) / ((w.s.n + a.ns - 1) / a.ns) * ZW;
            auto fetch = [&](int i) {
                int r = oob_row;
                if (i < w.nt) {
                    const int blk = pages[i];
                    if (blk >= 0 && blk < d.num_blocks)
                        r = blk * kBlockSize;
                    else
                        set_status(d.status, LRKV_DEV_BAD_BLOCK);
                }
                return r;
            };
            int cur = fetch(lane), nxt = fetch(32 + lane);
            for (int j = 0; j < w.nt; ++j) {
                if (j > 0 && (j & 31) == 0) {
                    cur = nxt;
                    nxt = fetch(j + 32 + lane);
                }
                const int prow = __shfl_sync(0xffffffffu, cur, j & 31);
                if ((issued >= depth && !wait_role(B(empty + st), phase, d)) || aborted()) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint32_t dst = ring + st * stage_bytes;
                    const uint32_t bar = B(full + st);
                    mbar_arrive_expect_tx(bar, stage_bytes);
                    for (int bk = 0; bk < nblk; ++bk, dst += cols * 128) tma_load_2d(dst, ms, cols * bk, prow, bar);
                    for (int bk = 0; bk < Lay::ZBLK; ++bk, dst += Lay::ZBLK_BYTES)
                        tma_load_2d(dst, mz, x0 + 64 * bk, prow, bar);
                }
                __syncwarp();
                ++issued;
                if (++st == depth) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) *abort_flag = 1;
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMAs
        // One thread issues all of them, so they run in this order: S_0 .. S_{NSB-1} | P_0 V_0, S_NSB | P_1 V_1, ..: S_{g+NSB}
        // overwrites the buffer that P_g V_g has read; while the rows work on S_g, the products of its neighbours run.
        // (128 heads x 64 tokens: 481 us with a vote of the warp at every wait and MMA and two S buffers, 357 from one
        // thread and with three.)
        constexpr uint32_t id_S = idesc_bf16_f32(128, 64);
        constexpr uint32_t id_PV = idesc_bf16_f32(128, D_H + ZW) | (1u << 16);  // B is MN-major
        if (elect_one_sync()) {
            constexpr uint32_t U128 = desc_upper(1024, 2), U64 = desc_upper(512, 4);
            const uint32_t dQ = desc_lower(S0, 16), dK = desc_lower(S0 + Lay::OFF_K, 16);
            const uint32_t dV = desc_lower(S0 + Lay::OFF_V, ZW == 32 ? 4096 : 8192);
            int kst = 0, vst = 0, sb = 0, pb = 0;  // stages and S buffers in turn
            uint32_t kphase = 0, vphase = 0, qphase = 0, pphase = 0;
            auto s_tile = [&]() -> bool {
                if (!wait_one(B(k_full + kst), kphase, d, abort_flag)) return false;
                tc_fence_after();
                const uint32_t bs = dK + kst * (Lay::K_BYTES >> 4), ts = Lay::TM_S + sb * 64;
#pragma unroll
                for (int kk = 0; kk < NBQ * 4; ++kk) {
                    // 16 columns of Q; q's against s^K, both pieces of q~ against the same z^K
                    const int col = kk * 16, z = (col - D_K) % ZW;
                    const uint32_t at = col < D_K ? col / 64 * 8192 + col % 64 * 2
                                        : ZW == 32 ? D_K / 64 * 8192 + z * 2
                                                   : (D_K + z) / 64 * 8192 + z % 64 * 2;
                    if (kk >= Lay::QBT * 4)
                        mma_ss_h<U128, U128>(ts, dQ + ((((kk >> 2) - Lay::QBT) * 16384 + (kk & 3) * 32) >> 4),
                                             bs + (at >> 4), id_S, 1);
                    else if (ZW == 32 && col >= D_K)
                        mma_ts_h<U64>(ts, Lay::TM_Q + kk * 8, bs + (at >> 4), id_S, kk > 0);
                    else
                        mma_ts_h<U128>(ts, Lay::TM_Q + kk * 8, bs + (at >> 4), id_S, kk > 0);
                }
                tc_commit(B(s_done + kst));
                if (++sb == NSB) sb = 0;
                if (++kst == KST) {
                    kst = 0;
                    kphase ^= 1;
                }
                return true;
            };
            auto pv_tile = [&](bool first) -> bool {
                if (!wait_one(B(v_full + vst), vphase, d, abort_flag) || !wait_one(B(p_full + pb), pphase, d, abort_flag))
                    return false;
                tc_fence_after();
                const uint32_t so = vst * (Lay::V_BYTES >> 4), tp = Lay::TM_S + pb * 64;
#pragma unroll
                for (int kk = 0; kk < kBlockSize / 16; ++kk)
                    mma_ts_h<ZW == 32 ? U64 : U128>(Lay::TM_O, tp + kk * 8, dV + so + (kk * (ZW == 32 ? 1024 : 2048) >> 4),
                                                    id_PV, !first || kk > 0);
                tc_commit(B(o_done + vst));
                if (++pb == NSB) {
                    pb = 0;
                    pphase ^= 1;
                }
                if (++vst == VST) {
                    vst = 0;
                    vphase ^= 1;
                }
                return true;
            };
            // (all 512 columns are this block's, so they begin at column 0 and the addresses above are constants)
            bool ok = tmem == 0;
            if (!ok) set_status(d.status, LRKV_DEV_TIMEOUT);
            for (; ok && w.next(a); w.step()) {
                ok = wait_one(B(q_ready), qphase, d, abort_flag);
                qphase ^= 1;
                tc_fence_after();
                for (int j = 0; ok && j < NSB && j < w.nt; ++j) ok = s_tile();
                for (int j = 0; ok && j < w.nt; ++j) ok = pv_tile(j == 0) && (j + NSB >= w.nt || s_tile());
            }
            if (!ok) *abort_flag = 1;
            tc_commit(B(mma_drain));
        }
        __syncwarp();
        // every MMA this warp issued has finished before the CTA tears TMEM down
        drain(B(mma_drain), 0, d.status);
    } else if (warp != 7) {
        // ---------------------------------------------------------------- query rows: softmax, partials
        // Two groups of four warps, a query row per thread in each; group g % 2 takes page g.  The reference maximum
        // goes from page to page, so a group decides on it once the other has for the page before; the exponentials of
        // two pages run side by side.
        const int qq = warp & 3, half = warp >> 3;  // TMEM lanes 32 qq ..
        const int row = qq * 32 + lane;
        const uint32_t tl = (uint32_t)(qq * 32) << 16;
        const int hl = row / a.ns, il = row - hl * a.ns;
        volatile float* const refs = reinterpret_cast<float*>(smem + Lay::OFF_ROW);
        float2* const sums2 = reinterpret_cast<float2*>(smem + Lay::OFF_ROW + 512);
        bool ok = true;
        int g0 = 0, sb0 = 0, kst0 = 0, vst0 = 0, piece = 0;  // pages so far, S buffer and stages of the next, pieces so far
        uint32_t kphase0 = 0, vphase0 = 0;
        // 64 columns of a block into TMEM (two columns a register), or K-major with 128-byte swizzle (16-byte chunk c
        // at c ^ (row mod 8))
        auto put_block = [&](int bk, const uint4* x) {
            if (bk < Lay::QBT) {
                tmem_st_32x32b_x32(tmem + tl + Lay::TM_Q + bk * 32, reinterpret_cast<const uint32_t*>(x));
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(smem + (bk - Lay::QBT) * 16384 + row * 128 + ((c ^ (row & 7)) << 4)) = x[c];
            }
        };
        bool have = w.next(a);
        if (have && half == 1) {
            const uint4 zeros[8] = {};
#pragma unroll
            for (int bk = D_K / 64; bk < NBQ; ++bk) put_block(bk, zeros);
            tmem_wait_st();
        }
        pdl_wait();  // q~ (and this grid's end stands for that of the launches before it)
        if (have) pdl_trigger();  // the merge may be set up: its blocks wait for this grid's end
        while (have) {
            const int b = w.b, L = w.s.L, n = w.s.n, st_b = (n + a.ns - 1) / a.ns;
            const int tile = w.tile(a), h = tile / st_b * a.hb + hl, i = tile % st_b * a.ns + il;
            const bool live = h < H && i < n;
            const size_t qr = live ? ((size_t)b * a.T + i) * H + h : 0;
            const int slot = (gang + b * a.gmax + w.t) * a.gang + member;
            const int p0 = w.p0, nt = w.nt;
            // the drafted tokens that the row sees
            unsigned long long tree = ~0ull >> (64 - n);  // (n >= 1)
            if (live) tree &= a.mask ? a.mask[(size_t)b * a.T + i] : ~0ull >> (63 - i);
            {
                // Its share of [Q | diag(Q~)]: group 0 has the first 128 columns of q, group 1 the last 64 of 192 and q~, of
                // which a row only ever writes its own head's columns (the others are zeroed once).
                uint4 qv[16];  // (of group 1: eight of q, eight of q~'s fp32 values)
                const uint4 zero = make_uint4(0, 0, 0, 0);
                const uint4* const q = reinterpret_cast<const uint4*>(d.q + qr * D_K) + (half == 0 ? 0 : 16);
                const uint4* const y = reinterpret_cast<const uint4*>(d.qt + qr * R);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    qv[c] = live && (half == 0 || D_K == 192) ? q[c] : zero;
                    qv[8 + c] = !live ? zero : half == 0 ? (D_K >= 128 ? q[8 + c] : zero) : c < R / 4 ? y[c] : zero;
                }
                if (half == 0) {
                    put_block(0, qv);
                    if (D_K >= 128) put_block(1, qv + 8);
                } else {
                    if (D_K == 192) put_block(2, qv);
                    // q~ rounded to bf16, and what that left, rounded: R / 2 registers each
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 y = make_float4(__uint_as_float(qv[8 + c].x), __uint_as_float(qv[8 + c].y),
                                                     __uint_as_float(qv[8 + c].z), __uint_as_float(qv[8 + c].w));
                        hi[2 * c] = pack_bf16x2(y.x, y.y);
                        hi[2 * c + 1] = pack_bf16x2(y.z, y.w);
                        lo[2 * c] = pack_bf16x2(y.x - bf16lo(hi[2 * c]), y.y - bf16hi(hi[2 * c]));
                        lo[2 * c + 1] = pack_bf16x2(y.z - bf16lo(hi[2 * c + 1]), y.w - bf16hi(hi[2 * c + 1]));
                    }
                    // (a warp's rows are of 32 / ns heads or of one, whose columns lie in one block)
                    const int h1 = (qq * 32) / a.ns, h2 = (qq * 32 + 31) / a.ns;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t* const x = part ? lo : hi;
                        const int col = D_K + part * ZW + h1 * R;
                        if (col / 64 < Lay::QBT) {
                            for (int hh = h1; hh <= h2; ++hh) {
                                uint32_t v[16];
#pragma unroll
                                for (int c = 0; c < 16; ++c) v[c] = hl == hh ? x[c] : 0u;
                                const uint32_t at = tmem + tl + Lay::TM_Q + (D_K + part * ZW + hh * R) / 2;
                                if (R == 8)
                                    tmem_st_32x32b_x4(at, v);
                                else if (R == 16)
                                    tmem_st_32x32b_x8(at, v);
                                else
                                    tmem_st_32x32b_x16(at, v);
                            }
                        } else {
                            const int mine = D_K + part * ZW + hl * R, c0 = mine % 64 / 8;
                            uint8_t* const r = smem + (mine / 64 - Lay::QBT) * 16384 + row * 128;
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c < R / 8)
                                    *reinterpret_cast<uint4*>(r + (((c0 + c) ^ (row & 7)) << 4)) =
                                        make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
                        }
                    }
                }
                tmem_wait_st();
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(q_ready);
            }
            if (p0 == 0 && warp == 2 && lane == 0) {
                const int last = work.range_of(w.seg + w.s.pages - 1);
                a.seg_table[b * a.tmax + tile] = make_int2(slot, last - gang + 1);
            }
            w.step();
            have = w.next(a);  // (from here on the walk shows the next piece)
            float mref = -INFINITY, l = 0.f;  // the reference that this group knows, and its sum relative to that
            // After an expired wait the loop goes on without work, so that the groups still meet at their barriers.
            // S buffer and stages of page g; the thread's own pages are every second one
            int sb = sb0, kst = kst0, vst = vst0;
            uint32_t kphase = kphase0, vphase = vphase0;
            auto advance = [&](int pages) {  // by 1 or 2
                sb += pages;
                sb -= sb >= NSB ? NSB : 0;
                kst += pages;
                kphase ^= kst >= KST;
                kst -= kst >= KST ? KST : 0;
                vst += pages;
                vphase ^= vst >= VST;
                vst -= vst >= VST ? VST : 0;
            };
            auto wait_before = [&]() {  // until the page before has been added to O
                return wait_warp(B(o_done + (vst > 0 ? vst - 1 : VST - 1)), vst > 0 ? vphase : vphase ^ 1, d, abort_flag);
            };
            const int32_t* const pages = d.block_table + (size_t)b * d.max_pages + p0;
            const int j0 = (g0 ^ half) & 1;
            if (j0) advance(1);
            // (a page's id is loaded a page ahead: some 700 cycles late, it was half of a page's time)
            int blk_next = j0 < nt ? pages[j0] : -1;
            for (int j = j0; j < nt; j += 2, advance(2)) {
                const int g = g0 + j, blk = blk_next;
                blk_next = j + 2 < nt ? pages[j + 2] : -1;
                const uint32_t tS = tmem + tl + Lay::TM_S + sb * 64;
                const int base = (p0 + j) * kBlockSize;
                const bool good = blk >= 0 && blk < d.num_blocks;
                const bool inner = good && base + kBlockSize <= L;  // every row sees every token
                ok = ok && wait_warp(B(s_done + kst), kphase, d, abort_flag);
                float mx = -INFINITY;
                if (ok) {
                    if (j == 0 && row == 0) poison[(piece + 1) & 1] = 0;  // (every row is done with the piece before)
                    tc_fence_after();
                    const int c = L - base;  // tokens of the page before the drafted ones
                    unsigned long long seen = ~0ull;
                    if (!inner) {
                        seen = c >= 0 ? (c < 64 ? tree << c : 0) | (c < 64 ? (1ull << c) - 1 : ~0ull)
                                      : (c > -64 ? tree >> -c : 0);
                        if (!good) seen = 0;
                        // Values that not every row sees, or none: cleared where they could spoil a product with a
                        // probability of 0.  Rows behind the end wholly; of a drafted token what is not finite,
                        // which is noted and added at the end to the rows that do see it.
                        ok = wait_warp(B(v_full + vst), vphase, d, abort_flag);
                        const int t = base + (row & 63) - L;
                        if (ok && t >= 0 &&
                            clean_values<D_H, ZW>(smem + Lay::OFF_V + vst * Lay::V_BYTES, row & 63, row >> 6, t >= n))
                            atomicOr(poison + (piece & 1), 1ull << t);
                        __syncwarp();
                    }
                    // (in halves, and again for the exponentials: a loop that stays in the instruction cache is worth
                    // more than the loads from TMEM)
                    mx = look(tS, inner, seen, d.scale_log2);
                    // diag(Q~)'s zeros times another head's NaN or infinity are NaN (and so is what rounding an
                    // infinite product left): such logits are formed again from the row's own head alone.  A
                    // second look is over numbers, or over what is NaN by itself, which decides through the sum.
                    if (__any_sync(0xffffffffu, mx != mx)) {
                        form_again(tS, live, (size_t)blk * kBlockSize, d.q + qr * D_K, d.qt + qr * R, a.sK, a.zK, D_K, R, H,
                                   h);
                        mx = look(tS, true, ~0ull, d.scale_log2);
                        mx = mx != mx ? INFINITY : mx;
                    }
                }
                if (g > 0) named_bar(1 + qq + 4 * half, 64);  // the other group has decided for the page before
                const float before = j > 0 ? refs[row] : -INFINITY;
                const bool raise = mx > before + kRescaleThreshold;  // or the row's first token
                const float now = raise ? mx : before;
                refs[row] = now;
                if (j + 1 < nt || have) named_arrive(1 + qq + 4 * (half ^ 1), 64);
                if (!ok) continue;
                if (mref != now) {
                    l = mref == -INFINITY ? 0.f : l * ex2_approx(mref - now);
                    mref = now;
                }
                // p = 2^(s scale log2 e - m), 0 everywhere as long as the row has seen no token
                const float nm = now == -INFINITY ? -INFINITY : -now;
                const uint64_t nm2 = pair(__float_as_uint(nm), __float_as_uint(nm));
                const uint64_t sc2 = pair(__float_as_uint(d.scale_log2), __float_as_uint(d.scale_log2));
                uint64_t l2[2] = {0, 0};
#pragma unroll 1
                for (int e0 = 0; e0 < 64; e0 += 32) {
                    uint32_t sv[32], pk[16];
                    tmem_ld_32x32b_x32(tS + e0, sv);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float x0, x1;
                        unpair(fma2(pair(sv[e], sv[e + 1]), sc2, nm2), x0, x1);
                        x0 = ex2_approx(x0);
                        x1 = ex2_approx(x1);
                        l2[e / 2 & 1] = add2(l2[e / 2 & 1], pair(__float_as_uint(x0), __float_as_uint(x1)));
                        pk[e / 2] = pack_bf16x2(x0, x1);
                    }
                    tmem_st_32x32b_x16(tS + e0 / 2, pk);
                }
                {
                    float x0, x1;
                    unpair(add2(l2[0], l2[1]), x0, x1);
                    l += x0 + x1;
                }
                // O may only be rescaled once P_{g-1} V_{g-1} has finished accumulating into it
                if (j > 0 && __any_sync(0xffffffffu, raise)) {
                    ok = wait_before();
                    if (ok) {
                        tc_fence_after();
                        const float alpha = raise && before != -INFINITY ? ex2_approx(before - now) : 1.f;
                        uint32_t v[32];
#pragma unroll 1
                        for (int c = 0; c < (D_H + ZW) / 32; ++c) {
                            tmem_ld_32x32b_x32(tmem + tl + Lay::TM_O + c * 32, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                            tmem_st_32x32b_x32(tmem + tl + Lay::TM_O + c * 32, v);
                        }
                    }
                }
                tmem_wait_st();
                if (!ok) continue;
                if (!inner) fence_proxy_async_smem();  // cleared values before the tensor cores read them
                tc_fence_before();
                arrive(p_full + sb);
            }
            g0 += nt;
            sb0 = (sb0 + nt) % NSB;
            kphase0 ^= (kst0 + nt) / KST & 1;
            kst0 = (kst0 + nt) % KST;
            vphase0 ^= (vst0 + nt) / VST & 1;
            vst0 = (vst0 + nt) % VST;
            // the row's sum over both groups' pages
            // (by the piece's parity: a group without a page in the next piece gets there while the other may still read)
            float2* const sums = sums2 + (piece & 1) * 256;
            sums[half * 128 + row] = make_float2(l, mref);
            named_bar(9 + qq, 64);
            const float2 other = sums[(half ^ 1) * 128 + row];
            const float M = fmaxf(mref, other.y);
            float ls = (mref == -INFINITY ? 0.f : l * ex2_approx(mref - M)) +
                       (other.y == -INFINITY ? 0.f : other.x * ex2_approx(other.y - M));
            // ---- partials, unnormalised: [column quad][row], so that a warp's stores are consecutive
            vst = vst0;
            vphase = vphase0;
            if (ok) ok = wait_before();
            if (ok) {
                tc_fence_after();
                const bool nan = ls != ls;  // handed on as NaN values with a weight, not as an empty part
                const float mo = nan && !(fabsf(M) < INFINITY) ? 0.f : M;
                // (rows without a drafted token or head are not stored)
                if (half == 0 && live) a.ml[(size_t)slot * a.rs + hl * a.tn + il] = make_float2(mo, nan ? 1.f : ls);
                float4* const dst = a.acc + (size_t)slot * (W / 4) * a.rs + hl * a.tn + il;
                const float bad = __uint_as_float(0x7fc00000u);
                auto put = [&](const uint32_t* v, int c) {  // columns c .. c + 3 of [s^V | z^V of the row's head]
                    if (live)
                        dst[(size_t)(c / 4) * a.rs] = nan ? make_float4(bad, bad, bad, bad)
                                                          : make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]),
                                                                        __uint_as_float(v[2]), __uint_as_float(v[3]));
                };
#pragma unroll 1
                for (int c = half; c < D_H / 32; c += 2) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem + tl + Lay::TM_O + c * 32, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) put(v + 4 * e, c * 32 + e * 4);
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
                    for (int e = 0; e < 8; ++e) {
                        const int col = c * 32 + e * 4 - hl * R;
                        if (col >= 0 && col < R) put(v + 4 * e, D_H + col);
                    }
                }
                tc_fence_before();
                const unsigned long long spoilt = live ? poison[piece & 1] & tree : 0ull;
                if (spoilt)
                    add_spoilt(dst, a.rs, spoilt, half, hl, d.block_table + (size_t)b * d.max_pages, L, a.sV, a.zV, D_H, R, H,
                               h);
            } else {
                *abort_flag = 1;
            }
            ++piece;
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

// Merge of a tile's pieces, B_h^V, division by the sum: grid (groups of 32 rows x D_H / DC groups of DC output columns, tiles,
// sequences), block (32, 8).  A lane is a row while the pieces are read (consecutive rows' quads lie side by
// side), output columns after.  Where there are few tiles a block takes few columns (and reads the latents' sums again) and
// has the loads of four pieces in flight; many tiles are of one or two pieces each, and more blocks fit with one.
template <int D_H, int R, int DC>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int W4 = (D_H + R) / 4, C4 = (DC + R) / 4, QPW = (C4 + 7) / 8, DPL = DC / 32, kPieces = DC == 32 ? 4 : 1;
    static_assert(DPL == 1 || DPL == 2, "output columns of a lane");
    const DecodeArgs& d = a.d;
    const int lane = threadIdx.x, warp = threadIdx.y, b = blockIdx.z, t = blockIdx.y;
    // rows: head x drafted token of the tile, tn tokens a head
    const int groups = a.rs / 32, row0 = blockIdx.x % groups * 32, row = row0 + lane, d0 = blockIdx.x / groups * DC;
    __shared__ float tile[32][DC + R + 1];
    const Seq s = seq_of(a, b);  // (the caller's, not of a launch before this one)
    const int st_b = max(1, (s.n + a.ns - 1) / a.ns), h0 = t / st_b * a.hb, i0 = t % st_b * a.ns;
    // four rows per warp, mostly of one head, DPL output columns per lane
    const int r0 = warp * 4;
    int h = h0 + (row0 + r0) / a.tn;
    uint4 f[DPL][R / 8];
    auto factors = [&]() {
        const uint16_t* bv = d.BV + ((size_t)h * D_H + d0 + lane * DPL) * R;
#pragma unroll
        for (int e = 0; e < DPL; ++e)
#pragma unroll
            for (int k = 0; k < R / 8; ++k) f[e][k] = *reinterpret_cast<const uint4*>(bv + e * R + k * 8);
    };
    if (!s.bad && t < tiles_of(a, s.n) && h < d.H) factors();
    pdl_wait();  // the scan (in every block: this grid's end stands for that of the launches before it)
    if (s.bad) {  // zeros in all T rows: the tiles of a full sequence share them
        if (t == 0 && blockIdx.x == 0 && lane == 0 && warp == 0) set_status(d.status, LRKV_DEV_BAD_SEQLEN);
        const size_t n = (size_t)a.T * d.H * D_H / 8, step = (size_t)gridDim.x * gridDim.y * 256;
        uint4* out = reinterpret_cast<uint4*>(d.out + (size_t)b * a.T * d.H * D_H);
        for (size_t i = (size_t)(t * gridDim.x + blockIdx.x) * 256 + warp * 32 + lane; i < n; i += step)
            out[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    if (t >= tiles_of(a, s.n) || h0 + row0 / a.tn >= d.H) return;
    const bool live = row < a.hb * a.tn && h0 + row / a.tn < d.H && i0 + row % a.tn < s.n;
    if (!__syncthreads_or(live)) return;
    const int2 fe = a.seg_table[b * a.tmax + t];
    float M = -INFINITY, ls = 0.f;
    float4 x[QPW];
#pragma unroll
    for (int e = 0; e < QPW; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    const float2* const ml0 = a.ml + (size_t)fe.x * a.rs + row;
    const float4* const acc0 = a.acc + (size_t)fe.x * W4 * a.rs + row;
    for (int k0 = 0; live && k0 < fe.y; k0 += kPieces) {
        float2 ml[kPieces];
        float4 y[kPieces][QPW];
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const bool there = k0 + k < fe.y;
            ml[k] = there ? ml0[(size_t)(k0 + k) * a.gang * a.rs] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < QPW; ++e) {
                const int c = e * 8 + warp, at = c < DC / 4 ? d0 / 4 + c : D_H / 4 + c - DC / 4;
                y[k][e] = there && c < C4 ? acc0[((size_t)(k0 + k) * a.gang * W4 + at) * a.rs]
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) mn = fmaxf(mn, ml[k].x);
        if (mn == -INFINITY) continue;
        const float sc = M == -INFINITY ? 0.f : exp2f(M - mn);
        M = mn;
        ls *= sc;
#pragma unroll
        for (int e = 0; e < QPW; ++e) {
            x[e].x *= sc;
            x[e].y *= sc;
            x[e].z *= sc;
            x[e].w *= sc;
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            if (ml[k].x == -INFINITY) continue;  // a piece of which the row sees nothing
            const float w = exp2f(ml[k].x - mn);
            ls = fmaf(w, ml[k].y, ls);
#pragma unroll
            for (int e = 0; e < QPW; ++e) {
                x[e].x = fmaf(w, y[k][e].x, x[e].x);
                x[e].y = fmaf(w, y[k][e].y, x[e].y);
                x[e].z = fmaf(w, y[k][e].z, x[e].z);
                x[e].w = fmaf(w, y[k][e].w, x[e].w);
            }
        }
    }
    // (the sum is 0 where the row sees no token: zeros)
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll
    for (int e = 0; e < QPW; ++e) {
        const int c = (e * 8 + warp) * 4;
        if (c >= DC + R) break;
        tile[lane][c] = x[e].x * inv;
        tile[lane][c + 1] = x[e].y * inv;
        tile[lane][c + 2] = x[e].z * inv;
        tile[lane][c + 3] = x[e].w * inv;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int rr = row0 + r0 + r, i = i0 + rr % a.tn, hr = h0 + rr / a.tn;
        if (rr >= a.hb * a.tn || i >= s.n || hr >= d.H) continue;
        if (hr != h) {
            h = hr;
            factors();
        }
        float y[DPL];
#pragma unroll
        for (int e = 0; e < DPL; ++e) y[e] = tile[r0 + r][lane * DPL + e];
#pragma unroll
        for (int k = 0; k < R / 8; ++k) {
            float z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = tile[r0 + r][DC + k * 8 + j];
#pragma unroll
            for (int e = 0; e < DPL; ++e) {
                y[e] = fmaf(bf16lo(f[e][k].x), z[0], fmaf(bf16hi(f[e][k].x), z[1], y[e]));
                y[e] = fmaf(bf16lo(f[e][k].y), z[2], fmaf(bf16hi(f[e][k].y), z[3], y[e]));
                y[e] = fmaf(bf16lo(f[e][k].z), z[4], fmaf(bf16hi(f[e][k].z), z[5], y[e]));
                y[e] = fmaf(bf16lo(f[e][k].w), z[6], fmaf(bf16hi(f[e][k].w), z[7], y[e]));
            }
        }
        uint16_t* out = d.out + (((size_t)b * a.T + i) * d.H + h) * D_H + d0 + lane * DPL;
        if constexpr (DPL == 2) {
            *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(y[0], y[1]);
        } else {
            const __nv_bfloat16 o = __float2bfloat16_rn(y[0]);
            *out = *reinterpret_cast<const uint16_t*>(&o);
        }
    }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// Which tile: the fewest columns of products, tiles x (d_k + d_h + 3 zw).
TreePlan tree_plan(int H, int D_H, int R, int D_R, int T) {
    TreePlan best{};
    long long least = -1;
    for (int zw = 32; zw <= 128; zw *= 2) {
        TreePlan p{};
        p.zw = zw;
        p.hb = zw / R;
        p.ns = 128 / p.hb;
        p.htiles = (H + p.hb - 1) / p.hb;
        p.stiles = (T + p.ns - 1) / p.ns;
        if (p.ns > 64) continue;
        const long long cost = (long long)p.htiles * p.stiles * (2 * D_H + D_R + 3 * zw);
        if (least < 0 || cost < least) {
            best = p;
            least = cost;
        }
    }
    return best;
}

// CTAs of a gang: as many as leave the fewest SMs and the fewest members without a tile (within 2%), up to 16, more
// rather than fewer.  (In a graph, us, at most 1 | 4 | 8 to 32: 24 ragged sequences of 32 heads 103 | 94 | 92, 4 of 16 to
// 32 K tokens 110 | 99 | 96, 128 heads 347 | 325 | 325; within 0 to 5% all alike, 10% 128 heads 344.)
static int tree_gang(int tiles, int sms) {
    int best = 1;
    double most = 0;
    for (int q = 1; q <= 16 && q <= tiles && q <= sms; ++q) {
        const double use = (double)(sms / q * q) / sms * tiles / ((tiles + q - 1) / q * q);
        if (use >= most - 0.02) {
            best = q;
            most = use > most ? use : most;
        }
    }
    return best;
}

struct TreeSizes {
    int gang, gangs, gmax;  // CTAs of a gang, gangs, groups of tiles of a sequence
    int tn, rs;             // drafted tokens of a tile at most, rows kept of it
    size_t qt, seg, ml, acc;
};
static TreeSizes tree_sizes(int H, int D_H, int R, int batch, int T, const TreePlan& p, int sms) {
    TreeSizes z{};
    const int tiles = p.htiles * p.stiles;
    z.gang = tree_gang(tiles, sms);
    z.gangs = sms / z.gang;
    z.gmax = (tiles + z.gang - 1) / z.gang;
    z.tn = T < p.ns ? T : p.ns;
    z.rs = (p.hb * z.tn + 31) / 32 * 32;
    const size_t slots = ((size_t)z.gangs + (size_t)batch * z.gmax) * z.gang;
    z.qt = align256((size_t)batch * T * H * R * sizeof(float));
    z.seg = align256((size_t)batch * tiles * sizeof(int2));
    z.ml = align256(slots * z.rs * sizeof(float2));
    z.acc = align256(slots * z.rs * (D_H + R) * sizeof(float));
    return z;
}

size_t tree_workspace_bytes(int H, int D_H, int R, int D_R, int batch, int T, int sms) {
    const TreeSizes z = tree_sizes(H, D_H, R, batch, T, tree_plan(H, D_H, R, D_R, T), sms);
    return z.qt + z.seg + z.ml + z.acc + 256;  // (never 0)
}

void tree_carve_workspace(TreeArgs* a, void* ws, int D_H, int R, int D_R, int sms) {
    const TreePlan p = tree_plan(a->d.H, D_H, R, D_R, a->T);
    const TreeSizes z = tree_sizes(a->d.H, D_H, R, a->batch, a->T, p, sms);
    a->zw = p.zw;
    a->hb = p.hb;
    a->ns = p.ns;
    a->htiles = p.htiles;
    a->tmax = p.htiles * p.stiles;
    a->gang = z.gang;
    a->gangs = z.gangs;
    a->gmax = z.gmax;
    a->tn = z.tn;
    a->rs = z.rs;
    uint8_t* at = static_cast<uint8_t*>(ws);
    a->d.qt = reinterpret_cast<float*>(at);
    a->seg_table = reinterpret_cast<int2*>(at += z.qt);
    a->ml = reinterpret_cast<float2*>(at += z.seg);
    a->acc = reinterpret_cast<float4*>(at += z.ml);
}

template <int D_H, int D_R, int ZW>
static cudaError_t launch_scan_t(const TreeMaps& maps, const TreeArgs& a, int R, cudaStream_t stream) {
    constexpr uint32_t smem = TrLayout<D_H, D_R, ZW>::SMEM;
    auto kern = tree_scan_kernel<D_H, D_R, ZW>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(a.gang * a.gangs), dim3(kThreads), smem, stream, maps, a, R);
}

cudaError_t launch_tree(const TreeMaps& maps, const TreeArgs& a, int D_H, int R, int D_R, cudaStream_t stream) {
    cudaError_t e = launch_decode_absorb(a.d, D_H, R, D_R, stream);
    if (e != cudaSuccess) return e;
    e = cudaErrorInvalidValue;
#define LRKV_TS(DH, DR)                                                        \
    if (D_H == DH && D_R == DR)                                                \
        e = a.zw == 128  ? launch_scan_t<DH, DR, 128>(maps, a, R, stream)      \
            : a.zw == 64 ? launch_scan_t<DH, DR, 64>(maps, a, R, stream)       \
                         : launch_scan_t<DH, DR, 32>(maps, a, R, stream);
    LRKV_TS(64, 0) LRKV_TS(64, 64) LRKV_TS(128, 0) LRKV_TS(128, 64)
#undef LRKV_TS
    if (e != cudaSuccess) return e;
    const int groups = a.rs / 32;
    // Up to one group of 32 rows for an SM: blocks of 32 output columns with four pieces in flight, else of 64 with one.  (In
    // a graph, us, 32 | 64 columns: 0.03 groups an SM 17.9 | 28.5, 0.2 95.7 | 101, 0.4 18.8 | 21.6; 1.2 58.0 | 53.2, 2.1
    // 31.6 | 26.8, 3.4 42.5 | 30.6, 5 109 | 92.)
    const bool few = (long long)a.tmax * a.batch * groups <= a.gang * a.gangs;
#define LRKV_TC(DH, RR)                                                                                             \
    if (D_H == DH && R == RR)                                                                                       \
        return few ? launch_dependent(tree_combine_kernel<DH, RR, 32>, dim3(groups * (DH / 32), a.tmax, a.batch),        \
                                      dim3(32, 8), 0, stream, a)                                                    \
                   : launch_dependent(tree_combine_kernel<DH, RR, 64>, dim3(groups * (DH / 64), a.tmax, a.batch), dim3(32, 8), 0,    \
                                      stream, a);
    LRKV_TC(64, 8) LRKV_TC(64, 16) LRKV_TC(64, 32) LRKV_TC(128, 8) LRKV_TC(128, 16) LRKV_TC(128, 32)
#undef LRKV_TC
    return cudaErrorInvalidValue;
}

}  // namespace lrkv
