// pages.cu -- pages of the cache: taken, shared, copied, compacted and given back on the device.
//
// The only state is a count per page (refs) beside the block table; a free page is one whose count is 0, and free
// pages are taken lowest first.  Counts change by atomic additions, whose order does not change the outcome, and taken
// pages go to the requests in the order of the call by a prefix sum, so results do not depend on timing.
#include <cooperative_groups.h>

#include <climits>

#include "draft.h"
#include "lrkv_internal.cuh"
#include "tile_attn.cuh"

namespace lrkv {

namespace {

// These kernels are short and follow one another: each is launched while the one before it on the stream still runs, waits
// for its end before it touches memory, and only then lets the next one be launched.
__device__ __forceinline__ void begin_dependent() {
    pdl_wait();
    pdl_trigger();
}

constexpr int kPlanThreads = 1024;
constexpr int kPerThread = 16;  // counts a thread looks at in one round of the search

__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// Inclusive prefix sum over the block's kPlanThreads threads; total to every thread.
__device__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_incl_scan(v, lane);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = warp_incl_scan(warp_sums[lane], lane);
    __syncthreads();
    *total = warp_sums[kPlanThreads / 32 - 1];
    const int r = v + (warp ? warp_sums[warp - 1] : 0);
    __syncthreads();
    return r;
}

// Sum of need[0..n) (shared memory) to every thread, in 64 bits: 8,192 requests of up to 2^24 + 1 pages each.
__device__ long long sum_of_needs(const int* need, int n) {
    __shared__ uint2 sums[kPlanThreads / 32];
    unsigned v = 0;  // (at most eight requests of a thread)
    for (int i = threadIdx.x; i < n; i += kPlanThreads) v += need[i];
    uint2 x = make_uint2(__reduce_add_sync(0xffffffffu, v & 0xffff), __reduce_add_sync(0xffffffffu, v >> 16));
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sums[threadIdx.x & 31];
    return (long long)__reduce_add_sync(0xffffffffu, x.y) * 65536 + __reduce_add_sync(0xffffffffu, x.x);
}

// need[0..n) (shared memory), at most num_blocks together: pages of request i -> exclusive prefix sums; returns their
// total.
__device__ int prefix_of_needs(int* need, int n, int* warp_sums) {
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x, v = i < n ? need[i] : 0;
        int total;
        const int incl = block_scan(v, warp_sums, &total);
        if (i < n) need[i] = base + incl - v;
        base += total;
    }
    __syncthreads();
    return base;
}

// Walks the counts from page 0 until `want` free pages are found; take(page, rank) for each of the first `want`.
// Returns how many there are (at most want).
template <class F>
__device__ int search_free(const int32_t* refs, int num_blocks, int want, int* warp_sums, F&& take) {
    int found = 0;
    for (int p0 = 0; p0 < num_blocks && found < want; p0 += kPlanThreads * kPerThread) {
        const int p = p0 + threadIdx.x * kPerThread;
        uint32_t free = 0;
        if (p + kPerThread <= num_blocks) {
            int4 r[kPerThread / 4];
#pragma unroll
            for (int k = 0; k < kPerThread / 4; ++k) r[k] = __ldcg(reinterpret_cast<const int4*>(refs + p) + k);
#pragma unroll
            for (int k = 0; k < kPerThread / 4; ++k)
                free |= ((uint32_t)(r[k].x == 0) | (uint32_t)(r[k].y == 0) << 1 | (uint32_t)(r[k].z == 0) << 2 |
                         (uint32_t)(r[k].w == 0) << 3)
                        << (4 * k);
        } else {
            for (int e = 0; e < kPerThread; ++e)
                if (p + e < num_blocks && __ldcg(refs + p + e) == 0) free |= 1u << e;
        }
        const int c = __popc(free);
        int total;
        int rank = found + block_scan(c, warp_sums, &total) - c;
        while (free && rank < want) {
            take(p + __ffs(free) - 1, rank++);
            free &= free - 1;
        }
        found += total;
    }
    return found < want ? found : want;
}

// The request that rank `rank` belongs to: the last i with pre[i] <= rank (requests without needs have
// their successor's sum).
__device__ __forceinline__ int owner(const int* pre, int n, int rank) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= rank)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// need[0..n) granted from the free pages, whole requests or none, in order (refused(i) for those that do not fit);
// give(i, k, granted, page) is called for the k-th of the `granted` pages of request i.  The first search keeps the pages it
// finds, up to kPicked: they are all that most calls need.
constexpr int kPicked = 2048;
template <class F, class G>
__device__ void grant(int* need, int n, const int32_t* refs, int num_blocks, int* warp_sums, int* picked, F&& refused,
                      G&& give) {
    const long long asked = sum_of_needs(need, n);
    if (asked == 0) return;
    int total = (int)(asked < num_blocks ? asked : num_blocks);
    const int have = search_free(refs, num_blocks, total, warp_sums, [&](int page, int rank) {
        if (rank < kPicked) picked[rank] = page;
    });
    if (have < asked) {
        __syncthreads();
        if (threadIdx.x == 0) {
            int left = have;
            for (int i = 0; i < n; ++i) {
                if (need[i] <= left) {
                    left -= need[i];
                } else {
                    refused(i);
                    need[i] = 0;
                }
            }
        }
        __syncthreads();
    }
    total = prefix_of_needs(need, n, warp_sums);
    auto hand = [&](int page, int rank) {
        const int i = owner(need, n, rank);
        give(i, rank - need[i], (i + 1 < n ? need[i + 1] : total) - need[i], page);
    };
    if (total <= kPicked) {
        for (int rank = threadIdx.x; rank < total; rank += kPlanThreads) hand(picked[rank], rank);
    } else {
        search_free(refs, num_blocks, total, warp_sums, hand);
    }
}

__device__ __forceinline__ int pages_of(long long tokens) { return (int)((tokens + kBlockSize - 1) / kBlockSize); }

// E pages (negative: none) given back, their atomics on the way together.
template <int E>
__device__ __forceinline__ void give_back(int32_t* refs, int num_blocks, const int* page, uint32_t* status) {
    int old[E];
#pragma unroll
    for (int e = 0; e < E; ++e) old[e] = page[e] >= 0 && page[e] < num_blocks ? atomicSub(refs + page[e], 1) : 1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (page[e] >= num_blocks) set_status(status, LRKV_DEV_BAD_BLOCK);
        if (old[e] <= 0) {
            atomicAdd(refs + page[e], 1);
            set_status(status, LRKV_DEV_BAD_INDEX);
        }
    }
}

// ---------------------------------------------------------------- reserve: one block
// The empty entries of a row are counted from its first one on: a caller may set a length before the row has pages for
// it.  They have to be the last ones of what is asked for, as in every row that these calls leave; a page that stands
// behind an empty entry is not written over.
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const PageArgs a) {
    __shared__ int need[LRKV_MAX_PAGE_BATCH], warp_sums[32], picked[kPicked];
    __shared__ int first_of[16], empty_of[16];
    begin_dependent();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // `parts` warps a sequence, kEntries x 32 entries at a time: several where there are few long rows (at most 16)
    constexpr int kWarps = kPlanThreads / 32, kEntries = 4;
    const int parts = a.batch < kWarps && a.max_pages > 32 * kEntries ? kWarps / a.batch : 1, part = warp % parts;
    if (parts > 1) {
        if (threadIdx.x < 16) {
            first_of[threadIdx.x] = INT_MAX;
            empty_of[threadIdx.x] = 0;
        }
        __syncthreads();
    }
    auto want_of = [&](int b) {
        const int L = a.lens[b], add = a.b[b];
        const int want = L >= 0 && add >= 0 ? pages_of((long long)L + add) : -1;
        return want <= a.max_pages ? want : -1;
    };
    auto decide = [&](int b, int want, int first, int empty) {
        need[b] = 0;
        if (want < 0)
            set_status(a.status, LRKV_DEV_BAD_SEQLEN);
        else if (empty > a.num_blocks)
            need[b] = a.num_blocks + 1;
        else if (empty > 0 && first + empty != want)
            set_status(a.status, LRKV_DEV_BAD_BLOCK);
        else
            need[b] = empty;
    };
    for (int b = warp / parts; b < a.batch && warp < parts * a.batch; b += kWarps / parts) {
        const int want = want_of(b);
        const int32_t* row = a.table + (size_t)b * a.max_pages;
        int first = INT_MAX, empty = 0;  // of this lane's entries
        for (int k0 = part * 32 * kEntries; k0 < want; k0 += parts * 32 * kEntries) {
            int page[kEntries];
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                const int k = k0 + e * 32 + lane;
                page[e] = k < want ? row[k] : 0;
            }
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                if (page[e] >= 0) continue;
                first = min(first, k0 + e * 32 + lane);
                ++empty;
            }
            // (looked for only where there is more to come)
            if (k0 + parts * 32 * kEntries < want && __reduce_add_sync(0xffffffffu, empty) > a.num_blocks) break;
        }
        first = __reduce_min_sync(0xffffffffu, first);
        empty = __reduce_add_sync(0xffffffffu, empty);
        if (lane != 0) continue;
        if (parts == 1) {
            decide(b, want, first, empty);
        } else {
            atomicMin(first_of + b, first);
            atomicAdd(empty_of + b, empty);
        }
    }
    __syncthreads();
    if (parts > 1) {
        if (threadIdx.x < a.batch) decide(threadIdx.x, want_of(threadIdx.x), first_of[threadIdx.x], empty_of[threadIdx.x]);
        __syncthreads();
    }
    grant(need, a.batch, a.refs, a.num_blocks, warp_sums, picked, [&](int) { set_status(a.status, LRKV_DEV_NO_PAGES); },
          [&](int b, int k, int granted, int page) {
              // (the granted entries are the last ones of what the sequence asked for)
              const int want = pages_of((long long)a.lens[b] + a.b[b]);
              a.table[(size_t)b * a.max_pages + want - granted + k] = page;
              a.refs[page] = 1;
          });
}

// ---------------------------------------------------------------- fork
// What stands against fork i (status bits; 0: it is done): its indices, the child named twice or also as a parent, the
// parent's length, a page of the part of its row that is passed on.  The threads of a warp or block share the
// look (`all` joins their bits).  Both kernels of the call ask and find the same, since parents are never children,
// so nothing has to be passed on.
template <class All>
__device__ uint32_t fork_refused(const PageArgs& a, int i, int lane, int lanes, All&& all) {
    const int p = a.a[i], c = a.b[i];
    if (p < 0 || p >= a.batch || c < 0 || c >= a.batch) return LRKV_DEV_BAD_INDEX;
    const int L = a.lens[p];
    const bool fits = L >= 0 && L <= a.max_pages * kBlockSize;
    uint32_t bad = fits ? 0u : LRKV_DEV_BAD_SEQLEN;
    for (int j = lane; j < a.n; j += lanes)
        if (a.a[j] == c || (j != i && a.b[j] == c)) bad |= LRKV_DEV_BAD_INDEX;
    for (int k = lane; fits && k < pages_of(L); k += lanes) {
        const int page = a.table[(size_t)p * a.max_pages + k];
        if (page < 0 || page >= a.num_blocks) bad |= LRKV_DEV_BAD_BLOCK;
    }
    return all(bad);
}

// One block: a warp per fork, or a half or quarter of one where there are more forks, looks, gives the child's pages
// back, and passes the parent's on; eight entries of a row per lane on their way at once (one after the other, a warp per
// fork: 64 forks of 100 pages 26 us).
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PageArgs a) {
    // need: pages asked for, then their prefix sums; full: the full pages that a fork passes on (-1: left out, -2: no
    // page was left for the last, partly filled one)
    extern __shared__ int sh[];
    int *const need = sh, *const full = sh + a.n;
    __shared__ int warp_sums[32], picked[kPicked];
    begin_dependent();
    const int lanes = a.n <= 32 ? 32 : a.n <= 64 ? 16 : 8, lane = threadIdx.x & (lanes - 1);
    const int first = threadIdx.x / lanes, step = kPlanThreads / lanes;
    const uint32_t mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
    auto row_of = [&](int s) { return a.table + (size_t)s * a.max_pages; };
    constexpr int E = 8;
    for (int i = first; i < a.n; i += step) {
        const uint32_t bad = fork_refused(a, i, lane, lanes, [&](uint32_t x) { return __reduce_or_sync(mask, x); });
        if (lane == 0) {
            if (bad) set_status(a.status, bad & LRKV_DEV_BAD_INDEX ? LRKV_DEV_BAD_INDEX : bad);
            const int L = bad ? 0 : a.lens[a.a[i]];
            full[i] = bad ? -1 : L / kBlockSize;
            need[i] = L % kBlockSize != 0;
        }
        if (bad) continue;
        // what the child held goes back (parents' rows are not written here: no child is a parent)
        int32_t* row = row_of(a.b[i]);
        for (int k0 = 0; k0 < a.max_pages; k0 += lanes * E) {
            int page[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int k = k0 + e * lanes + lane;
                page[e] = k < a.max_pages ? row[k] : -1;
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (page[e] >= 0) row[k0 + e * lanes + lane] = -1;
            give_back<E>(a.refs, a.num_blocks, page, a.status);
        }
    }
    __threadfence();
    __syncthreads();
    grant(need, a.n, a.refs, a.num_blocks, warp_sums, picked,
          [&](int i) {
              set_status(a.status, LRKV_DEV_NO_PAGES);
              full[i] = -2;  // the child stays empty
          },
          [&](int i, int, int, int page) {
              row_of(a.b[i])[full[i]] = page;
              a.refs[page] = 1;
          });
    __syncthreads();
    for (int i = first; i < a.n; i += step) {
        const int f = full[i];
        if (f == -1) continue;
        const int32_t* from = row_of(a.a[i]);
        int32_t* to = row_of(a.b[i]);
        for (int k0 = 0; k0 < f; k0 += lanes * E) {
            int page[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int k = k0 + e * lanes + lane;
                page[e] = k < f ? from[k] : -1;
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (page[e] >= 0) {
                    to[k0 + e * lanes + lane] = page[e];
                    atomicAdd(a.refs + page[e], 1);
                }
        }
        if (lane == 0) a.lens[a.b[i]] = f < 0 ? 0 : a.lens[a.a[i]];
    }
}

// 16-byte unit `u` of a token row over all pools: the pool, and the unit within its row.
__device__ __forceinline__ int pool_of(const PoolArgs& p, int* u) {
    int k = 0;
    while (k + 1 < p.pools && *u >= p.u[k]) *u -= p.u[k++];
    return k;
}

// Rows of the children's last pages: grid (forks, layers, parts of a page's rows), about as many blocks as run at once, since
// each begins with a chain of loads (in pieces of 32 KB, 64 forks of 4 layers 20 us).  The whole call, 64 forks, 35 us in a
// stream of others, 32 in a graph; 11 for the bytes, the rest is the plan's chain of loads and this one's.
constexpr int kForkThreads = 512;
__global__ void __launch_bounds__(kForkThreads) fork_copy_kernel(const PoolArgs p, const PageArgs a) {
    const int i = blockIdx.x;
    begin_dependent();
    if (fork_refused(a, i, threadIdx.x, kForkThreads, [](uint32_t x) { return (uint32_t)__syncthreads_or(x != 0); })) return;
    const int par = a.a[i], c = a.b[i], L = a.lens[c];  // (0 where no page was left for the child)
    if (L % kBlockSize == 0) return;
    const int k = L / kBlockSize, from = a.table[(size_t)par * a.max_pages + k], to = a.table[(size_t)c * a.max_pages + k];
    const int rows = L % kBlockSize, n = rows * p.units, step = gridDim.z * kForkThreads;
    constexpr int E = 6;
    for (int u0 = blockIdx.z * kForkThreads + threadIdx.x; u0 < n; u0 += step * E) {
        uint4 v[E];
        uint4* out[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            int pool = 0, u = u0 + e * step;
            out[e] = nullptr;
            if (u >= n) continue;
            while (pool + 1 < p.pools && u >= p.u[pool] * rows) u -= p.u[pool++] * rows;
            uint4* b = p.base[pool] + (size_t)blockIdx.y * p.layer[pool];
            const size_t page = (size_t)kBlockSize * p.u[pool];
            v[e] = b[from * page + u];
            out[e] = b + to * page + u;
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (out[e]) *out[e] = v[e];
    }
}

// ---------------------------------------------------------------- free: a block per sequence
__global__ void __launch_bounds__(256) free_kernel(const PageArgs a) {
    begin_dependent();
    const int b = a.a[blockIdx.x];
    if (b < 0 || b >= a.batch) {
        if (threadIdx.x == 0) set_status(a.status, LRKV_DEV_BAD_INDEX);
        return;
    }
    const int keep = a.b ? a.b[b] : 0;
    if (keep < 0) {
        if (threadIdx.x == 0) set_status(a.status, LRKV_DEV_BAD_SEQLEN);
        return;
    }
    int32_t* row = a.table + (size_t)b * a.max_pages;
    for (int k = pages_of(keep) + threadIdx.x; k < a.max_pages; k += 256) {
        if (row[k] < 0) continue;
        const int page = atomicExch(row + k, -1);  // (the sequence may be listed twice)
        give_back<1>(a.refs, a.num_blocks, &page, a.status);
    }
    if (threadIdx.x == 0) {
        const int L = a.lens[b];
        a.lens[b] = L < keep ? L : keep;
    }
}

// ---------------------------------------------------------------- copy of whole pages
// A page's rows lie together in each pool, so it is moved in pieces of up to 16 KB by bulk copies, through a ring of
// stages in shared memory.  A warp is a block: its lanes work out the next 32 pieces, one of them issues the copies.
// 1,024 pages of 295 KB: 99 us (89 for the bytes at the copy rate); 164 with four 16-byte loads a thread, whose blocks came
// and went.
constexpr uint32_t kPiece = 16384;
constexpr int kStages = 6, kLag = 4;  // stages; pieces between a load's issue and its store's
struct CopyArgs {
    PoolArgs src, dst;
    const int32_t *from, *to;
    long long items;
    int parts;  // pieces of a page in all pools
    uint32_t* status;
};
__global__ void __launch_bounds__(32) copy_kernel(const __grid_constant__ CopyArgs a) {
    extern __shared__ uint8_t raw[];
    uint8_t* const ring = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    __shared__ uint64_t full[kStages];
    __shared__ uint4* dst[kStages];
    __shared__ uint32_t size[kStages];
    begin_dependent();
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(full + i), 1);
        fence_mbar_init();
    }
    __syncwarp();
    int loaded = 0, stored = 0;
    bool ok = true;
    auto store = [&]() {  // the oldest piece on its way
        const int st = stored % kStages;
        if (!mbar_wait(smem_u32(full + st), (stored / kStages) & 1, a.status)) return false;
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst[st]),
                     "r"(smem_u32(ring) + st * kPiece), "r"(size[st])
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        ++stored;
        return true;
    };
    for (long long base = blockIdx.x; base < a.items; base += (long long)gridDim.x * 32) {
        const long long item = base + (long long)gridDim.x * lane;
        const uint4* s = nullptr;
        uint4* t = nullptr;
        uint32_t bytes = 0;
        if (item < a.items) {
            const long long page = item / a.parts, i = page / a.src.layers;
            int part = (int)(item - page * a.parts);
            const int layer = (int)(page - i * a.src.layers), f = a.from[i], to = a.to[i];
            if (f >= 0 && to >= 0) {
                if (f >= a.src.num_blocks || to >= a.dst.num_blocks) {
                    set_status(a.status, LRKV_DEV_BAD_BLOCK);
                } else {
                    int p = 0;
                    auto pieces = [&](int k) { return (int)((kBlockSize * a.src.u[k] * 16 + kPiece - 1) / kPiece); };
                    while (part >= pieces(p)) part -= pieces(p++);
                    const size_t u = (size_t)kBlockSize * a.src.u[p], at = (size_t)part * (kPiece / 16);
                    s = a.src.base[p] + (size_t)layer * a.src.layer[p] + f * u + at;
                    t = a.dst.base[p] + (size_t)layer * a.dst.layer[p] + to * u + at;
                    bytes = (uint32_t)((u - at < kPiece / 16 ? u - at : kPiece / 16) * 16);
                }
            }
        }
        for (int j = 0; j < 32; ++j) {
            const uint32_t n = __shfl_sync(0xffffffffu, bytes, j);
            const uint64_t sp = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(s), j);
            const uint64_t tp = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(t), j);
            if (lane != 0 || n == 0 || !ok) continue;
            const int st = loaded % kStages;
            // the stage's last store has read it: behind it kStages - kLag - 1 others have been issued
            if (loaded >= kStages) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kStages - kLag - 1) : "memory");
            dst[st] = reinterpret_cast<uint4*>(tp);
            size[st] = n;
            mbar_arrive_expect_tx(smem_u32(full + st), n);
            bulk_load(smem_u32(ring) + st * kPiece, reinterpret_cast<const void*>(sp), n, smem_u32(full + st));
            if (++loaded > kLag) ok = store();
        }
    }
    if (lane == 0) {
        while (ok && stored < loaded) ok = store();
        // (after an expired wait: what is still on its way lands before the block gives up its shared memory)
        for (; stored < loaded; ++stored) mbar_wait(smem_u32(full + stored % kStages), (stored / kStages) & 1, a.status);
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// ---------------------------------------------------------------- compact: a cluster per sequence
// Row i moves from L + path[i] >= L + i down; a path increases, so a row is read before it is written if every thread
// takes its 16-byte column through the rows in order (eight rows in flight: the sources of the next eight lie behind
// all rows written so far).  The length may be updated in place once every block of the cluster has read it.
constexpr int kCompactCtas = 8, kCompactBatch = 8;
__global__ void __cluster_dims__(kCompactCtas, 1, 1) __launch_bounds__(256) compact_kernel(const CompactArgs a) {
    __shared__ int from[1024], to[1024];
    begin_dependent();
    const int b = blockIdx.y, L = a.lens[b], n = a.path_lens[b];
    const int32_t* path = a.path + (size_t)b * a.max_path;
    const int32_t* row = a.table + (size_t)b * a.max_pages;
    const long long cap = (long long)a.max_pages * kBlockSize;
    uint32_t bad = 0;
    if (L < 0 || L > cap) {
        bad = LRKV_DEV_BAD_SEQLEN;
    } else if (n < 0 || n > a.max_path) {
        bad = LRKV_DEV_BAD_INDEX;
    } else {
        for (int i = threadIdx.x; i < n; i += 256) {
            const int x = path[i], before = i ? path[i - 1] : -1;
            from[i] = to[i] = 0;
            if (x <= before || x < i) {
                bad |= LRKV_DEV_BAD_INDEX;
            } else if ((long long)L + x >= cap) {
                bad |= LRKV_DEV_BAD_SEQLEN;
            } else {
                const int f = row[(L + x) / kBlockSize], t = row[(L + i) / kBlockSize];
                if (f < 0 || f >= a.p.num_blocks || t < 0 || t >= a.p.num_blocks) {
                    bad |= LRKV_DEV_BAD_BLOCK;
                } else {
                    // (slots fit 31 bits: 2^24 blocks of 64 rows at most)
                    from[i] = f * kBlockSize + (L + x) % kBlockSize;
                    to[i] = t * kBlockSize + (L + i) % kBlockSize;
                }
            }
        }
    }
    const bool skip = __syncthreads_or(bad != 0);
    if (bad && blockIdx.x == 0) set_status(a.status, bad);
    // every block of the cluster has read the length and the path
    cooperative_groups::this_cluster().sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.new_lens[b] = skip ? L : L + n;
    if (skip) return;
    const int cols = a.p.units * a.p.layers;
    for (int c = blockIdx.x * 256 + threadIdx.x; c < cols; c += kCompactCtas * 256) {
        int u = c % a.p.units;
        const int layer = c / a.p.units, pool = pool_of(a.p, &u), w = a.p.u[pool];
        uint4* base = a.p.base[pool] + (size_t)layer * a.p.layer[pool] + u;
        for (int i0 = 0; i0 < n; i0 += kCompactBatch) {
            uint4 v[kCompactBatch];
#pragma unroll
            for (int e = 0; e < kCompactBatch; ++e)
                if (i0 + e < n && from[i0 + e] != to[i0 + e]) v[e] = base[(size_t)from[i0 + e] * w];
#pragma unroll
            for (int e = 0; e < kCompactBatch; ++e)
                if (i0 + e < n && from[i0 + e] != to[i0 + e]) base[(size_t)to[i0 + e] * w] = v[e];
        }
    }
}

}  // namespace

cudaError_t launch_pages_reserve(const PageArgs& a, cudaStream_t stream) {
    return launch_dependent(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
}

cudaError_t launch_pages_fork(const PoolArgs& p, const PageArgs& a, int sms, cudaStream_t stream) {
    const size_t smem = 2 * (size_t)a.n * sizeof(int);
    if (smem > 32768) {  // (beside 8 KB of its own)
        const cudaError_t e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * LRKV_MAX_PAGE_BATCH * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_dependent(fork_plan_kernel, dim3(1), dim3(kPlanThreads), smem, stream, a);
    if (e != cudaSuccess) return e;
    const long long pages = (long long)a.n * p.layers;
    const int most = (kBlockSize * p.units + kForkThreads - 1) / kForkThreads;
    const int parts = pages >= 2 * sms ? 1 : (int)(2 * sms / pages) < most ? (int)(2 * sms / pages) : most;
    return launch_dependent(fork_copy_kernel, dim3(a.n, p.layers, parts), dim3(kForkThreads), 0, stream, p, a);
}

cudaError_t launch_pages_free(const PageArgs& a, cudaStream_t stream) {
    return launch_dependent(free_kernel, dim3(a.n), dim3(256), 0, stream, a);
}

cudaError_t launch_pages_copy(const PoolArgs& src, const PoolArgs& dst, const int32_t* src_pages,
                              const int32_t* dst_pages, int n, int sms, uint32_t* status, cudaStream_t stream) {
    CopyArgs a{src, dst, src_pages, dst_pages, 0, 0, status};
    for (int p = 0; p < src.pools; ++p) a.parts += (int)((kBlockSize * src.u[p] * 16 + kPiece - 1) / kPiece);
    a.items = (long long)n * src.layers * a.parts;
    constexpr int smem = kStages * (int)kPiece + 128;
    const cudaError_t e = cudaFuncSetAttribute(copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(copy_kernel, dim3((unsigned)(a.items < 2 * sms ? a.items : 2 * sms)), dim3(32), smem, stream, a);
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream) {
    return launch_dependent(compact_kernel, dim3(kCompactCtas, a.batch), dim3(256), 0, stream, a);
}

}  // namespace lrkv
