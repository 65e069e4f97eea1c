// pages.cu -- pages of the cache: taken, shared, copied, compacted and given back on the device.
//
// The only state is a count per page (refs) beside the block table; a free page is one whose count is 0, and free
// pages are taken lowest first.  Counts change by atomic additions, whose order does not change the outcome, and taken
// pages go to the requests in the order of the call by a prefix sum, so results do not depend on timing.
#include <cooperative_groups.h>

#include "draft.h"
#include "lrkv_internal.cuh"

namespace lrkv {

namespace {

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

// need[0..n) (shared memory): pages asked for by request i -> exclusive prefix sums; returns their total.
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
#pragma unroll
        for (int k = 0; k < kPerThread; k += 4) {
            if (p + k + 4 <= num_blocks) {
                const int4 r = __ldcg(reinterpret_cast<const int4*>(refs + p + k));
                free |= (uint32_t)(r.x == 0) << k | (uint32_t)(r.y == 0) << (k + 1) | (uint32_t)(r.z == 0) << (k + 2) |
                        (uint32_t)(r.w == 0) << (k + 3);
            } else {
                for (int e = k; e < k + 4; ++e)
                    if (p + e < num_blocks && __ldcg(refs + p + e) == 0) free |= 1u << e;
            }
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

// need[0..n) granted from the free pages, whole requests or none, in order; afterwards need holds exclusive
// prefix sums of what is granted.  Returns the total; refused(i) for requests that do not fit.
template <class F>
__device__ int grant(int* need, int n, const int32_t* refs, int num_blocks, int* warp_sums, F&& refused) {
    int total = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        int t;
        block_scan(i0 + (int)threadIdx.x < n ? need[i0 + threadIdx.x] : 0, warp_sums, &t);
        total += t;
    }
    const int have = search_free(refs, num_blocks, total, warp_sums, [](int, int) {});
    if (have < total) {
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
    return prefix_of_needs(need, n, warp_sums);
}

__device__ __forceinline__ int pages_of(long long tokens) { return (int)((tokens + kBlockSize - 1) / kBlockSize); }

__device__ __forceinline__ void give_back(int32_t* refs, int num_blocks, int page, uint32_t* status) {
    if (page >= num_blocks) {
        set_status(status, LRKV_DEV_BAD_BLOCK);
    } else if (atomicSub(refs + page, 1) <= 0) {
        atomicAdd(refs + page, 1);
        set_status(status, LRKV_DEV_BAD_INDEX);
    }
}

// ---------------------------------------------------------------- reserve: one block
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const PageArgs a) {
    __shared__ int need[LRKV_MAX_PAGE_BATCH], warp_sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a warp per sequence: its first empty entry from the page of its length on
    for (int b = warp; b < a.batch; b += kPlanThreads / 32) {
        const int L = a.lens[b], add = a.b[b];
        const int want = L >= 0 && add >= 0 ? pages_of((long long)L + add) : -1;
        int held = want;
        if (want < 0 || want > a.max_pages) {
            if (lane == 0) set_status(a.status, LRKV_DEV_BAD_SEQLEN);
            held = want;
        } else {
            for (int k = pages_of(L); k < want; k += 32) {
                const bool empty = k + lane < want && a.table[(size_t)b * a.max_pages + k + lane] < 0;
                const unsigned m = __ballot_sync(0xffffffffu, empty);
                if (m) {
                    held = k + __ffs(m) - 1;
                    break;
                }
            }
        }
        if (lane == 0) need[b] = want - held;
    }
    __syncthreads();
    const int total = grant(need, a.batch, a.refs, a.num_blocks, warp_sums,
                            [&](int) { set_status(a.status, LRKV_DEV_NO_PAGES); });
    search_free(a.refs, a.num_blocks, total, warp_sums, [&](int page, int rank) {
        const int b = owner(need, a.batch, rank);
        // the granted entries are the last ones of what the sequence asked for
        const int granted = (b + 1 < a.batch ? need[b + 1] : total) - need[b];
        const int last = pages_of((long long)a.lens[b] + a.b[b]);
        a.table[(size_t)b * a.max_pages + last - granted + (rank - need[b])] = page;
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

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PageArgs a) {
    // need: pages asked for, then their prefix sums; full: the full pages that a fork passes on (-1: left out)
    __shared__ int need[LRKV_MAX_PAGE_BATCH], warp_sums[32];
    extern __shared__ int full[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = warp; i < a.n; i += kPlanThreads / 32) {
        const uint32_t bad = fork_refused(a, i, lane, 32, [](uint32_t x) { return __reduce_or_sync(0xffffffffu, x); });
        if (lane == 0) {
            if (bad) set_status(a.status, bad & LRKV_DEV_BAD_INDEX ? LRKV_DEV_BAD_INDEX : bad);
            const int L = bad ? 0 : a.lens[a.a[i]];
            full[i] = bad ? -1 : L / kBlockSize;
            need[i] = L % kBlockSize != 0;
        }
    }
    __syncthreads();
    // what the children held goes back first
    for (int i = warp; i < a.n; i += kPlanThreads / 32) {
        if (full[i] < 0) continue;
        int32_t* row = a.table + (size_t)a.b[i] * a.max_pages;
        for (int k = lane; k < a.max_pages; k += 32) {
            const int page = row[k];
            if (page >= 0) give_back(a.refs, a.num_blocks, page, a.status);
            row[k] = -1;
        }
    }
    __threadfence();
    __syncthreads();
    const int total = grant(need, a.n, a.refs, a.num_blocks, warp_sums, [&](int i) {
        set_status(a.status, LRKV_DEV_NO_PAGES);
        full[i] = -2;  // the child stays empty
    });
    search_free(a.refs, a.num_blocks, total, warp_sums, [&](int page, int rank) {
        const int i = owner(need, a.n, rank);
        a.table[(size_t)a.b[i] * a.max_pages + full[i]] = page;
        a.refs[page] = 1;
    });
    __syncthreads();
    for (int i = warp; i < a.n; i += kPlanThreads / 32) {
        if (full[i] == -1) continue;
        const int p = a.a[i], c = a.b[i];
        for (int k = lane; k < full[i]; k += 32) {
            const int page = a.table[(size_t)p * a.max_pages + k];
            a.table[(size_t)c * a.max_pages + k] = page;
            atomicAdd(a.refs + page, 1);
        }
        if (lane == 0) a.lens[c] = full[i] < 0 ? 0 : a.lens[p];
    }
}

// 16-byte unit `u` of a token row over all pools: the pool, and the unit within its row.
__device__ __forceinline__ int pool_of(const PoolArgs& p, int* u) {
    int k = 0;
    while (k + 1 < p.pools && *u >= p.u[k]) *u -= p.u[k++];
    return k;
}

// Rows of the children's last pages: grid (units in pieces, forks, layers).
__global__ void __launch_bounds__(256) fork_copy_kernel(const PoolArgs p, const PageArgs a) {
    const int i = blockIdx.y;
    if (fork_refused(a, i, threadIdx.x, 256, [](uint32_t x) { return (uint32_t)__syncthreads_or(x != 0); })) return;
    const int par = a.a[i], c = a.b[i], L = a.lens[c];  // (0 where no page was left for the child)
    if (L % kBlockSize == 0) return;
    const int k = L / kBlockSize, from = a.table[(size_t)par * a.max_pages + k], to = a.table[(size_t)c * a.max_pages + k];
    const int rows = L % kBlockSize, n = rows * p.units;
    for (int e = blockIdx.x * 256 + threadIdx.x; e < n; e += gridDim.x * 256) {
        int pool = 0, u = e;
        while (pool + 1 < p.pools && u >= p.u[pool] * rows) u -= p.u[pool++] * rows;
        uint4* b = p.base[pool] + (size_t)blockIdx.z * p.layer[pool];
        const size_t page = (size_t)kBlockSize * p.u[pool];
        b[to * page + u] = b[from * page + u];
    }
}

// ---------------------------------------------------------------- free: a block per sequence
__global__ void __launch_bounds__(256) free_kernel(const PageArgs a) {
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
        if (page >= 0) give_back(a.refs, a.num_blocks, page, a.status);
    }
    if (threadIdx.x == 0) {
        const int L = a.lens[b];
        a.lens[b] = L < keep ? L : keep;
    }
}

// ---------------------------------------------------------------- copy of whole pages
constexpr int kCopyUnroll = 4;
__global__ void __launch_bounds__(256) copy_kernel(const PoolArgs src, const PoolArgs dst, const int32_t* from,
                                                   const int32_t* to, const int pieces, uint32_t* status) {
    const int i = blockIdx.x / pieces, piece = blockIdx.x - i * pieces;
    const int f = from[i], t = to[i];
    if (f < 0 || t < 0) return;
    if (f >= src.num_blocks || t >= dst.num_blocks) {
        if (threadIdx.x == 0) set_status(status, LRKV_DEV_BAD_BLOCK);
        return;
    }
    const int n = kBlockSize * src.units;
    uint4 v[kCopyUnroll];
    uint4* out[kCopyUnroll];
#pragma unroll
    for (int e = 0; e < kCopyUnroll; ++e) {
        int u = (piece * kCopyUnroll + e) * 256 + threadIdx.x;
        out[e] = nullptr;
        if (u >= n) continue;
        int p = 0;
        while (p + 1 < src.pools && u >= kBlockSize * src.u[p]) u -= kBlockSize * src.u[p++];
        const size_t page = (size_t)kBlockSize * src.u[p];
        v[e] = __ldcs(src.base[p] + (size_t)blockIdx.y * src.layer[p] + f * page + u);
        out[e] = dst.base[p] + (size_t)blockIdx.y * dst.layer[p] + t * page + u;
    }
#pragma unroll
    for (int e = 0; e < kCopyUnroll; ++e)
        if (out[e]) __stcs(out[e], v[e]);
}

// ---------------------------------------------------------------- compact: a cluster per sequence
// Row i moves from L + path[i] >= L + i down; a path increases, so a row is read before it is written if every thread
// takes its 16-byte column through the rows in order (eight rows in flight: the sources of the next eight lie behind
// all rows written so far).  The length may be updated in place once every block of the cluster has read it.
constexpr int kCompactCtas = 8, kCompactBatch = 8;
__global__ void __cluster_dims__(kCompactCtas, 1, 1) __launch_bounds__(256) compact_kernel(const CompactArgs a) {
    __shared__ int from[1024], to[1024];
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
    reserve_kernel<<<1, kPlanThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PoolArgs& p, const PageArgs& a, cudaStream_t stream) {
    const int smem = a.n * (int)sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               LRKV_MAX_PAGE_BATCH * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    fork_plan_kernel<<<1, kPlanThreads, smem, stream>>>(a);
    const int pieces = (kBlockSize * p.units + 256 * 8 - 1) / (256 * 8);
    fork_copy_kernel<<<dim3(pieces, a.n, p.layers), 256, 0, stream>>>(p, a);
    return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageArgs& a, cudaStream_t stream) {
    free_kernel<<<a.n, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PoolArgs& src, const PoolArgs& dst, const int32_t* src_pages,
                              const int32_t* dst_pages, int n, uint32_t* status, cudaStream_t stream) {
    const int pieces = (kBlockSize * src.units + 256 * kCopyUnroll - 1) / (256 * kCopyUnroll);
    copy_kernel<<<dim3((unsigned)pieces * n, src.layers), 256, 0, stream>>>(src, dst, src_pages, dst_pages, pieces,
                                                                            status);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream) {
    compact_kernel<<<dim3(kCompactCtas, a.batch), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace lrkv
