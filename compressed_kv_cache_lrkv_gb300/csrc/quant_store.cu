// quant_store.cu -- a cache quantised as it is written, and read back.
//
// Each block of 32 values x_i of a token's row has one scale 2^k:
//     k = exponent(max |x_i|) - 6,   q_i = min(127, max(-127, rint(x_i / 2^k)))
// so the largest magnitude lands in [64, 128).  bf16 has 8 significant bits, so the division (a
// power of two) is exact, the largest quotient is 127.5, and every value is stored to within half
// a step: |x_i - q_i 2^k| <= 2^(k-1) <= max|x| 2^-7.  q_i 2^k has 7 significant bits and is
// exact in bf16, so reading back rounds nothing.
// Both directions move each value once: bound by memory (by the launch and one chain of loads for a
// decode step's few rows), as long as the arithmetic stays small: 65,536 rows of 2,304 values keep every
// issue slot of the GPU busy for half the time the memory takes.  So magnitudes are compared and limited
// two at a time as 16-bit integers, rounded by adding 1.5 2^23 (whose low mantissa byte then is the
// result), and widened two at a time in bf16.
// A thread keeps to sixteen consecutive values (32 bytes of bf16, 16 of the row) of one place of the row and
// walks over rows, the next row's loads in flight; a block spans a row (up to 8192 values), so few rows still
// spread over many SMs.  The two lanes of a block of 32 agree on its scale with a shuffle; the scale
// bytes of four blocks leave in one word.
// 65,536 rows of 2,304 values in random order, there and back: 164 us, 5.6 TB/s (of 6.8 measured for a copy);
// with eight values a thread 179 us (a third more instructions per value); with streaming loads 171 us, streaming
// stores too 183; with registers for full occupancy 183; two rows in flight 188, a warp per row 204.  In a
// graph 1,000 rows of 1,344 values take 5.3 us there and back, 16 rows (a decode step's) 3.9, with a warp per row 11.6;
// called one after the other from the host both take 14, the calls themselves.
#include "lrkv_internal.cuh"
#include "quant.cuh"
#include "quant.h"

namespace lrkv {

namespace {

constexpr int kMaxThreads = 512;

// Where the sixteen values of chunk c of a row lie.  Chunks are counted part after part, each part
// padded to whole blocks (two chunks), so chunk c belongs to scale byte c / 2.
struct Chunk {
    uint16_t* base;   // the part's pool, at the chunk's first value of token slot 0
    int width;        // values of the part per token
    int off;          // byte offset of the chunk in a quantised row
    bool lo, hi;      // its first and last eight values exist (else padding; parts are multiples of eight)
};
__device__ __forceinline__ Chunk chunk_at(const QuantStoreArgs& a, int c) {
    const QuantLayout& q = a.q;
    const int c1 = q.nb_sK * 2, c2 = c1 + q.nb_sV * 2, c3 = c2 + q.nb_z * 2, c4 = c3 + q.nb_z * 2;
    const int first = (c < c1 ? c : c < c2 ? c - c1 : c < c3 ? c - c2 : c - c3) * 16;
    uint16_t* pool = c < c1 ? a.sK : c < c2 ? a.sV : c < c3 ? a.zK : a.zV;
    const int width = c < c1 ? q.d_k : c < c2 ? q.d_h : q.HR;
    const int off = c < c1 ? 0 : c < c2 ? q.off_sV : c < c3 ? q.off_zK : q.off_zV;
    return {pool + first, width, off + first, c < c4 && first < width, c < c4 && first + 8 < width};
}
__host__ __device__ __forceinline__ int total_chunks(const QuantLayout& q) {
    return (q.nb_sK + q.nb_sV + 2 * q.nb_z) * 2;
}

// Slots of row i, (-1, -1) behind the last row.
__device__ __forceinline__ int2 load_slots(const QuantStoreArgs& a, int i) {
    return i < a.n ? make_int2(__ldg(a.bf_slots + i), __ldg(a.q_slots + i)) : make_int2(-1, -1);
}

// (two unsigned 16-bit maxima / minima)
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) { return __vminu2(a, b); }

// Sixteen values of a row -> its bytes and, from one lane in eight, scale bytes.
__device__ __forceinline__ void quantize_chunk(const QuantStoreArgs& a, const Chunk& ch, int c, int nc, const uint4 v[2],
                                               uint8_t* row, bool row_ok) {
    const int lane = threadIdx.x & 31;
    // the largest magnitude of the block as bf16 bits (their order is that of the values; a NaN or infinity
    // ends with exponent 255)
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t mag[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) mag[k] = w[k] & 0x7fff7fffu;
    uint32_t m2 = max2(max2(max2(mag[0], mag[1]), max2(mag[2], mag[3])), max2(max2(mag[4], mag[5]), max2(mag[6], mag[7])));
    m2 = max2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
    const uint32_t mx = max(m2 & 0xffffu, m2 >> 16);
    const int ex = (int)(mx >> 7);
    // scale byte e: scale 2^(e - 127); at least 1 (2^-126: smaller values are rounded to multiples of it),
    // 255 for a block with a NaN or infinity
    const int e = ex == 255 ? 255 : max(ex - 6, 1);
    // 2^-(e - 127): e is in [1, 248] for a finite block, so its exponent field 254 - e is in [6, 253]
    const float inv = __uint_as_float((uint32_t)(254 - min(e, 253)) << 23);
    // Only a quotient of 127.5, the largest magnitude with all mantissa bits set, rounds beyond 127: such
    // values take the next smaller mantissa, 127 exactly.
    const uint32_t top = ex >= 7 ? (mx & 0x7f80u) | 0x7eu : 0x7fffu;
    const uint32_t top2 = top | (top << 16);
    uint32_t out[4];
#pragma unroll
    for (int k2 = 0; k2 < 4; ++k2) {
        uint32_t t[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t x = min2(mag[2 * k2 + k], top2) | (w[2 * k2 + k] & 0x80008000u);
            // 1.5 2^23 + 128 + q, q rounded to nearest even: the low byte is q + 128
            t[2 * k] = __float_as_uint(fmaf(bf16lo(x), inv, 12583040.0f));
            t[2 * k + 1] = __float_as_uint(fmaf(bf16hi(x), inv, 12583040.0f));
        }
        out[k2] = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
        out[k2] = ex == 255 ? 0x80808080u : out[k2];
    }
    uint32_t sc = (uint32_t)e << (8 * ((lane >> 1) & 3));
    sc |= __shfl_xor_sync(0xffffffffu, sc, 2);
    sc |= __shfl_xor_sync(0xffffffffu, sc, 4);
    if (!row_ok) return;
    // (a chunk that ends with padding writes zeros there: parts of a row are padded to 16)
    if (ch.lo) *reinterpret_cast<uint4*>(row + ch.off) = make_uint4(out[0], out[1], out[2], out[3]);
    // (the word may end in the row's padding: the scales start on 16 bytes, and so does the next row)
    if ((lane & 7) == 0 && c < nc) *reinterpret_cast<uint32_t*>(row + a.q.off_sc + (c >> 1)) = sc;
}

__device__ __forceinline__ uint4 dequantize8(uint32_t x, uint32_t y, uint32_t s2) {
    const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
    return make_uint4(bytes_bf16(__byte_perm(x, 0u, 0x4140), s), bytes_bf16(__byte_perm(x, 0u, 0x4342), s),
                      bytes_bf16(__byte_perm(y, 0u, 0x4140), s), bytes_bf16(__byte_perm(y, 0u, 0x4342), s));
}

// grid (blocks over rows, row chunks / threads): rows blockIdx.x, + gridDim.x, ...; slots are read one
// row ahead of the loads they address.
template <bool WRITE>
__global__ void __launch_bounds__(kMaxThreads) store_kernel(const QuantStoreArgs a) {
    const int nc = total_chunks(a.q);
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    const Chunk ch = chunk_at(a, c);
    const int step = gridDim.x;
    // The loads of the row with these slots: *to becomes the slot that is written (-1: none), v its values
    // (dequantised: v[0] the bytes, v[1].x the scale byte).  Slots out of range are reported.
    auto load = [&](int2 s, long long* to, uint4* v) {
        bool good = s.x >= 0 && s.y >= 0;
        if (good && (s.x >= a.bf_nslots || s.y >= a.q_nslots)) {
            if (threadIdx.x == 0) set_status(a.status, LRKV_DEV_BAD_SLOT);
            good = false;
        }
        *to = !good ? -1 : WRITE ? s.y : s.x;
        v[0] = v[1] = make_uint4(0, 0, 0, 0);
        if (!good || !ch.lo) return;
        if (WRITE) {
            const uint4* src = reinterpret_cast<const uint4*>(ch.base + (long long)s.x * ch.width);
            v[0] = __ldg(src);
            if (ch.hi) v[1] = __ldg(src + 1);
        } else {
            const uint8_t* row = a.rows + (long long)s.y * a.q.row_bytes;
            v[0] = *reinterpret_cast<const uint4*>(row + ch.off);
            v[1].x = row[a.q.off_sc + (c >> 1)];
        }
    };
    int r = blockIdx.x;
    long long to;
    uint4 v[2];
    load(load_slots(a, r), &to, v);
    int2 next = load_slots(a, r + step);
    for (; r < a.n; r += step) {
        const long long at = to;
        const uint4 x[2] = {v[0], v[1]};
        load(next, &to, v);
        next = load_slots(a, r + 2 * step);
        if (WRITE) {
            quantize_chunk(a, ch, c, nc, x, a.rows + at * a.q.row_bytes, at >= 0);
        } else if (at >= 0 && ch.lo) {
            uint4* dst = reinterpret_cast<uint4*>(ch.base + at * ch.width);
            const uint32_t s2 = scale_bf16x2(x[1].x);
            dst[0] = dequantize8(x[0].x, x[0].y, s2);
            if (ch.hi) dst[1] = dequantize8(x[0].z, x[0].w, s2);
        }
    }
}

template <bool WRITE>
cudaError_t launch_store(const QuantStoreArgs& a, int sms, cudaStream_t stream) {
    const int nc = total_chunks(a.q);
    const int ny = (nc + kMaxThreads - 1) / kMaxThreads;
    const int threads = ((nc + ny - 1) / ny + 31) & ~31;
    // some five waves of blocks: with 2048 threads per SM 203 us on the case above, with 16384 169.  (Rows are
    // counted up to n + 2 gridDim.x, below 2^31.)
    const int most = (int)((long long)sms * 8192 / (threads * ny)) + 1;
    store_kernel<WRITE><<<dim3(a.n < most ? a.n : most, ny), threads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_quantize(const QuantStoreArgs& a, int sms, cudaStream_t stream) {
    return launch_store<true>(a, sms, stream);
}

cudaError_t launch_cache_dequantize(const QuantStoreArgs& a, int sms, cudaStream_t stream) {
    return launch_store<false>(a, sms, stream);
}

}  // namespace lrkv
