// rope.cu -- rotation of part of the heads of rows: y = m R(pos f_i) x on pairs of neighbours or of halves.
//
// The angle pos f_i modulo a turn is an integer product: f_i / 2 pi as a fraction of a turn in 64 bits times the
// position, modulo 2^64, is exact to |pos| 2^-64 of a turn (2^-33 at the largest), where a product in fp32 would be
// off by whole turns from some 2^24 positions on and the narrow FP64 pipe would cost more than the memory.  The
// quadrant is its two leading bits (rounded to nearest); the rest, at most an eighth of a turn, goes to fp32 (2^-28 of
// a turn) and through the Taylor polynomials of sine and cosine.
#include "draft.h"
#include "lrkv_internal.cuh"

namespace lrkv {

namespace {

// Cosine and sine of 2 pi f / 2^64.  |x| <= pi / 4; the first term left out is below 2e-9 (sine), 2e-9 (cosine).
__device__ __forceinline__ void cos_sin_turn(unsigned long long f, float& c, float& s) {
    const unsigned long long r = f + (1ull << 61);
    const unsigned q = (unsigned)(r >> 62);
    const long long rest = (long long)(f - ((unsigned long long)q << 62));  // [-2^61, 2^61)
    const float x = (float)(int)(rest >> 30) * (6.283185307179586f / 17179869184.0f);  // / 2^34
    const float x2 = x * x;
    float sp = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
    sp = fmaf(x2, sp, 8.3333333e-3f);
    sp = fmaf(x2, sp, -1.6666667e-1f);
    sp = fmaf(x * x2, sp, x);
    float cp = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
    cp = fmaf(x2, cp, -1.3888889e-3f);
    cp = fmaf(x2, cp, 4.1666667e-2f);
    cp = fmaf(x2, cp, -0.5f);
    cp = fmaf(x2, cp, 1.0f);
    c = q & 1 ? sp : cp;
    s = q & 1 ? cp : sp;
    if (q == 1 || q == 2) c = -c;
    if (q >= 2) s = -s;
}

// N consecutive values of a row, as fp32: N = 4 or 8, the address a multiple of N elements.
template <int N>
struct Vals {
    float v[N];
};
template <int N>
__device__ __forceinline__ Vals<N> load(const uint16_t* p) {
    Vals<N> r;
    if constexpr (N == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[2 * i] = bf16lo(w[i]), r.v[2 * i + 1] = bf16hi(w[i]);
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        r.v[0] = bf16lo(x.x), r.v[1] = bf16hi(x.x), r.v[2] = bf16lo(x.y), r.v[3] = bf16hi(x.y);
    }
    return r;
}
template <int N>
__device__ __forceinline__ Vals<N> load(const float* p) {
    Vals<N> r;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 x = reinterpret_cast<const float4*>(p)[i];
        r.v[4 * i] = x.x, r.v[4 * i + 1] = x.y, r.v[4 * i + 2] = x.z, r.v[4 * i + 3] = x.w;
    }
    return r;
}
template <int N>
__device__ __forceinline__ void store(uint16_t* p, const Vals<N>& r) {
    if constexpr (N == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]),
                                                  pack_bf16x2(r.v[4], r.v[5]), pack_bf16x2(r.v[6], r.v[7]));
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]));
}
template <int N>
__device__ __forceinline__ void store(float* p, const Vals<N>& r) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(r.v[4 * i], r.v[4 * i + 1], r.v[4 * i + 2], r.v[4 * i + 3]);
}

// A block: x units (4 pairs, or 8 values that are copied) of a head, y heads, z rows; a thread takes its unit of
// every blockDim.y-th head, HB of them in flight, with the sines of its four pairs formed once.
// HALF: a unit's pairs are 4 values of the lower half and 4 of the upper one; else 8 neighbouring values.
template <typename T, bool HALF, int HB>
__global__ void __launch_bounds__(512) rope_kernel(const __grid_constant__ RopeArgs a) {
    const int un = threadIdx.x, rot = a.plan.d_rot / 8;
    // units: first the rotated ones, then 8 copied values each, those before `begin` and those behind the part
    const bool turns = un < rot;
    int at0, at1;
    if (turns) {
        at0 = a.begin + (HALF ? un * 4 : un * 8);
        at1 = HALF ? at0 + a.plan.d_rot / 2 : at0 + 4;
    } else {
        at0 = (un - rot) * 8;
        if (at0 >= a.begin) at0 += a.plan.d_rot;
        at1 = at0 + 4;
    }
    const T* xb = static_cast<const T*>(a.x);
    T* yb = static_cast<T*>(a.y);
    const int hstep = blockDim.y * gridDim.y;
    unsigned long long speed[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) speed[k] = turns ? a.plan.turn[un * 4 + k] : 0;
    for (long long i = (long long)blockIdx.x * blockDim.z + threadIdx.z; i < a.n;
         i += (long long)gridDim.x * blockDim.z) {
        const long long xr = a.x_index ? a.x_index[i] : i, yr = a.y_index ? a.y_index[i] : i;
        if (xr < 0 || yr < 0) continue;
        if (xr >= a.x_rows || yr >= a.y_rows) {
            set_status(a.status, LRKV_DEV_BAD_SLOT);
            continue;
        }
        float c[4], s[4];
        if (turns) {
            const long long pos = a.positions[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cos_sin_turn((unsigned long long)pos * speed[k], c[k], s[k]);
                c[k] *= a.plan.magnitude;
                s[k] *= a.transpose ? -a.plan.magnitude : a.plan.magnitude;
            }
        }
        const T* xp = xb + xr * a.x_row;
        T* yp = yb + yr * a.y_row;
        for (int h = blockIdx.y * blockDim.y + threadIdx.y; h < a.heads; h += hstep * HB) {
            Vals<8> v[HB];
#pragma unroll
            for (int b = 0; b < HB; ++b) {
                if (h + b * hstep >= a.heads) break;
                const T* p = xp + (h + b * hstep) * a.x_head;
                if (HALF && turns) {
                    const Vals<4> lo = load<4>(p + at0), hi = load<4>(p + at1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[b].v[k] = lo.v[k], v[b].v[4 + k] = hi.v[k];
                } else {
                    v[b] = load<8>(p + at0);
                }
            }
#pragma unroll
            for (int b = 0; b < HB; ++b) {
                if (h + b * hstep >= a.heads) break;
                T* p = yp + (h + b * hstep) * a.y_head;
                if (!turns) {
                    store<8>(p + at0, v[b]);
                    continue;
                }
                Vals<8> o;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i0 = HALF ? k : 2 * k, i1 = HALF ? 4 + k : 2 * k + 1;
                    const float x0 = v[b].v[i0], x1 = v[b].v[i1];
                    o.v[i0] = fmaf(x0, c[k], -(x1 * s[k]));
                    o.v[i1] = fmaf(x0, s[k], x1 * c[k]);
                }
                if (HALF) {
                    Vals<4> lo, hi;
#pragma unroll
                    for (int k = 0; k < 4; ++k) lo.v[k] = o.v[k], hi.v[k] = o.v[4 + k];
                    store<4>(p + at0, lo);
                    store<4>(p + at1, hi);
                } else {
                    store<8>(p + at0, o);
                }
            }
        }
    }
}

template <typename T, bool HALF>
cudaError_t launch_t(const RopeArgs& a, int sms, cudaStream_t stream) {
    const int units = a.in_place ? a.plan.d_rot / 8 : a.width / 8;
    // a head a thread while that fits on the GPU at once, else four in flight and the sines shared by all
    const bool few = (long long)a.n * a.heads * units <= (long long)sms * 2048;
    int ny = 1;
    while (ny * (few ? 1 : 4) < a.heads && units * ny * 2 <= 256) ny *= 2;
    int nz = 1;
    while (units * ny * nz * 2 <= 256 && nz < 64) nz *= 2;
    const long long rows = ((long long)a.n + nz - 1) / nz;
    const unsigned gx = (unsigned)(rows < (1 << 20) ? rows : 1 << 20);
    const unsigned gy = few ? (unsigned)((a.heads + ny - 1) / ny) : 1u;
    const dim3 grid(gx, gy), block(units, ny, nz);
    if (few)
        rope_kernel<T, HALF, 1><<<grid, block, 0, stream>>>(a);
    else
        rope_kernel<T, HALF, 4><<<grid, block, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool fp32, int sms, cudaStream_t stream) {
    if (a.plan.layout == LRKV_ROPE_HALF)
        return fp32 ? launch_t<float, true>(a, sms, stream) : launch_t<uint16_t, true>(a, sms, stream);
    return fp32 ? launch_t<float, false>(a, sms, stream) : launch_t<uint16_t, false>(a, sms, stream);
}

}  // namespace lrkv
