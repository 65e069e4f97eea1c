// rope.cu -- rotation of part of the heads of rows: y = m R(pos f_i) x on pairs of neighbours or of halves.
//
// The angle pos f_i modulo a turn is an integer product: f_i / 2 pi as a fraction of a turn in 64 bits times the
// position, modulo 2^64, is exact to |pos| 2^-64 of a turn (2^-33 at the largest), where a product in fp32 would be
// off by whole turns from some 2^24 positions on and the narrow FP64 pipe would cost more than the memory.  The
// quadrant is its two leading bits (rounded to nearest); the rest, at most an eighth of a turn, goes to fp32 (2^-28 of
// a turn) and through the Taylor polynomials of sine and cosine.
#include "draft.h"
#include "lrkv_internal.cuh"
#include "tile_attn.cuh"

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

// Eight values of a head as they lie in memory, four from p + at0 and four from p + at1.
template <typename T>
struct Raw {
    uint32_t r[2 * sizeof(T)];
};
template <bool HALF>
__device__ __forceinline__ void get(Raw<uint16_t>& v, const uint16_t* p, int at0, int at1) {
    if (HALF) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + at0), y = *reinterpret_cast<const uint2*>(p + at1);
        v.r[0] = x.x, v.r[1] = x.y, v.r[2] = y.x, v.r[3] = y.y;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p + at0);
        v.r[0] = x.x, v.r[1] = x.y, v.r[2] = x.z, v.r[3] = x.w;
    }
}
template <bool HALF>
__device__ __forceinline__ void put(const Raw<uint16_t>& v, uint16_t* p, int at0, int at1) {
    if (HALF) {
        *reinterpret_cast<uint2*>(p + at0) = make_uint2(v.r[0], v.r[1]);
        *reinterpret_cast<uint2*>(p + at1) = make_uint2(v.r[2], v.r[3]);
    } else {
        *reinterpret_cast<uint4*>(p + at0) = make_uint4(v.r[0], v.r[1], v.r[2], v.r[3]);
    }
}
template <bool HALF>
__device__ __forceinline__ void get(Raw<float>& v, const float* p, int at0, int at1) {
    const uint4 x = *reinterpret_cast<const uint4*>(p + at0), y = *reinterpret_cast<const uint4*>(p + at1);
    v.r[0] = x.x, v.r[1] = x.y, v.r[2] = x.z, v.r[3] = x.w, v.r[4] = y.x, v.r[5] = y.y, v.r[6] = y.z, v.r[7] = y.w;
}
template <bool HALF>
__device__ __forceinline__ void put(const Raw<float>& v, float* p, int at0, int at1) {
    *reinterpret_cast<uint4*>(p + at0) = make_uint4(v.r[0], v.r[1], v.r[2], v.r[3]);
    *reinterpret_cast<uint4*>(p + at1) = make_uint4(v.r[4], v.r[5], v.r[6], v.r[7]);
}
__device__ __forceinline__ void widen(const Raw<uint16_t>& v, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(v.r[i]), x[2 * i + 1] = bf16hi(v.r[i]);
}
__device__ __forceinline__ void widen(const Raw<float>& v, float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v.r[i]);
}
__device__ __forceinline__ void narrow(const float* x, Raw<uint16_t>& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.r[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float* x, Raw<float>& v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.r[i] = __float_as_uint(x[i]);
}

// A block: x units of a head (four pairs, or eight values that are copied), y heads, z rows; a thread takes its unit of
// RB rows and every blockDim.y-th head, HB of them, RB x HB units in flight at once and before the sines are formed
// (once for all heads of a row).  HALF: a unit's pairs are four values of the lower half and four of the upper one;
// else eight neighbouring values.  Bound by the memory: what carries it is bytes in flight, so the values wait in their
// own type.  8,192 rows x 32 heads of 192: 37 us (30 at the copy rate);
// with one unit after another behind the position's load 98.
template <typename T, bool HALF, int RB, int HB>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
    const int un = threadIdx.x, rot = a.plan.d_rot / 8;
    // units: first the rotated ones, then eight copied values each, those before `begin` and those behind the part
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
    const long long rstep = (long long)gridDim.x * blockDim.z;
    pdl_wait();  // (launched while the kernel before it on the stream still runs)
    pdl_trigger();
    for (long long i0 = (long long)blockIdx.x * blockDim.z + threadIdx.z; i0 < a.n; i0 += rstep * RB) {
        const T* xp[RB];
        T* yp[RB];
        int pos[RB];
        bool ok[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const long long i = i0 + r * rstep;
            ok[r] = i < a.n;
            long long xr = i, yr = i;
            if (ok[r] && a.x_index) xr = a.x_index[i];
            if (ok[r] && a.y_index) yr = a.y_index[i];
            if (ok[r] && xr >= 0 && yr >= 0 && (xr >= a.x_rows || yr >= a.y_rows)) set_status(a.status, LRKV_DEV_BAD_SLOT);
            pos[r] = ok[r] ? a.positions[i] : 0;
            ok[r] = ok[r] && xr >= 0 && yr >= 0 && xr < a.x_rows && yr < a.y_rows;
            xp[r] = xb + xr * a.x_row;
            yp[r] = yb + yr * a.y_row;
        }
        for (int h0 = blockIdx.y * blockDim.y + threadIdx.y; h0 < a.heads; h0 += hstep * HB) {
            Raw<T> v[RB][HB];
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int b = 0; b < HB; ++b)
                    if (ok[r] && h0 + b * hstep < a.heads) get<HALF>(v[r][b], xp[r] + (h0 + b * hstep) * a.x_head, at0, at1);
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                float c[4], s[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    cos_sin_turn((unsigned long long)(long long)pos[r] * speed[k], c[k], s[k]);
                    c[k] *= a.plan.magnitude;
                    s[k] *= a.transpose ? -a.plan.magnitude : a.plan.magnitude;
                }
#pragma unroll
                for (int b = 0; b < HB; ++b) {
                    if (!ok[r] || h0 + b * hstep >= a.heads) continue;
                    if (turns) {
                        float x[8], o[8];
                        widen(v[r][b], x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int e0 = HALF ? k : 2 * k, e1 = HALF ? 4 + k : 2 * k + 1;
                            o[e0] = fmaf(x[e0], c[k], -(x[e1] * s[k]));
                            o[e1] = fmaf(x[e0], s[k], x[e1] * c[k]);
                        }
                        narrow(o, v[r][b]);
                    }
                    put<HALF>(v[r][b], yp[r] + (h0 + b * hstep) * a.y_head, at0, at1);
                }
            }
        }
    }
}

template <typename T, bool HALF>
cudaError_t launch_t(const RopeArgs& a, int sms, cudaStream_t stream) {
    const int units = a.in_place ? a.plan.d_rot / 8 : a.width / 8;
    // One unit a thread up to 512 of them for an SM (latency counts), else four rows of one or two heads, or four
    // (fp32) or eight heads of a row.  In a graph, us, one unit | several: 1 head of 64, 500 an SM 2.4 | 3.1, 700
    // 3.6 | 3.2, 9,600 24 | 20; 8 heads of 128, 64 turned, 500 2.4 | 2.6, 700 3.6 | 2.8; 32 heads of 192, 300 2.2 | 2.5,
    // 500 3.3 | 2.6, 9,600 23 | 10.5; fp32, 8 heads of 128, 500 3.1 | 3.2, 700 4.2 | 3.5.  2,400 an SM by rows | by heads:
    // 2 heads of 64 7.1 | 8.0, 3 of 128 9.4 | 7.4; fp32, 2 of 128 8.9 | 9.1, 3 of 64 9.0 | 7.5.
    const bool few = (long long)a.n * a.heads * units <= (long long)sms * 512;
    constexpr int HB = sizeof(T) == 2 ? 8 : 4;
    const int rb = few || a.heads >= 3 ? 1 : 4, hb = few || a.heads < 3 ? 1 : HB;
    int ny = 1;
    while (ny * hb < a.heads && units * ny * 2 <= 256) ny *= 2;
    int nz = 1;
    while (units * ny * nz * 2 <= 256 && nz < 64) nz *= 2;
    const long long rows = ((long long)a.n + nz * rb - 1) / (nz * rb);
    const unsigned gx = (unsigned)(rows < (1 << 20) ? rows : 1 << 20);
    const unsigned gy = hb == 1 ? (unsigned)((a.heads + ny - 1) / ny) : 1u;
    const dim3 grid(gx, gy), block(units, ny, nz);
    if (rb == 4) return launch_dependent(rope_kernel<T, HALF, 4, 1>, grid, block, 0, stream, a);
    if (hb == 1) return launch_dependent(rope_kernel<T, HALF, 1, 1>, grid, block, 0, stream, a);
    return launch_dependent(rope_kernel<T, HALF, 1, HB>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool fp32, int sms, cudaStream_t stream) {
    if (a.plan.layout == LRKV_ROPE_HALF)
        return fp32 ? launch_t<float, true>(a, sms, stream) : launch_t<uint16_t, true>(a, sms, stream);
    return fp32 ? launch_t<float, false>(a, sms, stream) : launch_t<uint16_t, false>(a, sms, stream);
}

}  // namespace lrkv
