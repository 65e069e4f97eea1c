// tile_attn.cuh -- parts shared by the scans that treat heads x queries as one 128-row attention tile on tcgen05
// (prefix.cu, tree.cu).
#pragma once

#include "kernels.h"
#include "lrkv_internal.cuh"

namespace lrkv {

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Shared-memory operand tiles of 64 bf16 columns, 128-byte swizzle: K-major, and MN-major with the next 64 columns
// 8 KB on.
__device__ __forceinline__ uint64_t kdesc128(uint32_t a) { return sdesc(a, 16, 1024, 2); }
__device__ __forceinline__ uint64_t mndesc128(uint32_t a) { return sdesc(a, 8192, 1024, 2); }

// Shared-memory descriptors in two halves, the upper one (strides, swizzle) a constant: MMAs whose TMEM addresses and
// upper halves are constants leave their thread one operand to bring into a uniform register.
constexpr uint32_t desc_upper(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | (1u << 14) | (layout << 29); }
__device__ __forceinline__ uint32_t desc_lower(uint32_t smem_addr, uint32_t lbo) {
    return ((smem_addr >> 4) & 0x3FFFu) | ((lbo >> 4) & 0x3FFFu) << 16;
}
// D (TMEM) (+)= A (TMEM, or shared memory) . B (shared memory), bf16, fp32 sums.
template <uint32_t B_UPPER>
__device__ __forceinline__ void mma_ts_h(uint32_t d, uint32_t a, uint32_t b_lower, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lower), "n"(B_UPPER), "r"(idesc), "r"(accumulate)
        : "memory");
}
template <uint32_t A_UPPER, uint32_t B_UPPER>
__device__ __forceinline__ void mma_ss_h(uint32_t d, uint32_t a_lower, uint32_t b_lower, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lower), "n"(A_UPPER), "r"(b_lower), "n"(B_UPPER), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Wait of a role, with the call's limit, and one for what the block has in flight, with the full limit.
__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, const DecodeArgs& d) {
    const bool ok = mbar_look_wait(bar, parity, d.status, d.wait_ns);
    return __all_sync(0xffffffffu, ok);
}
// wait_role for a role that one thread plays: the stop flag and the timer only while it has to wait.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, const DecodeArgs& d, volatile int* stop) {
    if (mbar_test(bar, parity)) return true;
    const bool nap = d.wait_ns == kWaitLimitNs;
    if (nap && (mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (nap ? mbar_try_wait(bar, parity) : mbar_test(bar, parity)) return true;
        if (*stop) return false;
        if (((it & 255u) == 0 || !nap) && globaltimer_ns() - t0 > d.wait_ns) {
            set_status(d.status, LRKV_DEV_TIMEOUT);
            return false;
        }
    }
}
// The same for the 32 threads of a warp together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const DecodeArgs& d, volatile int* stop) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_one(bar, parity, d, stop));
}
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, uint32_t* status) {
    mbar_wait(bar, parity, status);
    __syncwarp();
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x4(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}

// Pairs of fp32 values in one register pair, and what works on both at once.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// max(a, b, c), NaN where one of them is one.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// max(a, b), NaN where either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// n (a multiple of 8) products of bf16 a with bf16 b, or of fp32 a, summed in fp32.
__device__ __forceinline__ float dot8(const uint16_t* a, const uint16_t* b, int n) {
    float s = 0.f;
#pragma unroll 1
    for (int i = 0; i < n; i += 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(a + i), y = *reinterpret_cast<const uint4*>(b + i);
        s = fmaf(bf16lo(x.x), bf16lo(y.x), fmaf(bf16hi(x.x), bf16hi(y.x), s));
        s = fmaf(bf16lo(x.y), bf16lo(y.y), fmaf(bf16hi(x.y), bf16hi(y.y), s));
        s = fmaf(bf16lo(x.z), bf16lo(y.z), fmaf(bf16hi(x.z), bf16hi(y.z), s));
        s = fmaf(bf16lo(x.w), bf16lo(y.w), fmaf(bf16hi(x.w), bf16hi(y.w), s));
    }
    return s;
}
__device__ __forceinline__ float dot8(const float* a, const uint16_t* b, int n) {
    float s = 0.f;
#pragma unroll 1
    for (int i = 0; i < n; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(a + i);
        const uint2 y = *reinterpret_cast<const uint2*>(b + i);
        s = fmaf(x.x, bf16lo(y.x), fmaf(x.y, bf16hi(y.x), fmaf(x.z, bf16lo(y.y), fmaf(x.w, bf16hi(y.y), s))));
    }
    return s;
}

// A launch that may start before the one before it on the stream has ended (programmatic dependent
// launch): the kernels wait for it where they first read what it writes, and in every block.
template <typename... Args>
inline cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                    Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace lrkv
