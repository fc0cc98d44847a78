// Element types of the layers around the attention, and the tcgen05 and TMA
// forms that only they use.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "sm100.cuh"

namespace h3 {

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ float from_f32(float x) { return x; }

// Two 16-bit values in a word, `lo` in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    return pack_bf16x2(lo, hi);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    __half2 h;
    *reinterpret_cast<uint32_t *>(&h) = w;
    return __half22float2(h);
}

// Instruction descriptor of tcgen05.mma kind::f16 for A and B of type T.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, bool a_mn, bool b_mn) {
    const uint32_t d = idesc_bf16_f32(M, N, a_mn, b_mn);
    return !std::is_same<T, __half>::value ? d : d & ~((1u << 7) | (1u << 10));
}

// 2-D tiled bulk tensor load global -> shared; c0 * 2 bytes is a multiple of 16.
__device__ __forceinline__ void tma_load_rows(void *smem_dst, const CUtensorMap *map,
                                              uint64_t *bar, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

// Barrier among `threads` threads of the block (ids 1..15).
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// mbar_wait, mbar_arrive and give_up with shared-memory addresses, for code that is
// short of registers.
__device__ __forceinline__ bool mbar_wait_at(uint32_t bar, uint32_t parity, uint32_t abort,
                                             long long limit_cycles = kWaitLimitCycles) {
    auto done = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        return ok != 0;
    };
    if (done()) return true;
    const long long t0 = clock64();
    while (true) {
        if (done()) return true;
        int stop;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(stop) : "r"(abort) : "memory");
        if (stop != 0 || clock64() - t0 > limit_cycles) return false;
    }
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b64 st;\n\t"
        "mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}

__device__ __forceinline__ int lds32(uint32_t addr) {
    int v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts32(uint32_t addr, int v) {
    asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// The first block starts about a second (kWaitLimitCycles) before any wait of the
// others can give up, so its reset never covers their code.
__device__ __forceinline__ void reset_status(int *status) {
    if (blockIdx.x == 0) atomicExch(status, 0);
}

// A wait that gave up: the block stops, the call's status word says why.
__device__ __forceinline__ void give_up(volatile int *abort, int *status) {
    *abort = 1;
    atomicCAS(status, 0, 6);
}

}  // namespace h3
