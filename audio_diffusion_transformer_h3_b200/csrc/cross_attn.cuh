// Packed varlen cross attention, one warp a (query token, head).
#pragma once

#include <cstdint>

#include "rope_qk.cuh"

namespace h3 {

struct CrossParams {
    const void *q, *k, *v;
    void *o;
    float *lse;
    int64_t ldq, ldk, ldv, ldo;
    const int32_t *cu_q, *cu_k;
    const uint8_t *mask;
    int *status;
    int32_t nseg, max_q, max_k, Nq, Nk, Hq, Hk;
    float scale_log2;
};

// Both boundary arrays, by the whole block: non-zero in every thread if bad.
__device__ __forceinline__ int cross_bad_seqlens(const CrossParams &p) {
    int bad = 0;
    for (int i = threadIdx.x; i <= p.nseg; i += blockDim.x) {
        const int a = p.cu_q[i], b = p.cu_k[i];
        if (i == 0 && (a != 0 || b != 0)) bad = 1;
        if (i == p.nseg && (a > p.Nq || b > p.Nk)) bad = 1;
        if (i > 0) {
            const int pa = p.cu_q[i - 1], pb = p.cu_k[i - 1];
            if (a < pa || a - pa > p.max_q || b < pb || b - pb > p.max_k) bad = 1;
        }
    }
    return __syncthreads_or(bad);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) cross_attn_kernel(const CrossParams p) {
    __shared__ float qs[4][D];
    if (cross_bad_seqlens(p)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, 7);
        return;
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int total = p.cu_q[p.nseg];
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + warp;
         at < static_cast<int64_t>(total) * p.Hq; at += static_cast<int64_t>(gridDim.x) * 4) {
        const int row = static_cast<int>(at / p.Hq), head = static_cast<int>(at % p.Hq);
        const int kvh = head / (p.Hq / p.Hk);
        int lo = 0, hi = p.nseg;   // last segment that begins at or before row and holds it
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (p.cu_q[mid] <= row) lo = mid; else hi = mid;
        }
        const int k0 = p.cu_k[lo], k1 = p.cu_k[lo + 1];
        __syncwarp();
        for (int d = lane; d < D; d += 32)
            qs[warp][d] = to_f32(static_cast<const T *>(p.q)[row * p.ldq + head * D + d]);
        __syncwarp();
        float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
        for (int j0 = k0; j0 < k1; j0 += 32) {
            const int j = j0 + lane;
            float s = -INFINITY;
            if (j < k1 && (p.mask == nullptr || p.mask[j] != 0)) {
                const T *kr = static_cast<const T *>(p.k) + j * p.ldk + kvh * D;
                float dot = 0.0f;
                for (int d = 0; d < D; ++d) dot = fmaf(qs[warp][d], to_f32(kr[d]), dot);
                s = dot * p.scale_log2;
            }
            const unsigned kept = __ballot_sync(0xffffffffu, s != -INFINITY);
            if (kept == 0) continue;
            float mx = s;
            for (int o = 16; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(mx, m);
            const float f = exp2f(m - mx), e = s == -INFINITY ? 0.0f : exp2f(s - mx);
            m = mx;
            float sum = e;
            for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = l * f + sum;
            for (int c = 0; c < D / 32; ++c) acc[c] *= f;
            for (int i = 0; i < 32; ++i) {
                const float pi = __shfl_sync(0xffffffffu, e, i);
                if (!((kept >> i) & 1)) continue;
                const T *vr = static_cast<const T *>(p.v) + (j0 + i) * p.ldv + kvh * D;
                for (int c = 0; c < D / 32; ++c)
                    acc[c] = fmaf(pi, to_f32(vr[c * 32 + lane]), acc[c]);
            }
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        T *orow = static_cast<T *>(p.o) + row * p.ldo + head * D;
        for (int c = 0; c < D / 32; ++c) orow[c * 32 + lane] = from_f32<T>(acc[c] * inv);
        if (p.lse != nullptr && lane == 0)
            p.lse[static_cast<int64_t>(head) * p.Nq + row] =
                l > 0.0f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
    }
}

}  // namespace h3
