// Linear layer with bias, activation and residual in its epilogue.
#pragma once

#include <cstdint>

#include "rope_qk.cuh"

namespace h3 {

struct LinearParams {
    const void *x, *w, *bias, *residual;
    void *y;
    int64_t ldx, ldw, ldr, ldy, M;
    int32_t N, K;
};

// Act: h3_act without the gate bit.
template <int Act>
__device__ __forceinline__ float activate(float x) {
    if constexpr (Act == 1) return x < 0.0f ? 0.0f : x;   // keeps NaN
    if constexpr (Act == 2) return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
    if constexpr (Act == 3) {
        // x/2 (1 + tanh u) = x / (1 + exp(-2u))
        const float u2 = 1.5957691216057308f * (x + 0.044715f * x * x * x);
        return x / (1.0f + __expf(-u2));
    }
    if constexpr (Act == 4) return x / (1.0f + __expf(-x));
    return x;
}

// 64 x 64 outputs a block, 4 x 4 a thread, fp32 FMAs.
template <typename T, int Act, bool Gated>
__global__ void __launch_bounds__(256) linear_kernel(const LinearParams p) {
    constexpr int B = 64, KB = 16, W = Gated ? 2 : 1;
    __shared__ float xs[KB][B + 1], ws[W][KB][B + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * B;
    const int n0 = blockIdx.x * B;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    float acc[W][4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += KB) {
        for (int i = threadIdx.x; i < B * KB; i += 256) {
            const int r = i / KB, k = i % KB;
            const bool kin = k0 + k < p.K;
            xs[k][r] = kin && m0 + r < p.M ? to_f32(x[(m0 + r) * p.ldx + k0 + k]) : 0.0f;
            for (int g = 0; g < W; ++g)
                ws[g][k][r] = kin && n0 + r < p.N
                    ? to_f32(w[(static_cast<int64_t>(g) * p.N + n0 + r) * p.ldw + k0 + k]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < KB; ++k)
            for (int g = 0; g < W; ++g)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j)
                        acc[g][i][j] = fmaf(xs[k][ty * 4 + i], ws[g][k][tx * 4 + j], acc[g][i][j]);
        __syncthreads();
    }
    const T *bias = static_cast<const T *>(p.bias), *res = static_cast<const T *>(p.residual);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i;
            const int n = n0 + tx * 4 + j;
            if (m >= p.M || n >= p.N) continue;
            float v = acc[0][i][j] + (bias ? to_f32(bias[n]) : 0.0f);
            v = activate<Act>(v);
            if (Gated) v *= acc[W - 1][i][j] + (bias ? to_f32(bias[p.N + n]) : 0.0f);
            if (res) v += to_f32(res[m * p.ldr + n]);
            static_cast<T *>(p.y)[m * p.ldy + n] = from_f32<T>(v);
        }
}

}  // namespace h3
