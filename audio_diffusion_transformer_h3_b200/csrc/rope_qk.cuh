// Rotary embedding with one whole-number position a token, for q and k.
//
// Pair j of the rotated channels turns by position * f_j. The angle per
// position is held as a 64-bit fixed-point fraction of a full turn, so
// position * phase modulo 2^64 is the angle modulo one turn without any range
// reduction: exact for every int32 position up to the phase's own rounding
// (2^-65 turns a position, 2^-34 turns at 2^31). An fp32 product would be off
// by 2^-8 radians at position 2^17.
#pragma once

#include <cstdint>

#include "layer_types.cuh"

namespace h3 {

constexpr int kRopeQkMaxPairs = 256;

struct RopeQkParams {
    const void *q, *k;
    void *qo, *ko;
    int64_t ldq, ldqo, ldk, ldko;   // elements
    const int32_t *positions;
    int64_t N;
    int32_t Hq, Hk, D, rot;
    int32_t half;                   // 1: pair (j, j + rot/2), 0: pair (2j, 2j + 1)
    float attn_factor;
    uint64_t phase[kRopeQkMaxPairs];   // turns per position * 2^64, modulo 2^64
};

// a * (cos, sin) of `position` times the pair's phase.
__device__ __forceinline__ float2 rope_qk_cos_sin(int32_t position, uint64_t phase, float a) {
    const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(position)) * phase;
    // the top 32 bits as a signed fraction of a turn in [-1/2, 1/2), times 2
    const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(a * c, a * s);
}

template <typename T>
__global__ void __launch_bounds__(256) rope_qk_kernel(const __grid_constant__ RopeQkParams p) {
    __shared__ float2 cs[kRopeQkMaxPairs];
    const int np = p.rot / 2, per_head = np + (p.D - p.rot);
    for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
        const int32_t pos = p.positions[n];
        __syncthreads();
        for (int j = threadIdx.x; j < np; j += blockDim.x)
            cs[j] = rope_qk_cos_sin(pos, p.phase[j], p.attn_factor);
        __syncthreads();
        for (int i = threadIdx.x; i < (p.Hq + p.Hk) * per_head; i += blockDim.x) {
            const int head = i / per_head, j = i - head * per_head;
            const bool is_q = head < p.Hq;
            const T *x = is_q ? static_cast<const T *>(p.q) + n * p.ldq + static_cast<int64_t>(head) * p.D
                              : static_cast<const T *>(p.k) + n * p.ldk + static_cast<int64_t>(head - p.Hq) * p.D;
            T *y = is_q ? static_cast<T *>(p.qo) + n * p.ldqo + static_cast<int64_t>(head) * p.D
                        : static_cast<T *>(p.ko) + n * p.ldko + static_cast<int64_t>(head - p.Hq) * p.D;
            if (j < np) {
                const int c0 = p.half ? j : 2 * j, c1 = p.half ? j + np : 2 * j + 1;
                const float a = to_f32(x[c0]), b = to_f32(x[c1]);
                y[c0] = from_f32<T>(a * cs[j].x - b * cs[j].y);
                y[c1] = from_f32<T>(a * cs[j].y + b * cs[j].x);
            } else {
                const int c = p.rot + j - np;
                y[c] = x[c];
            }
        }
    }
}

}  // namespace h3
