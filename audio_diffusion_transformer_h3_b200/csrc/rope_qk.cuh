// Rotary embedding with one whole-number position a token, for q and k.
//
// Pair j of the rotated channels turns by position * f_j. The angle per
// position is held as a 64-bit fixed-point fraction of a full turn, so
// position * phase modulo 2^64 is the angle modulo one turn without any range
// reduction, up to the phase's own rounding (2^-65 turns a position, 2^-34 turns at
// 2^31; the frequency it is made of, a double, is off by some 2^-53 of itself:
// |position| f_j 2^-52 radians). The top 32 bits of the fraction go to fp32: 2^-32
// turns are left out and 2^-26 rounded off, 1e-7 radians at every position. An fp32
// product would be off by 2^-8 radians at position 2^17.
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
    int32_t copy;                   // 1: channels [rot, D) are copied, 0: they are in place
    int32_t head_chunk;             // heads of one block
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

// One 16-byte vector of T, or one T where rows, halves or pointers do not allow it.
template <typename T, bool Wide> struct RopeVec {
    static constexpr int E = Wide ? 16 / sizeof(T) : 1;
    T v[E];
};

template <typename T, bool Wide>
__device__ __forceinline__ void rope_vec_load(RopeVec<T, Wide> &x, const T *p) {
    if constexpr (Wide) *reinterpret_cast<uint4 *>(x.v) = *reinterpret_cast<const uint4 *>(p);
    else x.v[0] = *p;
}
template <typename T, bool Wide>
__device__ __forceinline__ void rope_vec_store(T *p, const RopeVec<T, Wide> &x) {
    if constexpr (Wide) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(x.v);
    else *p = x.v[0];
}

// A thread holds the cos and sin of one place of the head (in two vectors: a
// pair's first and second members; interleaved vectors hold both, so one
// vector, or two scalars) for one token and walks the heads [y * head_chunk,
// ...) with it, four at a time, so that each angle is computed once for all of
// them and the loads of four heads are in flight together. Bound by HBM (one
// read and one write of q and k): 131072 tokens of 72 heads of 128 at 6.4 TB/s, 97 %
// of a plain copy's rate (a block a token, its angles in shared memory, scalar
// accesses: 2.3 TB/s).
template <typename T, bool Wide, bool Half>
__global__ void __launch_bounds__(256) rope_qk_kernel(const __grid_constant__ RopeQkParams p) {
    using Vec = RopeVec<T, Wide>;
    constexpr int E = Vec::E;
    constexpr bool TWO = Half || !Wide;          // the pair's members lie in two vectors
    constexpr int NP = TWO ? E : E / 2;          // pairs of a place
    constexpr int U = 4;
    const int turning = p.rot / 2 / NP;          // places of a head that rotate
    const int places = turning + (p.copy ? (p.D - p.rot) / E : 0);
    const int64_t f = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t n = f / places;
    if (n >= p.N) return;
    const int place = static_cast<int>(f - n * places);
    const bool turns = place < turning;
    int c0, c1 = 0;                              // first channels of the two vectors
    float2 cs[NP];
    if (turns) {
        const int32_t pos = p.positions[n];
#pragma unroll
        for (int i = 0; i < NP; ++i)
            cs[i] = rope_qk_cos_sin(pos, p.phase[place * NP + i], p.attn_factor);
        c0 = Half ? place * E : (TWO ? 2 * place : place * E);
        c1 = Half ? c0 + p.rot / 2 : c0 + 1;
    } else {
        c0 = p.rot + (place - turning) * E;
    }
    const int heads = p.Hq + p.Hk;
    const int first = blockIdx.y * p.head_chunk, end = min(first + p.head_chunk, heads);
    for (int h0 = first; h0 < end; h0 += U) {
        Vec a[U], b[U];
        T *to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u;
            if (h >= end) break;
            const bool is_q = h < p.Hq;
            const int64_t at = static_cast<int64_t>(is_q ? h : h - p.Hq) * p.D + c0;
            const T *from = static_cast<const T *>(is_q ? p.q : p.k) + n * (is_q ? p.ldq : p.ldk) + at;
            to[u] = static_cast<T *>(is_q ? p.qo : p.ko) + n * (is_q ? p.ldqo : p.ldko) + at;
            rope_vec_load<T, Wide>(a[u], from);
            if (TWO && turns) rope_vec_load<T, Wide>(b[u], from + (c1 - c0));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u >= end) break;
            if (turns) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    T &lo = TWO ? a[u].v[i] : a[u].v[2 * i], &hi = TWO ? b[u].v[i] : a[u].v[2 * i + 1];
                    const float x0 = to_f32(lo), x1 = to_f32(hi);
                    lo = from_f32<T>(x0 * cs[i].x - x1 * cs[i].y);
                    hi = from_f32<T>(x0 * cs[i].y + x1 * cs[i].x);
                }
                if (TWO) rope_vec_store<T, Wide>(to[u] + (c1 - c0), b[u]);
            }
            rope_vec_store<T, Wide>(to[u], a[u]);
        }
    }
}

}  // namespace h3
