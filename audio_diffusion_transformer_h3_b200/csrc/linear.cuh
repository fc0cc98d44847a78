// Linear layer with bias, activation and residual in the product's epilogue:
// y = act(x w^T + bias) + residual, or act(x wg^T + bg) (x wu^T + bu) + residual.
//
// Two kernels, both fed by TMA through a ring of 64-wide K steps, multiplied
// by tcgen05.mma into fp32 TMEM accumulators, every wait bounded:
//   linear_tile_kernel  rows of x are the 128 rows of the MMA, 32 to 256 weight rows
//       its columns. Persistent, two accumulators, so that a tile's epilogue
//       runs under the next tile's main loop. Bound by the tensor cores: 73 % of
//       their cycles in a single launch of 4160 x 7168 x 5376 (232 us), 1140 to
//       1350 TFLOP/s in a loop under the power cap (8320 rows).
//   linear_skinny_kernel  few rows of x: weight rows are the MMA's 128 rows
//       and x its 16..128 columns, so nothing of the MMA is spent on absent
//       rows. Bound by reading w once; to have all SMs read, the sum over K
//       is split over a cluster of up to 8 CTAs, which then share out the
//       columns: each adds the parts of its own, read from the others' shared
//       memory in their order (parts joined through global memory by the last
//       CTA took 45 us instead of 22 for 32 rows of 7168 x 5376). Measured: two
//       rows of 5376 x 32256 at 6.1 TB/s, 94 % of a plain copy's rate.
// A gated layer keeps the gate and the up product of the same outputs side by
// side in TMEM and multiplies them in the epilogue.
#pragma once

#include <cstdint>

#include "layer_types.cuh"

namespace h3 {

struct LinearParams {
    const void *bias, *residual;
    void *y;
    int64_t ldr, ldy;
    int *status;
    int32_t M, N, K, act;     // act: h3_act without the gate
    int32_t vec_y, vec_r;     // y / residual rows allow 16-byte accesses
    // tile kernel
    int32_t out_cols, stages, n_row_tiles, n_col_tiles, n_tiles, group_m;
    int32_t whole, pieces;    // whole tiles, then the rest of them in `pieces` parts each
    // skinny kernel
    int32_t cols, splits;     // splits: the cluster's CTAs
};

// (1 + erf(x / sqrt 2)) / 2, relatively accurate also where it is small (1 + erff cancels
// there: 10 % at x = -5). Method: with z = |x| / sqrt 2 and t = 1 / (1 + 0.4 z),
// erfc(z) exp(z^2) / t is a polynomial in t on (0, 1]: degree 8, fitted for the least
// relative error (iteratively reweighted least squares: 1.3e-7, 4.4e-7 in fp32), its
// coefficients halved; exp(-z^2) adds 2^-23 (z^2 + 2). Measured: 8320 x 14336 x 512,
// where the epilogue counts most, 375 us (1 + erff 390, erfcf 685).
__device__ __forceinline__ float normal_cdf(float x) {
    const float t = __fdividef(1.0f, fmaf(fabsf(x), 0.28284271247461901f, 1.0f));
    float p = 0.0251363218f;
    p = fmaf(p, t, -0.0914719701f);
    p = fmaf(p, t, 0.0845777988f);
    p = fmaf(p, t, -0.00283428328f);
    p = fmaf(p, t, 0.0707306936f);
    p = fmaf(p, t, 0.0842668638f);
    p = fmaf(p, t, 0.103921942f);
    p = fmaf(p, t, 0.112834759f);
    p = fmaf(p, t, 0.112837933f);
    const float h = p * t * ex2_approx(x * x * -0.72134752044448170f);   // exp(-z^2)
    return x < 0.0f ? h : 1.0f - h;
}

// act in place on V values; the switch is uniform over the grid. Each keeps its relative
// accuracy where it is small. __expf is off by up to 2 + 1.2 |t| units of 2^-23 and
// __fdividef by 2, far below the result's rounding (2^-9, 2^-12) until the quotient
// itself is below x 2^-126.
template <int V>
__device__ __forceinline__ void activate(float (&x)[V], int act) {
    switch (act) {
        case 1:
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = x[i] < 0.0f ? 0.0f : x[i];   // keeps NaN
            break;
        case 2:
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] *= normal_cdf(x[i]);
            break;
        case 3:
            // x/2 (1 + tanh u) = x / (1 + exp(-2u))
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float u2 = 1.5957691216057308f * (x[i] + 0.044715f * x[i] * x[i] * x[i]);
                x[i] = __fdividef(x[i], 1.0f + __expf(-u2));
            }
            break;
        case 4:
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = __fdividef(x[i], 1.0f + __expf(-x[i]));
            break;
        default: break;
    }
}

// --------------------------------------------------------------- tile kernel

struct LinearTile {
    static constexpr int BM = 128, BK = 64, MAX_BN = 256;
    static constexpr int A_BYTES = BM * BK * 2;
    static constexpr int MAX_STAGES = 8;
    static constexpr int RING_BYTES = 4 * (A_BYTES + MAX_BN * BK * 2);   // 192 KB
    static constexpr int OFF_BIAS = RING_BYTES;                          // 256 fp32
    static constexpr int OFF_OUT = OFF_BIAS + MAX_BN * 4;                // 4 KB a warp
    static constexpr int OFF_BAR = OFF_OUT + 4 * 4096;
    static constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;              // + alignment slack
    static constexpr int THREADS = 192, TMA_WARP = 4, MMA_WARP = 5;
};

enum : int {
    LT_FULL = 0, LT_EMPTY = 8, LT_ACC_FULL = 16, LT_ACC_EMPTY = 18, LT_DRAIN = 20, LT_COUNT = 21
};

struct LinearTileAt {
    int row, col, width;   // row tile, first output column, output columns
};

// Tile number -> its place: group_m row tiles sweep the columns together, so the x
// rows and w slices in flight stay in L2; the tiles of the last, partial round of
// SMs come in parts.
__device__ __forceinline__ LinearTileAt linear_tile_at(const LinearParams &p, int tile) {
    int piece = 0, width = p.out_cols;
    if (tile >= p.whole) {
        const int i = tile - p.whole;
        tile = p.whole + i / p.pieces;
        piece = i % p.pieces;
        width = p.out_cols / p.pieces;
    }
    const int per_group = p.group_m * p.n_col_tiles;
    const int group = tile / per_group, first = group * p.group_m;
    const int left = p.n_row_tiles - first, gm = left < p.group_m ? left : p.group_m;
    const int in_group = tile - group * per_group;
    return {first + in_group % gm, in_group / gm * p.out_cols + piece * width, width};
}

// 32 rows x 64 columns of 16-bit values of a warp in shared memory: row r's
// 16-byte piece i at r * 128 + ((i ^ r % 8) * 16), so that a lane's own row and
// four rows of 128 bytes are both free of bank conflicts.
__device__ __forceinline__ uint32_t linear_piece(uint32_t stage, int r, int i) {
    return stage + r * 128 + ((i ^ (r & 7)) << 4);
}

// Columns [0, width) of rows [0, rows) between `stage` and memory (g: the first
// row's first column), by the whole warp: four rows of 16-byte pieces at a time
// where the rows allow it, else 32 elements of a row at a time.
template <typename T>
__device__ __forceinline__ void linear_rows_out(uint32_t stage, T *g, int64_t ld, int rows, int width,
                                                bool wide, int lane) {
    if (wide) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lds128(linear_piece(stage, i * 4 + lane / 8, lane & 7));
        const int left = width - (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + lane / 8;
            if (r >= rows || left <= 0) continue;
            T *at = g + r * ld + (lane & 7) * 8;
            if (left >= 8) {
                *reinterpret_cast<uint4 *>(at) = v[i];
            } else {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < left)
                        reinterpret_cast<uint16_t *>(at)[e] = static_cast<uint16_t>(w[e / 2] >> (e % 2 * 16));
            }
        }
        return;
    }
    for (int r = 0; r < rows; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = h * 32 + lane;
            uint16_t x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(linear_piece(stage, r, c >> 3) + (c & 7) * 2));
            if (c < width) reinterpret_cast<uint16_t *>(g + r * ld)[c] = x;
        }
}

// The first half of reading such rows: what this lane fetches (wide rows only).
template <typename T>
__device__ __forceinline__ void linear_rows_fetch(uint4 (&v)[8], const T *g, int64_t ld, int rows,
                                                  int width, int lane) {
    const int left = width - (lane & 7) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + lane / 8;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r >= rows || left <= 0) continue;
        const T *at = g + r * ld + (lane & 7) * 8;
        if (left >= 8) {
            v[i] = *reinterpret_cast<const uint4 *>(at);
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < left)
                    w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at)[e]) << (e % 2 * 16);
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// The second half: into shared memory (rows that are not wide are read here).
template <typename T>
__device__ __forceinline__ void linear_rows_in(uint32_t stage, const uint4 (&v)[8], const T *g,
                                               int64_t ld, int rows, int width, bool wide, int lane) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sts128(linear_piece(stage, i * 4 + lane / 8, lane & 7), v[i].x, v[i].y, v[i].z, v[i].w);
        return;
    }
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = h * 32 + lane;
            const uint16_t x = c < width ? reinterpret_cast<const uint16_t *>(g + r * ld)[c] : 0;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(linear_piece(stage, r, c >> 3) + (c & 7) * 2), "h"(x)
                         : "memory");
        }
}

template <typename T, bool Gated>
__global__ void __launch_bounds__(192, 1)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmWPiece, const LinearParams p) {
    using C = LinearTile;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_k = (p.K + C::BK - 1) / C::BK;
    constexpr int W = Gated ? 2 : 1;                    // products
    const int stage_bytes = C::A_BYTES + W * p.out_cols * C::BK * 2;

    float *bias_s = reinterpret_cast<float *>(smem + C::OFF_BIAS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + LT_COUNT);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (tid == 0) {
        reset_status(p.status);
        for (int s = 0; s < C::MAX_STAGES; ++s) {
            mbar_init(&bars[LT_FULL + s], 1);
            mbar_init(&bars[LT_EMPTY + s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars[LT_ACC_FULL + b], 1);
            mbar_init(&bars[LT_ACC_EMPTY + b], 4);   // one arrival per epilogue warp
        }
        mbar_init(&bars[LT_DRAIN], 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == C::TMA_WARP && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == C::TMA_WARP) {
        const uint32_t leader = elect_one();
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < p.n_tiles; tile += gridDim.x) {
            const LinearTileAt x = linear_tile_at(p, tile);
            const CUtensorMap *w_map = x.width == p.out_cols ? &tmW : &tmWPiece;
            const int w_bytes = x.width * C::BK * 2;
            for (int ks = 0; ks < n_k; ++ks) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars[LT_EMPTY + stage], phase ^ 1, abort))) {
                    ok = false;
                    break;
                }
                if (leader) {
                    uint8_t *a = smem + stage * stage_bytes, *b = a + C::A_BYTES;
                    mbar_arrive_expect_tx(&bars[LT_FULL + stage], C::A_BYTES + W * w_bytes);
                    tma_load_rows(a, &tmX, &bars[LT_FULL + stage], ks * C::BK, x.row * C::BM);
                    tma_load_rows(b, w_map, &bars[LT_FULL + stage], ks * C::BK, x.col);
                    if (Gated)
                        tma_load_rows(b + w_bytes, w_map, &bars[LT_FULL + stage], ks * C::BK, p.N + x.col);
                }
                ++issued;
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
        }
        if (!ok) {
            if (leader) give_up(abort, p.status);
            // copies still in flight land before the CTA leaves
            for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; ++j)
                mbar_wait(&bars[LT_FULL + j % p.stages], (j / p.stages) & 1, nullptr);
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP) {
        const uint32_t leader = elect_one();
        const uint64_t d0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        int stage = 0, count = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < p.n_tiles; tile += gridDim.x, ++count) {
            const int buf = count & 1;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&bars[LT_ACC_EMPTY + buf], ((count >> 1) & 1) ^ 1, abort));
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + static_cast<uint32_t>(buf) * 256;
            const uint32_t idesc = idesc_f32<T>(C::BM, 0, false, false) |
                                   (static_cast<uint32_t>(W * linear_tile_at(p, tile).width >> 3) << 17);
            for (int ks = 0; ks < n_k; ++ks) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[LT_FULL + stage], phase, abort));
                if (!ok) break;
                tc_fence_after();
                const uint64_t ad = d0 + static_cast<uint64_t>((stage * stage_bytes) >> 4);
                const uint64_t bd = ad + (C::A_BYTES >> 4);
#pragma unroll
                for (int kk = 0; kk < C::BK / 16; ++kk)
                    umma_ss_w(acc, ad + kk * 2, bd + kk * 2, idesc, (ks > 0 || kk > 0) ? 1u : 0u,
                              leader);
                umma_commit_w(&bars[LT_EMPTY + stage], leader);
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
            if (!ok) break;
            umma_commit_w(&bars[LT_ACC_FULL + buf], leader);
        }
        if (!ok) {
            if (leader) give_up(abort, p.status);
            // MMAs in flight complete before the accumulators are released
            umma_commit_w(&bars[LT_DRAIN], leader);
            mbar_wait(&bars[LT_DRAIN], 0, nullptr);
        }
        __syncwarp();
    } else {
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const T *bias = static_cast<const T *>(p.bias);
        const uint32_t stage = smem_u32(smem + C::OFF_OUT) + warp * 4096;
        int count = 0;
        bool ok = true;   // after a wait that gave up the warps still meet at named_sync
        for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x, ++count) {
            const int buf = count & 1;
            const LinearTileAt x = linear_tile_at(p, tile);
            const int col0 = x.col, out_cols = x.width;
            named_sync(1, 128);   // the last tile's bias has been read
            for (int c = tid; c < W * out_cols; c += 128) {
                const int half = Gated && c >= out_cols;
                const int n = col0 + c - half * out_cols;
                bias_s[c] = bias != nullptr && n < p.N ? to_f32(bias[half * p.N + n]) : 0.0f;
            }
            named_sync(1, 128);
            // this warp's rows, 64 columns at a time: the residual comes and the result
            // goes through shared memory, in whole lines; the next residual is on its way
            // while these columns are at work
            const int row0 = x.row * C::BM + warp * 32, rows = min(p.M - row0, 32);
            const int cols = rows > 0 ? min(out_cols, p.N - col0) : 0;
            const T *res = p.residual == nullptr
                ? nullptr : static_cast<const T *>(p.residual) + row0 * p.ldr + col0;
            T *y = static_cast<T *>(p.y) + row0 * p.ldy + col0;
            uint4 fetched[8];
            if (res != nullptr && p.vec_r && cols > 0)
                linear_rows_fetch<T>(fetched, res, p.ldr, rows, min(cols, 64), lane);
            ok = ok && __all_sync(0xffffffffu,
                                  mbar_wait(&bars[LT_ACC_FULL + buf], (count >> 1) & 1, abort));
            if (!ok) {
                if (lane == 0) give_up(abort, p.status);
                continue;
            }
            tc_fence_after();
            const uint32_t acc = tmem + lane_off + static_cast<uint32_t>(buf) * 256;
#pragma unroll 1
            for (int c = 0; c < cols; c += 64) {
                const int width = min(cols - c, 64);
                if (res != nullptr) {
                    linear_rows_in<T>(stage, fetched, res + c, p.ldr, rows, width, p.vec_r, lane);
                    __syncwarp();
                    if (p.vec_r && c + 64 < cols)
                        linear_rows_fetch<T>(fetched, res + c + 64, p.ldr, rows, min(cols - c - 64, 64), lane);
                }
#pragma unroll 1
                for (int h = 0; h < 64 && h < width; h += 32) {
                    uint32_t a[32];
                    float v[32];
                    tmem_ld32(acc + c + h, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(a[i]) + bias_s[c + h + i];
                    activate(v, p.act);
                    if constexpr (Gated) {
                        tmem_ld32(acc + out_cols + c + h, a);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] *= __uint_as_float(a[i]) + bias_s[out_cols + c + h + i];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // 8 columns, this lane's row
                        const uint32_t at = linear_piece(stage, lane, h / 8 + i);
                        if (res != nullptr) {
                            const uint4 w = lds128(at);
                            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = unpack2<T>(ww[e]);
                                v[8 * i + 2 * e] += f.x;
                                v[8 * i + 2 * e + 1] += f.y;
                            }
                        }
                        sts128(at, pack2<T>(v[8 * i], v[8 * i + 1]), pack2<T>(v[8 * i + 2], v[8 * i + 3]),
                               pack2<T>(v[8 * i + 4], v[8 * i + 5]), pack2<T>(v[8 * i + 6], v[8 * i + 7]));
                    }
                }
                __syncwarp();
                linear_rows_out<T>(stage, y + c, p.ldy, rows, width, p.vec_y, lane);
                __syncwarp();
            }
            // accumulator reads done -> the MMA warp may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[LT_ACC_EMPTY + buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------- skinny kernel

struct LinearSkinny {
    static constexpr int BM = 128, BK = 64;
    static constexpr int W_BYTES = BM * BK * 2;
    static constexpr int MAX_STAGES = 6;
    static constexpr int RING_BYTES = 108 * 1024;                 // two CTAs an SM
    static constexpr int OFF_BAR = RING_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;       // + alignment slack
    static constexpr int THREADS = 192, TMA_WARP = 4, MMA_WARP = 5;
};

enum : int { LS_FULL = 0, LS_EMPTY = 6, LS_ACC = 12, LS_COUNT = 13 };

// V outputs of weight row n (this thread's), x rows c, c + 1, ...: bias,
// activation, gate, residual, store.
template <typename T, bool Gated, int V>
__device__ __forceinline__ void linear_skinny_store(const LinearParams &p, int n, int c, int end,
                                                    float (&v)[V], float (&u)[V]) {
    const T *bias = static_cast<const T *>(p.bias), *res = static_cast<const T *>(p.residual);
    if (bias != nullptr) {
        const float b = to_f32(bias[n]);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += b;
    }
    activate(v, p.act);
    if constexpr (Gated) {
        const float b = bias != nullptr ? to_f32(bias[p.N + n]) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= u[i] + b;
    }
    if (res != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < end) v[i] += to_f32(res[(c + i) * p.ldr + n]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c + i < end) static_cast<T *>(p.y)[(c + i) * p.ldy + n] = from_f32<T>(v[i]);
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A float of the cluster's CTA `rank` at the address that `addr` is in this CTA.
__device__ __forceinline__ float cluster_read(uint32_t addr, uint32_t rank) {
    uint32_t there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
}

template <typename T, bool Gated>
__global__ void __launch_bounds__(192)
    linear_skinny_kernel(const __grid_constant__ CUtensorMap tmX,
                         const __grid_constant__ CUtensorMap tmW, const LinearParams p) {
    using C = LinearSkinny;
    constexpr int W = Gated ? 2 : 1;   // products
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;   // a cluster's CTAs are neighbours
    const int n_k = (p.K + C::BK - 1) / C::BK;
    const int k_first = static_cast<int>(static_cast<int64_t>(n_k) * split / p.splits);
    const int k_count = static_cast<int>(static_cast<int64_t>(n_k) * (split + 1) / p.splits) - k_first;
    const int x_bytes = p.cols * C::BK * 2, stage_bytes = W * C::W_BYTES + x_bytes;
    uint32_t tmem_cols = 32;
    while (tmem_cols < static_cast<uint32_t>(W * p.cols)) tmem_cols *= 2;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + LS_COUNT);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (tid == 0) {
        reset_status(p.status);
        for (int s = 0; s < C::MAX_STAGES; ++s) {
            mbar_init(&bars[LS_FULL + s], 1);
            mbar_init(&bars[LS_EMPTY + s], 1);
        }
        mbar_init(&bars[LS_ACC], 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == C::TMA_WARP) {
        const uint32_t leader = elect_one();
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int ks = 0; ks < k_count; ++ks) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[LS_EMPTY + stage], phase ^ 1, abort));
            if (!ok) break;
            if (leader) {
                uint8_t *a = smem + stage * stage_bytes;
                const int k = (k_first + ks) * C::BK;
                mbar_arrive_expect_tx(&bars[LS_FULL + stage], stage_bytes);
                tma_load_rows(a, &tmW, &bars[LS_FULL + stage], k, tile * C::BM);
                if (Gated)
                    tma_load_rows(a + C::W_BYTES, &tmW, &bars[LS_FULL + stage], k,
                                  p.N + tile * C::BM);
                tma_load_rows(a + W * C::W_BYTES, &tmX, &bars[LS_FULL + stage], k, 0);
            }
            ++issued;
            if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
        if (!ok) {
            if (leader) give_up(abort, p.status);
            for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; ++j)
                mbar_wait(&bars[LS_FULL + j % p.stages], (j / p.stages) & 1, nullptr);
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP) {
        const uint32_t leader = elect_one();
        const uint32_t idesc = idesc_f32<T>(C::BM, 0, false, false) |
                               (static_cast<uint32_t>(p.cols >> 3) << 17);
        const uint64_t d0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int ks = 0; ks < k_count; ++ks) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[LS_FULL + stage], phase, abort));
            if (!ok) break;
            tc_fence_after();
            const uint64_t wd = d0 + static_cast<uint64_t>((stage * stage_bytes) >> 4);
            const uint64_t xd = wd + ((W * C::W_BYTES) >> 4);
#pragma unroll
            for (int kk = 0; kk < C::BK / 16; ++kk)
#pragma unroll
                for (int g = 0; g < W; ++g)
                    umma_ss_w(tmem + g * p.cols, wd + ((g * C::W_BYTES) >> 4) + kk * 2, xd + kk * 2,
                              idesc, (ks > 0 || kk > 0) ? 1u : 0u, leader);
            umma_commit_w(&bars[LS_EMPTY + stage], leader);
            if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
        if (!ok && leader) give_up(abort, p.status);
        // also after a wait that gave up: the MMAs in flight complete first
        umma_commit_w(&bars[LS_ACC], leader);
        if (!ok) mbar_wait(&bars[LS_ACC], 0, nullptr);
        __syncwarp();
    } else {
        const int n = tile * C::BM + tid;
        bool ok = __all_sync(0xffffffffu, mbar_wait(&bars[LS_ACC], 0, abort));
        if (!ok && lane == 0) give_up(abort, p.status);
        tc_fence_after();
        ok = ok && *abort == 0;
        const uint32_t acc = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        if (p.splits == 1) {
            for (int c = 0; ok && c < p.cols; c += 16) {
                uint32_t a[16], b[16];
                float v[16], u[16];
                tmem_ld16(acc + c, a);
                if constexpr (Gated) tmem_ld16(acc + p.cols + c, b);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[i] = __uint_as_float(a[i]);
                    if constexpr (Gated) u[i] = __uint_as_float(b[i]);
                }
                if (n < p.N) linear_skinny_store<T, Gated>(p, n, c, p.M, v, u);
            }
        } else {
            // the ring is done with: this CTA's part goes there, [product, column][row]
            float *part = reinterpret_cast<float *>(smem) + tid;
            for (int c = 0; ok && c < W * p.cols; c += 16) {
                uint32_t a[16];
                tmem_ld16(acc + c, a);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * C::BM] = __uint_as_float(a[i]);
            }
        }
    }
    if (p.splits > 1) {
        // every thread of every CTA of the cluster comes by here, whatever gave up
        cluster_sync_all();
        const int n = tile * C::BM + tid;
        if (tid < C::BM && n < p.N && *abort == 0) {
            const int each = (p.M + p.splits - 1) / p.splits;
            const int end = min((split + 1) * each, p.M);
            const uint32_t at = smem_u32(smem) + tid * 4;
            constexpr int V = 4;   // columns at a time: 4 x splits loads in flight
            for (int c = split * each; c < end; c += V) {
                float v[V] = {}, u[V] = {};
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    if (s >= p.splits) break;
#pragma unroll
                    for (int i = 0; i < V; ++i) {   // (columns behind the last hold zeros or other columns' sums)
                        const int col = min(c + i, p.cols - 1);
                        v[i] += cluster_read(at + col * C::BM * 4, s);
                        if constexpr (Gated) u[i] += cluster_read(at + (p.cols + col) * C::BM * 4, s);
                    }
                }
                linear_skinny_store<T, Gated>(p, n, c, end, v, u);
            }
        }
        cluster_sync_all();   // nobody leaves while the others still read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols);
    }
}

}  // namespace h3
