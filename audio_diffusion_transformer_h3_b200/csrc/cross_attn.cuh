// Packed varlen cross attention, forward, sm_100a: the queries of segment s
// attend to the keys of segment s of another packed sequence.
//
// One work item is two 128-row query tiles of one segment and one key head,
// against the segment's keys or a chunk of them. A tile's rows are (token,
// query head) pairs of one key head's group, token by token, so that every key
// tile is read once for the whole group; a tile of 128 rows holds 128/G tokens.
// The kernel is persistent: a CTA per SM takes items in turn, and the loads and
// the first score product of an item run under the softmax and the output of
// the one before.
//   warps 0-7   softmax, one thread a row (warpgroup t owns tile t and TMEM
//               lanes 0..127): online softmax in the log2 domain, the running
//               maximum m and sum l in fp32, the accumulator rescaled only when
//               m grows by more than 2^8; P in the operands' type into the
//               first 64 columns of S_t, in two halves of 64 keys; then O / l.
//               (Taking turns on the exponential unit, as the dense kernel's
//               tiles do over thousands of keys, cost 3 to 4 % here.)
//   warp 8      tcgen05.mma issuer: S_t = Q_t K^T, O_t += P_t V.
//   warp 9      where a value tile holds rows that must not count (behind the
//               segment's end, or masked) it writes zeros over them: P is 0
//               there, but 0 times a NaN or an infinity is not.
//   warp 10     TMA producer.
//   warp 11     finds the items (a search over the segments) ahead of the others
//               and hands them over in a ring of four.
// A key tile's products stop at its last key (in steps of 16).
//
// Few rows: an item with no more rows than one tile gives both tiles the same
// rows and every other key tile, and the keys of a segment are split into
// chunks so that all SMs read. Each tile then leaves its unnormalised O, m and
// l in fp32, and cross_join_kernel adds a row's parts up in their order.
//
// Measured, in a loop that leaves K, V and the output's memory in L2: 8320 rows x 56
// heads of 128 on 2048 keys 421 us (1160 TFLOP/s, the dense self attention's rate), on
// 512 keys 127 us (145 to 151 where the output's lines are not in L2): a key tile costs 1.9 us for
// both query tiles, bound by the softmax, an item another 2 us, in which the
// tensor cores wait for the last P, the output and the next first scores. 64 rows
// on 33280 keys of 24 heads of 64: 63 us (3.2 TB/s), with a mask 74.
//
// Every wait is bounded; one that gives up sets H3_ERR_DEVICE_TIMEOUT, stops
// the CTA, and leaves TMEM and shared memory only after the copies and MMAs in
// flight have landed.
#pragma once

#include <cstdint>

#include "layer_types.cuh"

namespace h3 {

struct CrossParams {
    void *o;
    float *lse;
    int64_t ldo;
    const int32_t *cu_q, *cu_k;
    const uint8_t *mask;
    int *status;
    int32_t nseg, max_q, max_k, Nq, Nk, Hq, Hk;
    int32_t hp, tokens, heads_blocks;   // heads and tokens of a tile, Hq / hp
    int32_t split;                      // 1: keys may be split
    float scale_log2;
    float *parts;                       // [item][tile][slot_rows][m, l, O]
    int2 *rows;                         // [token][query head]: first part, parts (split)
    int32_t slot_rows;
};

constexpr int kCrossTable = 256;        // entries of the segment table
// items that a split aims at: two for each of B200's 148 SMs (a constant: the workspace's
// size hangs on it, which is asked for without a device)
constexpr int kCrossItems = 296;
constexpr int kCrossMinChunk = 2;       // key tiles of a chunk at least

// An item in the ring (byte offsets).
enum : int {
    CX_Q0 = 0,         // first query token
    CX_Q_LEFT = 4,     // query tokens of this item (at most two tiles)
    CX_HEAD = 8,       // block of hp query heads
    CX_K0 = 12,        // first key token
    CX_K_LEFT = 16,    // keys from there to the segment's end
    CX_N_KV = 20,      // key tiles; negative: no more items
    CX_SPLITS = 24,    // chunks that these rows' keys are split into
    CX_GROUP = 28,     // item number of the first of them
    CX_ITEM = 32,      // item number
    CX_MODE = 36,      // CM_*
    CX_BYTES = 48
};
// How an item uses its two tiles: one only; the first and the second half of its
// rows; the same rows for the even and the odd key tiles.
enum : int { CM_ONE = 0, CM_ROWS = 1, CM_KEYS = 2 };
constexpr int kCrossRing = 4;

template <int D>
struct CrossCfg {
    static constexpr int NBOX = D / 64;
    static constexpr int BOX_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = NBOX * BOX_BYTES;
    // key and value tiles in flight each (what shared memory holds; a power of 2)
    static constexpr int STAGES = D == 64 ? 4 : 2, LOG_STAGES = D == 64 ? 2 : 1;
    static constexpr int OFF_Q = 0, OFF_K = 2 * TILE_BYTES, OFF_V = OFF_K + STAGES * TILE_BYTES;
    static constexpr int OFF_OUT = OFF_V + STAGES * TILE_BYTES;            // 4 KB for each softmax warp
    static constexpr int SMEM_BYTES = OFF_OUT + 8 * 4096 + 1024;   // + alignment slack
    static constexpr uint32_t COL_S = 0, COL_O = 256;   // S_t at 128 t, O_t at 256 + 128 t
    static constexpr int THREADS = 384;
    // 168 registers a thread at launch; the producer warpgroup drops to 56 and
    // the two softmax warpgroups rise to 224: 2 * 128 * 224 + 128 * 56 = 384 * 168
    // (with 232 and 40 masked keys took 11 % longer, the rest the same)
    static constexpr int REGS_SOFTMAX = 224, REGS_PRODUCER = 56;
};

enum : int {
    CB_QFULL = 0, CB_QEMPTY = 2, CB_KFULL = 4, CB_KEMPTY = 8, CB_VFULL = 12, CB_VEMPTY = 16,
    CB_VFIX = 20, CB_SFULL = 24, CB_P1 = 26, CB_P2 = 28, CB_OFULL = 30, CB_DRAIN = 32,
    CB_IFULL = 33, CB_IEMPTY = 37, CB_COUNT = 41
};

// The plan of a launch in shared memory, from one address on: the key tiles of a
// chunk at most, the items in all, then the table: items (without the head blocks)
// before entry i, an entry holding cross_stride(nseg) segments.
enum : int { CP_CHUNK = 0, CP_TOTAL = 4, CP_TABLE = 8 };
__device__ __forceinline__ int cross_stride(int nseg) { return (nseg + kCrossTable - 1) / kCrossTable; }

__device__ __forceinline__ void cross_segment(const CrossParams &p, int chunk, int s, int &blocks,
                                              int &tiles, int &splits) {
    const int lq = p.cu_q[s + 1] - p.cu_q[s], lk = p.cu_k[s + 1] - p.cu_k[s];
    blocks = (lq + 2 * p.tokens - 1) / (2 * p.tokens);
    tiles = (lk + 127) / 128;
    splits = tiles == 0 ? 1 : (tiles + chunk - 1) / chunk;
}

// Writes item `it` to the ring slot `to`.
__device__ __forceinline__ void cross_find_item(const CrossParams &p, uint32_t plan, int it,
                                                uint32_t to) {
    const int unit = it / p.heads_blocks, chunk = lds32(plan + CP_CHUNK);
    const int stride = cross_stride(p.nseg);
    int lo = 0, hi = (p.nseg + stride - 1) / stride;   // the last entry that begins at or before unit
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (lds32(plan + CP_TABLE + mid * 4) <= unit) lo = mid; else hi = mid;
    }
    int s = lo * stride, before = lds32(plan + CP_TABLE + lo * 4), blocks, tiles, splits;
    while (true) {
        cross_segment(p, chunk, s, blocks, tiles, splits);
        if (unit < before + blocks * splits || s + 1 >= p.nseg) break;
        before += blocks * splits;
        ++s;
    }
    const int in_seg = unit - before, block = in_seg / splits, split = in_seg - block * splits;
    // chunks of tiles / splits key tiles, the first ones of one more
    const int each = tiles / splits, more = tiles - each * splits;
    const int first = split * each + min(split, more);
    const int head = it - unit * p.heads_blocks;
    const int q0 = p.cu_q[s] + block * 2 * p.tokens, k0 = p.cu_k[s] + first * 128;
    sts32(to + CX_Q0, q0);
    const int q_left = min(p.cu_q[s + 1] - q0, 2 * p.tokens);
    sts32(to + CX_Q_LEFT, q_left);
    sts32(to + CX_MODE, q_left > p.tokens ? CM_ROWS : (p.split && tiles > 1 ? CM_KEYS : CM_ONE));
    sts32(to + CX_HEAD, head);
    sts32(to + CX_K0, k0);
    sts32(to + CX_K_LEFT, p.cu_k[s + 1] - k0);
    sts32(to + CX_N_KV, each + (split < more));
    sts32(to + CX_SPLITS, splits);
    sts32(to + CX_GROUP, (before + block * splits) * p.heads_blocks + head);
    sts32(to + CX_ITEM, it);
}

// 3-D tile of a [N, H, D] tensor's map (dims D, H, N).
__device__ __forceinline__ void cross_load(uint8_t *dst, const CUtensorMap *map, uint64_t *bar,
                                           int boxes, int head, int token) {
    for (int b = 0; b < boxes; ++b)
        tma_load_3d(dst + b * 128 * 128, map, bar, b * 64, head, token);
}

// s = -infinity unless `keep`. In place: written as a select, the compiler kept two
// copies of the score registers and spilled.
__device__ __forceinline__ void drop_unless(uint32_t &s, uint32_t keep) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.u32 p, %1, 0;\n\t"
        "@p mov.b32 %0, 0xff800000;\n\t}" : "+r"(s) : "r"(keep));
}

__device__ __forceinline__ int lane_now() {
    int v;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(v));
    return v;
}
__device__ __forceinline__ int threadIdx_x_now() {
    int v;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(v));
    return v;
}

// (y0, y1) = (x0, x1) * s, lane-wise, s a packed pair
__device__ __forceinline__ void fmul2(float &y0, float &y1, float x0, float x1, uint64_t s) {
    asm("{\n\t.reg .b64 xa, da;\n\t"
        "mov.b64 xa, {%2, %3};\n\t"
        "mul.rn.f32x2 da, xa, %4;\n\t"
        "mov.b64 {%0, %1}, da;\n\t}"
        : "=f"(y0), "=f"(y1) : "f"(x0), "f"(x1), "l"(s));
}

template <typename T, int D>
__global__ void __launch_bounds__(384, 1)
    cross_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const CrossParams p) {
    using C = CrossCfg<D>;
    // fp16: P is scaled by 2^6 so that values down to 2^-20 of the row's
    // largest stay normal; with the 2^8 of slack the largest is 2^14
    constexpr float P_SHIFT = std::is_same<T, __half>::value ? 6.0f : 0.0f;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // static, so that their addresses take no registers
    __shared__ __align__(64) uint64_t bars[CB_COUNT];
    __shared__ __align__(16) int ring_s[kCrossRing * CX_BYTES / 4];
    __shared__ int plan_s[2 + kCrossTable + 1];
    __shared__ int flags_s[2];                    // abort, TMEM address
    __shared__ unsigned long long units_s;
    volatile int *abort = flags_s;
    int *table = plan_s + CP_TABLE / 4;
    const uint32_t plan = smem_u32(plan_s);

    // ---- the boundaries, checked by every CTA; the work they make
    const int stride = cross_stride(p.nseg), entries = (p.nseg + stride - 1) / stride;
    int chunk = 1 << 24;   // more than any segment has: no split
    if (tid == 0) {
        reset_status(p.status);
        units_s = 0;
    }
    int bad = 0;
    unsigned long long units = 0;
    for (int i = tid; i <= p.nseg; i += C::THREADS) {
        const int a = p.cu_q[i], b = p.cu_k[i];
        if (i == 0 && (a != 0 || b != 0)) bad = 1;
        if (i == p.nseg && (a > p.Nq || b > p.Nk)) bad = 1;
        if (i > 0) {
            const int pa = p.cu_q[i - 1], pb = p.cu_k[i - 1];
            if (a < pa || a - pa > p.max_q || b < pb || b - pb > p.max_k) bad = 1;
            units += static_cast<unsigned long long>((a - pa + 2 * p.tokens - 1) / (2 * p.tokens)) *
                     static_cast<unsigned>((b - pb + 127) / 128);
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.x == 0) atomicCAS(p.status, 0, 7);
        return;
    }
    if (p.split) {
        if (units) atomicAdd(&units_s, units);
        __syncthreads();
        const unsigned long long all = units_s * static_cast<unsigned>(p.heads_blocks);
        chunk = static_cast<int>(max((all + kCrossItems - 1) / kCrossItems,
                                     static_cast<unsigned long long>(kCrossMinChunk)));
    }
    for (int e = tid; e < entries; e += C::THREADS) {
        int sum = 0;
        for (int s = e * stride; s < min((e + 1) * stride, p.nseg); ++s) {
            int blocks, tiles, splits;
            cross_segment(p, chunk, s, blocks, tiles, splits);
            sum += blocks * splits;
        }
        table[e + 1] = sum;
    }
    if (tid == 0) {
        table[0] = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[CB_QFULL + s], 1);
            mbar_init(&bars[CB_QEMPTY + s], 1);
            mbar_init(&bars[CB_SFULL + s], 1);
            mbar_init(&bars[CB_P1 + s], 4);
            mbar_init(&bars[CB_P2 + s], 4);
            mbar_init(&bars[CB_OFULL + s], 1);
        }
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bars[CB_KFULL + s], 1);
            mbar_init(&bars[CB_KEMPTY + s], 2);   // one commit for each tile
            mbar_init(&bars[CB_VFULL + s], 1);
            mbar_init(&bars[CB_VEMPTY + s], 3);   // and warp 9, which passes every value tile
            mbar_init(&bars[CB_VFIX + s], 1);
        }
        mbar_init(&bars[CB_DRAIN], 1);
        for (int i = 0; i < kCrossRing; ++i) {
            mbar_init(&bars[CB_IFULL + i], 1);
            mbar_init(&bars[CB_IEMPTY + i], 11);   // every warp but the one that fills it
        }
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(reinterpret_cast<uint32_t *>(flags_s + 1), 512);
        tmem_relinquish();
    }
    if (warp == 10 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncthreads();
    if (warp == 0) {   // running sums of the table
        int carry = 0;
        for (int e = 0; e < entries; e += 32) {
            int x = e + lane < entries ? table[e + lane + 1] : 0;
            for (int d = 1; d < 32; d *= 2) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            x += carry;
            if (e + lane < entries) table[e + lane + 1] = x;
            carry = __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            sts32(plan + CP_CHUNK, chunk);
            sts32(plan + CP_TOTAL, carry * p.heads_blocks);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(lds32(smem_u32(flags_s + 1)));

    const uint32_t bar0 = smem_u32(bars), abort_at = smem_u32(flags_s);
    const uint32_t ring = smem_u32(ring_s);
    auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_at(bar0 + bar * 8, parity, abort_at));
    };
    // The n-th item: its ring slot, when it is there, and its release by this warp.
    // (These waits last as long as items do, so their limit is that of many tiles' waits;
    // a wait that gives up elsewhere in the CTA ends them at once.)
    constexpr long long kItemLimit = 64 * kWaitLimitCycles;
    auto item_wait = [&](uint32_t n) {
        return __all_sync(0xffffffffu, mbar_wait_at(bar0 + (CB_IFULL + n % kCrossRing) * 8,
                                                    (n / kCrossRing) & 1, abort_at, kItemLimit));
    };
    auto item_done = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) mbar_arrive_at(bar0 + (CB_IEMPTY + n % kCrossRing) * 8);
    };
    // stage of key tile number n of this CTA, and the parity of its phase there
    auto stage_of = [](int n) { return n & (C::STAGES - 1); };
    auto phase_of = [](int n) { return static_cast<uint32_t>(n >> C::LOG_STAGES) & 1u; };
    // keys of key tile j
    auto keys_in = [](int k_left, int j) { return min(k_left - j * 128, 128); };
    // which of a key tile's 32 keys from `c` on count, for all lanes
    auto keys_valid = [&](int k0, int keys, int c) {
        c += lane;
        return __ballot_sync(0xffffffffu, c < keys && (p.mask == nullptr || p.mask[k0 + c] != 0));
    };

    if (warp == 11) {
        // ============================ items ===================================
        reg_dealloc<C::REGS_PRODUCER>();
        uint32_t n = 0;
        bool ok = true;
        for (int it = blockIdx.x; ok; it += gridDim.x, ++n) {
            const bool more = it < lds32(plan + CP_TOTAL);
            ok = __all_sync(0xffffffffu, mbar_wait_at(bar0 + (CB_IEMPTY + n % kCrossRing) * 8,
                                                      ((n / kCrossRing) & 1) ^ 1, abort_at, kItemLimit));
            if (!ok) break;
            if (lane == 0) {
                const uint32_t to = ring + (n % kCrossRing) * CX_BYTES;
                if (more) cross_find_item(p, plan, it, to);
                else sts32(to + CX_N_KV, -1);
                mbar_arrive_at(bar0 + (CB_IFULL + n % kCrossRing) * 8);
            }
            if (!more) break;
        }
        if (!ok && lane == 0) give_up(abort, p.status);
        __syncwarp();
    } else if (warp == 10) {
        // ============================ TMA producer ============================
        reg_dealloc<C::REGS_PRODUCER>();
        const uint32_t leader = elect_one();
        const uint32_t q_bytes = static_cast<uint32_t>(C::NBOX * 128 * p.hp * p.tokens);
        int nq[2] = {0, 0}, nk = 0, nv = 0;   // loads issued
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            if (!ok) break;
            const uint32_t x = ring + (n % kCrossRing) * CX_BYTES;
            const int n_kv = lds32(x + CX_N_KV), head = lds32(x + CX_HEAD) * p.hp;
            const int kv_head = head / (p.Hq / p.Hk), q0 = lds32(x + CX_Q0), k0 = lds32(x + CX_K0);
            const int n_t = lds32(x + CX_MODE) == CM_ROWS ? 2 : 1;
            item_done(n);
            if (n_kv < 0) break;
            for (int j = 0; ok && j < n_kv; ++j) {
                const int s = stage_of(nk);
                ok = wait(CB_KEMPTY + s, phase_of(nk) ^ 1);
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&bars[CB_KFULL + s], C::TILE_BYTES);
                    cross_load(smem + C::OFF_K + s * C::TILE_BYTES, &tmK, &bars[CB_KFULL + s],
                               C::NBOX, kv_head, k0 + j * 128);
                }
                ++nk;
                // behind the keys, whose room is free earlier
                if (j == 0)
                    for (int t = 0; ok && t < n_t; ++t) {
                        ok = wait(CB_QEMPTY + t, (nq[t] & 1) ^ 1);
                        if (!ok) break;
                        if (leader) {
                            mbar_arrive_expect_tx(&bars[CB_QFULL + t], q_bytes);
                            cross_load(smem + C::OFF_Q + t * C::TILE_BYTES, &tmQ,
                                       &bars[CB_QFULL + t], C::NBOX, head, q0 + t * p.tokens);
                        }
                        ++nq[t];
                    }
                if (!ok) break;
                ok = wait(CB_VEMPTY + s, phase_of(nv) ^ 1);
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(&bars[CB_VFULL + s], C::TILE_BYTES);
                    cross_load(smem + C::OFF_V + s * C::TILE_BYTES, &tmV, &bars[CB_VFULL + s],
                               C::NBOX, kv_head, k0 + j * 128);
                }
                ++nv;
            }
        }
        if (!ok && leader) give_up(abort, p.status);
        if (*abort) {
            // the copies still in flight land before shared memory is released
            for (int t = 0; t < 2; ++t)
                if (nq[t] > 0) mbar_wait(&bars[CB_QFULL + t], (nq[t] - 1) & 1, nullptr);
            for (int j = max(nk - C::STAGES, 0); j < nk; ++j)
                mbar_wait(&bars[CB_KFULL + stage_of(j)], phase_of(j), nullptr);
            for (int j = max(nv - C::STAGES, 0); j < nv; ++j)
                mbar_wait(&bars[CB_VFULL + stage_of(j)], phase_of(j), nullptr);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ============================ value rows that must not count ==========
        reg_dealloc<C::REGS_PRODUCER>();
        int nv = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            if (!ok) break;
            const uint32_t x = ring + (n % kCrossRing) * CX_BYTES;
            const int n_kv = lds32(x + CX_N_KV), k0 = lds32(x + CX_K0), k_left = lds32(x + CX_K_LEFT);
            item_done(n);
            if (n_kv < 0) break;
            // the mask of a key tile is read while the tile before is at work
            uint32_t bytes = 0;   // of keys lane, lane + 32, lane + 64, lane + 96
            auto mask_of = [&](int j) {
                uint32_t b = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = j * 128 + i * 32 + lane;
                    if (c < k_left && (p.mask == nullptr || p.mask[k0 + c] != 0)) b |= 1u << i;
                }
                return b;
            };
            if (n_kv > 0) bytes = mask_of(0);
            for (int j = 0; ok && j < n_kv; ++j, ++nv) {
                const int keys = keys_in(k_left, j), s = stage_of(nv);
                const bool fix = p.mask != nullptr || keys % 16 != 0;
                const uint32_t now = bytes;
                if (j + 1 < n_kv) bytes = mask_of(j + 1);
                // every phase is waited for, those of tiles that need nothing too, and
                // the stage is filled again only after that: a parity tells a phase
                // from its neighbours only, so a turn of the ring behind, this warp
                // would take a later tile for its own
                ok = wait(CB_VFULL + s, phase_of(nv));
                if (!ok) break;
                if (!fix) {
                    if (lane == 0) mbar_arrive_at(bar0 + (CB_VEMPTY + s) * 8);
                    continue;
                }
                uint8_t *v = smem + C::OFF_V + s * C::TILE_BYTES + (lane & 7) * 16;
                // four rows a step, eight lanes a row
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t valid = __ballot_sync(0xffffffffu, (now >> i) & 1u) >> (lane / 8);
#pragma unroll
                    for (int r = 0; r < 32; r += 4)
                        if (!((valid >> r) & 1u))
                            for (int b = 0; b < C::NBOX; ++b)
                                *reinterpret_cast<uint4 *>(v + b * C::BOX_BYTES + (i * 32 + r + lane / 8) * 128) =
                                    make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_at(bar0 + (CB_VFIX + s) * 8);
                    mbar_arrive_at(bar0 + (CB_VEMPTY + s) * 8);
                }
            }
        }
        if (!ok && lane == 0) give_up(abort, p.status);
        __syncwarp();
    } else if (warp == 8) {
        // ============================ MMA issuer ==============================
        reg_dealloc<C::REGS_PRODUCER>();
        const uint32_t leader = elect_one();
        constexpr uint32_t IDESC_S = idesc_f32<T>(128, 0, false, false);
        constexpr uint32_t IDESC_O = idesc_f32<T>(128, D, false, true);
        const uint64_t dQ = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
        const uint64_t dK = sdesc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
        const uint64_t dV = sdesc_sw128(smem_u32(smem + C::OFF_V), C::BOX_BYTES, 1024);
        auto mma_wait = [&](int bar, uint32_t parity) {
            const bool r = wait(bar, parity);
            tc_fence_after();
            return r;
        };
        auto issue_s = [&](int t, int tq, int stage, int keys) {
            const uint32_t n16 = static_cast<uint32_t>((keys + 15) / 16);
            const uint64_t dq = dQ + static_cast<uint64_t>((tq * C::TILE_BYTES) >> 4);
            const uint64_t dk = dK + static_cast<uint64_t>((stage * C::TILE_BYTES) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
                umma_ss_w(tmem + C::COL_S + t * 128, dq + off, dk + off, IDESC_S | ((n16 * 2) << 17),
                          kk > 0 ? 1u : 0u, leader);
            }
        };
        auto issue_pv = [&](int t, int stage, int from, int to, bool add) {
            const uint64_t dv = dV + static_cast<uint64_t>((stage * C::TILE_BYTES + from * 2048) >> 4);
            const uint32_t o = tmem + C::COL_O + t * 128, a = tmem + C::COL_S + t * 128 + from * 8;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                if (from + kk < to)
                    umma_ts_w(o, a + kk * 8, dv + static_cast<uint64_t>((kk * 2048) >> 4), IDESC_O,
                              (add || kk > 0) ? 1u : 0u, leader);
        };
        uint32_t nq = 0, g = 0;              // parities of the next Q and P phases, a bit a tile
        int nkv = 0;                         // key tiles so far
        uint32_t fixes = 0;                  // parity of the next VFIX phase, a bit a stage
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            if (!ok) break;
            const uint32_t x = ring + (n % kCrossRing) * CX_BYTES;
            const int n_kv = lds32(x + CX_N_KV), k_left = lds32(x + CX_K_LEFT);
            const bool keys_mode = lds32(x + CX_MODE) == CM_KEYS;
            const int n_t = lds32(x + CX_MODE) == CM_ROWS ? 2 : 1;
            item_done(n);
            if (n_kv < 0) break;
            if (keys_mode) {
                ok = mma_wait(CB_QFULL, nq & 1);
                nq ^= 1u;
                for (int j = -2; ok && j < n_kv; ++j) {   // key tile j: values of j, scores of j + 2
                    const int t = j & 1, s = stage_of(nkv);
                    if (j >= 0) {
                        const int keys = keys_in(k_left, j), n16 = (keys + 15) / 16;
                        ok = mma_wait(CB_VFULL + s, phase_of(nkv));
                        if (ok && (p.mask != nullptr || keys % 16 != 0)) {
                            ok = mma_wait(CB_VFIX + s, (fixes >> s) & 1);
                            fixes ^= 1u << s;
                        }
                        ok = ok && mma_wait(CB_P1 + t, (g >> t) & 1);
                        if (!ok) break;
                        issue_pv(t, s, 0, n16, j >= 2);
                        ok = mma_wait(CB_P2 + t, (g >> t) & 1);
                        if (!ok) break;
                        issue_pv(t, s, 4, n16, true);
                        umma_commit_w(&bars[CB_VEMPTY + s], leader);
                        umma_commit_w(&bars[CB_VEMPTY + s], leader);
                        if (j + 2 >= n_kv) umma_commit_w(&bars[CB_OFULL + t], leader);
                        g ^= 1u << t;
                        ++nkv;
                    }
                    if (j + 2 < n_kv) {
                        const int at = j < 0 ? nkv + j + 2 : nkv + 1;   // = this item's key tile j + 2
                        ok = mma_wait(CB_KFULL + stage_of(at), phase_of(at));
                        if (!ok) break;
                        issue_s(t, 0, stage_of(at), keys_in(k_left, j + 2));
                        umma_commit_w(&bars[CB_SFULL + t], leader);
                        umma_commit_w(&bars[CB_KEMPTY + stage_of(at)], leader);
                        umma_commit_w(&bars[CB_KEMPTY + stage_of(at)], leader);
                        if (j + 3 == n_kv) umma_commit_w(&bars[CB_QEMPTY], leader);
                    }
                }
                continue;
            }
            for (int t = 0; ok && n_kv > 0 && t < n_t; ++t) {
                ok = mma_wait(CB_QFULL + t, (nq >> t) & 1) && mma_wait(CB_KFULL + stage_of(nkv), phase_of(nkv));
                if (!ok) break;
                issue_s(t, t, stage_of(nkv), keys_in(k_left, 0));
                umma_commit_w(&bars[CB_SFULL + t], leader);
                umma_commit_w(&bars[CB_KEMPTY + stage_of(nkv)], leader);
                if (n_t == 1) umma_commit_w(&bars[CB_KEMPTY + stage_of(nkv)], leader);
                if (n_kv == 1) umma_commit_w(&bars[CB_QEMPTY + t], leader);
                nq ^= 1u << t;
            }
            for (int j = 0; ok && j < n_kv; ++j, ++nkv) {
                // everything but P is waited for ahead of P, whose arrival is what the
                // tensor cores wait for
                const int s = stage_of(nkv), s1 = stage_of(nkv + 1), keys = keys_in(k_left, j), n16 = (keys + 15) / 16;
                const bool more = j + 1 < n_kv;
                ok = mma_wait(CB_VFULL + s, phase_of(nkv));
                if (ok && (p.mask != nullptr || keys % 16 != 0)) {
                    ok = mma_wait(CB_VFIX + s, (fixes >> s) & 1);
                    fixes ^= 1u << s;
                }
                const int next_keys = keys_in(k_left, j + 1);
                for (int t = 0; ok && t < n_t; ++t) {
                    ok = mma_wait(CB_P1 + t, (g >> t) & 1);
                    if (!ok) break;
                    issue_pv(t, s, 0, n16, j > 0);
                    if (more && t == 0) ok = mma_wait(CB_KFULL + s1, phase_of(nkv + 1));
                    ok = ok && mma_wait(CB_P2 + t, (g >> t) & 1);
                    if (!ok) break;
                    issue_pv(t, s, 4, n16, true);
                    if (more) {
                        umma_commit_w(&bars[CB_VEMPTY + s], leader);
                        issue_s(t, t, s1, next_keys);
                        umma_commit_w(&bars[CB_SFULL + t], leader);
                        umma_commit_w(&bars[CB_KEMPTY + s1], leader);
                        if (n_t == 1) umma_commit_w(&bars[CB_KEMPTY + s1], leader);
                        if (j + 2 == n_kv) umma_commit_w(&bars[CB_QEMPTY + t], leader);
                    } else {
                        umma_commit_w(&bars[CB_OFULL + t], leader);
                        umma_commit_w(&bars[CB_VEMPTY + s], leader);
                    }
                    if (n_t == 1) umma_commit_w(&bars[CB_VEMPTY + s], leader);
                    g ^= 1u << t;
                }
            }
        }
        if (!ok) {
            if (leader) give_up(abort, p.status);
            umma_commit_w(&bars[CB_DRAIN], leader);
            mbar_wait(&bars[CB_DRAIN], 0, nullptr);
        }
        __syncwarp();
    } else {
        // ============================ softmax / output ========================
        reg_alloc<C::REGS_SOFTMAX>();
        const int t = warp >> 2;                 // query tile of this warpgroup
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + C::COL_S + t * 128;
        const uint32_t tO = tS + (C::COL_O - C::COL_S);
        const float sl2 = p.scale_log2;
        uint32_t par = 0;   // parities of the next phases: 1 S, 2 O
        const uint32_t bar_t = bar0 + t * 8;   // of this tile's barriers, less their number * 8
        auto wait_t = [&](int bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_at(bar_t + bar * 8, parity, abort_at));
        };
        bool ok = true;   // false from the first wait that gave up
        for (uint32_t n = 0; ; item_done(n), ++n) {
            if (!ok || !item_wait(n)) {
                if (lane == 0) give_up(abort, p.status);
                break;
            }
            const uint32_t xs = ring + (n % kCrossRing) * CX_BYTES;   // read again after the loop
            const int mode = lds32(xs + CX_MODE);
            int n_kv = lds32(xs + CX_N_KV), k_left = lds32(xs + CX_K_LEFT);
            if (n_kv < 0) break;
            if (mode == CM_ONE && t == 1) continue;
            const bool two = mode == CM_ROWS;
            int step = 128;   // keys from one key tile of this query tile to its next
            if (mode == CM_KEYS) {
                step = 256;
                k_left -= t * 128;
                n_kv = (n_kv + 1 - t) >> 1;
            }
            // a warp without rows only signals
            const bool active = (warp & 3) * 32 <
                                min(lds32(xs + CX_Q_LEFT) - (two ? t * p.tokens : 0), p.tokens) * p.hp;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; ok && !active && j < n_kv; ++j) {
                ok = wait_t(CB_SFULL, par & 1);
                par ^= 1u;
                if (lane == 0) {
                    mbar_arrive_at(bar_t + CB_P1 * 8);
                    mbar_arrive_at(bar_t + CB_P2 * 8);
                }
            }
            // One key tile of this warp's rows, `keys` of them left; `part`: not all count.
            // Two copies of the code, so that only one of them pays for the masking.
            auto softmax_tile = [&](auto part, int keys, int j) {
                uint32_t valid[4];
                if constexpr (decltype(part)::value) {
                    const int k0 = lds32(xs + CX_K0) + lds32(xs + CX_K_LEFT) - keys;
#pragma unroll
                    for (int i = 0; i < 4; ++i) valid[i] = keys_valid(k0, keys, i * 32);
                }
                ok = wait_t(CB_SFULL, par & 1);
                par ^= 1u;
                if (!ok) return;
                tc_fence_after();
                uint32_t s[128];
                tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
                tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
                tmem_wait_ld();
                if constexpr (decltype(part)::value) {
#pragma unroll
                    for (int q = 0; q < 128; ++q) drop_unless(s[q], valid[q >> 5] & (1u << (q & 31)));
                    // no key of this tile counts: P = 0, nothing else changes
                    if ((valid[0] | valid[1] | valid[2] | valid[3]) == 0) {
                        uint32_t z[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[i] = 0u;
                        tmem_st32(tS + 0, z);
                        tmem_st32(tS + 32, z);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive_at(bar_t + CB_P1 * 8);
                            mbar_arrive_at(bar_t + CB_P2 * 8);
                        }
                        return;
                    }
                }
                float mq[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mq[i] = __uint_as_float(s[i]);
#pragma unroll
                for (int c = 8; c < 120; c += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mq[i] = fmax3(mq[i], __uint_as_float(s[c + i]), __uint_as_float(s[c + 8 + i]));
#pragma unroll
                for (int i = 0; i < 8; ++i) mq[i] = fmaxf(mq[i], __uint_as_float(s[120 + i]));
                const float mx = fmaxf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])),
                                       fmaxf(fmaxf(mq[4], mq[5]), fmaxf(mq[6], mq[7])));
                const float m_new = mx * sl2;
                // (false while no score is above -infinity: m stays there.) The
                // accumulator holds something from the item's second key tile on
                const bool grow = m_new > m + 8.0f;
                const bool need = grow && j > 0;
                const float f = need ? ex2_approx(m - m_new) : 1.0f;
                if (grow) {
                    l *= need ? f : 0.0f;
                    m = m_new;
                }
                // scores of -infinity weigh 0 also before any other score
                const float nm = P_SHIFT - (m == -INFINITY ? 0.0f : m);
                uint64_t acc0 = 0, acc1 = 0;
                const uint64_t s2 = f2_splat(sl2), n2 = f2_splat(nm);
                // P of keys [32 h, 32 h + 32): to T for the PV product (kind::f16 takes A
                // and B of one 16-bit type), into the sum as it is. That rounding adds about
                // as much error as O's own (bf16, against 64 bits: 1.7e-3 with P in fp32,
                // 2.3e-3 so). All exponentials on MUFU: with three pairs of
                // eight as polynomials on the FMA pipe, as the dense kernel has them, the
                // packed clips took 2 % longer
                auto exp_part = [&](const int h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float x0, x1, p0, p1;
                        ffma2(x0, x1, __uint_as_float(s[32 * h + 2 * c]),
                              __uint_as_float(s[32 * h + 2 * c + 1]), s2, n2);
                        p0 = ex2_approx(x0);
                        p1 = ex2_approx(x1);
                        if (c & 1) fadd2(acc1, p0, p1); else fadd2(acc0, p0, p1);
                        pk[c] = pack2<T>(p0, p1);
                    }
                    tmem_st16(tS + 16 * h, pk);
                };
                exp_part(0);
                exp_part(1);
                if (__any_sync(0xffffffffu, need)) {
                    // O holds P V up to the tile before; rescale it before P is released
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(tO + c * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(bar_t + CB_P1 * 8);
                exp_part(2);
                exp_part(3);
                l += f2_sum(acc0) + f2_sum(acc1);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(bar_t + CB_P2 * 8);
            };
            for (int j = 0; ok && active && j < n_kv; ++j) {
                const int keys = k_left - j * step;   // and more, behind the tile
                if (keys < 128 || p.mask != nullptr) softmax_tile(std::true_type{}, keys, j);
                else softmax_tile(std::false_type{}, keys, j);
            }
            if (n_kv > 0) {
                ok = ok && wait_t(CB_OFULL, (par >> 1) & 1);
                par ^= 2u;
                tc_fence_after();
            }
            if (!ok && lane == 0) give_up(abort, p.status);
            const int t_first = two ? t * p.tokens : 0;   // first token of this tile
            const int rows = min(lds32(xs + CX_Q_LEFT) - t_first, p.tokens) * p.hp;
            // read anew, or what depends on them alone (a dozen addresses) is kept in
            // registers through the score loop, which then spills
            const int lane = lane_now(), warp = threadIdx_x_now() >> 5;
            const int r = (warp & 3) * 32 + lane;
            const bool row_ok = r < rows;
            const int tok = r / p.hp;
            const int qrow = lds32(xs + CX_Q0) + t_first + tok, head = lds32(xs + CX_HEAD) * p.hp + r - tok * p.hp;
            const int parts = lds32(xs + CX_SPLITS) * (mode == CM_KEYS ? 2 : 1);
            if (!ok || !active) continue;
            if (parts == 1) {
                // a row without keys: O is 0 or, without a single key tile, not there (a
                // sum of NaN is neither: it shows in O and in the LSE)
                const uint64_t inv2 = f2_splat(l == 0.0f ? 0.0f : 1.0f / l);
                // 64 channels at a time through shared memory (16-byte pieces, their
                // place exclusive-or'ed with the row), so that a store writes four
                // whole 128-byte lines; 16 bytes of each of 32 rows at a time took 4 to
                // 5 thousand cycles a tile and left sectors half written
                const int64_t at = row_ok ? qrow * p.ldo + static_cast<int64_t>(head) * D : -1;
                const uint32_t out = smem_u32(smem) + C::OFF_OUT + warp * 4096;
#pragma unroll 1
                for (int c = 0; c < D; c += 64) {
                    __syncwarp();
#pragma unroll 1
                    for (int q = 0; q < 64; q += 32) {
                        uint32_t o[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                        if (n_kv > 0) tmem_ld32(tO + c + q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            fmul2(y0, y1, __uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]), inv2);
                            o[i] = pack2<T>(y0, y1);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sts128(out + lane * 128 + (((q / 8 + i) ^ (lane & 7)) << 4), o[4 * i],
                                   o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                    __syncwarp();
                    // loads, then stores: their latencies overlap
                    uint4 v[8];
                    int64_t row_at[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = i * 4 + lane / 8;
                        v[i] = lds128(out + rr * 128 + (((lane ^ rr) & 7) << 4));
                        row_at[i] = __shfl_sync(0xffffffffu, at, rr);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (row_at[i] >= 0)
                            *reinterpret_cast<uint4 *>(static_cast<T *>(p.o) + row_at[i] + c +
                                                       (lane & 7) * 8) = v[i];
                }
                if (row_ok && p.lse != nullptr)
                    p.lse[static_cast<int64_t>(head) * p.Nq + qrow] =
                        l == 0.0f ? -INFINITY : (m + (log2f(l) - P_SHIFT)) * 0.69314718055994530942f;
                if (p.split && row_ok)   // not among the parts
                    p.rows[static_cast<int64_t>(qrow) * p.Hq + head] = make_int2(0, 0);
                continue;
            }
            // ---- one of several parts of these rows: O, m and l as they are
            const int64_t first = static_cast<int64_t>(lds32(xs + CX_ITEM)) * 2 + t;
            float *mine = p.parts + (first * p.slot_rows + r) * (D + 2);
            if (row_ok) {
                *reinterpret_cast<float2 *>(mine) = make_float2(m, l);
                // the rows' first part says where they are
                if (lds32(xs + CX_ITEM) == lds32(xs + CX_GROUP) && (mode != CM_KEYS || t == 0))
                    p.rows[static_cast<int64_t>(qrow) * p.Hq + head] = make_int2(
                        static_cast<int>(first * p.slot_rows) + r, mode == CM_KEYS ? -parts : parts);
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0u;   // without a key tile
                if (n_kv > 0) tmem_ld16(tO + c, o);
                tmem_wait_ld();
                if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        *reinterpret_cast<uint2 *>(mine + 2 + c + i) = make_uint2(o[i], o[i + 1]);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the rows that have several: a block a row, every fourth part
// a warp, lane i the weight of its warp's i-th, then all lanes the channels; the
// warps' sums in the warps' order. Part i of a row lies one item's slots (both
// tiles') behind the other or, where an item's two tiles share rows (count
// negative), tile by tile.
template <typename T, int D>
__global__ void __launch_bounds__(128) cross_join_kernel(const CrossParams p) {
    constexpr float P_SHIFT = std::is_same<T, __half>::value ? 6.0f : 0.0f;
    __shared__ float m_s[4], sum_s[4], o_s[4][D];
    if (*p.status != 0) return;   // the main kernel has not written what is read here
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t row = blockIdx.x;
    if (row >= static_cast<int64_t>(p.cu_q[p.nseg]) * p.Hq) return;
    const int2 at = p.rows[row];
    const bool pairs = at.y < 0;
    const int parts = pairs ? -at.y : at.y;
    if (parts == 0) return;
    const int64_t tile = static_cast<int64_t>(p.slot_rows) * (D + 2);   // floats
    const int64_t item = 2 * tile * p.heads_blocks;
    const float *all = p.parts + static_cast<int64_t>(at.x) * (D + 2);
    auto part = [&](int i) { return all + (pairs ? (i >> 1) * item + (i & 1) * tile : i * item); };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < parts; i += 128) m = fmaxf(m, part(i)[0]);
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) m_s[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
    const float m0 = m == -INFINITY ? 0.0f : m;   // then every part weighs 0
    float sum = 0.0f, o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = 0.0f;
    for (int i0 = warp; i0 < parts; i0 += 128) {
        float w = 0.0f;
        const int mine = i0 + lane * 4;
        if (mine < parts) {
            const float2 ml = *reinterpret_cast<const float2 *>(part(mine));
            w = ex2_approx(ml.x - m0);
            sum = fmaf(w, ml.y, sum);
        }
        const int n = min((parts - i0 + 3) / 4, 32);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const float *a = part(i0 + 4 * i) + 2 + lane * 2;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float2 v = *reinterpret_cast<const float2 *>(a + c * 64);
                o[2 * c] = fmaf(wi, v.x, o[2 * c]);
                o[2 * c + 1] = fmaf(wi, v.y, o[2 * c + 1]);
            }
        }
    }
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) sum_s[warp] = sum;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        o_s[warp][c * 64 + lane * 2] = o[2 * c];
        o_s[warp][c * 64 + lane * 2 + 1] = o[2 * c + 1];
    }
    __syncthreads();
    sum = ((sum_s[0] + sum_s[1]) + sum_s[2]) + sum_s[3];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int token = static_cast<int>(row / p.Hq), head = static_cast<int>(row - static_cast<int64_t>(token) * p.Hq);
    T *to = static_cast<T *>(p.o) + token * p.ldo + static_cast<int64_t>(head) * D;
    const int c = threadIdx.x;
    if (c < D) to[c] = from_f32<T>((((o_s[0][c] + o_s[1][c]) + o_s[2][c]) + o_s[3][c]) * inv);
    if (c == 0 && p.lse != nullptr)
        p.lse[static_cast<int64_t>(head) * p.Nq + token] =
            sum == 0.0f ? -INFINITY : (m + (log2f(sum) - P_SHIFT)) * 0.69314718055994530942f;
}

}  // namespace h3
