// C-ABI entry points of the layers around the attention (declared in
// include/h3attn.h): 1-D rotary positions, linear layers, cross attention.
// Host side only: argument checks, frequency tables, launches on the caller's
// stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>
#include <mutex>

#include "h3attn.h"
#include "host_util.h"
#include "cross_attn.cuh"
#include "linear.cuh"
#include "rope_qk.cuh"

namespace {

using h3host::aligned;
using h3host::cuda_fail;
using h3host::kStatusBytes;

struct Device {
    bool ready = false, sm100 = false;
    bool cross_regs_ok = false;   // see set_up_kernels
    int sms = 0;
};
// Shared memory of the kernels that need more than the default, on the current
// device. *cross_regs_ok: the launch allocation of every cross attention kernel
// covers what its softmax warpgroups raise themselves to (the raise waits for
// registers that the block holds from launch, so it would wait forever else).
template <typename Kernel>
cudaError_t big_smem(Kernel kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int D>
cudaError_t set_up_cross(bool *regs_ok) {
    using C = h3::CrossCfg<D>;
    cudaFuncAttributes a{};
    cudaError_t e = big_smem(h3::cross_attn_kernel<T, D>, C::SMEM_BYTES);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, h3::cross_attn_kernel<T, D>);
    if (a.numRegs * C::THREADS < 2 * 128 * C::REGS_SOFTMAX + 128 * C::REGS_PRODUCER) *regs_ok = false;
    return e;
}

template <typename T>
cudaError_t set_up_typed(bool *regs_ok) {
    cudaError_t e;
    if ((e = big_smem(h3::linear_tile_kernel<T, false>, h3::LinearTile::SMEM_BYTES)) != cudaSuccess ||
        (e = big_smem(h3::linear_tile_kernel<T, true>, h3::LinearTile::SMEM_BYTES)) != cudaSuccess ||
        (e = big_smem(h3::linear_skinny_kernel<T, false>, h3::LinearSkinny::SMEM_BYTES)) != cudaSuccess ||
        (e = big_smem(h3::linear_skinny_kernel<T, true>, h3::LinearSkinny::SMEM_BYTES)) != cudaSuccess ||
        (e = set_up_cross<T, 64>(regs_ok)) != cudaSuccess)
        return e;
    return set_up_cross<T, 128>(regs_ok);
}

cudaError_t set_up_kernels(bool *cross_regs_ok) {
    *cross_regs_ok = true;
    const cudaError_t e = set_up_typed<__nv_bfloat16>(cross_regs_ok);
    return e != cudaSuccess ? e : set_up_typed<__half>(cross_regs_ok);
}

constexpr int kMaxDevices = 64;
Device g_dev[kMaxDevices];
std::mutex g_dev_mu;

h3_status device_info(const Device **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return H3_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_dev_mu);
    Device &d = g_dev[dev];
    if (!d.ready) {
        int major = 0, minor = 0;
        if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return cuda_fail(e);
        d.sm100 = (major == 10 && minor == 0);
        if (d.sm100 && (e = set_up_kernels(&d.cross_regs_ok)) != cudaSuccess) return cuda_fail(e);
        d.ready = true;
    }
    if (!d.sm100) return H3_ERR_UNSUPPORTED;
    *out = &d;
    return H3_OK;
}

h3_status launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? H3_OK : cuda_fail(e);
}

// ---------------------------------------------------------------- frequencies

bool positive(double x) { return x > 0.0 && std::isfinite(x); }

// Angle per position of each pair, or false for a cfg that is refused.
bool rope_freqs(const h3_rope_qk_cfg &c, double *f) {
    const int r = c.rot_dim;
    if (r < 2 || r > 2 * h3::kRopeQkMaxPairs || (r & 1) || c.reserved != 0) return false;
    if (c.layout != H3_ROPE_INTERLEAVED && c.layout != H3_ROPE_HALF) return false;
    // (the kernel multiplies by it in fp32)
    if (!positive(c.theta) || !(std::fabs(c.attn_factor) <= FLT_MAX)) return false;
    if (c.scaling < H3_ROPE_SCALE_NONE || c.scaling > H3_ROPE_SCALE_YARN) return false;
    const double pi = 3.14159265358979323846;
    double theta = c.theta, lo = 0.0, hi = 0.0;
    if (c.scaling != H3_ROPE_SCALE_NONE && !positive(c.factor)) return false;
    if (c.scaling == H3_ROPE_SCALE_NTK) {
        if (r <= 2) return false;
        theta = c.theta * std::pow(c.factor, static_cast<double>(r) / (r - 2));
        if (!positive(theta)) return false;
    }
    if (c.scaling == H3_ROPE_SCALE_TURNS || c.scaling == H3_ROPE_SCALE_YARN) {
        if (!positive(c.original_len) || !positive(c.beta_fast) || !positive(c.beta_slow) ||
            c.beta_fast <= c.beta_slow)
            return false;
    }
    if (c.scaling == H3_ROPE_SCALE_YARN) {
        if (c.theta <= 1.0) return false;
        auto at = [&](double turns) {
            return r * std::log(c.original_len / (turns * 2.0 * pi)) / (2.0 * std::log(c.theta));
        };
        lo = std::max(std::floor(at(c.beta_fast)), 0.0);
        hi = std::min(std::ceil(at(c.beta_slow)), static_cast<double>(r - 1));
    }
    for (int j = 0; j < r / 2; ++j) {
        const double base = std::pow(theta, -2.0 * j / static_cast<double>(r));
        double keep = 1.0;
        if (c.scaling == H3_ROPE_SCALE_LINEAR) keep = 0.0;
        if (c.scaling == H3_ROPE_SCALE_TURNS)
            keep = (c.original_len * base / (2.0 * pi) - c.beta_slow) / (c.beta_fast - c.beta_slow);
        if (c.scaling == H3_ROPE_SCALE_YARN) keep = 1.0 - (j - lo) / std::max(hi - lo, 0.001);
        keep = std::min(std::max(keep, 0.0), 1.0);
        f[j] = keep == 1.0 ? base : keep * base + (1.0 - keep) * base / c.factor;
        if (!std::isfinite(f[j])) return false;
    }
    return true;
}

// f / (2 pi) turns a position, the fraction of a turn in units of 2^-64.
uint64_t phase_of(double f) {
    const long double turns = static_cast<long double>(f) / 6.283185307179586476925286766559L;
    const long double whole = turns < 9e18L ? static_cast<long double>(static_cast<int64_t>(turns))
                                            : std::floor(turns);
    const long double scaled = (turns - whole) * 18446744073709551616.0L + 0.5L;
    return scaled >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(scaled);
}

// The phases of a cfg's pairs, or false for a cfg that is refused. A thread keeps
// those of the last cfg it used: the powers cost more than the launch.
bool rope_phases(const h3_rope_qk_cfg &c, uint64_t *phase) {
    static thread_local h3_rope_qk_cfg last{};   // rot_dim 0: none
    static thread_local uint64_t kept[h3::kRopeQkMaxPairs];
    if (last.rot_dim == 0 || std::memcmp(&last, &c, sizeof(c)) != 0) {
        double f[h3::kRopeQkMaxPairs];
        if (!rope_freqs(c, f)) return false;
        for (int j = 0; j < c.rot_dim / 2; ++j) kept[j] = phase_of(f[j]);
        last = c;
    }
    std::memcpy(phase, kept, static_cast<size_t>(c.rot_dim / 2) * sizeof(uint64_t));
    return true;
}

// Blocks of 256 places; the heads are split so that an SM gets about 16 blocks, for
// even shares (8320 tokens of 72 heads: 5.87 TB/s with 16 blocks an SM, 5.20 with
// 2); a block computes its angles anew, so no further.
template <typename T, bool Wide>
void launch_rope_qk(h3::RopeQkParams &p, bool half, int sms, cudaStream_t st) {
    constexpr int E = h3::RopeVec<T, Wide>::E;
    const int pairs = half || !Wide ? E : E / 2;
    const int places = p.rot / 2 / pairs + (p.copy ? (p.D - p.rot) / E : 0);
    const int64_t blocks = (p.N * places + 255) / 256;
    const int heads = p.Hq + p.Hk;
    const int64_t parts = std::min<int64_t>(std::max<int64_t>(1, 16 * sms / blocks), (heads + 3) / 4);
    p.head_chunk = static_cast<int32_t>((heads + parts - 1) / parts + 3) / 4 * 4;
    const dim3 grid(static_cast<unsigned>(blocks),
                    static_cast<unsigned>((heads + p.head_chunk - 1) / p.head_chunk));
    if (half) h3::rope_qk_kernel<T, Wide, true><<<grid, 256, 0, st>>>(p);
    else h3::rope_qk_kernel<T, Wide, false><<<grid, 256, 0, st>>>(p);
}

// 16-byte vectors where every row, head and (for the half layout) half of the
// rotated part begins on one.
template <typename T>
void launch_rope_qk(h3::RopeQkParams &p, bool half, int sms, cudaStream_t st) {
    constexpr int E = 16 / sizeof(T);
    bool wide = p.D % E == 0 && (half ? p.rot / 2 : p.rot) % E == 0 && p.ldq % E == 0 &&
                p.ldqo % E == 0 && aligned(p.q, 16) && aligned(p.qo, 16);
    if (p.Hk > 0)
        wide = wide && p.ldk % E == 0 && p.ldko % E == 0 && aligned(p.k, 16) && aligned(p.ko, 16);
    if (wide) launch_rope_qk<T, true>(p, half, sms, st);
    else launch_rope_qk<T, false>(p, half, sms, st);
}

// --------------------------------------------------------------------- linear

bool linear_sizes_ok(int64_t M, int32_t N, int32_t K, int32_t act) {
    const int a = act & ~H3_ACT_GATED;
    return M >= 0 && M < INT32_MAX - 256 && N >= 1 && N <= (1 << 20) && K >= 1 &&
           K <= (1 << 20) && a >= H3_ACT_NONE && a <= H3_ACT_SILU;
}

// Rows of x up to which the weight rows are the MMA's rows (linear_skinny_kernel):
// 128 is its widest MMA, and a gated layer's two parts of 96 columns still fit the
// ring that they are joined in.
int64_t skinny_rows(bool gated) { return gated ? 96 : 128; }

int skinny_tiles(int32_t N) { return (N + 127) / 128; }

// CTAs that share the sum over K, a cluster: those that end first, with two CTAs
// on each SM, a step of 64 as the unit and six steps for a CTA's start and end.
int skinny_splits(int32_t N, int32_t K, int sms) {
    const int n_k = (K + 63) / 64;
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int s = 1; s <= 8 && n_k / s >= 4; s *= 2) {
        const int64_t waves = (static_cast<int64_t>(skinny_tiles(N)) * s + 2 * sms - 1) / (2 * sms);
        const int64_t cost = waves * ((n_k + s - 1) / s + 6);
        if (cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return best;
}

int skinny_cols(int64_t M) { return static_cast<int>((M + 15) / 16 * 16); }

// Output columns of a tile and the parts that the last, partial round's tiles come
// in: the cheapest sum over the rounds, a round costing its products' columns plus
// 80 (8320 x 7168 x 5376 with tiles of 128, 192, 224 and 256 columns: 19, 13, 11
// and 10 rounds of 35, 48, 53 and 57 us).
struct TileShape {
    int out_cols, pieces;
};

TileShape tile_shape(int64_t M, int32_t N, bool gated, int sms) {
    TileShape best{};
    int64_t best_cost = INT64_MAX;
    const int products = gated ? 2 : 1;
    for (int cols = 256 / products; cols >= 32; cols -= 32) {   // whole chunks of 32 outputs
        const int64_t tiles = (M + 127) / 128 * ((static_cast<int64_t>(N) + cols - 1) / cols);
        for (int pieces = 1; pieces <= 4; pieces *= 2) {
            // (without a whole round, smaller tiles do the same with a deeper ring)
            if (pieces > 1 && (cols % (32 * pieces) != 0 || tiles < sms)) break;
            const int64_t cost = tiles / sms * (products * cols + 80) +
                                 (tiles % sms * pieces + sms - 1) / sms * (products * cols / pieces + 80);
            if (cost < best_cost) {
                best_cost = cost;
                best = {cols, pieces};
            }
        }
    }
    return best;
}

// TMA map over `rows` x `cols` 16-bit elements, row stride ld, box 64 x box_rows,
// 128-byte swizzle, zeros out of bounds.
h3_status make_rows_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols,
                        int64_t ld, uint32_t box_rows) {
    const h3host::EncodeTiledFn enc = h3host::encode_tiled();
    if (enc == nullptr) return cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims,
                           strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? H3_OK : cuda_fail(cudaErrorInvalidValue);
}

template <typename Kernel, typename... Args>
h3_status launch_mma(Kernel kernel, int grid, int cluster, int threads, int smem, cudaStream_t st,
                     const Args &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();   // not to be found by the next call
    return e == cudaSuccess ? H3_OK : cuda_fail(e);
}

template <typename T, bool Gated>
h3_status launch_linear(h3::LinearParams &p, const void *x, int64_t ldx, const void *w, int64_t ldw,
                        int sms, cudaStream_t st) {
    const int64_t w_rows = Gated ? 2 * static_cast<int64_t>(p.N) : p.N;
    CUtensorMap tx, tw;
    h3_status s;
    if (p.splits > 0) {
        using C = h3::LinearSkinny;
        if ((s = make_rows_map(&tx, x, p.M, p.K, ldx, p.cols)) != H3_OK ||
            (s = make_rows_map(&tw, w, w_rows, p.K, ldw, C::BM)) != H3_OK)
            return s;
        return launch_mma(h3::linear_skinny_kernel<T, Gated>, skinny_tiles(p.N) * p.splits, p.splits,
                          C::THREADS, C::SMEM_BYTES, st, tx, tw, p);
    }
    using C = h3::LinearTile;
    CUtensorMap tw_piece;
    if ((s = make_rows_map(&tx, x, p.M, p.K, ldx, C::BM)) != H3_OK ||
        (s = make_rows_map(&tw, w, w_rows, p.K, ldw, p.out_cols)) != H3_OK ||
        (s = make_rows_map(&tw_piece, w, w_rows, p.K, ldw, p.out_cols / p.pieces)) != H3_OK)
        return s;
    return launch_mma(h3::linear_tile_kernel<T, Gated>, std::min(p.n_tiles, sms), 1, C::THREADS,
                      C::SMEM_BYTES, st, tx, tw, tw_piece, p);
}

// ------------------------------------------------------------ cross attention

bool cross_sizes_ok(int64_t Nq, int64_t Nk, int32_t Hq, int32_t Hk, int32_t nseg) {
    return Nq >= 0 && Nq <= INT32_MAX - 1 && Nk >= 0 && Nk <= INT32_MAX - 1 && Hk >= 1 &&
           Hq >= Hk && Hq <= 65535 && Hq % Hk == 0 && nseg >= 1 && nseg <= 65535;
}

struct CrossPlanHost {
    int32_t hp, tokens;       // heads and tokens of a 128-row tile
    int64_t items;            // bound on the items without a split
    bool split;
    int64_t slots;            // bound on the items with it
    int32_t slot_rows;        // of one of an item's two tiles
    int64_t rows;             // (token, query head) pairs at most
};

// A tile takes the whole group of query heads of a key head where the group
// fits, else single heads. The keys are split where the items alone could not
// give each SM two and a segment may have more than one key tile.
CrossPlanHost cross_plan(int64_t Nq, int32_t Hq, int32_t Hk, int32_t nseg, int32_t max_q,
                         int32_t max_k) {
    CrossPlanHost c;
    const int32_t group = Hq / Hk;
    c.hp = group <= 128 ? group : 1;
    c.tokens = 128 / c.hp;
    const int64_t two = 2 * c.tokens;
    c.items = std::min(nseg * ((max_q + two - 1) / two), Nq / two + nseg) * (Hq / c.hp);
    c.split = c.items < h3::kCrossItems && max_k > 128;
    c.slots = c.split ? c.items + h3::kCrossItems : 0;
    c.slot_rows = std::min(c.tokens, max_q) * c.hp;
    c.rows = std::min<int64_t>(Nq, static_cast<int64_t>(nseg) * max_q) * Hq;
    return c;
}

// Behind the status block: where each row's parts are, then the parts.
size_t cross_rows_bytes(const CrossPlanHost &c) {
    return c.split ? h3host::round_up(static_cast<size_t>(c.rows) * 8, 256) : 0;
}

// TMA map over a [N, H, D] tensor of 16-bit elements, token stride ld, box
// 64 channels x `heads` x `tokens`, 128-byte swizzle, zeros out of bounds.
h3_status make_heads_map(CUtensorMap *map, const void *base, int64_t N, int32_t H, int32_t D,
                         int64_t ld, uint32_t heads, uint32_t tokens) {
    const h3host::EncodeTiledFn enc = h3host::encode_tiled();
    if (enc == nullptr) return cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                                static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[3] = {64, heads, tokens};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims,
                           strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? H3_OK : cuda_fail(cudaErrorInvalidValue);
}

template <typename T, int D>
h3_status launch_cross(const h3::CrossParams &p, int grid, int64_t rows, const CUtensorMap &tq,
                       const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
    using C = h3::CrossCfg<D>;
    h3::cross_attn_kernel<T, D><<<grid, C::THREADS, C::SMEM_BYTES, st>>>(tq, tk, tv, p);
    if (p.split) {
        // a block a row: fewer than 296 items of at most 256 rows each
        h3::cross_join_kernel<T, D><<<static_cast<unsigned>(rows), 128, 0, st>>>(p);
    }
    return launched();
}

}  // namespace

extern "C" {

h3_status h3_rope_qk_freqs(const h3_rope_qk_cfg *cfg, double *freqs) {
    if (cfg == nullptr || freqs == nullptr || !rope_freqs(*cfg, freqs)) return H3_ERR_INVALID_ARG;
    return H3_OK;
}

h3_status h3_rope_qk_apply(const void *q, int64_t ldq, void *q_out, int64_t ldq_out,
                           const void *k, int64_t ldk, void *k_out, int64_t ldk_out,
                           const int32_t *positions, const h3_rope_qk_cfg *cfg, int64_t N,
                           int32_t Hq, int32_t Hk, int32_t D, int32_t dtype,
                           h3_stream_t stream) {
    if (cfg == nullptr || N < 0 || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 65535)
        return H3_ERR_INVALID_ARG;
    if (D < 2 || D > 512 || dtype < H3_BF16 || dtype > H3_FP32) return H3_ERR_UNSUPPORTED;
    h3::RopeQkParams p;
    if (!rope_phases(*cfg, p.phase) || cfg->rot_dim > D) return H3_ERR_INVALID_ARG;
    const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hk) * D;
    if (ldq < wq || ldq_out < wq || (Hk > 0 && (ldk < wk || ldk_out < wk)))
        return H3_ERR_INVALID_ARG;
    const int64_t widest = std::max(std::max(ldq, ldq_out), Hk > 0 ? std::max(ldk, ldk_out) : 0);
    if (N > 0 && widest >= (int64_t{1} << 47) / N) return H3_ERR_INVALID_ARG;
    if (N > (int64_t{1} << 30)) return H3_ERR_INVALID_ARG;   // blocks of a grid
    if (N > 0 && (q == nullptr || q_out == nullptr || positions == nullptr ||
                  (Hk > 0 && (k == nullptr || k_out == nullptr))))
        return H3_ERR_INVALID_ARG;
    if (q == q_out && ldq != ldq_out && q != nullptr) return H3_ERR_INVALID_ARG;
    if (Hk > 0 && k == k_out && ldk != ldk_out && k != nullptr) return H3_ERR_INVALID_ARG;
    if (Hk > 0 && N > 0 && (q_out == k_out || q_out == k || k_out == q)) return H3_ERR_INVALID_ARG;
    const uintptr_t size = dtype == H3_FP32 ? 4 : 2;
    if (!aligned(q, size) || !aligned(q_out, size) || !aligned(positions, 4) ||
        (Hk > 0 && (!aligned(k, size) || !aligned(k_out, size))))
        return H3_ERR_MISALIGNED;
    if (N == 0) return H3_OK;
    const Device *d = nullptr;
    h3_status st = device_info(&d);
    if (st != H3_OK) return st;
    p.q = q; p.qo = q_out; p.ldq = ldq; p.ldqo = ldq_out;
    p.k = k; p.ko = k_out; p.ldk = ldk; p.ldko = ldk_out;
    p.positions = positions;
    p.N = N;
    p.Hq = Hq; p.Hk = Hk; p.D = D; p.rot = cfg->rot_dim;
    const bool half = cfg->layout == H3_ROPE_HALF;
    // channels behind the rotated part are in place already where q and k are
    p.copy = q != q_out || (Hk > 0 && k != k_out);
    p.attn_factor = static_cast<float>(cfg->attn_factor);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == H3_BF16) launch_rope_qk<__nv_bfloat16>(p, half, d->sms, cs);
    else if (dtype == H3_FP16) launch_rope_qk<__half>(p, half, d->sms, cs);
    else launch_rope_qk<float>(p, half, d->sms, cs);
    return launched();
}

size_t h3_linear_workspace_size(int64_t M, int32_t N, int32_t K, int32_t act) {
    return linear_sizes_ok(M, N, K, act) ? kStatusBytes : 0;
}

h3_status h3_linear_fwd(const void *x, int64_t ldx, const void *w, int64_t ldw,
                        const void *bias, const void *residual, int64_t ldr, void *y,
                        int64_t ldy, int64_t M, int32_t N, int32_t K, int32_t act,
                        int32_t dtype, void *workspace, size_t workspace_bytes,
                        h3_stream_t stream) {
    if (!linear_sizes_ok(M, N, K, act)) return H3_ERR_INVALID_ARG;
    if (dtype != H3_BF16 && dtype != H3_FP16) return H3_ERR_UNSUPPORTED;
    if (ldx < K || ldw < K || ldy < N || (residual != nullptr && ldr < N))
        return H3_ERR_INVALID_ARG;
    if (w == nullptr || (M > 0 && (x == nullptr || y == nullptr))) return H3_ERR_INVALID_ARG;
    if (y != nullptr && (y == x || y == w || (y == residual && ldy != ldr)))
        return H3_ERR_INVALID_ARG;
    if (ldx >= (int64_t{1} << 39) || ldw >= (int64_t{1} << 39) || ldy >= (int64_t{1} << 31) ||
        (residual != nullptr && ldr >= (int64_t{1} << 31)))
        return H3_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || ldx % 8 != 0 || ldw % 8 != 0 || !aligned(bias, 2) ||
        !aligned(residual, 2) || !aligned(y, 2))
        return H3_ERR_MISALIGNED;
    if (workspace == nullptr || !aligned(workspace, 256) ||
        workspace_bytes < h3_linear_workspace_size(M, N, K, act))
        return H3_ERR_WORKSPACE;
    const Device *d = nullptr;
    h3_status st = device_info(&d);
    if (st != H3_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool gated = (act & H3_ACT_GATED) != 0;
    if (M == 0) {   // else the kernel's first block resets the status word
        const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int), cs);
        return e == cudaSuccess ? H3_OK : cuda_fail(e);
    }
    h3::LinearParams p;
    std::memset(&p, 0, sizeof(p));
    p.bias = bias; p.residual = residual; p.y = y;
    p.ldr = ldr; p.ldy = ldy;
    p.status = static_cast<int *>(workspace);
    p.M = static_cast<int32_t>(M); p.N = N; p.K = K; p.act = act & ~H3_ACT_GATED;
    p.vec_y = aligned(y, 16) && ldy % 8 == 0;
    p.vec_r = aligned(residual, 16) && ldr % 8 == 0;
    if (M <= skinny_rows(gated)) {
        using C = h3::LinearSkinny;
        p.cols = skinny_cols(M);
        p.splits = skinny_splits(N, K, d->sms);
        p.stages = std::min(C::MAX_STAGES, C::RING_BYTES / ((gated ? 2 : 1) * C::W_BYTES + p.cols * C::BK * 2));
    } else {
        using C = h3::LinearTile;
        const TileShape shape = tile_shape(M, N, gated, d->sms);
        p.out_cols = shape.out_cols;
        p.pieces = shape.pieces;
        p.stages = std::min(C::MAX_STAGES,
                            C::RING_BYTES / (C::A_BYTES + (gated ? 2 : 1) * p.out_cols * C::BK * 2));
        p.n_row_tiles = static_cast<int32_t>((M + C::BM - 1) / C::BM);
        p.n_col_tiles = (N + p.out_cols - 1) / p.out_cols;
        const int64_t tiles = static_cast<int64_t>(p.n_row_tiles) * p.n_col_tiles;
        if (tiles > INT32_MAX / 8) return H3_ERR_INVALID_ARG;
        const int rest = static_cast<int>(tiles % d->sms);
        p.whole = static_cast<int32_t>(tiles) - rest;
        p.n_tiles = p.whole + rest * p.pieces;
        // the x rows and w slices that a round of SMs reads are fewest near
        // sqrt(148 * 256 / 128) = 17 row tiles together; 8320 x 7168 x 5376 and the
        // gated 8320 x 5376 x 14336 took 550 and 2021 us with 12, 546 and 1988 with
        // 16, 546 and 1977 with 20, 555 and 1965 with 32
        p.group_m = 20;
    }
    if (dtype == H3_BF16)
        return gated ? launch_linear<__nv_bfloat16, true>(p, x, ldx, w, ldw, d->sms, cs)
                     : launch_linear<__nv_bfloat16, false>(p, x, ldx, w, ldw, d->sms, cs);
    return gated ? launch_linear<__half, true>(p, x, ldx, w, ldw, d->sms, cs)
                 : launch_linear<__half, false>(p, x, ldx, w, ldw, d->sms, cs);
}

size_t h3_cross_workspace_size(int64_t Nq, int32_t Hq, int32_t Hk, int32_t D, int32_t nseg,
                               int32_t max_q, int32_t max_k) {
    if (!cross_sizes_ok(Nq, 0, Hq, Hk, nseg) || (D != 64 && D != 128) || max_q < 0 || max_k < 0)
        return 0;
    const CrossPlanHost c = cross_plan(Nq, Hq, Hk, nseg, max_q, max_k);
    return kStatusBytes + cross_rows_bytes(c) +
           static_cast<size_t>(c.slots) * 2 * c.slot_rows * (D + 2) * 4;
}

h3_status h3_cross_attn_fwd(const void *q, int64_t ldq, const void *k, int64_t ldk,
                            const void *v, int64_t ldv, void *o, int64_t ldo, float *lse,
                            const int32_t *cu_q, const int32_t *cu_k, int32_t nseg,
                            int32_t max_q, int32_t max_k, const uint8_t *key_mask, int64_t Nq,
                            int64_t Nk, int32_t Hq, int32_t Hk, int32_t D,
                            float softmax_scale, int32_t dtype, void *workspace,
                            size_t workspace_bytes, h3_stream_t stream) {
    if (!cross_sizes_ok(Nq, Nk, Hq, Hk, nseg)) return H3_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || (dtype != H3_BF16 && dtype != H3_FP16))
        return H3_ERR_UNSUPPORTED;
    if (!std::isfinite(softmax_scale * 1.4426950408889634f) || softmax_scale < 0.0f)
        return H3_ERR_INVALID_ARG;
    if (cu_q == nullptr || cu_k == nullptr) return H3_ERR_INVALID_ARG;
    if (Nq > 0 && (q == nullptr || o == nullptr || max_q < 1 || max_q > Nq))
        return H3_ERR_INVALID_ARG;
    if (max_k < 0 || max_k > Nk || (Nk > 0 && (k == nullptr || v == nullptr)))
        return H3_ERR_INVALID_ARG;
    const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hk) * D;
    constexpr int64_t kMaxLd = int64_t{1} << 31;
    if (ldq < wq || ldo < wq || ldk < wk || ldv < wk || ldq >= kMaxLd || ldo >= kMaxLd ||
        ldk >= kMaxLd || ldv >= kMaxLd)
        return H3_ERR_INVALID_ARG;
    if (o != nullptr && (o == q || o == k || o == v)) return H3_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
        ldq % 8 != 0 || ldk % 8 != 0 || ldv % 8 != 0 || ldo % 8 != 0 || !aligned(lse, 4) ||
        !aligned(cu_q, 4) || !aligned(cu_k, 4))
        return H3_ERR_MISALIGNED;
    if (workspace == nullptr || !aligned(workspace, 256) ||
        workspace_bytes < h3_cross_workspace_size(Nq, Hq, Hk, D, nseg, max_q, max_k))
        return H3_ERR_WORKSPACE;
    const Device *d = nullptr;
    h3_status st = device_info(&d);
    if (st != H3_OK) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (!d->cross_regs_ok) return H3_ERR_UNSUPPORTED;
    const CrossPlanHost c = cross_plan(Nq, Hq, Hk, nseg, max_q, max_k);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (Nq == 0) {   // else the kernel's first block resets the status word
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), cs);
        return e == cudaSuccess ? H3_OK : cuda_fail(e);
    }
    h3::CrossParams p;
    std::memset(&p, 0, sizeof(p));
    p.o = o; p.lse = lse; p.ldo = ldo;
    p.cu_q = cu_q; p.cu_k = cu_k; p.mask = key_mask;
    p.status = reinterpret_cast<int *>(ws);
    p.nseg = nseg; p.max_q = max_q; p.max_k = max_k;
    p.Nq = static_cast<int32_t>(Nq); p.Nk = static_cast<int32_t>(Nk);
    p.Hq = Hq; p.Hk = Hk;
    p.hp = c.hp; p.tokens = c.tokens; p.heads_blocks = Hq / c.hp;
    p.split = c.split;
    // a scale of 0 (the mean of the values) as one that no score survives (fp32's
    // largest times it is 5e-7), so that a masked score of -infinity stays one
    p.scale_log2 = std::max(softmax_scale * 1.4426950408889634f,
                            std::numeric_limits<float>::denorm_min());
    p.rows = reinterpret_cast<int2 *>(ws + kStatusBytes);
    p.parts = reinterpret_cast<float *>(ws + kStatusBytes + cross_rows_bytes(c));
    p.slot_rows = c.slot_rows;
    CUtensorMap tq, tk, tv;
    if ((st = make_heads_map(&tq, q, Nq, Hq, D, ldq, c.hp, c.tokens)) != H3_OK) return st;
    // without keys nothing is loaded: any valid map will do
    if ((st = Nk > 0 ? make_heads_map(&tk, k, Nk, Hk, D, ldk, 1, 128)
                     : make_heads_map(&tk, q, Nq, Hq, D, ldq, 1, 128)) != H3_OK) return st;
    if ((st = Nk > 0 ? make_heads_map(&tv, v, Nk, Hk, D, ldv, 1, 128)
                     : make_heads_map(&tv, q, Nq, Hq, D, ldq, 1, 128)) != H3_OK) return st;
    const int grid = static_cast<int>(std::min<int64_t>(d->sms, c.items + c.slots));
    if (dtype == H3_BF16)
        return D == 128 ? launch_cross<__nv_bfloat16, 128>(p, grid, c.rows, tq, tk, tv, cs)
                        : launch_cross<__nv_bfloat16, 64>(p, grid, c.rows, tq, tk, tv, cs);
    return D == 128 ? launch_cross<__half, 128>(p, grid, c.rows, tq, tk, tv, cs)
                    : launch_cross<__half, 64>(p, grid, c.rows, tq, tk, tv, cs);
}

}  // extern "C"
