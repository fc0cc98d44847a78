// C-ABI entry points of the layers around the attention (declared in
// include/h3attn.h): 1-D rotary positions, linear layers, cross attention.
// Host side only: argument checks, frequency tables, launches on the caller's
// stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
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
    int sms = 0;
};
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
    if (!positive(c.theta) || !std::isfinite(c.attn_factor)) return false;
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
    const long double frac = turns - std::floor(turns);
    const long double scaled = std::nearbyint(std::ldexp(frac, 64));
    return scaled >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(scaled);
}

template <typename T>
void launch_rope_qk(const h3::RopeQkParams &p, int sms, cudaStream_t st) {
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    h3::rope_qk_kernel<T><<<static_cast<int>(std::min(p.N, cap)), 256, 0, st>>>(p);
}

// --------------------------------------------------------------------- linear

bool linear_sizes_ok(int64_t M, int32_t N, int32_t K, int32_t act) {
    const int a = act & ~H3_ACT_GATED;
    return M >= 0 && M < INT32_MAX - 256 && N >= 1 && N <= (1 << 20) && K >= 1 &&
           K <= (1 << 20) && a >= H3_ACT_NONE && a <= H3_ACT_SILU;
}

template <typename T, int Act>
void launch_linear_act(const h3::LinearParams &p, bool gated, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((p.N + 63) / 64), static_cast<unsigned>((p.M + 63) / 64));
    if (gated) h3::linear_kernel<T, Act, true><<<grid, 256, 0, st>>>(p);
    else h3::linear_kernel<T, Act, false><<<grid, 256, 0, st>>>(p);
}

template <typename T>
void launch_linear(const h3::LinearParams &p, int act, cudaStream_t st) {
    const bool gated = (act & H3_ACT_GATED) != 0;
    switch (act & ~H3_ACT_GATED) {
        case H3_ACT_RELU: return launch_linear_act<T, 1>(p, gated, st);
        case H3_ACT_GELU: return launch_linear_act<T, 2>(p, gated, st);
        case H3_ACT_GELU_TANH: return launch_linear_act<T, 3>(p, gated, st);
        case H3_ACT_SILU: return launch_linear_act<T, 4>(p, gated, st);
        default: return launch_linear_act<T, 0>(p, gated, st);
    }
}

// ------------------------------------------------------------ cross attention

bool cross_sizes_ok(int64_t Nq, int64_t Nk, int32_t Hq, int32_t Hk, int32_t nseg) {
    return Nq >= 0 && Nq <= INT32_MAX - 1 && Nk >= 0 && Nk <= INT32_MAX - 1 && Hk >= 1 &&
           Hq >= Hk && Hq <= 65535 && Hq % Hk == 0 && nseg >= 1 && nseg <= 65535;
}

template <typename T>
void launch_cross(const h3::CrossParams &p, int D, int sms, cudaStream_t st) {
    const int64_t blocks = (static_cast<int64_t>(p.Nq) * p.Hq + 3) / 4;
    const int grid = static_cast<int>(std::min<int64_t>(blocks, static_cast<int64_t>(sms) * 64));
    if (D == 128) h3::cross_attn_kernel<T, 128><<<grid, 128, 0, st>>>(p);
    else h3::cross_attn_kernel<T, 64><<<grid, 128, 0, st>>>(p);
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
    double f[h3::kRopeQkMaxPairs];
    if (!rope_freqs(*cfg, f) || cfg->rot_dim > D) return H3_ERR_INVALID_ARG;
    const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hk) * D;
    if (ldq < wq || ldq_out < wq || (Hk > 0 && (ldk < wk || ldk_out < wk)))
        return H3_ERR_INVALID_ARG;
    const int64_t widest = std::max(std::max(ldq, ldq_out), Hk > 0 ? std::max(ldk, ldk_out) : 0);
    if (N > 0 && widest >= (int64_t{1} << 47) / N) return H3_ERR_INVALID_ARG;
    if (N > 0 && (q == nullptr || q_out == nullptr || positions == nullptr ||
                  (Hk > 0 && (k == nullptr || k_out == nullptr))))
        return H3_ERR_INVALID_ARG;
    if (q == q_out && ldq != ldq_out && q != nullptr) return H3_ERR_INVALID_ARG;
    if (Hk > 0 && k == k_out && ldk != ldk_out && k != nullptr) return H3_ERR_INVALID_ARG;
    const uintptr_t size = dtype == H3_FP32 ? 4 : 2;
    if (!aligned(q, size) || !aligned(q_out, size) || !aligned(positions, 4) ||
        (Hk > 0 && (!aligned(k, size) || !aligned(k_out, size))))
        return H3_ERR_MISALIGNED;
    if (N == 0) return H3_OK;
    const Device *d = nullptr;
    h3_status st = device_info(&d);
    if (st != H3_OK) return st;
    h3::RopeQkParams p;
    p.q = q; p.qo = q_out; p.ldq = ldq; p.ldqo = ldq_out;
    p.k = k; p.ko = k_out; p.ldk = ldk; p.ldko = ldk_out;
    p.positions = positions;
    p.N = N;
    p.Hq = Hq; p.Hk = Hk; p.D = D; p.rot = cfg->rot_dim;
    p.half = cfg->layout == H3_ROPE_HALF;
    p.attn_factor = static_cast<float>(cfg->attn_factor);
    for (int j = 0; j < h3::kRopeQkMaxPairs; ++j)
        p.phase[j] = j < cfg->rot_dim / 2 ? phase_of(f[j]) : 0;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == H3_BF16) launch_rope_qk<__nv_bfloat16>(p, d->sms, cs);
    else if (dtype == H3_FP16) launch_rope_qk<__half>(p, d->sms, cs);
    else launch_rope_qk<float>(p, d->sms, cs);
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
    const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int), cs);
    if (e != cudaSuccess) return cuda_fail(e);
    if (M == 0) return H3_OK;
    h3::LinearParams p;
    p.x = x; p.w = w; p.bias = bias; p.residual = residual; p.y = y;
    p.ldx = ldx; p.ldw = ldw; p.ldr = ldr; p.ldy = ldy;
    p.M = M; p.N = N; p.K = K;
    if (dtype == H3_BF16) launch_linear<__nv_bfloat16>(p, act, cs);
    else launch_linear<__half>(p, act, cs);
    return launched();
}

size_t h3_cross_workspace_size(int64_t Nq, int32_t Hq, int32_t Hk, int32_t D, int32_t nseg,
                               int32_t max_q, int32_t max_k) {
    if (!cross_sizes_ok(Nq, 0, Hq, Hk, nseg) || (D != 64 && D != 128) || max_q < 0 || max_k < 0)
        return 0;
    return kStatusBytes;
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
    if (!std::isfinite(softmax_scale) || softmax_scale < 0.0f) return H3_ERR_INVALID_ARG;
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
    const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int), cs);
    if (e != cudaSuccess) return cuda_fail(e);
    if (Nq == 0) return H3_OK;
    h3::CrossParams p;
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    p.ldq = ldq; p.ldk = ldk; p.ldv = ldv; p.ldo = ldo;
    p.cu_q = cu_q; p.cu_k = cu_k; p.mask = key_mask;
    p.status = static_cast<int *>(workspace);
    p.nseg = nseg; p.max_q = max_q; p.max_k = max_k;
    p.Nq = static_cast<int32_t>(Nq); p.Nk = static_cast<int32_t>(Nk);
    p.Hq = Hq; p.Hk = Hk;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    if (dtype == H3_BF16) launch_cross<__nv_bfloat16>(p, D, d->sms, cs);
    else launch_cross<__half>(p, D, d->sms, cs);
    return launched();
}

}  // extern "C"
