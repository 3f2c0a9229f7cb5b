// Query / key norm of each head with the rotary position in the same pass: the step between a
// layer's projections and the cache (keys are cached after rotation) or the attention call.
//
//   y = x * rsqrt(mean(x^2) + eps) * w                      (per head of D; w NULL: y = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t) * rot_scale,   t = position * inv_freq[i]
// over the pairs i < rot_dim / 2 of the head's first rot_dim elements: (2i, 2i + 1) interleaved,
// or (i, i + rot_dim / 2) by halves. Rotary embedding: Su et al. 2021 (RoFormer); the frequency
// scalings of tg_rope_frequencies: Chen et al. 2023 (position interpolation), the base change of
// NTK-aware scaling, Peng et al. 2023 (YaRN).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "tg.h"
#include "tg_internal.h"
#include "tg_ptx.cuh"

namespace tg {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 3;    // head rows of a lane group in flight
constexpr int kRopeMaxD = 256;  // a head row is at most one warp of 16-byte slices

struct RopeArgs {
    const __nv_bfloat16 *x[2];   // q, k
    const __nv_bfloat16 *w[2];
    __nv_bfloat16 *y[2];
    int64_t in_stride[2], out_stride[2];
    int32_t heads[2];
    int32_t D, rot;
    float eps, rot_scale;
    const int32_t *pos;
    const double *inv_freq;
};

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
    f[0] = lo16(v.x); f[1] = hi16(v.x); f[2] = lo16(v.y); f[3] = hi16(v.y);
    f[4] = lo16(v.z); f[5] = hi16(v.z); f[6] = lo16(v.w); f[7] = hi16(v.w);
}

// One CTA per token. A head row of D bf16 is D/8 16-byte slices, one per lane of a group of LPH
// lanes (LPH = D/8 rounded up to a power of two), so a row is read and written once, a norm is a
// few xor-shuffles, and the partner of a half-layout pair sits rot/16 lanes away (rot % 16 == 0).
// The token's angles are the same for all heads: rot/2 of them in 64 bits (position * frequency
// in turns, reduced to one turn before it is rounded to 32 bits: a position of 10^6 keeps its
// angle to 2^-24 of a turn), their sines and cosines once in shared memory while the rows' loads
// are in flight. Norm, weight and rotation stay in fp32; the only rounding is the output's.
// Bound: DRAM (4 D bytes per head row).
template <int LPH, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 cs[kRopeMaxD / 2];
    constexpr int GROUPS = kRopeThreads / LPH;  // head rows per pass
    const int64_t n = blockIdx.x;
    const int sub = threadIdx.x % LPH, grp = threadIdx.x / LPH;
    const int H = a.heads[0] + a.heads[1];
    const int nvec = a.D / 8;
    const int half = a.rot / 2;
    ptx::grid_wait();
    ptx::grid_launch();

    auto row_in = [&](int hd) {
        const int s = hd >= a.heads[0];
        return reinterpret_cast<const uint4 *>(a.x[s] + n * a.in_stride[s] + static_cast<int64_t>(hd - s * a.heads[0]) * a.D);
    };
    for (int h0 = 0; h0 < H; h0 += GROUPS * kRopeRows) {
        uint4 v[kRopeRows];
#pragma unroll
        for (int j = 0; j < kRopeRows; ++j) {
            const int hd = h0 + j * GROUPS + grp;
            v[j] = hd < H && sub < nvec ? row_in(hd)[sub] : make_uint4(0u, 0u, 0u, 0u);
        }
        if (h0 == 0) {
            for (int i = threadIdx.x; i < half; i += kRopeThreads) {
                double t = static_cast<double>(a.pos[n]) * a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
                t -= rint(t);
                float s, c;
                sincospif(static_cast<float>(2.0 * t), &s, &c);
                cs[i] = make_float2(c * a.rot_scale, s * a.rot_scale);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kRopeRows; ++j) {
            const int hd = h0 + j * GROUPS + grp;
            const int s = hd >= a.heads[0];
            float x[8];
            unpack(v[j], x);
            float r = 1.f;
            const __nv_bfloat16 *w = a.w[s];
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int d = LPH / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            if (w) r = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
            const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
            float wf[8];
            unpack(w && sub < nvec ? __ldg(reinterpret_cast<const uint4 *>(w) + sub) : one, wf);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= r * wf[e];
            if (INTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * sub + e;
                    if (i < half) {
                        const float2 t = cs[i];
                        const float x0 = x[2 * e], x1 = x[2 * e + 1];
                        x[2 * e] = x0 * t.x - x1 * t.y;
                        x[2 * e + 1] = x0 * t.y + x1 * t.x;
                    }
                }
            } else {
                // the partner slice sits half / 8 lanes up (first half) or down (second half)
                const int step = half / 8;
                const bool first = sub < step, turned = sub < 2 * step;
                const int other = !turned ? sub : (first ? sub + step : sub - step);
                const float sign = first ? -1.f : 1.f;
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xffffffffu, x[e], other, LPH);
                if (turned) {
                    const int i = 8 * (first ? sub : sub - step);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = cs[i + e];
                        x[e] = x[e] * t.x + sign * p[e] * t.y;
                    }
                }
            }
            if (hd < H && sub < nvec) {
                uint4 o;
                o.x = ptx::pack_bf16(x[0], x[1]);
                o.y = ptx::pack_bf16(x[2], x[3]);
                o.z = ptx::pack_bf16(x[4], x[5]);
                o.w = ptx::pack_bf16(x[6], x[7]);
                reinterpret_cast<uint4 *>(a.y[s] + n * a.out_stride[s] + static_cast<int64_t>(hd - s * a.heads[0]) * a.D)[sub] = o;
            }
        }
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int LPH>
cudaError_t launch(const RopeArgs &a, int64_t n, bool inter, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return inter ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<LPH, true>, a)
                 : cudaLaunchKernelEx(&cfg, norm_rope_kernel<LPH, false>, a);
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, int64_t orig_len,
                                   double beta_fast, double beta_slow, double *inv_freq, float *rot_scale) {
    if (rot_dim < 0 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base) || (rot_dim > 0 && !inv_freq) ||
        !rot_scale || scaling < TG_ROPE_NONE || scaling > TG_ROPE_YARN)
        return TG_EINVAL;
    if (scaling != TG_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return TG_EINVAL;
    if (scaling == TG_ROPE_YARN && (orig_len < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0))) return TG_EINVAL;
    if (scaling == TG_ROPE_NTK && rot_dim == 2) return TG_EINVAL;  // its exponent rot / (rot - 2)
    const int32_t half = rot_dim / 2;
    if (scaling == TG_ROPE_NTK && rot_dim > 2)
        base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    double low = 0.0, high = 0.0;
    if (scaling == TG_ROPE_YARN) {
        // pair index at which a dimension turns `beta` times over the original length
        auto pair_of = [&](double beta) {
            return rot_dim * std::log(static_cast<double>(orig_len) / (beta * 2.0 * M_PI)) / (2.0 * std::log(base));
        };
        low = std::max(0.0, std::floor(pair_of(beta_fast)));
        high = std::min(rot_dim - 1.0, std::ceil(pair_of(beta_slow)));
        if (high <= low) high = low + 0.001;
    }
    for (int32_t i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == TG_ROPE_LINEAR) f /= factor;
        if (scaling == TG_ROPE_YARN) {
            const double ramp = std::min(1.0, std::max(0.0, (i - low) / (high - low)));
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        inv_freq[i] = f;
    }
    *rot_scale = scaling == TG_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return TG_OK;
}

extern "C" int tg_qk_norm_rope(int64_t n_tokens, int32_t Hq, int32_t Hkv, int32_t D, const void *q, int64_t q_stride,
                               const void *k, int64_t k_stride, const void *q_weight, const void *k_weight, float eps,
                               const int32_t *position, const double *inv_freq, int32_t rot_dim, int32_t interleaved,
                               float rot_scale, void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                               tg_stream stream) {
    if (n_tokens < 0 || n_tokens > INT32_MAX || Hq < 0 || Hkv < 0 || Hq > 65536 || Hkv > 65536 || Hq + Hkv < 1 || D < 8 ||
        rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0 || !(eps >= 0.f))
        return TG_EINVAL;
    if (D % 8 != 0 || D > kRopeMaxD || (!interleaved && rot_dim % 16 != 0)) return TG_EUNSUPPORTED;
    if (n_tokens == 0) return TG_OK;
    if ((rot_dim > 0 && (!position || !inv_freq)) || !al16(q) || !al16(k) || !al16(q_out) || !al16(k_out) ||
        !al16(q_weight) || !al16(k_weight))
        return TG_EINVAL;
    RopeArgs a{};
    const void *x[2] = {q, k}, *w[2] = {q_weight, k_weight};
    void *y[2] = {q_out, k_out};
    const int64_t is[2] = {q_stride, k_stride}, os[2] = {q_out_stride, k_out_stride};
    const int32_t hs[2] = {Hq, Hkv};
    for (int s = 0; s < 2; ++s) {
        a.heads[s] = hs[s];
        if (hs[s] == 0) continue;
        const int64_t width = static_cast<int64_t>(hs[s]) * D;
        if (!x[s] || !y[s] || is[s] < width || os[s] < width || is[s] % 8 != 0 || os[s] % 8 != 0) return TG_EINVAL;
        a.x[s] = static_cast<const __nv_bfloat16 *>(x[s]);
        a.w[s] = static_cast<const __nv_bfloat16 *>(w[s]);
        a.y[s] = static_cast<__nv_bfloat16 *>(y[s]);
        a.in_stride[s] = is[s];
        a.out_stride[s] = os[s];
    }
    a.D = D;
    a.rot = rot_dim;
    a.eps = eps;
    a.rot_scale = rot_scale;
    a.pos = position;
    a.inv_freq = inv_freq;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int nvec = D / 8;
    const bool inter = interleaved != 0;
    cudaError_t e = nvec > 16  ? launch<32>(a, n_tokens, inter, st)
                    : nvec > 8 ? launch<16>(a, n_tokens, inter, st)
                    : nvec > 4 ? launch<8>(a, n_tokens, inter, st)
                    : nvec > 2 ? launch<4>(a, n_tokens, inter, st)
                    : nvec > 1 ? launch<2>(a, n_tokens, inter, st)
                               : launch<1>(a, n_tokens, inter, st);
    if (e != cudaSuccess) {
        set_cuda_error("norm_rope_kernel", static_cast<int>(e));
        return TG_ECUDA;
    }
    return TG_OK;
}
