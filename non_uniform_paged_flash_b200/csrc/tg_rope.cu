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

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 5;    // head rows of a lane group in flight
constexpr int kRopeMaxD = 256;  // a head row is at most one warp of 8-element lanes

struct RopeArgs {
    const __nv_bfloat16 *x[2];   // q, k
    const __nv_bfloat16 *w[2];
    __nv_bfloat16 *y[2];
    int64_t in_stride[2], out_stride[2];
    int32_t heads[2];
    int32_t D, rot;
    float inv_d, eps, rot_scale;
    const int32_t *pos;
    const double *inv_freq;
};

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// A lane's 8 elements of a head row as four pairs (a_i, b_i) that turn together: A = a_0..3, B = b_0..3.
// Interleaved: words hold (a_i, b_i). Halves: the first two words hold a_0..3, the last two b_0..3.
template <bool INTER>
__device__ __forceinline__ void unpack(const uint4 &v, ptx::f2 (&A)[2], ptx::f2 (&B)[2]) {
    if (INTER) {
        A[0] = ptx::pair(lo16(v.x), lo16(v.y));
        A[1] = ptx::pair(lo16(v.z), lo16(v.w));
        B[0] = ptx::pair(hi16(v.x), hi16(v.y));
        B[1] = ptx::pair(hi16(v.z), hi16(v.w));
    } else {
        A[0] = ptx::pair(lo16(v.x), hi16(v.x));
        A[1] = ptx::pair(lo16(v.y), hi16(v.y));
        B[0] = ptx::pair(lo16(v.z), hi16(v.z));
        B[1] = ptx::pair(lo16(v.w), hi16(v.w));
    }
}

template <bool INTER>
__device__ __forceinline__ uint4 repack(const ptx::f2 (&A)[2], const ptx::f2 (&B)[2]) {
    float a[4], b[4];
    ptx::split(A[0], a[0], a[1]);
    ptx::split(A[1], a[2], a[3]);
    ptx::split(B[0], b[0], b[1]);
    ptx::split(B[1], b[2], b[3]);
    if (INTER)
        return make_uint4(ptx::pack_bf16(a[0], b[0]), ptx::pack_bf16(a[1], b[1]), ptx::pack_bf16(a[2], b[2]), ptx::pack_bf16(a[3], b[3]));
    return make_uint4(ptx::pack_bf16(a[0], a[1]), ptx::pack_bf16(a[2], a[3]), ptx::pack_bf16(b[0], b[1]), ptx::pack_bf16(b[2], b[3]));
}

// One CTA per token. A head row of D bf16 takes D/8 lanes of a group of LPH (D/8 rounded up to a power
// of two): 16 bytes a lane, or for halves 8 bytes from each half of the rotated part, so that both
// elements of a pair are in one lane and rotating needs no shuffle; a row is read and written once.
// The token's angles are the same for all heads: rot/2 of them in 64 bits (position * frequency
// in turns, reduced to one turn before it is rounded to 32 bits: a position of 10^6 keeps its
// angle to 2^-24 of a turn), their sines and cosines once in shared memory while the rows' loads
// are in flight. Norm, weight and rotation stay in fp32, two elements an instruction; the only
// rounding is the output's. Bound: DRAM (4 D bytes per head row): 32001 tokens of 32 + 8 heads of
// D = 128 take 120 us, 5.46 TB/s, and 134 us in 1 s loops, where the power limit takes the clock to
// 1.75 GHz. 8 CTAs per SM of 5 rows a lane measured best (3 rows of 256 threads 145 us, 10 CTAs at fewer
// registers 128 us, 64 threads 122 us, persistent CTAs that load the next token ahead 157 us).
template <int LPH, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 8) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    using ptx::f2;
    __shared__ float2 cs[kRopeMaxD / 2];
    constexpr int GROUPS = kRopeThreads / LPH;  // head rows per pass
    const int64_t n = blockIdx.x;
    const int sub = threadIdx.x % LPH, grp = threadIdx.x / LPH;
    const int warp_grp = (threadIdx.x & ~31) / LPH;  // the warp's first group
    const int H = a.heads[0] + a.heads[1];
    const bool on = sub < a.D / 8;
    const int half = a.rot / 2;
    // element offsets of the lane's two 8-byte parts
    const int turning = a.rot / 8;  // lanes that hold pairs of halves
    const int e0 = INTER || sub >= turning ? 8 * sub : 4 * sub;
    const int e1 = INTER || sub >= turning ? 8 * sub + 4 : half + 4 * sub;
    ptx::grid_wait();
    ptx::grid_launch();

    auto load = [&](const __nv_bfloat16 *row) {
        if (INTER) return *reinterpret_cast<const uint4 *>(row + e0);
        const uint2 u = *reinterpret_cast<const uint2 *>(row + e0), w = *reinterpret_cast<const uint2 *>(row + e1);
        return make_uint4(u.x, u.y, w.x, w.y);
    };
    auto offset = [&](int hd, const int64_t (&stride)[2]) {
        const int s = hd >= a.heads[0];
        return n * stride[s] + static_cast<int64_t>(hd - (s ? a.heads[0] : 0)) * a.D;
    };
    const f2 one = ptx::pair(1.f, 1.f);
    f2 C[2] = {one, one}, S[2], NS[2];
    bool turn[4] = {false, false, false, false};
    for (int h0 = 0; h0 < H; h0 += GROUPS * kRopeRows) {
        uint4 v[kRopeRows];
#pragma unroll
        for (int j = 0; j < kRopeRows; ++j) {
            const int hd = h0 + j * GROUPS + grp;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (hd < H && on) v[j] = load(a.x[hd >= a.heads[0]] + offset(hd, a.in_stride));
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
            float c[4], s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                turn[i] = 4 * sub + i < half;
                const float2 t = turn[i] ? cs[4 * sub + i] : make_float2(1.f, 0.f);
                c[i] = t.x;
                s[i] = t.y;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                C[k] = ptx::pair(c[2 * k], c[2 * k + 1]);
                S[k] = ptx::pair(s[2 * k], s[2 * k + 1]);
                NS[k] = ptx::pair(-s[2 * k], -s[2 * k + 1]);
            }
        }
#pragma unroll
        for (int j = 0; j < kRopeRows; ++j) {
            if (h0 + j * GROUPS + warp_grp >= H) break;  // no row of this warp
            const int hd = h0 + j * GROUPS + grp;
            const int side = hd >= a.heads[0];
            f2 A[2], B[2];
            unpack<INTER>(v[j], A, B);
            const __nv_bfloat16 *w = a.w[side];
            if (a.w[0] || a.w[1]) {
                const f2 q = ptx::add2(ptx::fma2(A[0], A[0], ptx::mul2(A[1], A[1])), ptx::fma2(B[0], B[0], ptx::mul2(B[1], B[1])));
                float s0, s1;
                ptx::split(q, s0, s1);
                float ss = s0 + s1;
#pragma unroll
                for (int d = LPH / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                if (w && on) {
                    const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
                    f2 WA[2], WB[2];
                    unpack<INTER>(load(w), WA, WB);
                    const f2 rr = ptx::pair(r, r);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        A[k] = ptx::mul2(ptx::mul2(A[k], rr), WA[k]);
                        B[k] = ptx::mul2(ptx::mul2(B[k], rr), WB[k]);
                    }
                }
            }
            if (turn[0]) {
                f2 U[2], V[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    U[k] = ptx::fma2(B[k], NS[k], ptx::mul2(A[k], C[k]));
                    V[k] = ptx::fma2(A[k], S[k], ptx::mul2(B[k], C[k]));
                }
                if (turn[3]) {
                    A[0] = U[0]; A[1] = U[1]; B[0] = V[0]; B[1] = V[1];
                } else {  // the rotated part ends inside this lane
                    float a0[4], b0[4], u[4], w0[4];
                    ptx::split(A[0], a0[0], a0[1]); ptx::split(A[1], a0[2], a0[3]);
                    ptx::split(B[0], b0[0], b0[1]); ptx::split(B[1], b0[2], b0[3]);
                    ptx::split(U[0], u[0], u[1]); ptx::split(U[1], u[2], u[3]);
                    ptx::split(V[0], w0[0], w0[1]); ptx::split(V[1], w0[2], w0[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (turn[i]) {
                            a0[i] = u[i];
                            b0[i] = w0[i];
                        }
                    A[0] = ptx::pair(a0[0], a0[1]); A[1] = ptx::pair(a0[2], a0[3]);
                    B[0] = ptx::pair(b0[0], b0[1]); B[1] = ptx::pair(b0[2], b0[3]);
                }
            }
            if (hd < H && on) {
                __nv_bfloat16 *row = a.y[side] + offset(hd, a.out_stride);
                const uint4 o = repack<INTER>(A, B);
                if (INTER) {
                    *reinterpret_cast<uint4 *>(row + e0) = o;
                } else {
                    *reinterpret_cast<uint2 *>(row + e0) = make_uint2(o.x, o.y);
                    *reinterpret_cast<uint2 *>(row + e1) = make_uint2(o.z, o.w);
                }
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
        if (pair_of(beta_slow) < 0.0) low = -1.0, high = -0.5;  // even the first pair turns less: all are slow
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
    a.inv_d = 1.f / static_cast<float>(D);
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
