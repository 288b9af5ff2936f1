// kda_norm.cu -- norm of queries and keys per head with the position rotation in
// the same pass, and its gradients (sm_100a).
//
// Per token and head, over the d channels of a row x, with weight w:
//
//   r = (m sum x^2 + eps)^{-1/2},   n = r x w,      m = 1 / d (RMS) or 1 (L2)
//   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin    for the pairs (a, b) of the
//                                                        first rotary_dim channels
//
// and backwards, with g the cotangent of n (the rotation turned back) and h = g w:
//
//   dx = r h - m r^3 <h, x> x,   dw = sum over tokens and heads of g r x
//
// Both read each row once and write it once: HBM bandwidth bounds them at size,
// launch latency for a handful of tokens.  A lane holds eight channels of a row, so
// LPR = d / 8 lanes (rounded up to 8, 16 or 32) share a row and a warp takes
// 32 / LPR rows at a time; the sums are butterflies over those lanes.  A warp works
// on the heads of one token (or a slab of them when there are few tokens), so its
// angles are computed once per token and kept in registers.  An angle is
// pos * freq in fp64, reduced to a turn before it is rounded to fp32: positions of
// 10^6 keep every bit of the angle that fp32 can hold.
#include "kda_common.cuh"
#include "kda_launch.h"
#include "../../include/kda.h"

#include <algorithm>

namespace kda {
namespace {

constexpr int kWarps = 8;              // per CTA
constexpr int kMaxCtas = 1024;         // partial weight gradients are sized for this many
constexpr int kUnroll = 4;             // rows in flight per lane

struct NormSide {
    const void* x; const void* dy;     // dy: backward only
    void* out;                         // y, or dx
    const float* w;                    // [d], nullable
    int64_t sb, st, sh;                // element strides of x (batch, token, head)
    int heads;
};
struct NormArgs {
    NormSide side[2];                  // queries, keys
    const float* inv_freq; const int32_t* positions;
    int T, d, rot, slab, slabs;        // heads of one unit of work, units per token
    int64_t tokens;
    int interleaved;
    float m, eps;
    float* partial;                    // [CTAs][2][d], backward with weights only
};

template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
        __align__(16) __nv_bfloat162 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    }
};
template <> struct Vec8<float> {
    float4 lo, hi;
    __device__ __forceinline__ void load(const float* p) {
        lo = __ldcs(reinterpret_cast<const float4*>(p));
        hi = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
        x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LPR / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Turns this lane's eight channels by (c, s).  Pairs lie in one lane
// (interleaved) or `hop` lanes apart (first half with second half).  All lanes of
// the warp call it; `in` says whether this lane's channels turn.
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[8], const float (&s)[8], bool in, int interleaved,
                                     int partner, bool second) {
    if (interleaved) {
        if (in) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = fmaf(a, c[i], -b * s[i]);
                x[2 * i + 1] = fmaf(b, c[i], a * s[i]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(0xffffffffu, x[i], partner);
        if (in) x[i] = fmaf(x[i], c[i], (second ? other : -other) * s[i]);
    }
}

template <typename T, int LPR, bool BWD>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_rope_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int RPW = 32 / LPR;
    __shared__ float angle[kWarps][2][128];
    __shared__ float red[BWD ? kWarps : 1][2][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, e0 = 8 * (lane % LPR);
    const bool mine = e0 < a.d;                    // lanes past the row's end only take part in shuffles
    const int half = a.rot / 2;
    const bool in = e0 < a.rot, second = e0 >= half;
    const int partner = (in && !a.interleaved) ? (second ? lane - half / 8 : lane + half / 8) : lane;
    const int heads = a.side[0].heads + a.side[1].heads;

    float w[2][8], dw[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[q][i] = (mine && a.side[q].w) ? a.side[q].w[e0 + i] : 1.f;
            dw[q][i] = 0.f;
        }
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }

    const int64_t units = a.tokens * a.slabs, stride = (int64_t)gridDim.x * kWarps;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += stride) {
        const int64_t tok = u / a.slabs;
        const int first = (int)(u - tok * a.slabs) * a.slab, end = min(heads, first + a.slab);
        const int64_t b = tok / a.T, t = tok - b * a.T;
        if (a.rot) {
            const double pos = a.positions ? (double)a.positions[tok] : (double)t;
            __syncwarp();
            for (int j = lane; j < half; j += 32) {
                double turns = pos * (double)a.inv_freq[j] * 0.15915494309189535;   // 1 / (2 pi)
                turns -= rint(turns);
                float sn, cs;
                sincospif(2.f * (float)turns, &sn, &cs);
                angle[warp][0][j] = cs;
                angle[warp][1][j] = BWD ? -sn : sn;
            }
            __syncwarp();
            if (in) {
                const int j0 = a.interleaved ? e0 / 2 : (second ? e0 - half : e0);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < 4 || !a.interleaved) { c[i] = angle[warp][0][j0 + i]; s[i] = angle[warp][1][j0 + i]; }
            }
        }
        for (int r0 = first; r0 < end; r0 += RPW * kUnroll) {
            Vec8<T> xv[kUnroll], gv[BWD ? kUnroll : 1];
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) {     // all loads first
                const int r = r0 + n * RPW + sub;
                if (r < end && mine) {
                    const int q = r >= a.side[0].heads, hd = r - (q ? a.side[0].heads : 0);
                    const NormSide& z = a.side[q];
                    xv[n].load(static_cast<const T*>(z.x) + b * z.sb + t * z.st + hd * z.sh + e0);
                    if constexpr (BWD)
                        gv[n].load(static_cast<const T*>(z.dy) + (tok * z.heads + hd) * (int64_t)a.d + e0);
                }
            }
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) {
                if (r0 + n * RPW >= end) break;     // uniform over the warp
                const int r = r0 + n * RPW + sub;
                const bool on = r < end && mine;
                const int q = r >= a.side[0].heads, hd = r - (q ? a.side[0].heads : 0);
                float x[8], ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
                if (on) xv[n].get(x);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                ss = row_sum<LPR>(ss);
                const float rs = rsqrtf(fmaf(ss, a.m, a.eps));
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= rs * (q ? w[1][i] : w[0][i]);
                    if (a.rot) turn(x, c, s, in, a.interleaved, partner, second);
                    if (on) Vec8<T>::store(static_cast<T*>(a.side[q].out) + (tok * a.side[q].heads + hd) * (int64_t)a.d + e0, x);
                } else {
                    float g[8], dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = 0.f;
                    if (on) gv[n].get(g);
                    if (a.rot) turn(g, c, s, in, a.interleaved, partner, second);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p = g[i] * x[i] * rs;
                        if (q) dw[1][i] += p; else dw[0][i] += p;
                        g[i] *= q ? w[1][i] : w[0][i];
                        dot = fmaf(g[i], x[i], dot);
                    }
                    dot = row_sum<LPR>(dot) * a.m * rs * rs;
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = rs * fmaf(-dot, x[i], g[i]);
                    if (on) Vec8<T>::store(static_cast<T*>(a.side[q].out) + (tok * a.side[q].heads + hd) * (int64_t)a.d + e0, g);
                }
            }
        }
    }

    if constexpr (BWD) {
        if (!a.partial) return;
        // sums of the CTA in a fixed order: lanes of one channel, then warps
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v = dw[q][i];
#pragma unroll
                for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                if (sub == 0 && mine) red[warp][q][e0 + i] = v;
            }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * a.d; e += kWarps * 32) {
            const int q = e / a.d, i = e - q * a.d;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += red[k][q][i];
            a.partial[((size_t)blockIdx.x * 2 + q) * a.d + i] = v;
        }
    }
}

// dw of one side, 32 channels per CTA: the CTAs' partial sums in a fixed order.
__global__ void __launch_bounds__(256)
norm_weight_grad_kernel(const float* __restrict__ partial, int ctas, int d, float* dwq, float* dwk)
{
    __shared__ double red[8][33];
    const int q = blockIdx.y, lane = threadIdx.x & 31, part = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float* dw = q ? dwk : dwq;
    if (!dw) return;
    double v = 0.0;
    if (i < d)
        for (int n = part; n < ctas; n += 8) v += (double)partial[((size_t)n * 2 + q) * d + i];
    red[part][lane] = v;
    __syncthreads();
    if (part == 0 && i < d) {
        for (int k = 1; k < 8; ++k) v += red[k][lane];
        dw[i] = (float)v;
    }
}

template <typename T, bool BWD>
cudaError_t launch_norm_t(const NormArgs& a, int ctas, cudaStream_t s) {
    auto kern = a.d <= 64 ? qk_norm_rope_kernel<T, 8, BWD>
              : a.d <= 128 ? qk_norm_rope_kernel<T, 16, BWD> : qk_norm_rope_kernel<T, 32, BWD>;
    kern<<<ctas, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t partial_bytes(int d) { return sizeof(float) * 2 * (size_t)d * kMaxCtas; }

kda_status check_sizes(int B, int T, int Hq, int Hk, int d, int rot, kda_dtype dtype, kda_norm norm, float eps) {
    if (dtype != KDA_F32 && dtype != KDA_BF16) return (kda_status)set_error(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (norm != KDA_NORM_RMS && norm != KDA_NORM_L2) return (kda_status)set_error(KDA_ERR_INVALID_ARG, "unknown norm %d", (int)norm);
    if (B < 0 || T < 0 || Hq <= 0 || Hk <= 0)
        return (kda_status)set_error(KDA_ERR_INVALID_ARG, "bad sizes B=%d T=%d Hq=%d Hk=%d", B, T, Hq, Hk);
    if (d <= 0 || d > 256 || d % 8) return (kda_status)set_error(KDA_ERR_UNSUPPORTED, "head size d=%d is not a multiple of 8 up to 256", d);
    if (rot < 0 || rot > d || rot % 16)
        return (kda_status)set_error(KDA_ERR_UNSUPPORTED, "rotary_dim=%d is not a multiple of 16 up to d=%d", rot, d);
    if (!(eps > 0.f) || eps > 3.0e38f) return (kda_status)set_error(KDA_ERR_INVALID_ARG, "eps=%g must be positive and finite", (double)eps);
    if ((int64_t)B * T >= (int64_t)1 << 31 || Hq > 65536 || Hk > 65536)
        return (kda_status)set_error(KDA_ERR_UNSUPPORTED, "B*T or the head count is too large");
    return KDA_OK;
}

kda_status run_norm(const void* q, const void* k, const void* dyq, const void* dyk, const float* wq, const float* wk,
                    const float* inv_freq, const int32_t* positions, int B, int T, int Hq, int Hk, int d, int rot,
                    const int64_t* qs, const int64_t* ks, kda_dtype dtype, kda_norm norm, float eps, int interleaved,
                    void* oq, void* ok_, float* dwq, float* dwk, void* workspace, size_t workspace_bytes, void* stream,
                    bool bwd) {
    const kda_status st = check_sizes(B, T, Hq, Hk, d, rot, dtype, norm, eps);
    if (st != KDA_OK) return st;
    const int64_t tokens = (int64_t)B * T;
    const bool sums = bwd && (dwq || dwk);
    if (tokens > 0) {
        if (!q || !k || !oq || !ok_ || !qs || !ks || (bwd && (!dyq || !dyk)) || (rot && !inv_freq))
            return (kda_status)set_error(KDA_ERR_INVALID_ARG, "null pointer");
        const int per16 = dtype == KDA_BF16 ? 8 : 4;
        if (!aligned16(q) || !aligned16(k) || !aligned16(oq) || !aligned16(ok_) || (bwd && (!aligned16(dyq) || !aligned16(dyk))))
            return (kda_status)set_error(KDA_ERR_INVALID_ARG, "queries, keys and outputs must be 16-byte aligned");
        for (int i = 0; i < 3; ++i)
            if (qs[i] % per16 || ks[i] % per16)
                return (kda_status)set_error(KDA_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
    }
    if (sums) {
        if (!workspace || workspace_bytes < partial_bytes(d))
            return (kda_status)set_error(KDA_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", workspace ? workspace_bytes : (size_t)0, partial_bytes(d));
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return (kda_status)set_error(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    NormArgs a{};
    a.side[0] = {q, dyq, oq, wq, qs ? qs[0] : 0, qs ? qs[1] : 0, qs ? qs[2] : 0, Hq};
    a.side[1] = {k, dyk, ok_, wk, ks ? ks[0] : 0, ks ? ks[1] : 0, ks ? ks[2] : 0, Hk};
    a.inv_freq = inv_freq; a.positions = positions;
    a.T = T > 0 ? T : 1; a.d = d; a.rot = rot; a.tokens = tokens; a.interleaved = interleaved != 0;
    a.m = norm == KDA_NORM_RMS ? 1.f / (float)d : 1.f;
    a.eps = eps;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    // all heads of a token by one warp; fewer when the tokens alone would not give
    // every SM sixteen warps
    const int heads = Hq + Hk, rpw = d <= 64 ? 4 : d <= 128 ? 2 : 1;
    a.slab = heads;
    while (a.slab > rpw && tokens * ((heads + a.slab - 1) / a.slab) < (int64_t)sms * 16) a.slab = (a.slab + 1) / 2;
    a.slab = (a.slab + rpw - 1) / rpw * rpw;
    a.slabs = (heads + a.slab - 1) / a.slab;
    const int64_t want = (tokens * a.slabs + kWarps - 1) / kWarps;
    const int ctas = (int)std::min<int64_t>(want, std::min(kMaxCtas, sms * (bwd ? 4 : 6)));
    if (e == cudaSuccess && ctas > 0) {
        if (dtype == KDA_BF16)
            e = bwd ? launch_norm_t<__nv_bfloat16, true>(a, ctas, static_cast<cudaStream_t>(stream))
                    : launch_norm_t<__nv_bfloat16, false>(a, ctas, static_cast<cudaStream_t>(stream));
        else
            e = bwd ? launch_norm_t<float, true>(a, ctas, static_cast<cudaStream_t>(stream))
                    : launch_norm_t<float, false>(a, ctas, static_cast<cudaStream_t>(stream));
    }
    if (e == cudaSuccess && sums) {
        norm_weight_grad_kernel<<<dim3((d + 31) / 32, 2), 256, 0, static_cast<cudaStream_t>(stream)>>>(
            a.partial, ctas, d, dwq, dwk);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return (kda_status)set_error(KDA_ERR_CUDA, "kda_qk_norm_rope launch failed: %s", cudaGetErrorString(e));
    return (kda_status)set_error(KDA_OK, "");
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight,
                            const float* inv_freq, const int32_t* positions, int B, int T, int Hq, int Hk, int d,
                            int rotary_dim, const int64_t* q_strides, const int64_t* k_strides, kda_dtype dtype,
                            kda_norm norm, float eps, int interleaved, void* q_out, void* k_out, void* stream) {
    return kda::run_norm(q, k, nullptr, nullptr, q_weight, k_weight, inv_freq, positions, B, T, Hq, Hk, d, rotary_dim,
                         q_strides, k_strides, dtype, norm, eps, interleaved, q_out, k_out, nullptr, nullptr, nullptr, 0,
                         stream, false);
}

size_t kda_qk_norm_rope_bwd_workspace_size(int d) {
    return d > 0 && d <= 256 && d % 8 == 0 ? kda::partial_bytes(d) : 0;
}

kda_status kda_qk_norm_rope_bwd(const void* q, const void* k, const void* d_q_out, const void* d_k_out,
                                const float* q_weight, const float* k_weight, const float* inv_freq,
                                const int32_t* positions, int B, int T, int Hq, int Hk, int d, int rotary_dim,
                                const int64_t* q_strides, const int64_t* k_strides, kda_dtype dtype, kda_norm norm,
                                float eps, int interleaved, void* dq, void* dk, float* dq_weight, float* dk_weight,
                                void* workspace, size_t workspace_bytes, void* stream) {
    return kda::run_norm(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions, B, T, Hq, Hk, d, rotary_dim,
                         q_strides, k_strides, dtype, norm, eps, interleaved, dq, dk, dq_weight, dk_weight, workspace,
                         workspace_bytes, stream, true);
}

}  // extern "C"
