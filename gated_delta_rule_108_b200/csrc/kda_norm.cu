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
// Both read each row once and write it once: HBM bandwidth bounds them at size (65,536
// tokens of 32 + 8 heads, d = 128: 225 us in short runs, 91 % of a plain copy's rate, and
// 240 us, 85 %, at the clock that the power limit leaves in long ones, issue 54 %; the
// gradients of 4 x 4096 tokens of 16 + 16 heads 82 us, 75 %, and 86 us, 71 %, where the
// weights' sums hold 128 registers and leave two CTAs an SM), launch latency for a
// handful of tokens.  A lane holds eight channels of a row, in
// two groups of four chosen so that the two channels of a pair lie in one lane
// (4 l.. and 4 l + rotary_dim / 2.. where halves are paired), so LPR = d / 8 lanes
// (rounded up to 8, 16 or 32) share a row, a warp takes 32 / LPR rows at a time and
// the row's sums are the only exchange.  A warp works on the heads of one token (or
// a slab of them when there are few tokens): angle and weight of each channel are
// one pair of factors, formed once per token for queries and once for keys.  An
// angle is pos * freq in fp64, reduced to a turn before it is rounded to fp32:
// positions of 10^6 keep every bit of the angle that fp32 can hold.
#include "kda_common.cuh"
#include "kda_launch.h"
#include "../../include/kda.h"

#include <algorithm>
#include <cstdlib>

namespace kda {
namespace {

constexpr int kWarps = 8;              // per CTA
constexpr int kMaxCtas = 1024;         // partial weight gradients are sized for this many

struct NormSide {
    const void* x; const void* dy;     // dy: backward only
    void* out;                         // y, or dx
    const float* w;                    // [d], nullable
    int64_t sb, st;                    // element strides of x (batch, token)
    int sh, heads;                     // and head
};
struct NormArgs {
    NormSide side[2];                  // queries, keys
    const float* inv_freq; const int32_t* positions;
    int T, d, rot, slab, slabs;        // heads of one unit of work, units per token
    int64_t tokens;
    float m, eps;
    float* partial;                    // [CTAs][2][d], backward with weights only
};

// Four consecutive channels as loaded, and as fp32.
template <typename T> struct Vec4;
template <> struct Vec4<__nv_bfloat16> {
    uint2 raw;
    __device__ __forceinline__ void zero() { raw = make_uint2(0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldcs(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void get(float2 (&x)[2]) const { x[0] = unpack_bf16(raw.x); x[1] = unpack_bf16(raw.y); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&x)[2]) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y));
    }
};
template <> struct Vec4<float> {
    float4 raw;
    __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) { raw = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void get(float2 (&x)[2]) const { x[0] = make_float2(raw.x, raw.y); x[1] = make_float2(raw.z, raw.w); }
    static __device__ __forceinline__ void store(float* p, const float2 (&x)[2]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LPR / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The other channel of each pair of a lane's 2 x 4 channels.
template <bool INTER>
__device__ __forceinline__ float2 other_of(const float2 (&x)[4], int i) {
    return INTER ? make_float2(x[i].y, x[i].x) : x[i ^ 2];
}

template <typename T, int LPR, bool BWD, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, BWD ? 2 : 3)
qk_norm_rope_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int RPW = 32 / LPR;
    // rows in flight per lane, as registers allow for three (backward two) CTAs an SM
    constexpr int kUnroll = 8 / (int)sizeof(T);
    __shared__ __align__(8) float angle[kWarps][2][128];
    __shared__ double red[BWD ? kWarps : 1][2][BWD ? 256 : 1];   // each warp's weight gradients
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, l = lane % LPR;
    const bool mine = 8 * l < a.d;                 // lanes past the row's end only take part in sums
    const int half = a.rot / 2;
    // first channels of the lane's two groups
    const bool paired = !INTER && 4 * l < half;    // (j, j + half)
    const int e0 = paired ? 4 * l : 8 * l;
    const int e1 = paired ? e0 + half : e0 + 4;
    const bool turns = mine && (INTER ? e0 < a.rot : paired);

    float2 dw[BWD ? 2 : 1][4];                     // gradients of the weights of queries and keys
#pragma unroll
    for (int q = 0; q < (BWD ? 2 : 1); ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[q][i] = make_float2(0.f, 0.f);
    // Adds the lanes' sums, in a fixed order, to the warp's in 64 bits: every kRun terms, so
    // that the rounding of a sum does not grow with the batch (400,000 tokens of 8 equal
    // rows: 335 roundings off with one run, under 100 now; 85 and 87 us at 4 x 4096 x 16).
    auto join = [&]() {
#pragma unroll
        for (int q = 0; q < (BWD ? 2 : 1); ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 v = dw[q][i];
                dw[q][i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int off = LPR; off < 32; off <<= 1) {
                    v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
                    v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
                }
                const int e = (i < 2 ? e0 : e1) + 2 * (i & 1);
                if (sub == 0 && mine) {
                    red[warp][q][e] += (double)v.x;
                    red[warp][q][e + 1] += (double)v.y;
                }
            }
    };
    constexpr int kRun = 64;
    int terms = 0;                                 // since the last join
    if constexpr (BWD) {
        for (int e = lane; e < 512; e += 32) red[warp][e >> 8][e & 255] = 0.0;
        __syncwarp();
    }

    const int heads = a.side[0].heads + a.side[1].heads;
    const int64_t units = a.tokens * a.slabs, stride = (int64_t)gridDim.x * kWarps;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += stride) {
        const int64_t tok = u / a.slabs;
        const int first = (int)(u - tok * a.slabs) * a.slab, end = min(heads, first + a.slab);
        const int64_t b = tok / a.T, t = tok - b * a.T;
        if (a.rot) {
            const double pos = a.positions ? (double)a.positions[tok] : (double)t;
            __syncwarp();
            for (int j = lane; j < half; j += 32) {
                double rounds = pos * (double)a.inv_freq[j] * 0.15915494309189535;   // 1 / (2 pi)
                rounds -= rint(rounds);
                float sn, cs;
                sincospif(2.f * (float)rounds, &sn, &cs);
                angle[warp][0][j] = cs;
                angle[warp][1][j] = BWD ? -sn : sn;
            }
            __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const NormSide& z = a.side[q];
            const int shift = q ? a.side[0].heads : 0;
            const int lo = max(first - shift, 0), hi = min(end - shift, z.heads);    // this unit's heads of this side
            if (lo >= hi) continue;
            const T* x_tok = static_cast<const T*>(z.x) + b * z.sb + t * z.st + e0;
            const T* g_tok = BWD ? static_cast<const T*>(z.dy) + tok * z.heads * (int64_t)a.d + e0 : nullptr;
            T* out_tok = static_cast<T*>(z.out) + tok * z.heads * (int64_t)a.d + e0;
            const int sh = z.sh, to1 = e1 - e0;
            // y = n c + (other of n's pair) s, with c and s times the weights in the forward
            float2 w[4], c[4], s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = (i < 2 ? e0 : e1) + 2 * (i & 1);
                w[i] = (mine && z.w) ? *reinterpret_cast<const float2*>(z.w + e) : make_float2(1.f, 1.f);
                c[i] = make_float2(1.f, 1.f);
                s[i] = make_float2(0.f, 0.f);
                if (!turns) continue;
                if constexpr (INTER) {             // pair (x, y) of one float2
                    const float cs = angle[warp][0][e / 2], sn = angle[warp][1][e / 2];
                    c[i] = make_float2(cs, cs);
                    s[i] = make_float2(-sn, sn);
                } else {                           // pairs (x[0], x[2]), (x[1], x[3])
                    const int j = e0 + 2 * (i & 1);
                    const float2 sn = *reinterpret_cast<const float2*>(&angle[warp][1][j]);
                    c[i] = *reinterpret_cast<const float2*>(&angle[warp][0][j]);
                    s[i] = i < 2 ? make_float2(-sn.x, -sn.y) : sn;
                }
            }
            if constexpr (!BWD) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[i] = mul2(w[i], c[i]);
                    s[i] = mul2(other_of<INTER>(w, i), s[i]);
                }
            }
            for (int r0 = lo; r0 < hi; r0 += RPW * kUnroll) {
                Vec4<T> xv[kUnroll][2], gv[BWD ? kUnroll : 1][2];
#pragma unroll
                for (int n = 0; n < kUnroll; ++n) {     // all loads first
                    const int r = r0 + n * RPW + sub;
                    xv[n][0].zero();
                    xv[n][1].zero();
                    if constexpr (BWD) {
                        gv[n][0].zero();
                        gv[n][1].zero();
                    }
                    if (r < hi && mine) {
                        const T* p = x_tok + r * sh;
                        xv[n][0].load(p);
                        xv[n][1].load(p + to1);
                        if constexpr (BWD) {
                            const T* g = g_tok + r * a.d;
                            gv[n][0].load(g);
                            gv[n][1].load(g + to1);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < kUnroll; ++n) {
                    if (r0 + n * RPW >= hi) break;      // uniform over the warp
                    const int r = r0 + n * RPW + sub;
                    float2 x[4], h[4];
                    xv[n][0].get(*reinterpret_cast<float2(*)[2]>(&x[0]));
                    xv[n][1].get(*reinterpret_cast<float2(*)[2]>(&x[2]));
                    float2 ss = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
                    const float rs = rsqrtf(fmaf(row_sum<LPR>(ss.x + ss.y), a.m, a.eps));
                    const float2 rr = make_float2(rs, rs);
                    if constexpr (!BWD) {
                        // a channel that does not turn takes nothing from its neighbour, be it infinite
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 y = mul2(x[i], c[i]);
                            h[i] = mul2(rr, turns ? fma2(other_of<INTER>(x, i), s[i], y) : y);
                        }
                    } else {
                        float2 g[4], dot = make_float2(0.f, 0.f);
                        gv[n][0].get(*reinterpret_cast<float2(*)[2]>(&g[0]));
                        gv[n][1].get(*reinterpret_cast<float2(*)[2]>(&g[2]));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 y = mul2(g[i], c[i]);
                            h[i] = turns ? fma2(other_of<INTER>(g, i), s[i], y) : y;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            dw[q][i] = fma2(mul2(h[i], x[i]), rr, dw[q][i]);
                            h[i] = mul2(h[i], w[i]);
                            dot = fma2(h[i], x[i], dot);
                        }
                        const float k = -row_sum<LPR>(dot.x + dot.y) * a.m * rs * rs;
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = mul2(rr, fma2(make_float2(k, k), x[i], h[i]));
                    }
                    if (r < hi && mine) {
                        T* out = out_tok + r * a.d;
                        Vec4<T>::store(out, *reinterpret_cast<const float2(*)[2]>(&h[0]));
                        Vec4<T>::store(out + to1, *reinterpret_cast<const float2(*)[2]>(&h[2]));
                    }
                }
            }
        }
        if constexpr (BWD) {
            terms += (end - first + RPW - 1) / RPW;
            if (terms >= kRun && a.partial) {
                join();
                terms = 0;
            }
        }
    }

    if constexpr (BWD) {
        if (!a.partial) return;
        // sums of the CTA in a fixed order: lanes of one channel, then warps
        join();
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * a.d; e += kWarps * 32) {
            const int q = e / a.d, i = e - q * a.d;
            double v = 0.0;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += red[k][q][i];
            a.partial[((size_t)blockIdx.x * 2 + q) * a.d + i] = (float)v;
        }
    }
}

// dw of one side, 32 channels per CTA: the CTAs' partial sums in a fixed order.
__global__ void __launch_bounds__(1024)
norm_weight_grad_kernel(const float* __restrict__ partial, int ctas, int d, float* dwq, float* dwk)
{
    __shared__ double red[32][33];
    const int q = blockIdx.y, lane = threadIdx.x & 31, part = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float* dw = q ? dwk : dwq;
    if (!dw) return;
    double v = 0.0;
    if (i < d) {
#pragma unroll 4
        for (int n = part; n < ctas; n += 32) v += (double)partial[((size_t)n * 2 + q) * d + i];
    }
    red[part][lane] = v;
    __syncthreads();
    v = red[lane][part];                       // this warp's channel, one part a lane
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0 && blockIdx.x * 32 + part < d) dw[blockIdx.x * 32 + part] = (float)v;
}

template <typename T, bool BWD, bool INTER>
cudaError_t launch_norm_t(const NormArgs& a, int ctas, cudaStream_t s) {
    auto kern = a.d <= 64 ? qk_norm_rope_kernel<T, 8, BWD, INTER>
              : a.d <= 128 ? qk_norm_rope_kernel<T, 16, BWD, INTER> : qk_norm_rope_kernel<T, 32, BWD, INTER>;
    kern<<<ctas, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_norm(const NormArgs& a, bool bwd, bool interleaved, int ctas, cudaStream_t s) {
    if (bwd) return interleaved ? launch_norm_t<T, true, true>(a, ctas, s) : launch_norm_t<T, true, false>(a, ctas, s);
    return interleaved ? launch_norm_t<T, false, true>(a, ctas, s) : launch_norm_t<T, false, false>(a, ctas, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes [lo, hi) that a tensor's elements lie in.
struct Extent { const char* lo; const char* hi; };
Extent dense(const void* p, int64_t bytes) { return {static_cast<const char*>(p), static_cast<const char*>(p) + bytes}; }
Extent strided(const void* p, const int64_t* s, int B, int T, int H, int d, int es) {
    const int64_t n[3] = {B, T, H};
    int64_t lo = 0, hi = d;
    for (int i = 0; i < 3; ++i) (s[i] < 0 ? lo : hi) += s[i] * (n[i] - 1);
    return {static_cast<const char*>(p) + lo * es, static_cast<const char*>(p) + hi * es};
}
bool is_dense(const int64_t* s, int B, int T, int H, int d) {
    return (H == 1 || s[2] == d) && (T == 1 || s[1] == (int64_t)H * d) && (B == 1 || s[0] == (int64_t)T * H * d);
}
// A step of s elements, n - 1 times, stays below `reach` (without a product that could wrap).
bool within(int64_t s, int64_t n, int64_t reach) { return s > -reach && s < reach && (n < 2 || std::abs(s) <= (reach - 1) / n); }
bool meet(const Extent& a, const Extent& b) { return a.lo && b.lo && a.lo < b.hi && b.lo < a.hi; }

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
    const int64_t wbytes = (int64_t)sizeof(float) * d;
    const Extent shared_in[4] = {dense(wq, wbytes), dense(wk, wbytes), dense(inv_freq, (int64_t)sizeof(float) * (rot / 2)),
                                 dense(positions, (int64_t)sizeof(int32_t) * tokens)};
    Extent rows[6] = {};               // inputs, outputs, cotangents
    if (tokens > 0) {
        if (!q || !k || !oq || !ok_ || (bwd && (!dyq || !dyk)) || (rot && !inv_freq))
            return (kda_status)set_error(KDA_ERR_INVALID_ARG, "null pointer");
        const int per16 = dtype == KDA_BF16 ? 8 : 4;
        if (!aligned16(q) || !aligned16(k) || !aligned16(oq) || !aligned16(ok_) || !aligned16(wq) || !aligned16(wk) || (bwd && (!aligned16(dyq) || !aligned16(dyk))))
            return (kda_status)set_error(KDA_ERR_INVALID_ARG, "queries, keys, weights and outputs must be 16-byte aligned");
        for (int i = 0; i < 3; ++i)
            if (qs[i] % per16 || ks[i] % per16)
                return (kda_status)set_error(KDA_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
        const int64_t reach = (int64_t)1 << 31;   // of a token's heads, whose offsets are 32 bits
        if (!within(qs[2], Hq, reach) || !within(ks[2], Hk, reach) || (int64_t)std::max(Hq, Hk) * d >= reach)
            return (kda_status)set_error(KDA_ERR_UNSUPPORTED, "the heads of one token span 2^31 elements or more");
        const int64_t memory = (int64_t)1 << 46;  // elements; no GPU's addresses reach further
        const int64_t n[2] = {B, T};
        for (int i = 0; i < 2; ++i)
            if (n[i] > 1 && (!within(qs[i], n[i], memory) || !within(ks[i], n[i], memory)))
                return (kda_status)set_error(KDA_ERR_UNSUPPORTED, "queries or keys span 2^46 elements or more");
        // an output may be its own input, contiguous: each row is read before it is written
        const int es = dtype == KDA_BF16 ? 2 : 4;
        const Extent xq = strided(q, qs, B, T, Hq, d, es), xk = strided(k, ks, B, T, Hk, d, es);
        const Extent yq = dense(oq, tokens * Hq * d * es), yk = dense(ok_, tokens * Hk * d * es);
        const bool own_q = !bwd && oq == q && is_dense(qs, B, T, Hq, d), own_k = !bwd && ok_ == k && is_dense(ks, B, T, Hk, d);
        if ((!own_q && meet(yq, xq)) || (!own_k && meet(yk, xk)) || meet(yq, xk) || meet(yk, xq) || meet(yq, yk))
            return (kda_status)set_error(KDA_ERR_INVALID_ARG, "an output overlaps an input or the other output");
        if (bwd) {
            const Extent gq = dense(dyq, tokens * Hq * d * es), gk = dense(dyk, tokens * Hk * d * es);
            if (meet(yq, gq) || meet(yq, gk) || meet(yk, gq) || meet(yk, gk))
                return (kda_status)set_error(KDA_ERR_INVALID_ARG, "an output overlaps a cotangent");
            rows[4] = gq;
            rows[5] = gk;
        }
        for (const Extent& x : shared_in)
            if (meet(yq, x) || meet(yk, x))
                return (kda_status)set_error(KDA_ERR_INVALID_ARG, "an output overlaps a weight, the frequencies or the positions");
        rows[0] = xq; rows[1] = xk; rows[2] = yq; rows[3] = yk;
    }
    if (sums) {
        if (!workspace || workspace_bytes < partial_bytes(d))
            return (kda_status)set_error(KDA_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", workspace ? workspace_bytes : (size_t)0, partial_bytes(d));
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return (kda_status)set_error(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
        const Extent out[3] = {dense(dwq, wbytes), dense(dwk, wbytes), dense(workspace, (int64_t)partial_bytes(d))};
        bool bad = meet(out[0], out[1]) || meet(out[0], out[2]) || meet(out[1], out[2]);
        for (const Extent& y : out) {
            for (const Extent& x : shared_in) bad |= meet(y, x);
            for (const Extent& x : rows) bad |= meet(y, x);
        }
        if (bad) return (kda_status)set_error(KDA_ERR_INVALID_ARG, "a weight gradient or the workspace overlaps another tensor");
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    NormArgs a{};
    a.side[0] = {q, dyq, oq, wq, qs[0], qs[1], (int)qs[2], Hq};
    a.side[1] = {k, dyk, ok_, wk, ks[0], ks[1], (int)ks[2], Hk};
    a.inv_freq = inv_freq; a.positions = positions;
    a.T = T > 0 ? T : 1; a.d = d; a.rot = rot; a.tokens = tokens;
    a.m = norm == KDA_NORM_RMS ? 1.f / (float)d : 1.f;
    a.eps = eps;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    // all heads of a token by one warp; fewer when the tokens alone would not give
    // every SM sixteen warps (40 heads, not cut / cut: 1 token 6.3 / 2.7 us, 64 7.2 / 3.0,
    // 256 7.3 / 3.6, 1024 7.6 / 7.1; with a bound of 8 warps 256 take 3.9, of 32 4.7 us)
    const int heads = Hq + Hk, rpw = d <= 64 ? 4 : d <= 128 ? 2 : 1;
    a.slab = heads;
    while (a.slab > rpw && tokens * ((heads + a.slab - 1) / a.slab) < (int64_t)sms * 16) a.slab = (a.slab + 1) / 2;
    a.slab = (a.slab + rpw - 1) / rpw * rpw;
    a.slabs = (heads + a.slab - 1) / a.slab;
    const int64_t want = (tokens * a.slabs + kWarps - 1) / kWarps;
    const int ctas = (int)std::min<int64_t>(want, std::min(kMaxCtas, sms * (bwd ? 2 : 3)));
    if (e == cudaSuccess && ctas > 0) {
        e = dtype == KDA_BF16
            ? launch_norm<__nv_bfloat16>(a, bwd, interleaved != 0, ctas, static_cast<cudaStream_t>(stream))
            : launch_norm<float>(a, bwd, interleaved != 0, ctas, static_cast<cudaStream_t>(stream));
    }
    if (e == cudaSuccess && sums) {
        norm_weight_grad_kernel<<<dim3((d + 31) / 32, 2), 1024, 0, static_cast<cudaStream_t>(stream)>>>(
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
                            int rotary_dim, int64_t q_stride_b, int64_t q_stride_t, int64_t q_stride_h, int64_t k_stride_b,
                            int64_t k_stride_t, int64_t k_stride_h, kda_dtype dtype,
                            kda_norm norm, float eps, int interleaved, void* q_out, void* k_out, void* stream) {
    const int64_t q_strides[3] = {q_stride_b, q_stride_t, q_stride_h}, k_strides[3] = {k_stride_b, k_stride_t, k_stride_h};
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
                                int64_t q_stride_b, int64_t q_stride_t, int64_t q_stride_h, int64_t k_stride_b,
                                int64_t k_stride_t, int64_t k_stride_h, kda_dtype dtype, kda_norm norm,
                                float eps, int interleaved, void* dq, void* dk, float* dq_weight, float* dk_weight,
                                void* workspace, size_t workspace_bytes, void* stream) {
    const int64_t q_strides[3] = {q_stride_b, q_stride_t, q_stride_h}, k_strides[3] = {k_stride_b, k_stride_t, k_stride_h};
    return kda::run_norm(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions, B, T, Hq, Hk, d, rotary_dim,
                         q_strides, k_strides, dtype, norm, eps, interleaved, dq, dk, dq_weight, dk_weight, workspace,
                         workspace_bytes, stream, true);
}

}  // extern "C"
