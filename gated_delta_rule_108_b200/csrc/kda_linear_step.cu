// kda_linear_step.cu -- one token of the linear attention with one fixed decay per
// head, for B x H independent states (sm_100a):
//
//   S <- lambda S + k v^T,   o = dk^{-1/2} S^T q
//
// The state is read once and written once, 4 dk dv bytes each way per head, and
// that traffic bounds the step: B=256, H=32 takes 160 us, 6.8 TB/s, 3 % above a plain
// copy's rate.  Each thread holds four value columns of ROWS rows, all loaded before
// the first is used, so the update and the read need no exchange; the column sums are
// joined across the lanes of a warp that share columns, then across warps.
//
// One CTA per (sequence, head, NS value columns).  NS = dv reads whole rows; with fewer
// than four pairs per SM the columns are cut into slices of 32, which spreads a state
// over 2 or 4 SMs and evens out the last wave.  Whole rows and slices, dk = dv = 128:
// 16 pairs 2.5 and 1.7 us, 64 2.6 and 2.1, 256 4.7 and 4.7, 288 4.8 and 5.1, 320 6.3 and
// 5.5, 512 7.8 and 7.7, 1024 13.7 and 13.8.
#include "kda_common.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace {

template <typename T, int DK, int DV, int NS>
__global__ void __launch_bounds__(256)
linear_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                   const float* __restrict__ log_decay, float* __restrict__ state, T* __restrict__ o,
                   float scale, int H)
{
    constexpr int LANES = NS / 4;              // lanes across one row's columns
    constexpr int STEP = 256 / LANES;          // rows per pass of the CTA
    constexpr int ROWS = DK / STEP;            // rows per thread
    __shared__ float sk[DK], sq[DK];
    __shared__ float4 red[8][LANES];
    const int bh = blockIdx.x / (DV / NS);
    const int j0 = (blockIdx.x - bh * (DV / NS)) * NS;
    const int tid = threadIdx.x, col = tid % LANES, row = tid / LANES;
    float* S = state + (size_t)bh * DK * DV + j0 + 4 * col;

    float4 s[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        s[r] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)(row + r * STEP) * DV));
    for (int i = tid; i < DK; i += 256) {
        sk[i] = to_f32(k[(size_t)bh * DK + i]);
        sq[i] = to_f32(q[(size_t)bh * DK + i]);
    }
    float vj[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) vj[c] = to_f32(v[(size_t)bh * DV + j0 + 4 * col + c]);
    // lambda = m + keep with m = lambda - 1 where that is small: rounded to fp32 itself, a slow
    // decay is off by the same 2^-25 in every token (10,000 tokens at -1e-6: 3e-4 of the state)
    const float l = log_decay ? log_decay[bh % H] : 0.f;
    const bool slow = l > -0.5f;
    const float m = slow ? expm1f(l) : expf(l), keep = slow ? 1.f : 0.f;
    __syncthreads();

    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int i = row + r * STEP;
        const float ki = sk[i], qi = sq[i];
        s[r].x = fmaf(ki, vj[0], fmaf(m, s[r].x, keep * s[r].x));
        s[r].y = fmaf(ki, vj[1], fmaf(m, s[r].y, keep * s[r].y));
        s[r].z = fmaf(ki, vj[2], fmaf(m, s[r].z, keep * s[r].z));
        s[r].w = fmaf(ki, vj[3], fmaf(m, s[r].w, keep * s[r].w));
        __stcs(reinterpret_cast<float4*>(S + (size_t)i * DV), s[r]);
        acc.x = fmaf(qi, s[r].x, acc.x);
        acc.y = fmaf(qi, s[r].y, acc.y);
        acc.z = fmaf(qi, s[r].z, acc.z);
        acc.w = fmaf(qi, s[r].w, acc.w);
    }
#pragma unroll
    for (int off = 16; off >= LANES; off >>= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
    }
    if ((tid & 31) < LANES) red[tid >> 5][col] = acc;
    __syncthreads();
    if (tid < LANES) {
        float4 t = red[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) {
            const float4 x = red[w][tid];
            t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
        }
        T* dst = o + (size_t)bh * DV + j0 + 4 * tid;
        dst[0] = from_f32<T>(scale * t.x);
        dst[1] = from_f32<T>(scale * t.y);
        dst[2] = from_f32<T>(scale * t.z);
        dst[3] = from_f32<T>(scale * t.w);
    }
}

template <typename T, int DK, int DV>
cudaError_t launch_step_t(const LinStepArgs& a) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const unsigned pairs = (unsigned)(a.B * a.H);
    const T *q = static_cast<const T*>(a.q), *k = static_cast<const T*>(a.k), *v = static_cast<const T*>(a.v);
    if ((int)pairs < 4 * sms)
        linear_step_kernel<T, DK, DV, 32><<<pairs * (DV / 32), 256, 0, a.stream>>>(
            q, k, v, a.log_decay, a.state, static_cast<T*>(a.o), a.scale, a.H);
    else
        linear_step_kernel<T, DK, DV, DV><<<pairs, 256, 0, a.stream>>>(
            q, k, v, a.log_decay, a.state, static_cast<T*>(a.o), a.scale, a.H);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_dt(const LinStepArgs& a) {
    if (a.dk == 128 && a.dv == 128) return launch_step_t<T, 128, 128>(a);
    if (a.dk == 128 && a.dv == 64) return launch_step_t<T, 128, 64>(a);
    if (a.dk == 64 && a.dv == 128) return launch_step_t<T, 64, 128>(a);
    if (a.dk == 64 && a.dv == 64) return launch_step_t<T, 64, 64>(a);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_linear_step(const LinStepArgs& a) {
    if (a.B == 0) return cudaSuccess;
    return a.bf16 ? launch_step_dt<__nv_bfloat16>(a) : launch_step_dt<float>(a);
}

}  // namespace kda
