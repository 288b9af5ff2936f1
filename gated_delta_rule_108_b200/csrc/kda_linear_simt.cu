// kda_linear_simt.cu -- linear attention with one fixed decay per head: the
// segment table, the scan over segments, and the chunk kernel on CUDA cores that
// serves fp32 inputs (sm_100a).
//
// Per chunk of 64 tokens with entering state Z, local index r, lengths L, and the
// processing direction's order (kda_linear.cuh names the roles a, b, c, y):
//
//   P_ri = lambda^{|r - i|} <a_r, b_i>          i <= r  (i >= r last to first)
//   y_r  = c_intra sum_i P_ri c_i + c_inter lambda^{n_r} Z^T a_r
//   Z'   = lambda^L Z + c_upd sum_i lambda^{m_i} b_i c_i^T
//
// with n_r = r + 1, m_i = L - 1 - i first to last and n_r = L - 1 - r,
// m_i = i + 1 last to first (a cotangent decays when it leaves its token, a state
// before it enters).
#include "kda_linear.cuh"

namespace kda {
namespace {

// ------------------------------------------------------------- segments --
// Packed sequences: checks cu, orders the sequences longest first (up to 4096 of
// them; more are taken as they come) and writes the segment table.  One segment
// per sequence when the longest has at most `balance_tokens` tokens, the share of
// one SM: then the sequences alone balance and the extra pass over b and c is
// saved.
__global__ void __launch_bounds__(1024)
linear_prep_kernel(WsHeader* hdr, int32_t* tab, const int32_t* __restrict__ cu, int N, int T, int seg_tok,
                   int balance_tokens)
{
    __shared__ int warp_sums[32];
    __shared__ int s_carry, s_bad, s_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (cu == nullptr) {
        if (tid == 0) { hdr->status = kStatusOk; hdr->runtime_err = 0; }
        return;
    }
    if (tid == 0) { s_carry = 0; s_max = 0; s_bad = (cu[0] != 0 || cu[N] != T) ? 1 : 0; }
    __syncthreads();
    for (int s = tid; s < N; s += 1024) {
        const int lo = cu[s], hi = cu[s + 1];
        if (hi < lo) atomicOr(&s_bad, 1);
        else atomicMax(&s_max, hi - lo);
    }
    __syncthreads();
    if (s_bad) {
        if (tid == 0) { hdr->status = kStatusBadSeqlens; hdr->runtime_err = 0; }
        return;
    }
    const int size = s_max <= balance_tokens ? max(s_max, 1) : seg_tok;
    int32_t* first = tab + 1;
    int32_t* order = tab + 2 + N;
    for (int s = tid; s < N; s += 1024) {
        int rank = s;
        if (N <= 4096) {
            const int len = cu[s + 1] - cu[s];
            rank = 0;
            for (int t = 0; t < N; ++t) {
                const int lt = cu[t + 1] - cu[t];
                rank += (lt > len) || (lt == len && t < s);
            }
        }
        order[rank] = s;
    }
    __syncthreads();
    for (int base = 0; base < N; base += 1024) {   // exclusive scan of the segment counts
        const int r = base + tid;
        int cnt = 0;
        if (r < N) {
            const int s = order[r], len = cu[s + 1] - cu[s];
            cnt = len > size ? (len - 1) / size + 1 : 1;
        }
        int incl = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const int w = warp_sums[lane];
            int wi = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, wi, off);
                if (lane >= off) wi += y;
            }
            warp_sums[lane] = wi - w;
        }
        __syncthreads();
        const int excl = s_carry + warp_sums[warp] + incl - cnt;
        if (r < N) first[r] = excl;
        __syncthreads();
        if (tid == 1023) s_carry = excl + cnt;
        __syncthreads();
    }
    if (tid == 0) {
        first[N] = s_carry;
        tab[0] = size;
        hdr->status = kStatusOk;
        hdr->runtime_err = 0;
    }
}

// Each segment's own sum becomes its entering state, in processing order:
// E_0 = initial state, E_{j+1} = lambda^{len_j} E_j + (segment j's sum).
// One thread per four elements of Z; grid (sequence * H + h, element groups, role).
__global__ void __launch_bounds__(256)
linear_scan_kernel(const __grid_constant__ LinArgs a)
{
    if (a.hdr->status != kStatusOk) return;
    const LinRole& role = a.role[blockIdx.z];
    const int r = blockIdx.x / a.H, h = blockIdx.x - r * a.H;
    int seq, first, count;
    a.map.range(r, seq, first, count);
    if (count < 2) return;                      // the main pass reads the initial state itself
    const int size = a.dk * a.dv, e = 4 * (blockIdx.y * 256 + threadIdx.x);
    if (e >= size) return;
    const double l = lin_log_decay(a.log_decay, h);
    float4 E = make_float4(0.f, 0.f, 0.f, 0.f);
    if (role.s_in) {
        const float* src = role.s_in + ((size_t)seq * a.H + h) * size;
        if (!role.transposed) {
            E = *reinterpret_cast<const float4*>(src + e);
        } else {                                // Z is [dv, dk]: element (j, i) is the user's (i, j)
            const int j = e / a.dk, i = e - j * a.dk;
            E = make_float4(src[(size_t)i * a.dv + j], src[(size_t)(i + 1) * a.dv + j],
                            src[(size_t)(i + 2) * a.dv + j], src[(size_t)(i + 3) * a.dv + j]);
        }
    }
    for (int n = 0; n < count; ++n) {
        const int s = first + (role.reverse ? count - 1 - n : n);
        float4* p = reinterpret_cast<float4*>(role.seg + ((size_t)s * a.H + h) * size + e);
        float4 own = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n + 1 < count) own = *p;            // the last segment's own sum is not computed
        *p = E;
        const float w = lin_pow(l, a.map.locate(s).len);
        E.x = fmaf(w, E.x, own.x);
        E.y = fmaf(w, E.y, own.y);
        E.z = fmaf(w, E.z, own.z);
        E.w = fmaf(w, E.w, own.w);
    }
}

// ------------------------------------------------------------ CUDA cores --
constexpr int kSimtChunk = 64, kSimtCols = 64;   // tokens per chunk, value columns per CTA

template <int D1>
struct LinSimtSmem {
    static constexpr int LDA = D1 + 4;           // rows 16 bytes apart in the banks: float4 reads of 8 rows do not clash
    static constexpr int LDC = kSimtCols, LDP = kSimtChunk + 4;
    float a[kSimtChunk][LDA], b[kSimtChunk][LDA];
    float c[kSimtChunk][LDC], p[kSimtChunk][LDP], z[D1][LDC];
    float pw[kSimtChunk + 1];
};

// One CTA per (segment, head, 64 columns of D2); 256 threads.  A thread owns 4 x 4
// of P and of y (rows ty + 16 n) and D1 / 16 x 4 of Z, which stays in registers
// with a copy in shared memory for the read.  Bound by FMA issue: 64 FMAs per 8
// 16-byte shared-memory reads.
template <typename T, int D1, int D2>
__global__ void __launch_bounds__(256)
linear_simt_kernel(const __grid_constant__ LinArgs args, int states_only)
{
    using Sm = LinSimtSmem<D1>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    if (args.hdr->status != kStatusOk) return;
    constexpr int SL = D2 / kSimtCols, ZR = D1 / 16;
    int x = blockIdx.x;
    const int slice = x % SL;
    x /= SL;
    const LinRole& role = args.role[x % args.roles];
    x /= args.roles;
    const int H = args.H, h = x % H, sidx = x / H;
    if (sidx >= args.map.segments()) return;
    const LinMap::Seg g = args.map.locate(sidx);
    const bool rev = role.reverse;
    const bool last = g.index == (rev ? 0 : g.count - 1);        // the segment processed last
    if (states_only && last) return;
    const int j0 = slice * kSimtCols;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const double l = lin_log_decay(args.log_decay, h);
    for (int n = tid; n <= kSimtChunk; n += 256) sm.pw[n] = lin_pow(l, n);

    const size_t zsize = (size_t)D1 * D2;
    const size_t user = ((size_t)g.seq * H + h) * zsize;
    float* seg = role.seg ? role.seg + ((size_t)sidx * H + h) * zsize : nullptr;
    float4 z[ZR];
    const float* from = states_only ? nullptr : (g.count > 1 ? seg : (role.s_in ? role.s_in + user : nullptr));
    const bool tr_in = g.count == 1 && role.transposed;
#pragma unroll
    for (int n = 0; n < ZR; ++n) {
        const int i = ty * ZR + n, j = j0 + 4 * tx;
        z[n] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from)
            z[n] = tr_in ? make_float4(from[(size_t)j * D1 + i], from[(size_t)(j + 1) * D1 + i],
                                       from[(size_t)(j + 2) * D1 + i], from[(size_t)(j + 3) * D1 + i])
                         : *reinterpret_cast<const float4*>(from + (size_t)i * D2 + j);
    }
    const T* pa = static_cast<const T*>(args.x[role.a]);
    const T* pb = static_cast<const T*>(args.x[role.b]);
    const T* pc = static_cast<const T*>(args.x[role.c]);
    T* py = static_cast<T*>(role.y);
    const int nch = (g.len + kSimtChunk - 1) / kSimtChunk;
    for (int n = 0; n < nch; ++n) {
        const int ch = rev ? nch - 1 - n : n;
        const int tok0 = g.begin + ch * kSimtChunk, L = min(kSimtChunk, g.len - ch * kSimtChunk);
        __syncthreads();                         // the previous chunk's reads are done
        for (int e = tid; e < kSimtChunk * D1; e += 256) {
            const int r = e / D1, i = e - r * D1;
            const size_t at = ((size_t)(tok0 + r) * H + h) * D1 + i;
            sm.b[r][i] = r < L ? to_f32(pb[at]) : 0.f;
            if (!states_only) sm.a[r][i] = r < L ? to_f32(pa[at]) : 0.f;
        }
        for (int e = tid; e < kSimtChunk * kSimtCols; e += 256) {
            const int r = e / kSimtCols, j = e - r * kSimtCols;
            sm.c[r][j] = r < L ? to_f32(pc[((size_t)(tok0 + r) * H + h) * D2 + j0 + j]) : 0.f;
        }
        if (!states_only) {
#pragma unroll
            for (int i = 0; i < ZR; ++i) *reinterpret_cast<float4*>(&sm.z[ty * ZR + i][4 * tx]) = z[i];
        }
        __syncthreads();
        if (!states_only) {
            float acc[4][4] = {};
            for (int i = 0; i < D1; i += 4) {
                float4 av[4], bv[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    av[m] = *reinterpret_cast<const float4*>(&sm.a[ty + 16 * m][i]);
                    bv[m] = *reinterpret_cast<const float4*>(&sm.b[tx + 16 * m][i]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        acc[m][k] = fmaf(av[m].x, bv[k].x, acc[m][k]);
                        acc[m][k] = fmaf(av[m].y, bv[k].y, acc[m][k]);
                        acc[m][k] = fmaf(av[m].z, bv[k].z, acc[m][k]);
                        acc[m][k] = fmaf(av[m].w, bv[k].w, acc[m][k]);
                    }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int lag = rev ? (tx + 16 * k) - (ty + 16 * m) : (ty + 16 * m) - (tx + 16 * k);
                    sm.p[ty + 16 * m][tx + 16 * k] = lag >= 0 ? sm.pw[lag] * acc[m][k] : 0.f;
                }
            __syncthreads();
            float4 in[4], out[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                in[m] = make_float4(0.f, 0.f, 0.f, 0.f);
                out[m] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            auto axpy = [](float4& y, float p, const float4& c) {
                y.x = fmaf(p, c.x, y.x); y.y = fmaf(p, c.y, y.y);
                y.z = fmaf(p, c.z, y.z); y.w = fmaf(p, c.w, y.w);
            };
            for (int i = 0; i < kSimtChunk; i += 4) {
                float4 c0 = *reinterpret_cast<const float4*>(&sm.c[i][4 * tx]);
                float4 c1 = *reinterpret_cast<const float4*>(&sm.c[i + 1][4 * tx]);
                float4 c2 = *reinterpret_cast<const float4*>(&sm.c[i + 2][4 * tx]);
                float4 c3 = *reinterpret_cast<const float4*>(&sm.c[i + 3][4 * tx]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 p = *reinterpret_cast<const float4*>(&sm.p[ty + 16 * m][i]);
                    axpy(in[m], p.x, c0); axpy(in[m], p.y, c1); axpy(in[m], p.z, c2); axpy(in[m], p.w, c3);
                }
            }
            for (int i = 0; i < D1; i += 4) {
                float4 c0 = *reinterpret_cast<const float4*>(&sm.z[i][4 * tx]);
                float4 c1 = *reinterpret_cast<const float4*>(&sm.z[i + 1][4 * tx]);
                float4 c2 = *reinterpret_cast<const float4*>(&sm.z[i + 2][4 * tx]);
                float4 c3 = *reinterpret_cast<const float4*>(&sm.z[i + 3][4 * tx]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 p = *reinterpret_cast<const float4*>(&sm.a[ty + 16 * m][i]);
                    axpy(out[m], p.x, c0); axpy(out[m], p.y, c1); axpy(out[m], p.z, c2); axpy(out[m], p.w, c3);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int r = ty + 16 * m;
                if (r < L) {
                    const float w = role.c_inter * sm.pw[rev ? L - 1 - r : r + 1];
                    T* dst = py + ((size_t)(tok0 + r) * H + h) * D2 + j0 + 4 * tx;
                    dst[0] = from_f32<T>(fmaf(w, out[m].x, role.c_intra * in[m].x));
                    dst[1] = from_f32<T>(fmaf(w, out[m].y, role.c_intra * in[m].y));
                    dst[2] = from_f32<T>(fmaf(w, out[m].z, role.c_intra * in[m].z));
                    dst[3] = from_f32<T>(fmaf(w, out[m].w, role.c_intra * in[m].w));
                }
            }
            __syncthreads();                     // c is weighted in place next
        }
        for (int e = tid; e < kSimtChunk * kSimtCols; e += 256) {
            const int r = e / kSimtCols;
            if (r < L) sm.c[r][e - r * kSimtCols] *= role.c_upd * sm.pw[rev ? r + 1 : L - 1 - r];
        }
        __syncthreads();
        const float w = sm.pw[L];
#pragma unroll
        for (int i = 0; i < ZR; ++i) { z[i].x *= w; z[i].y *= w; z[i].z *= w; z[i].w *= w; }
        for (int r = 0; r < kSimtChunk; ++r) {
            const float4 c = *reinterpret_cast<const float4*>(&sm.c[r][4 * tx]);
#pragma unroll
            for (int i = 0; i < ZR; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(&sm.b[r][ty * ZR + i]);
                const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    z[i + m].x = fmaf(bb[m], c.x, z[i + m].x);
                    z[i + m].y = fmaf(bb[m], c.y, z[i + m].y);
                    z[i + m].z = fmaf(bb[m], c.z, z[i + m].z);
                    z[i + m].w = fmaf(bb[m], c.w, z[i + m].w);
                }
            }
        }
    }
    float* to = states_only ? seg : (last && role.s_out ? role.s_out + user : nullptr);
    if (!to) return;
    const bool tr_out = !states_only && role.transposed;
#pragma unroll
    for (int n = 0; n < ZR; ++n) {
        const int i = ty * ZR + n, j = j0 + 4 * tx;
        if (tr_out) {
            to[(size_t)j * D1 + i] = z[n].x;
            to[(size_t)(j + 1) * D1 + i] = z[n].y;
            to[(size_t)(j + 2) * D1 + i] = z[n].z;
            to[(size_t)(j + 3) * D1 + i] = z[n].w;
        } else {
            *reinterpret_cast<float4*>(to + (size_t)i * D2 + j) = z[n];
        }
    }
}

template <typename T, int D1, int D2>
cudaError_t launch_simt_t(const LinArgs& a, bool states_only) {
    auto kern = linear_simt_kernel<T, D1, D2>;
    const int smem = (int)sizeof(LinSimtSmem<D1>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const size_t grid = (size_t)a.max_segments * a.H * a.roles * (D2 / kSimtCols);
    kern<<<(unsigned)grid, 256, smem, a.stream>>>(a, states_only ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_prep(const LinArgs& a, int32_t* tab, int seg_tok, int balance_tokens) {
    linear_prep_kernel<<<1, a.map.cu ? 1024 : 32, 0, a.stream>>>(a.hdr, tab, a.map.cu, a.map.N, a.map.T, seg_tok,
                                                                 balance_tokens);
    return cudaGetLastError();
}

cudaError_t launch_linear_scan(const LinArgs& a) {
    const dim3 grid((unsigned)((size_t)a.map.N * a.H), (unsigned)((a.dk * a.dv + 1023) / 1024), (unsigned)a.roles);
    linear_scan_kernel<<<grid, 256, 0, a.stream>>>(a);
    return cudaGetLastError();
}

// All roles of one launch have the same (D1, D2): those of its first role's inputs.
cudaError_t launch_linear_simt(const LinArgs& a, bool states_only) {
    const int d1 = a.dim[a.role[0].a], d2 = a.dim[a.role[0].c];
    if (d1 == 128 && d2 == 128) return launch_simt_t<float, 128, 128>(a, states_only);
    if (d1 == 128 && d2 == 64) return launch_simt_t<float, 128, 64>(a, states_only);
    if (d1 == 64 && d2 == 128) return launch_simt_t<float, 64, 128>(a, states_only);
    if (d1 == 64 && d2 == 64) return launch_simt_t<float, 64, 64>(a, states_only);
    return cudaErrorInvalidValue;
}

}  // namespace kda
