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
#include <algorithm>

#include "kda_linear.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

using namespace ptx;

// ------------------------------------------------------------- segments --
// Exclusive sum over the block's 1024 threads.
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    __syncthreads();                               // the sums of the scan before have been read
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
    return warp_sums[warp] + incl - v;
}

// Packed sequences: checks cu, orders the sequences longest first, by 1024 classes of
// length (within a class as the threads come: the order says when a segment is worked
// on, not what it gives), and writes the segment table.  One segment per sequence when
// the longest has at most `balance_tokens` tokens, the share of one SM: then the
// sequences alone balance and the extra pass over b and c is saved.
__global__ void __launch_bounds__(1024)
linear_prep_kernel(WsHeader* hdr, int32_t* tab, const int32_t* __restrict__ cu, int N, int T, int seg_tok,
                   int balance_tokens)
{
    __shared__ int warp_sums[32], place[1024];
    __shared__ int s_bad, s_max;
    const int tid = threadIdx.x;
    if (tid == 0) { s_max = 0; s_bad = (cu[0] != 0 || cu[N] != T) ? 1 : 0; }
    place[tid] = 0;
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
    const int width = s_max / 1024 + 1;
    int32_t* first = tab + 1;
    int32_t* order = tab + 2 + N;
    for (int s = tid; s < N; s += 1024) atomicAdd(&place[1023 - (cu[s + 1] - cu[s]) / width], 1);
    __syncthreads();
    place[tid] = block_scan(place[tid], warp_sums);
    __syncthreads();
    for (int s = tid; s < N; s += 1024) order[atomicAdd(&place[1023 - (cu[s + 1] - cu[s]) / width], 1)] = s;
    __syncthreads();
    int carry = 0;                                 // the same in every thread
    for (int base = 0; base < N; base += 1024) {   // exclusive scan of the segment counts
        const int r = base + tid;
        int cnt = 0;
        if (r < N) {
            const int s = order[r], len = cu[s + 1] - cu[s];
            cnt = len > size ? (len - 1) / size + 1 : 1;
        }
        const int excl = carry + block_scan(cnt, warp_sums);
        if (r < N) first[r] = excl;
        if (tid == 1023) place[0] = excl + cnt;
        __syncthreads();
        carry = place[0];
    }
    if (tid == 0) {
        first[N] = carry;
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
    if (!lin_begin(a)) return;
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
        if (role.transposed == a.bf16) {        // the sums lie as the user's state does
            E = *reinterpret_cast<const float4*>(src + e);
        } else {                                // as [dv, dk]: element (j, i) is the user's (i, j)
            const int j = e / a.dk, i = e - j * a.dk;
            E = make_float4(src[(size_t)i * a.dv + j], src[(size_t)(i + 1) * a.dv + j],
                            src[(size_t)(i + 2) * a.dv + j], src[(size_t)(i + 3) * a.dv + j]);
        }
    }
    // only a sequence's last segment may be short; it is the first one processed in reverse
    const int tail = first + count - 1;
    const float w_full = lin_pow(l, a.map.locate(first).len), w_tail = lin_pow(l, a.map.locate(tail).len);
    constexpr int AHEAD = 8;                    // sums in flight
    for (int n0 = 0; n0 < count; n0 += AHEAD) {
        float4 own[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int n = n0 + k, s = role.reverse ? tail - n : first + n;
            own[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (n + 1 < count)                  // the last segment's own sum is not computed
                own[k] = *reinterpret_cast<const float4*>(role.seg + ((size_t)s * a.H + h) * size + e);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int n = n0 + k, s = role.reverse ? tail - n : first + n;
            if (n >= count) break;
            *reinterpret_cast<float4*>(role.seg + ((size_t)s * a.H + h) * size + e) = E;
            const float w = s == tail ? w_tail : w_full;
            E.x = fmaf(w, E.x, own[k].x);
            E.y = fmaf(w, E.y, own[k].y);
            E.z = fmaf(w, E.z, own[k].z);
            E.w = fmaf(w, E.w, own[k].w);
        }
    }
}

// ------------------------------------------------------------ CUDA cores --
constexpr int kSimtChunk = 64, kSimtCols = 64;   // tokens per chunk, value columns per CTA

template <int D1>
struct LinSimtSmem {
    static constexpr int LDA = D1 + 4;           // rows 16 bytes apart in the banks: float4 reads of 8 rows do not clash
    static constexpr int LDC = kSimtCols, LDP = kSimtChunk + 4;
    struct Tile { float a[kSimtChunk][LDA], b[kSimtChunk][LDA], c[kSimtChunk][LDC]; } tile[2];
    float p[kSimtChunk][LDP], z[D1][LDC];
    float pw[kSimtChunk + 1];
};

// y += p c, a row's four columns.
__device__ __forceinline__ void axpy(float2 (&y)[2], float p, const float4& c) {
    y[0] = fma2(make_float2(p, p), make_float2(c.x, c.y), y[0]);
    y[1] = fma2(make_float2(p, p), make_float2(c.z, c.w), y[1]);
}

// One CTA per (segment, head, 64 columns of D2); 256 threads.  A thread owns 4 x 4
// of P and of y (rows ty + 16 n) and D1 / 16 x 4 of Z, which stays in registers
// with a copy in shared memory for the read.  Bound by FMA issue (two at a time,
// 32 instructions per 8 16-byte shared-memory reads); the next chunk's tiles arrive
// by cp.async meanwhile, rows past a segment's end as zeros.
template <int D1, int D2>
__device__ __forceinline__ void linear_simt_body(const LinArgs& args, int ri, int x, int states_only)
{
    using Sm = LinSimtSmem<D1>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    constexpr int SL = D2 / kSimtCols, ZR = D1 / 16;
    const int slice = x % args.slices;
    x /= args.slices;
    if (slice >= SL) return;                     // a role with fewer columns than another
    const LinRole& role = args.role[ri];
    const int H = args.H, h = x % H, sidx = x / H;
    if (sidx >= args.map.segments()) return;
    const LinMap::Seg g = args.map.locate(sidx);
    const bool rev = role.reverse;
    const bool last = g.index == (rev ? 0 : g.count - 1);        // the segment processed last
    if (states_only && last) return;
    const int j0 = slice * kSimtCols;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const float c_inter = role.c_inter, c_intra = role.c_intra, c_upd = role.c_upd;
    const double l = lin_log_decay(args.log_decay, h);
    for (int n = tid; n <= kSimtChunk; n += 256) sm.pw[n] = lin_pow(l, n);

    const size_t zsize = (size_t)D1 * D2;
    const size_t user = ((size_t)g.seq * H + h) * zsize;
    float* seg = role.seg ? role.seg + ((size_t)sidx * H + h) * zsize : nullptr;
    const float* pa = static_cast<const float*>(args.x[role.a]);
    const float* pb = static_cast<const float*>(args.x[role.b]);
    const float* pc = static_cast<const float*>(args.x[role.c]);
    float* py = static_cast<float*>(role.y);
    const int chunks = (g.len + kSimtChunk - 1) / kSimtChunk;
    const int skip = states_only ? lin_skip(l, g.len, kSimtChunk, chunks, rev) : 0, nch = chunks - skip;
    auto chunk_of = [&](int n) { return rev ? nch - 1 - n : skip + n; };
    auto fetch = [&](int n) {                    // chunk n's tiles on their way
        if (n < nch) {
            typename Sm::Tile& t = sm.tile[n & 1];
            const int off = chunk_of(n) * kSimtChunk, L = min(kSimtChunk, g.len - off), tok0 = g.begin + off;
            for (int e = tid; e < kSimtChunk * (D1 / 4); e += 256) {
                const int r = e / (D1 / 4), i = 4 * (e % (D1 / 4));
                const size_t at = ((size_t)(tok0 + min(r, L - 1)) * H + h) * D1 + i;
                cp_async16(&t.b[r][i], pb + at, r < L ? 16 : 0);
                if (!states_only) cp_async16(&t.a[r][i], pa + at, r < L ? 16 : 0);
            }
            for (int e = tid; e < kSimtChunk * (kSimtCols / 4); e += 256) {
                const int r = e / (kSimtCols / 4), j = 4 * (e % (kSimtCols / 4));
                cp_async16(&t.c[r][j], pc + ((size_t)(tok0 + min(r, L - 1)) * H + h) * D2 + j0 + j, r < L ? 16 : 0);
            }
        }
        cp_async_commit();
    };
    fetch(0);

    float2 z[ZR][2];
    const bool scanned = args.scanned && g.count > 1;
    const float* from = states_only ? nullptr : (scanned ? seg : (role.s_in ? role.s_in + user : nullptr));
    const bool tr_in = !scanned && role.transposed;
#pragma unroll
    for (int n = 0; n < ZR; ++n) {
        const int i = ty * ZR + n, j = j0 + 4 * tx;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from)
            v = tr_in ? make_float4(from[(size_t)j * D1 + i], from[(size_t)(j + 1) * D1 + i],
                                    from[(size_t)(j + 2) * D1 + i], from[(size_t)(j + 3) * D1 + i])
                      : *reinterpret_cast<const float4*>(from + (size_t)i * D2 + j);
        z[n][0] = make_float2(v.x, v.y);
        z[n][1] = make_float2(v.z, v.w);
    }
    if (!states_only && !scanned)
        lin_enter(g, sidx, rev, l, [&](int slot, float w) {
            const float* own = role.seg + ((size_t)slot * H + h) * zsize + (size_t)ty * ZR * D2 + j0 + 4 * tx;
#pragma unroll
            for (int n = 0; n < ZR; ++n) {
                const float4 u = *reinterpret_cast<const float4*>(own + (size_t)n * D2);
                z[n][0] = fma2(make_float2(w, w), z[n][0], make_float2(u.x, u.y));
                z[n][1] = fma2(make_float2(w, w), z[n][1], make_float2(u.z, u.w));
            }
        });
    for (int n = 0; n < nch; ++n) {
        const int ch = chunk_of(n);
        const int tok0 = g.begin + ch * kSimtChunk, L = min(kSimtChunk, g.len - ch * kSimtChunk);
        typename Sm::Tile& t = sm.tile[n & 1];
        cp_async_wait<0>();
        if (!states_only) {
#pragma unroll
            for (int i = 0; i < ZR; ++i)
                *reinterpret_cast<float4*>(&sm.z[ty * ZR + i][4 * tx]) = make_float4(z[i][0].x, z[i][0].y, z[i][1].x, z[i][1].y);
        }
        __syncthreads();                         // chunk n has landed; chunk n - 1 has been read by all
        fetch(n + 1);
        if (!states_only) {
            float2 acc[4][4] = {};
#pragma unroll 4
            for (int i = 0; i < D1; i += 4) {
                float4 av[4], bv[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    av[m] = *reinterpret_cast<const float4*>(&t.a[ty + 16 * m][i]);
                    bv[m] = *reinterpret_cast<const float4*>(&t.b[tx + 16 * m][i]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        acc[m][k] = fma2(make_float2(av[m].x, av[m].y), make_float2(bv[k].x, bv[k].y), acc[m][k]);
                        acc[m][k] = fma2(make_float2(av[m].z, av[m].w), make_float2(bv[k].z, bv[k].w), acc[m][k]);
                    }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int lag = rev ? (tx + 16 * k) - (ty + 16 * m) : (ty + 16 * m) - (tx + 16 * k);
                    sm.p[ty + 16 * m][tx + 16 * k] = lag >= 0 ? c_intra * sm.pw[lag] * (acc[m][k].x + acc[m][k].y) : 0.f;
                }
            __syncthreads();
            float2 out[4][2] = {};
#pragma unroll 4
            for (int i = 0; i < D1; i += 4) {
                const float4 c0 = *reinterpret_cast<const float4*>(&sm.z[i][4 * tx]);
                const float4 c1 = *reinterpret_cast<const float4*>(&sm.z[i + 1][4 * tx]);
                const float4 c2 = *reinterpret_cast<const float4*>(&sm.z[i + 2][4 * tx]);
                const float4 c3 = *reinterpret_cast<const float4*>(&sm.z[i + 3][4 * tx]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 p = *reinterpret_cast<const float4*>(&t.a[ty + 16 * m][i]);
                    axpy(out[m], p.x, c0); axpy(out[m], p.y, c1); axpy(out[m], p.z, c2); axpy(out[m], p.w, c3);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int r = ty + 16 * m;
                const float w = c_inter * sm.pw[r < L ? (rev ? L - 1 - r : r + 1) : 0];
                out[m][0] = mul2(make_float2(w, w), out[m][0]);
                out[m][1] = mul2(make_float2(w, w), out[m][1]);
            }
#pragma unroll 4
            for (int i = 0; i < kSimtChunk; i += 4) {
                const float4 c0 = *reinterpret_cast<const float4*>(&t.c[i][4 * tx]);
                const float4 c1 = *reinterpret_cast<const float4*>(&t.c[i + 1][4 * tx]);
                const float4 c2 = *reinterpret_cast<const float4*>(&t.c[i + 2][4 * tx]);
                const float4 c3 = *reinterpret_cast<const float4*>(&t.c[i + 3][4 * tx]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 p = *reinterpret_cast<const float4*>(&sm.p[ty + 16 * m][i]);
                    axpy(out[m], p.x, c0); axpy(out[m], p.y, c1); axpy(out[m], p.z, c2); axpy(out[m], p.w, c3);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int r = ty + 16 * m;
                if (r < L)
                    *reinterpret_cast<float4*>(py + ((size_t)(tok0 + r) * H + h) * D2 + j0 + 4 * tx) =
                        make_float4(out[m][0].x, out[m][0].y, out[m][1].x, out[m][1].y);
            }
        }
        const float w = sm.pw[L];
#pragma unroll
        for (int i = 0; i < ZR; ++i) {
            z[i][0] = mul2(make_float2(w, w), z[i][0]);
            z[i][1] = mul2(make_float2(w, w), z[i][1]);
        }
#pragma unroll 4
        for (int r = 0; r < kSimtChunk; ++r) {
            const float m = r < L ? c_upd * sm.pw[rev ? r + 1 : L - 1 - r] : 0.f;
            float4 c = *reinterpret_cast<const float4*>(&t.c[r][4 * tx]);
            c.x *= m; c.y *= m; c.z *= m; c.w *= m;
#pragma unroll
            for (int i = 0; i < ZR; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(&t.b[r][ty * ZR + i]);
                axpy(z[i], b.x, c); axpy(z[i + 1], b.y, c); axpy(z[i + 2], b.z, c); axpy(z[i + 3], b.w, c);
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
            to[(size_t)j * D1 + i] = z[n][0].x;
            to[(size_t)(j + 1) * D1 + i] = z[n][0].y;
            to[(size_t)(j + 2) * D1 + i] = z[n][1].x;
            to[(size_t)(j + 3) * D1 + i] = z[n][1].y;
        } else {
            *reinterpret_cast<float4*>(to + (size_t)i * D2 + j) = make_float4(z[n][0].x, z[n][0].y, z[n][1].x, z[n][1].y);
        }
    }
}

// One launch for all roles: those over (DK, DV) and those over (DV, DK).
template <int DK, int DV>
__global__ void __launch_bounds__(256, 1)
linear_simt_kernel(const __grid_constant__ LinArgs args, int states_only)
{
    if (!lin_begin(args)) return;
    const int ri = blockIdx.x % args.roles, x = blockIdx.x / args.roles;
    if (DK == DV || !args.role[ri].transposed) linear_simt_body<DK, DV>(args, ri, x, states_only);
    else linear_simt_body<DV, DK>(args, ri, x, states_only);
}

template <int DK, int DV>
cudaError_t launch_simt_t(const LinArgs& a, bool states_only) {
    auto kern = linear_simt_kernel<DK, DV>;
    const int smem = (int)std::max(sizeof(LinSimtSmem<DK>), sizeof(LinSimtSmem<DV>));
    LinArgs b = a;
    b.slices = 1;
    for (int i = 0; i < a.roles; ++i) b.slices = std::max(b.slices, a.dim[a.role[i].c] / kSimtCols);
    static std::atomic<uint64_t> done;
    int only = states_only ? 1 : 0;
    void* args[] = {&b, &only};
    return lin_launch(reinterpret_cast<const void*>(kern), (size_t)a.max_segments * a.H * a.roles * b.slices, 256, smem,
                      args, a.stream, done);
}

}  // namespace

cudaError_t launch_linear_prep(const LinArgs& a, int32_t* tab, int seg_tok, int balance_tokens) {
    linear_prep_kernel<<<1, 1024, 0, a.stream>>>(a.hdr, tab, a.map.cu, a.map.N, a.map.T, seg_tok,
                                                                 balance_tokens);
    return cudaGetLastError();
}

cudaError_t launch_linear_scan(const LinArgs& a) {
    const dim3 grid((unsigned)((size_t)a.map.N * a.H), (unsigned)((a.dk * a.dv + 1023) / 1024), (unsigned)a.roles);
    linear_scan_kernel<<<grid, 256, 0, a.stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_linear_simt(const LinArgs& a, bool states_only) {
    if (a.dk == 128 && a.dv == 128) return launch_simt_t<128, 128>(a, states_only);
    if (a.dk == 128 && a.dv == 64) return launch_simt_t<128, 64>(a, states_only);
    if (a.dk == 64 && a.dv == 128) return launch_simt_t<64, 128>(a, states_only);
    if (a.dk == 64 && a.dv == 64) return launch_simt_t<64, 64>(a, states_only);
    return cudaErrorInvalidValue;
}

}  // namespace kda
