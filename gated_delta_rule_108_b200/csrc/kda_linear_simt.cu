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

// The same for at most 32 sequences by one warp, a lane each: a forward of 5 sequences takes 29.8
// us with it and 31.8 with the kernel above, of 32 40.6 and 42.5.
__global__ void __launch_bounds__(32)
linear_prep_few_kernel(WsHeader* hdr, int32_t* tab, const int32_t* __restrict__ cu, int N, int T, int seg_tok,
                       int balance_tokens)
{
    const unsigned all = 0xffffffffu;
    const int s = threadIdx.x;
    const int lo = cu[min(s, N)], hi = cu[min(s + 1, N)], len = hi - lo;
    const bool bad = hi < lo || (s == 0 && lo != 0) || (s == N - 1 && hi != T) || (N == 0 && T != 0);
    if (__any_sync(all, bad)) {
        if (s == 0) { hdr->status = kStatusBadSeqlens; hdr->runtime_err = 0; }
        return;
    }
    const int longest = __reduce_max_sync(all, len), size = longest <= balance_tokens ? max(longest, 1) : seg_tok;
    const int cnt = s >= N ? 0 : len > size ? (len - 1) / size + 1 : 1;
    int rank = 0, before = 0;
    for (int t = 0; t < N; ++t) {
        const int lt = __shfl_sync(all, len, t), ct = __shfl_sync(all, cnt, t);
        if (lt > len || (lt == len && t < s)) {
            ++rank;
            before += ct;
        }
    }
    const int total = __reduce_add_sync(all, cnt);
    if (s < N) {
        tab[1 + rank] = before;
        tab[2 + N + rank] = s;
    }
    if (s == 0) {
        tab[0] = size;
        tab[1 + N] = total;
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
    const float2 w_full = lin_pow2(l, a.map.locate(first).len), w_tail = lin_pow2(l, a.map.locate(tail).len);
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
            const float2 w = s == tail ? w_tail : w_full;
            E.x = decay_add(w, E.x, own[k].x);
            E.y = decay_add(w, E.y, own[k].y);
            E.z = decay_add(w, E.z, own[k].z);
            E.w = decay_add(w, E.w, own[k].w);
        }
    }
}

// ------------------------------------------------------------ CUDA cores --
constexpr int kSimtChunk = 64, kSimtCols = 64;   // tokens per chunk, value columns per CTA

// Rows of 16-byte groups whose place within a row depends on the row, so that the eight
// lanes of a 16-byte access fall on different banks: in a and b two rows eight apart with
// four groups each, or four rows four apart; in c and Z four rows four apart with two
// groups each.
template <int D1>
struct LinSimtSmem {
    struct Tile { float a[kSimtChunk * D1], b[kSimtChunk * D1], c[kSimtChunk * kSimtCols]; } tile[2];
    float p[kSimtChunk * kSimtChunk], z[D1 * kSimtCols];
    float pw[kSimtChunk + 1], pw_rest[2];       // powers; second parts of those of a whole chunk and of the short one

    static __device__ __forceinline__ int at(int r, int group) {          // a, b
        return r * D1 + 4 * (group ^ (((r >> 2) & 3) | ((r >> 1) & 4)));
    }
    static __device__ __forceinline__ int at_c(int r, int group) {        // c, Z
        return r * kSimtCols + 4 * (group ^ (((r >> 2) & 3) << 1));
    }
};

__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Sums of the four lanes 4 n .. 4 n + 3 over eight rows of eight values, two rows left to
// each: rows 4 bit0 + 2 bit1 + {0, 1} of the lane's number.
__device__ __forceinline__ void sum_of_four(const float2 (&x)[8][4], int lane, float2 (&y)[2][4]) {
    float2 h[4][4];
    const bool hi = lane & 1, up = lane & 2;
    auto swap = [](float2 keep, float2 send, int mask) {
        return make_float2(keep.x + __shfl_xor_sync(0xffffffffu, send.x, mask), keep.y + __shfl_xor_sync(0xffffffffu, send.y, mask));
    };
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) h[m][k] = swap(hi ? x[m + 4][k] : x[m][k], hi ? x[m][k] : x[m + 4][k], 1);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) y[m][k] = swap(up ? h[m + 2][k] : h[m][k], up ? h[m][k] : h[m + 2][k], 2);
}

// y[m] += p[m] * (eight columns in c0, c1), eight rows.
__device__ __forceinline__ void outer(float2 (&y)[8][4], const float (&p)[8], const float4& c0, const float4& c1) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const float2 q = make_float2(p[m], p[m]);
        y[m][0] = fma2(q, make_float2(c0.x, c0.y), y[m][0]);
        y[m][1] = fma2(q, make_float2(c0.z, c0.w), y[m][1]);
        y[m][2] = fma2(q, make_float2(c1.x, c1.y), y[m][2]);
        y[m][3] = fma2(q, make_float2(c1.z, c1.w), y[m][3]);
    }
}
// Four steps of that, the rows' factors contiguous in memory.
__device__ __forceinline__ void outer4(float2 (&y)[8][4], const float4 (&a)[8], const float* c, const int (&c_at)[4][2]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float p[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) p[m] = e == 0 ? a[m].x : e == 1 ? a[m].y : e == 2 ? a[m].z : a[m].w;
        outer(y, p, lds4(c + c_at[e][0]), lds4(c + c_at[e][1]));
    }
}

// One CTA per (segment, head, 64 columns of D2); 256 threads, a warp for every eighth
// row.  Every product of a chunk gives tiles of 64 x 64, a thread 8 x 8 of them from a
// quarter of the terms: the four lanes of one place share them out by groups of four and
// join their sums by shuffles.  Two things hold it: FMA issue, and the way from shared
// memory into registers, 128 bytes a cycle whatever the lanes share, of which 8 x 8 takes
// 16 16-byte reads for 128 paired FMAs.  B=4, T=4096, H=16, dk = dv = 128: 968 us, FMA
// pipes 56 %, reads 47 %, and the two warps of a scheduler do not fill the gaps; 8 x 4 by
// 512 threads takes 1,084 us (reads 62 %), 4 x 4 without the quarters 978 (dk = dv = 64:
// 8 x 8 574, 4 x 4 664).  The next chunk's tiles arrive by cp.async meanwhile, rows past a
// segment's end as zeros.
template <int D1, int D2>
__device__ __forceinline__ void linear_simt_body(const LinArgs& args, int ri, int x, int states_only)
{
    using Sm = LinSimtSmem<D1>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    constexpr int SL = D2 / kSimtCols, HALVES = D1 / 64;
    const int slice = x % args.slices;
    x /= args.slices;
    if (slice >= SL) return;                     // a role with fewer columns than another
    const LinRole& role = args.role[ri];
    const int H = args.H, h = x % H, slot = x / H, sidx = states_only ? slot / args.map.pieces : slot;
    if (sidx >= args.map.segments()) return;
    const LinMap::Seg g = states_only ? args.map.locate_piece(slot) : args.map.locate(sidx);
    const bool rev = role.reverse;
    const bool last = g.index == (rev ? 0 : g.count - 1);        // the segment processed last
    if (states_only && (last || g.len <= 0)) return;
    const int j0 = slice * kSimtCols;
    const int tid = threadIdx.x, lane = tid & 31, ty = tid >> 5, tx = lane >> 2, part = lane & 3;
    const float c_inter = role.c_inter, c_intra = role.c_intra, c_upd = role.c_upd;
    const double l = lin_log_decay(args.log_decay, h);
    for (int n = tid; n <= kSimtChunk; n += 256) sm.pw[n] = lin_pow(l, n);
    if (tid >= 128 && tid < 130) sm.pw_rest[tid - 128] = lin_pow2(l, tid == 128 ? kSimtChunk : g.len % kSimtChunk).y;

    const size_t zsize = (size_t)D1 * D2;
    const size_t user = ((size_t)g.seq * H + h) * zsize;
    float* seg = role.seg ? role.seg + ((size_t)slot * H + h) * zsize : nullptr;
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
                const int r = e / (D1 / 4), i = e % (D1 / 4);
                const size_t at = ((size_t)(tok0 + min(r, L - 1)) * H + h) * D1 + 4 * i;
                cp_async16(t.b + Sm::at(r, i), pb + at, r < L ? 16 : 0);
                if (!states_only) cp_async16(t.a + Sm::at(r, i), pa + at, r < L ? 16 : 0);
            }
            for (int e = tid; e < kSimtChunk * (kSimtCols / 4); e += 256) {
                const int r = e / (kSimtCols / 4), j = e % (kSimtCols / 4);
                cp_async16(t.c + Sm::at_c(r, j), pc + ((size_t)(tok0 + min(r, L - 1)) * H + h) * D2 + j0 + 4 * j, r < L ? 16 : 0);
            }
        }
        cp_async_commit();
    };
    fetch(0);

    // this thread's part of Z: rows row_z(half, 0 and 1), columns 4 tx.. and 32 + 4 tx..
    auto row_z = [&](int half, int m) { return 64 * half + 32 * (part & 1) + 4 * ty + (part & 2) + m; };
    float2 z[HALVES][2][4];
    const bool scanned = args.scanned && g.count > 1;
    const float* from = states_only ? nullptr : (scanned ? seg : (role.s_in ? role.s_in + user : nullptr));
    const bool tr_in = !scanned && role.transposed;
#pragma unroll
    for (int n = 0; n < HALVES; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = row_z(n, m), j = j0 + 32 * q + 4 * tx;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (from)
                    v = tr_in ? make_float4(from[(size_t)j * D1 + i], from[(size_t)(j + 1) * D1 + i],
                                            from[(size_t)(j + 2) * D1 + i], from[(size_t)(j + 3) * D1 + i])
                              : *reinterpret_cast<const float4*>(from + (size_t)i * D2 + j);
                z[n][m][2 * q] = make_float2(v.x, v.y);
                z[n][m][2 * q + 1] = make_float2(v.z, v.w);
            }
    if (!states_only && !scanned)
        lin_enter(args.map, g, sidx, rev, l, [&](int slot, float2 w) {
            const float* own = role.seg + ((size_t)slot * H + h) * zsize;
#pragma unroll
            for (int n = 0; n < HALVES; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float4 u = *reinterpret_cast<const float4*>(own + (size_t)row_z(n, m) * D2 + j0 + 32 * q + 4 * tx);
                        z[n][m][2 * q] = decay_add(w, z[n][m][2 * q], make_float2(u.x, u.y));
                        z[n][m][2 * q + 1] = decay_add(w, z[n][m][2 * q + 1], make_float2(u.z, u.w));
                    }
        });
    for (int n = 0; n < nch; ++n) {
        const int ch = chunk_of(n);
        const int tok0 = g.begin + ch * kSimtChunk, L = min(kSimtChunk, g.len - ch * kSimtChunk);
        typename Sm::Tile& t = sm.tile[n & 1];
        cp_async_wait<0>();
        if (!states_only) {
#pragma unroll
            for (int k = 0; k < HALVES; ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        *reinterpret_cast<float4*>(sm.z + Sm::at_c(row_z(k, m), 8 * q + tx)) =
                            make_float4(z[k][m][2 * q].x, z[k][m][2 * q].y, z[k][m][2 * q + 1].x, z[k][m][2 * q + 1].y);
        }
        __syncthreads();                         // chunk n has landed; chunk n - 1 has been read by all
        fetch(n + 1);
        if (!states_only) {
            // P: rows ty + 8 m, columns 8 tx + k, channels in groups of four, every fourth group
            {
                float2 acc[8][8] = {};
#pragma unroll 1
                for (int i = part; i < D1 / 4; i += 4) {
                    float4 av[8];
#pragma unroll
                    for (int m = 0; m < 8; ++m) av[m] = lds4(t.a + Sm::at(ty + 8 * m, i));
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 bv = lds4(t.b + Sm::at(8 * tx + k, i));
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            acc[m][k] = fma2(make_float2(av[m].x, av[m].y), make_float2(bv.x, bv.y), acc[m][k]);
                            acc[m][k] = fma2(make_float2(av[m].z, av[m].w), make_float2(bv.z, bv.w), acc[m][k]);
                        }
                    }
                }
                float2 sum[8][4], own[2][4];
#pragma unroll
                for (int m = 0; m < 8; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sum[m][k] = make_float2(acc[m][2 * k].x + acc[m][2 * k].y, acc[m][2 * k + 1].x + acc[m][2 * k + 1].y);
                sum_of_four(sum, lane, own);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int r = ty + 8 * (4 * (part & 1) + (part & 2) + m);
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int lag = rev ? 8 * tx + k - r : r - 8 * tx - k;
                        v[k] = lag >= 0 ? c_intra * sm.pw[lag] * (k & 1 ? own[m][k >> 1].y : own[m][k >> 1].x) : 0.f;
                    }
                    float* dst = sm.p + r * kSimtChunk + 8 * tx;
                    *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            __syncwarp();                        // a warp reads the rows of P that it has written
            float2 out[8][4] = {};
#pragma unroll 1
            for (int i = part; i < D1 / 4; i += 4) {
                float4 av[8];
                int at[4][2];
#pragma unroll
                for (int m = 0; m < 8; ++m) av[m] = lds4(t.a + Sm::at(ty + 8 * m, i));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    at[e][0] = Sm::at_c(4 * i + e, tx);
                    at[e][1] = Sm::at_c(4 * i + e, 8 + tx);
                }
                outer4(out, av, sm.z, at);
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const int r = ty + 8 * m;
                const float w = c_inter * sm.pw[r < L ? (rev ? L - 1 - r : r + 1) : 0];
#pragma unroll
                for (int k = 0; k < 4; ++k) out[m][k] = mul2(make_float2(w, w), out[m][k]);
            }
#pragma unroll 1
            for (int i = part; i < kSimtChunk / 4; i += 4) {
                float4 pv[8];
                int at[4][2];
#pragma unroll
                for (int m = 0; m < 8; ++m) pv[m] = lds4(sm.p + (ty + 8 * m) * kSimtChunk + 4 * i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    at[e][0] = Sm::at_c(4 * i + e, tx);
                    at[e][1] = Sm::at_c(4 * i + e, 8 + tx);
                }
                outer4(out, pv, t.c, at);
            }
            float2 own[2][4];
            sum_of_four(out, lane, own);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int r = ty + 8 * (4 * (part & 1) + (part & 2) + m);
                if (r >= L) continue;
                float* dst = py + ((size_t)(tok0 + r) * H + h) * D2 + j0 + 4 * tx;
                *reinterpret_cast<float4*>(dst) = make_float4(own[m][0].x, own[m][0].y, own[m][1].x, own[m][1].y);
                *reinterpret_cast<float4*>(dst + 32) = make_float4(own[m][2].x, own[m][2].y, own[m][3].x, own[m][3].y);
            }
            __syncthreads();                     // Z has been read by all: the next chunk's goes in its place
        }
        // the chunk's sum: rows 4 ty.. and 32 + 4 ty.. of each half, tokens in groups of four
        const float2 w = make_float2(sm.pw[L], sm.pw_rest[L < kSimtChunk]);
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
            float2 u[8][4] = {}, own[2][4];
#pragma unroll 1
            for (int q = part; q < kSimtChunk / 4; q += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * q + e;
                    const float m = r < L ? c_upd * sm.pw[rev ? r + 1 : L - 1 - r] : 0.f;
                    const float4 b0 = lds4(t.b + Sm::at(r, 16 * half + ty)), b1 = lds4(t.b + Sm::at(r, 16 * half + 8 + ty));
                    const float b[8] = {m * b0.x, m * b0.y, m * b0.z, m * b0.w, m * b1.x, m * b1.y, m * b1.z, m * b1.w};
                    outer(u, b, lds4(t.c + Sm::at_c(r, tx)), lds4(t.c + Sm::at_c(r, 8 + tx)));
                }
            }
            sum_of_four(u, lane, own);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) z[half][m][k] = decay_add(w, z[half][m][k], own[m][k]);
        }
    }
    float* to = states_only ? seg : (last && role.s_out ? role.s_out + user : nullptr);
    if (!to) return;
    const bool tr_out = !states_only && role.transposed;
#pragma unroll
    for (int n = 0; n < HALVES; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = row_z(n, m), j = j0 + 32 * q + 4 * tx;
                const float2 lo = z[n][m][2 * q], hi = z[n][m][2 * q + 1];
                if (tr_out) {
                    to[(size_t)j * D1 + i] = lo.x;
                    to[(size_t)(j + 1) * D1 + i] = lo.y;
                    to[(size_t)(j + 2) * D1 + i] = hi.x;
                    to[(size_t)(j + 3) * D1 + i] = hi.y;
                } else {
                    *reinterpret_cast<float4*>(to + (size_t)i * D2 + j) = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
}

// One launch for all roles: those over (DK, DV) and those over (DV, DK), one after the
// other, those with more rows of Z and so more work a block first (gradients of B=4,
// T=1021, H=16, dk 64, dv 128: 401 us, 509 with the roles in turn).
template <int DK, int DV>
__global__ void __launch_bounds__(256, 1)
linear_simt_kernel(const __grid_constant__ LinArgs args, int states_only)
{
    if (!lin_begin(args)) return;
    const int blocks = gridDim.x / args.roles, nth = blockIdx.x / blocks, x = blockIdx.x % blocks;
    const int ri = DK > DV ? args.roles - 1 - nth : nth;
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
    return lin_launch(reinterpret_cast<const void*>(kern), (size_t)a.max_segments * (states_only ? a.map.pieces : 1) * a.H * a.roles * b.slices, 256, smem,
                      args, a.follows, a.stream, done);
}

}  // namespace

cudaError_t launch_linear_prep(const LinArgs& a, int32_t* tab, int seg_tok, int balance_tokens) {
    if (a.map.N <= 32)
        linear_prep_few_kernel<<<1, 32, 0, a.stream>>>(a.hdr, tab, a.map.cu, a.map.N, a.map.T, seg_tok, balance_tokens);
    else
        linear_prep_kernel<<<1, 1024, 0, a.stream>>>(a.hdr, tab, a.map.cu, a.map.N, a.map.T, seg_tok, balance_tokens);
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
