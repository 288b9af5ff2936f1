// kda_linear_tc.cu -- linear attention with one fixed decay per head on the sm_100a
// tensor cores (bf16 inputs): the chunk kernel and the pass that sums a segment's
// contribution to the state.  kda_linear.cuh says how the forward and its three
// gradients map onto the roles a, b, c -> y used here.
//
// Per chunk of 128 tokens with entering state Z (D1 x D2), local index r, length L:
//
//   P_ri = lambda^{|r - i|} <a_r, b_i>          i <= r  (i >= r last to first)
//   y_r  = c_intra sum_i P_ri c_i + c_inter lambda^{n_r} Z^T a_r
//   Z'   = lambda^L Z + sum_i b_i (c_upd lambda^{m_i} c_i)^T
//
// n_r = r + 1, m_i = L - 1 - i first to last; n_r = L - 1 - r, m_i = i + 1 last to
// first.  Four products of 128-row tiles, all kind::f16 with bf16 operands and fp32
// accumulators in TMEM; a, b and c are exact in bf16, so only P, Z and the
// weighted c are rounded:
//  - P in two bf16 parts (2^-17), the A operand in TMEM, in place of its fp32 values;
//  - Z in one part as operand: it only reaches y, itself bf16, and adds at most its
//    own rounding to y's; the state itself stays fp32 in TMEM;
//  - the weighted c in three parts (2^-25) where the state is a result, in two where
//    it only reaches y: a state is a sum over the whole sequence, and fp32 is what
//    it is returned in.
//
// One CTA per (segment, head, role), one per SM (TMEM: Z, P and two accumulators of
// y, 512 columns).  Warp 9 loads tiles by TMA, warp 8 issues the MMAs, warps 0-3
// weight P and write y, warps 4-7 weight c, convert and decay Z.  The chain from
// chunk to chunk (Z -> operand -> Z^T a, update) and the rest overlap: b and c tiles
// go through a ring of three buffers, so the next chunk's b is in flight while this
// one is worked on, and a's buffer frees as soon as P and Z^T a are done.
//
// Every wait is bounded; one that gives up sets a flag that ends the CTA's other
// waits, records KDA_ERR_TIMEOUT, and the CTA waits for its own copies and MMAs,
// frees its TMEM and returns.
#include "kda_linear.cuh"
#include "kda_tc_common.cuh"

namespace kda {
namespace {

constexpr int C = kLinChunk;
constexpr uint32_t kTile = 128 * 128;          // 128 tokens x 64 bf16 channels, 128-byte swizzle

struct LinTcParams {
    CUtensorMap map[4];                        // q, k, v, d_o
    LinArgs a;
};

// Bounded wait that also gives up when another thread of the CTA has.
__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t parity, int* s_abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*(volatile int*)s_abort) return false;
        if (clock64() - t0 > kWaitCycles) {
            *(volatile int*)s_abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool lin_wait_warp(uint64_t* bar, uint32_t parity, int* s_abort) {
    return __all_sync(0xffffffffu, lin_wait(bar, parity, s_abort));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

template <int D>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, uint64_t* bar, int h, int tok) {
    mbar_arrive_expect_tx(bar, (D / 64) * kTile);
#pragma unroll
    for (int t = 0; t < D / 64; ++t) tma_load_3d(dst + t * kTile, map, bar, 64 * t, h, tok);
}

// Zeroes rows L..127 of a tile (another sequence's tokens): they are contracted
// over with weights of zero, which must not meet an infinity or a NaN.
__device__ __forceinline__ void clear_rows(unsigned char* tile, int D, int L, int lo, int hi, int t, int nthreads) {
    const int first = max(L, lo), n = max(hi - first, 0);
    for (int e = t; e < n * (D / 8); e += nthreads) {
        const int r = first + e / (D / 8), c = e % (D / 8);
        *reinterpret_cast<uint4*>(tile + (c >> 3) * kTile + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// Tokens [64 half, 64 half + 64) of c, weighted, in `parts` bf16 parts of
// D2 / 64 tiles of 64 rows each; 128 threads.  A row past L becomes zero.
template <int D2>
__device__ __forceinline__ void weight_c(const unsigned char* ct, unsigned char* out, int half, int parts, int L,
                                         const float* pw, float c_upd, bool rev, int t) {
    constexpr uint32_t PART = (D2 / 64) * 8192;
    const int chunk = t & 7;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int r = pass * 16 + (t >> 3), i = 64 * half + r;
        const bool on = i < L;
        const float w = on ? c_upd * pw[rev ? i + 1 : L - 1 - i] : 0.f;
#pragma unroll
        for (int tile = 0; tile < D2 / 64; ++tile) {
            const uint4 raw = *reinterpret_cast<const uint4*>(ct + tile * kTile + sw128_offset(i, chunk * 16));
            const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t p[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = on ? w * bf16_lo(u[e]) : 0.f, y = on ? w * bf16_hi(u[e]) : 0.f;
                p[0][e] = pack_bf16(x, y);
                x -= bf16_lo(p[0][e]);
                y -= bf16_hi(p[0][e]);
                p[1][e] = pack_bf16(x, y);
                x -= bf16_lo(p[1][e]);
                y -= bf16_hi(p[1][e]);
                p[2][e] = pack_bf16(x, y);
            }
            unsigned char* dst = out + tile * 8192 + sw128_offset(r, chunk * 16);
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (q < parts) *reinterpret_cast<uint4*>(dst + q * PART) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
        }
    }
}

// Z += b^T (weighted c) over 64 tokens.
template <int D2>
__device__ __forceinline__ void issue_update(uint32_t zacc, uint32_t bt, uint32_t cw, int half, int parts, bool first) {
    constexpr uint32_t idesc = instr_desc(kFmtBF16, 128, D2, true, true);
    constexpr uint32_t PART = (D2 / 64) * 8192;
    for (int q = 0; q < parts; ++q)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            mma_f16(zacc, smem_desc(bt + half * 8192 + ks * 2048, kTile, 1024, kLayoutSW128),
                    smem_desc(cw + q * PART + ks * 2048, 8192, 1024, kLayoutSW128), idesc, !(first && q == 0 && ks == 0));
}

// A thread's row of Z between global memory (the user's layout or its transpose)
// and 32 registers.
template <int D1, int D2>
__device__ __forceinline__ void read_state(const float* s, bool transposed, int i, int j0, float (&v)[32]) {
    if (!s) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
    } else if (transposed) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = s[(size_t)(j0 + j) * D1 + i];
    } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(s + (size_t)i * D2 + j0 + j);
            v[j] = x.x; v[j + 1] = x.y; v[j + 2] = x.z; v[j + 3] = x.w;
        }
    }
}
template <int D1, int D2>
__device__ __forceinline__ void write_state(float* s, bool transposed, int i, int j0, const float (&v)[32]) {
    if (transposed) {
#pragma unroll
        for (int j = 0; j < 32; ++j) s[(size_t)(j0 + j) * D1 + i] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(s + (size_t)i * D2 + j0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
}

// ------------------------------------------------------------- chunk kernel --
template <int D1, int D2>
struct LinSmem {
    static constexpr uint32_t AT = (D1 / 64) * kTile, CT = (D2 / 64) * kTile;
    static constexpr uint32_t SLOT = AT > CT ? AT : CT;
    static constexpr uint32_t A = 0;
    static constexpr uint32_t BC = A + AT;                       // ring of three b / c tiles
    static constexpr uint32_t Z = BC + 3 * SLOT;                 // bf16 Z: D2 / 64 tiles of D1 rows
    static constexpr uint32_t CW = Z + (D2 / 64) * D1 * 128;     // weighted c of 64 tokens, three parts
    static constexpr uint32_t END = CW + 3 * (D2 / 64) * 8192;
    static_assert(END + 1024 + 1200 <= 232448, "shared memory");
};

template <int D1, int D2>
__global__ void __launch_bounds__(320, 1)
linear_tc_kernel(const __grid_constant__ LinTcParams prm)
{
    using Sm = LinSmem<D1, D2>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t full_a, empty_a, full_bc[3], p_done, p_ready, y_done, y_free, cw_ready[2],
        upd_done[2], z_ready, drained;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ float pw[C + 1];
    __shared__ __align__(16) float colw[32];

    const LinArgs& args = prm.a;
    if (args.hdr->status != kStatusOk) return;
    int x = blockIdx.x;
    const LinRole& role = args.role[x % args.roles];
    x /= args.roles;
    const int H = args.H, h = x % H, sidx = x / H;
    if (sidx >= args.map.segments()) return;
    const LinMap::Seg g = args.map.locate(sidx);
    const bool rev = role.reverse;
    const int nch = (g.len + C - 1) / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t zsize = (size_t)D1 * D2, user = ((size_t)g.seq * H + h) * zsize;
    const int parts = role.s_out ? 3 : 2;

    if (tid == 0) {
        s_abort = 0;
        mbar_init(&full_a, 1);
        mbar_init(&empty_a, 1);
        for (int i = 0; i < 3; ++i) mbar_init(&full_bc[i], 1);
        mbar_init(&p_done, 1);
        mbar_init(&p_ready, 128);
        mbar_init(&y_done, 1);
        mbar_init(&y_free, 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&cw_ready[i], 128);
            mbar_init(&upd_done[i], 1);
        }
        mbar_init(&z_ready, 128);
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    {
        const double l = lin_log_decay(args.log_decay, h);
        if (tid <= C) pw[tid] = lin_pow(l, tid);
        if (tid < 32) colw[tid] = lin_pow(l, rev ? tid : 31 - tid);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t ZACC = tmem, PACC = tmem + 128, YZ = tmem + 256, YP = tmem + 384;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const int row = (warp & 3) * 32 + lane;
    auto chunk_of = [&](int n) { return rev ? nch - 1 - n : n; };

    if (warp == 9) {                                    // ---- TMA loads
        if (lane == 0) {
            int issued[3] = {0, 0, 0}, issued_a = 0;
            bool ok = true;
            for (int n = 0; ok && n < nch; ++n) {
                const int tok = g.begin + chunk_of(n) * C;
                int j = 2 * n;                          // b: the buffer of chunk n - 2's c, waited for with chunk n - 1's c
                load_tile<D1>(sm + Sm::BC + (j % 3) * Sm::SLOT, &prm.map[role.b], &full_bc[j % 3], h, tok);
                ++issued[j % 3];
                if (n > 0) ok = lin_wait(&empty_a, (n - 1) & 1, &s_abort);
                if (!ok) break;
                load_tile<D1>(sm + Sm::A, &prm.map[role.a], &full_a, h, tok);
                ++issued_a;
                if (n > 0) ok = lin_wait(&upd_done[1], (n - 1) & 1, &s_abort);
                if (!ok) break;
                j = 2 * n + 1;                          // c: the buffer of chunk n - 1's b
                load_tile<D2>(sm + Sm::BC + (j % 3) * Sm::SLOT, &prm.map[role.c], &full_bc[j % 3], h, tok);
                ++issued[j % 3];
            }
            // every copy issued has landed before the CTA's memory goes away
            if (issued_a) (void)mbar_wait_cycles(&full_a, (issued_a - 1) & 1, kWaitCycles);
            for (int i = 0; i < 3; ++i)
                if (issued[i]) (void)mbar_wait_cycles(&full_bc[i], (issued[i] - 1) & 1, kWaitCycles);
        }
    } else if (warp == 8) {                             // ---- MMA issue
        if (lane == 0) {
            const uint32_t at = smem_u32(sm + Sm::A), zt = smem_u32(sm + Sm::Z), cw = smem_u32(sm + Sm::CW);
            for (int n = 0; n < nch; ++n) {
                const uint32_t ph = n & 1, prev = (n - 1) & 1;
                const int jb = 2 * n, jc = 2 * n + 1;
                const uint32_t bt = smem_u32(sm + Sm::BC + (jb % 3) * Sm::SLOT);
                const uint32_t ct = smem_u32(sm + Sm::BC + (jc % 3) * Sm::SLOT);
                // P = a b^T, over the previous chunk's weighted P once y has been formed from it
                if (!lin_wait(&full_a, ph, &s_abort) || !lin_wait(&full_bc[jb % 3], (jb / 3) & 1, &s_abort)) break;
                if (n > 0 && !lin_wait(&y_done, prev, &s_abort)) break;
                tc_fence_after();
                constexpr uint32_t id_p = instr_desc(kFmtBF16, 128, 128);
#pragma unroll
                for (int k = 0; k < D1 / 16; ++k) {
                    const uint32_t off = (k >> 2) * kTile + (k & 3) * 32;
                    mma_f16(PACC, smem_desc(at + off, 16, 1024, kLayoutSW128), smem_desc(bt + off, 16, 1024, kLayoutSW128),
                            id_p, k != 0);
                }
                mma_commit(&p_done);
                // a Z
                if (!lin_wait(&z_ready, ph, &s_abort)) break;
                if (n > 0 && !lin_wait(&y_free, prev, &s_abort)) break;
                tc_fence_after();
                constexpr uint32_t id_y = instr_desc(kFmtBF16, 128, D2, false, true);
#pragma unroll
                for (int k = 0; k < D1 / 16; ++k)
                    mma_f16(YZ, smem_desc(at + (k >> 2) * kTile + (k & 3) * 32, 16, 1024, kLayoutSW128),
                            smem_desc(zt + k * 2048, D1 * 128, 1024, kLayoutSW128), id_y, k != 0);
                mma_commit(&empty_a);
                // first half of the update
                if (!lin_wait(&cw_ready[0], ph, &s_abort)) break;
                tc_fence_after();
                issue_update<D2>(ZACC, bt, cw, 0, parts, false);
                mma_commit(&upd_done[0]);
                // P c, both parts of P (16 columns of 32 each)
                if (!lin_wait(&p_ready, ph, &s_abort)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        mma_f16_ts(YP, PACC + (k >> 1) * 32 + q * 16 + (k & 1) * 8,
                                   smem_desc(ct + k * 2048, kTile, 1024, kLayoutSW128), id_y, (k | q) != 0);
                mma_commit(&y_done);
                // second half of the update
                if (!lin_wait(&cw_ready[1], ph, &s_abort)) break;
                tc_fence_after();
                issue_update<D2>(ZACC, bt, cw, 1, parts, false);
                mma_commit(&upd_done[1]);
            }
            mma_commit(&drained);
            (void)mbar_wait_cycles(&drained, 0, kWaitCycles);
        }
    } else if (warp < 4) {                              // ---- P and y
        for (int n = 0; n < nch; ++n) {
            const uint32_t ph = n & 1;
            const int ch = chunk_of(n), L = min(C, g.len - ch * C);
            if (!lin_wait_warp(&p_done, ph, &s_abort)) break;
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                const uint32_t at = PACC + lane_base + 32 * b;
                float v[32];
                uint32_t pk[32];
                const bool some = rev ? b >= warp : b <= warp;      // this warp's rows see this block of columns
                if (some) {
                    tmem_ld32_sync(at, v);
                    if (b == warp) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int lag = rev ? j - lane : lane - j;
                            v[j] = (lag >= 0 && 32 * b + j < L) ? pw[max(lag, 0)] * v[j] : 0.f;
                        }
                    } else {
                        // |r - i| = (distance to the block's near edge) + (distance within it): both factors <= 1
                        const float f = pw[rev ? 32 * b - row : row - (32 * b + 31)];
                        const int left = L - 32 * b;
#pragma unroll
                        for (int j4 = 0; j4 < 8; ++j4) {
                            const float4 w = *reinterpret_cast<const float4*>(&colw[4 * j4]);
                            v[4 * j4] = 4 * j4 < left ? f * w.x * v[4 * j4] : 0.f;
                            v[4 * j4 + 1] = 4 * j4 + 1 < left ? f * w.y * v[4 * j4 + 1] : 0.f;
                            v[4 * j4 + 2] = 4 * j4 + 2 < left ? f * w.z * v[4 * j4 + 2] : 0.f;
                            v[4 * j4 + 3] = 4 * j4 + 3 < left ? f * w.w * v[4 * j4 + 3] : 0.f;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        pk[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                        pk[16 + j] = pack_bf16(v[2 * j] - bf16_lo(pk[j]), v[2 * j + 1] - bf16_hi(pk[j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = 0;
                }
                float out[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) out[j] = __uint_as_float(pk[j]);
                tmem_st32_sync(at, out);
            }
            tc_fence_before();
            mbar_arrive(&p_ready);
            if (!lin_wait_warp(&y_done, ph, &s_abort)) break;
            tc_fence_after();
            const float wz = role.c_inter * pw[row < L ? (rev ? L - 1 - row : row + 1) : 0], wp = role.c_intra;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(role.y) +
                                 ((size_t)(g.begin + ch * C + row) * H + h) * D2;
#pragma unroll 1
            for (int j0 = 0; j0 < D2; j0 += 32) {
                float vz[32], vp[32];
                tmem_ld32_sync(YZ + lane_base + j0, vz);
                tmem_ld32_sync(YP + lane_base + j0, vp);
                if (row < L) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = pack_bf16(fmaf(wz, vz[j + 2 * e], wp * vp[j + 2 * e]),
                                             fmaf(wz, vz[j + 2 * e + 1], wp * vp[j + 2 * e + 1]));
                        *reinterpret_cast<uint4*>(dst + j0 + j) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&y_free);
        }
    } else {                                            // ---- weighted c and Z
        const int t = tid - 128;
        bool ok = true;
        if (row < D1 || D1 == 128) {
            const float* from = g.count > 1 ? role.seg + ((size_t)sidx * H + h) * zsize
                                            : (role.s_in ? role.s_in + user : nullptr);
#pragma unroll 1
            for (int j0 = 0; j0 < D2; j0 += 32) {
                float v[32];
                read_state<D1, D2>(from, g.count == 1 && role.transposed, row, j0, v);
                tmem_st32_sync(ZACC + lane_base + j0, v);
            }
        }
        for (int n = 0; n < nch; ++n) {
            const uint32_t ph = n & 1;
            const int L = min(C, g.len - chunk_of(n) * C), jb = 2 * n, jc = 2 * n + 1;
            unsigned char* bt = sm + Sm::BC + (jb % 3) * Sm::SLOT;
            unsigned char* ct = sm + Sm::BC + (jc % 3) * Sm::SLOT;
            if (n > 0) {
                ok = lin_wait_warp(&upd_done[1], (n - 1) & 1, &s_abort);
                if (!ok) break;
                tc_fence_after();
            }
            if (row < D1 || D1 == 128) {                // Z -> bf16 operand, decayed in place
                const float gam = pw[L];
#pragma unroll 1
                for (int j0 = 0; j0 < D2; j0 += 32) {
                    float v[32];
                    tmem_ld32_sync(ZACC + lane_base + j0, v);
                    unsigned char* zt = sm + Sm::Z + (j0 >> 6) * (D1 * 128);
#pragma unroll
                    for (int j8 = 0; j8 < 4; ++j8)
                        *reinterpret_cast<uint4*>(zt + sw128_offset(row, ((j0 & 63) + 8 * j8) * 2)) =
                            make_uint4(pack_bf16(v[8 * j8], v[8 * j8 + 1]), pack_bf16(v[8 * j8 + 2], v[8 * j8 + 3]),
                                       pack_bf16(v[8 * j8 + 4], v[8 * j8 + 5]), pack_bf16(v[8 * j8 + 6], v[8 * j8 + 7]));
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= gam;
                    tmem_st32_sync(ZACC + lane_base + j0, v);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&z_ready);
            ok = lin_wait_warp(&full_bc[jb % 3], (jb / 3) & 1, &s_abort) &&
                 lin_wait_warp(&full_bc[jc % 3], (jc / 3) & 1, &s_abort);
            if (!ok) break;
            if (L < C) {        // P's MMA may still read b: its columns past L are dropped when P is weighted
                clear_rows(bt, D1, L, 0, C, t, 128);
                clear_rows(ct, D2, L, 0, C, t, 128);
            }
            weight_c<D2>(ct, sm + Sm::CW, 0, parts, L, pw, role.c_upd, rev, t);
            fence_proxy_async_smem();
            mbar_arrive(&cw_ready[0]);
            ok = lin_wait_warp(&upd_done[0], ph, &s_abort);
            if (!ok) break;
            weight_c<D2>(ct, sm + Sm::CW, 1, parts, L, pw, role.c_upd, rev, t);
            fence_proxy_async_smem();
            mbar_arrive(&cw_ready[1]);
        }
        if (ok && nch > 0) ok = lin_wait_warp(&upd_done[1], (nch - 1) & 1, &s_abort);
        if (ok && role.s_out && g.index == (rev ? 0 : g.count - 1) && (row < D1 || D1 == 128)) {
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 0; j0 < D2; j0 += 32) {
                float v[32];
                tmem_ld32_sync(ZACC + lane_base + j0, v);
                write_state<D1, D2>(role.s_out + user, role.transposed, row, j0, v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && s_abort) flag_error(args.hdr, kStatusTimeout);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------- segment's sum --
// Z of one segment from zero: sum_i lambda^{tokens from i to the segment's end}
// b_i c_i^T.  The weights count to the segment's end, so nothing is rescaled and
// the MMAs only accumulate; warps 0-3 weight the first 64 tokens of each chunk,
// warps 4-7 the other 64, each into a buffer of its own.
template <int D1, int D2>
struct LinSumSmem {
    static constexpr uint32_t BT = (D1 / 64) * kTile, CT = (D2 / 64) * kTile;
    static constexpr uint32_t STAGE = BT + CT;
    static constexpr uint32_t CWH = 3 * (D2 / 64) * 8192;
    static constexpr uint32_t CW = 2 * STAGE;
    static constexpr uint32_t END = CW + 2 * CWH;
    static_assert(END + 1024 + 1200 <= 232448, "shared memory");
};

template <int D1, int D2>
__global__ void __launch_bounds__(320, 1)
linear_sum_tc_kernel(const __grid_constant__ LinTcParams prm)
{
    using Sm = LinSumSmem<D1, D2>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t full[2], empty[2], cw_ready[2], upd_done[2], drained;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ float pw[C + 1];

    const LinArgs& args = prm.a;
    if (args.hdr->status != kStatusOk) return;
    int x = blockIdx.x;
    const LinRole& role = args.role[x % args.roles];
    x /= args.roles;
    const int H = args.H, h = x % H, sidx = x / H;
    if (sidx >= args.map.segments()) return;
    const LinMap::Seg g = args.map.locate(sidx);
    const bool rev = role.reverse;
    if (g.index == (rev ? 0 : g.count - 1)) return;     // processed last: its sum enters no other segment
    const int nch = (g.len + C - 1) / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = role.s_out ? 3 : 2;
    const double l = lin_log_decay(args.log_decay, h);

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], 1);
            mbar_init(&cw_ready[i], 128);
            mbar_init(&upd_done[i], 1);
        }
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, 128);
        tmem_relinquish();
    }
    if (tid <= C) pw[tid] = lin_pow(l, tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto chunk_of = [&](int n) { return rev ? nch - 1 - n : n; };

    if (warp == 9) {
        if (lane == 0) {
            int n = 0;
            for (; n < nch; ++n) {
                const int tok = g.begin + chunk_of(n) * C, st = n & 1;
                if (n > 1 && !lin_wait(&empty[st], ((n >> 1) - 1) & 1, &s_abort)) break;
                load_tile<D1>(sm + st * Sm::STAGE, &prm.map[role.b], &full[st], h, tok);
                load_tile<D2>(sm + st * Sm::STAGE + Sm::BT, &prm.map[role.c], &full[st], h, tok);
            }
            for (int i = 0; i < 2; ++i) {
                const int count = (n - i + 1) >> 1;     // loads into stage i
                if (count > 0) (void)mbar_wait_cycles(&full[i], (count - 1) & 1, kWaitCycles);
            }
        }
    } else if (warp == 8) {
        if (lane == 0) {
            bool ok = true;
            for (int n = 0; ok && n < nch; ++n) {
                const uint32_t bt = smem_u32(sm + (n & 1) * Sm::STAGE);
                ok = lin_wait(&full[n & 1], (n >> 1) & 1, &s_abort);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    ok = ok && lin_wait(&cw_ready[half], n & 1, &s_abort);
                    if (!ok) break;
                    tc_fence_after();
                    issue_update<D2>(tmem, bt, smem_u32(sm + Sm::CW + half * Sm::CWH), half, parts, n == 0 && half == 0);
                    mma_commit(&upd_done[half]);
                }
                if (ok) mma_commit(&empty[n & 1]);
            }
            mma_commit(&drained);
            (void)mbar_wait_cycles(&drained, 0, kWaitCycles);
        }
    } else {
        const int half = warp >> 2, t = tid & 127;
        bool ok = true;
        int after = 0;                                  // tokens of this segment after the chunk, in its direction
        for (int n = 0; n < nch; ++n) {
            const int ch = chunk_of(n), L = min(C, g.len - ch * C);
            after = rev ? ch * C : g.len - ch * C - L;
            unsigned char* bt = sm + (n & 1) * Sm::STAGE;
            ok = lin_wait_warp(&full[n & 1], (n >> 1) & 1, &s_abort) &&
                 (n == 0 || lin_wait_warp(&upd_done[half], (n - 1) & 1, &s_abort));
            if (!ok) break;
            if (L < C) clear_rows(bt, D1, L, 64 * half, 64 * half + 64, t, 128);
            weight_c<D2>(bt + Sm::BT, sm + Sm::CW + half * Sm::CWH, half, parts, L, pw, role.c_upd * lin_pow(l, after), rev, t);
            fence_proxy_async_smem();
            mbar_arrive(&cw_ready[half]);
        }
        ok = ok && lin_wait_warp(&upd_done[1], (nch - 1) & 1, &s_abort);
        const int row = (warp & 3) * 32 + lane;
        if (ok && half == 0 && (row < D1 || D1 == 128)) {
            tc_fence_after();
            float* to = role.seg + ((size_t)sidx * H + h) * D1 * D2;
#pragma unroll 1
            for (int j0 = 0; j0 < D2; j0 += 32) {
                float v[32];
                tmem_ld32_sync(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + j0, v);
                write_state<D1, D2>(to, false, row, j0, v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && s_abort) flag_error(args.hdr, kStatusTimeout);
    if (warp == 0) tmem_dealloc(tmem, 128);
}

template <int D1, int D2>
cudaError_t launch_tc_t(const LinTcParams& p, bool states_only) {
    const LinArgs& a = p.a;
    auto kern = states_only ? linear_sum_tc_kernel<D1, D2> : linear_tc_kernel<D1, D2>;
    const int smem = (int)(states_only ? LinSumSmem<D1, D2>::END : LinSmem<D1, D2>::END) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((size_t)a.max_segments * a.H * a.roles), 320, smem, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_tc(const LinArgs& a, bool states_only) {
    LinTcParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    auto fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    for (int i = 0; i < 4; ++i) {
        if (!a.x[i] || a.tokens == 0) continue;
        // [tokens, H, d] in boxes of 64 channels x 1 head x 128 tokens
        const cuuint64_t dims[3] = {(cuuint64_t)a.dim[i], (cuuint64_t)a.H, (cuuint64_t)a.tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)a.dim[i] * 2, (cuuint64_t)a.H * a.dim[i] * 2};
        const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)C}, estr[3] = {1u, 1u, 1u};
        if (fn(&p.map[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.x[i]), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const int d1 = a.dim[a.role[0].a], d2 = a.dim[a.role[0].c];   // the same for all roles of one launch
    if (d1 == 128 && d2 == 128) return launch_tc_t<128, 128>(p, states_only);
    if (d1 == 128 && d2 == 64) return launch_tc_t<128, 64>(p, states_only);
    if (d1 == 64 && d2 == 128) return launch_tc_t<64, 128>(p, states_only);
    if (d1 == 64 && d2 == 64) return launch_tc_t<64, 64>(p, states_only);
    return cudaErrorInvalidValue;
}

}  // namespace kda
