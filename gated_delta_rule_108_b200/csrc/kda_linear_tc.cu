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
//  - P in two bf16 parts (2^-16), the A operand in TMEM, in place of its fp32 values;
//  - Z in two parts (2^-16) as operand, one after the other; the state itself stays
//    fp32 in TMEM.  y's own rounding is no measure for it: a row of a may read Z from
//    a direction in which Z holds little, and what a part leaves out scales with
//    |Z| |a|, not with y (one part, and keys within 0.1 of a direction that the queries
//    are orthogonal to: o off by ten times its rounding).  The second part costs 8 to
//    14 % of a forward;
//  - the weighted c in three parts (2^-24) in the roles whose state is a result (of the
//    forward, of dv), in two where it only reaches y: a state is a sum over the whole
//    sequence, and fp32 is what it is returned in (two parts everywhere would save 6 %:
//    B=9, T=4096, H=16 153 instead of 163 us).
// The tensor core cuts its sums off instead of rounding them, always towards zero.
// So each chunk's sum U starts from zero and is added to Z in registers, rounded:
// after 16,384 tokens without decay the state is off by 1.8e-7 of its size, 5.7e-6
// where the MMAs add to Z itself.
//
// One CTA per (segment, head, role), one per SM: 512 columns of TMEM hold Z, U, P and
// y.  Warp 17 loads tiles by TMA, warp 16 issues the MMAs, warps 0-7 weight P and y's
// rows of Z^T a, weight the last quarter of c and take y out, warps 8-15 keep Z, write
// its operands and weight the other quarters.  The chain from chunk to chunk (Z ->
// operands -> Z^T a, U) and the rest overlap: b and c have two buffers each, so the next
// chunk's tiles are in flight while this one is worked on; a's buffer frees as soon as
// P and Z^T a are done; y leaves through the buffer of its own chunk's c (warp 18 sends
// it out by TMA; stored straight from registers a chunk took 5.2 us instead of 4.6).
//
// What bounds it is shared memory: a chunk's MMAs read 448 KB of operands (3,584
// cycles), TMA moves 128 KB (1,024) and the warps 3,260 wavefronts, 7,870 cycles
// together, and a chunk takes 8,050.  B=9, T=4096, H=16 (144 CTAs of 32 chunks): 151 us
// under the counters (tensor pipe 49 %, issue 46 %, DRAM 3.9 TB/s), 168 us in short runs,
// 192 us at the clock that the power limit leaves in long ones.
//
// Every wait is bounded; one that gives up sets a flag that ends the CTA's other
// waits, records KDA_ERR_TIMEOUT, and the CTA waits for its own copies and MMAs,
// frees its TMEM and returns.
#include <algorithm>

#include "kda_linear.cuh"
#include "kda_tc_common.cuh"

namespace kda {
namespace {

constexpr int C = kLinChunk;
constexpr uint32_t kTile = 128 * 128;          // 128 tokens x 64 bf16 channels, 128-byte swizzle

struct LinTcParams {
    CUtensorMap map[4];                        // q, k, v, d_o
    CUtensorMap ymap[kLinMaxRoles];            // each role's output
    LinArgs a;
};

// What the waits of a CTA share: whether one has given up, and after how many cycles
// one does.
struct LinWait {
    int abort;
    long long cap;
};

// Bounded wait that also gives up when another thread of the CTA has.
__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t parity, LinWait* w) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_for(bar, parity, 1000000u)) {
        if (*(volatile int*)&w->abort) return false;
        if (clock64() - t0 > w->cap) {
            *(volatile int*)&w->abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool lin_wait_warp(uint64_t* bar, uint32_t parity, LinWait* w) {
    return __all_sync(0xffffffffu, lin_wait(bar, parity, w));
}

template <int D>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, uint64_t* bar, int h, int tok) {
    mbar_arrive_expect_tx(bar, (D / 64) * kTile);
#pragma unroll
    for (int t = 0; t < D / 64; ++t) tma_load_3d(dst + t * kTile, map, bar, 64 * t, h, tok);
}

// Zeroes rows L..127 of a tile (another sequence's tokens): they are contracted
// over with weights of zero, which must not meet an infinity or a NaN.
__device__ __forceinline__ void clear_rows(unsigned char* tile, int D, int L, int t, int nthreads) {
    for (int e = t; e < (C - L) * (D / 8); e += nthreads) {
        const int r = L + e / (D / 8), c = e % (D / 8);
        *reinterpret_cast<uint4*>(tile + (c >> 3) * kTile + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// Tokens of c from row i0 on, weighted, in `parts` bf16 parts of D2 / 64 tiles of ROWS
// rows each; eight threads a row (32 rows with 256 threads), eight channels of each
// tile a thread.  A row past L becomes zero.
template <int D2, int ROWS>
__device__ __forceinline__ void weight_c(const unsigned char* ct, unsigned char* out, int i0, int parts, int L,
                                         const float* pw, float c_upd, bool rev, int t) {
    constexpr uint32_t PART = (D2 / 64) * ROWS * 128;
    const int i = i0 + (t >> 3);
    const uint32_t src = sw128_offset(i, (t & 7) * 16);
    const bool on = i < L;
    uint4 raw[D2 / 64];
#pragma unroll
    for (int tile = 0; tile < D2 / 64; ++tile) raw[tile] = *reinterpret_cast<const uint4*>(ct + tile * kTile + src);
    const float w = on ? c_upd * pw[rev ? i + 1 : L - 1 - i] : 0.f;
    out += sw128_offset(t >> 3, (t & 7) * 16);
#pragma unroll
    for (int tile = 0; tile < D2 / 64; ++tile) {
        if (!on) raw[tile] = make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {raw[tile].x, raw[tile].y, raw[tile].z, raw[tile].w};
        uint32_t p[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 x = mul2(make_float2(w, w), unpack_bf16(u[k]));
            p[0][k] = pack_bf16(x.x, x.y);
            x = rest_of(x, p[0][k]);
            p[1][k] = pack_bf16(x.x, x.y);
            x = rest_of(x, p[1][k]);
            p[2][k] = pack_bf16(x.x, x.y);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
            if (q < parts)
                *reinterpret_cast<uint4*>(out + tile * (ROWS * 128) + q * PART) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
    }
}

// A shared-memory descriptor and the one `bytes` further on (the address field
// never carries: all tiles lie below 256 KB).
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

// D (+)= b^T (weighted c) over ROWS tokens from row i0 of b on: bd the descriptor of b
// as MN-major A, cd that of the weighted c as MN-major B.  The smallest parts first:
// the tensor core cuts each sum off, which costs least while the sum is small.
template <int D2, int ROWS, int PARTS>
__device__ __forceinline__ void issue_update_parts(uint32_t acc, uint64_t bd, uint64_t cd, int i0, bool first) {
    constexpr uint32_t idesc = instr_desc(kFmtBF16, 128, D2, true, true);
    constexpr uint32_t PART = (D2 / 64) * ROWS * 128;
#pragma unroll
    for (int q = PARTS - 1; q >= 0; --q)
#pragma unroll
        for (int ks = 0; ks < ROWS / 16; ++ks)
            mma_f16(acc, desc_at(bd, i0 * 128 + ks * 2048), desc_at(cd, q * PART + ks * 2048), idesc,
                    !(first && q == PARTS - 1 && ks == 0));
}
template <int D2, int ROWS>
__device__ __forceinline__ void issue_update(uint32_t acc, uint64_t bd, uint64_t cd, int i0, int parts, bool first) {
    if (parts == 3) issue_update_parts<D2, ROWS, 3>(acc, bd, cd, i0, first);
    else issue_update_parts<D2, ROWS, 2>(acc, bd, cd, i0, first);
}

// 32 columns from j0 on of a thread's row of Z, from and to a state [D2][D1]: the lanes
// of a warp hold rows that follow one another, so each column is one line of 128 bytes.
// Past L1: another block of this launch may have written it.
template <int D1>
__device__ __forceinline__ void read_columns(const float* s, int row, int j0, float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __ldcg(s + (size_t)(j0 + j) * D1 + row);
}
template <int D1>
__device__ __forceinline__ void write_columns(float* s, int row, int j0, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) s[(size_t)(j0 + j) * D1 + row] = v[j];
}

// The same for a state [D1][D2], whose rows lie apart: four lanes take 64 bytes of a row
// and hand them over through 2 KB of shared memory of the warp's own, 16 columns at a
// time.  (Each lane reading its own row touches 32 lines an instruction: 8,000 cycles
// for a state of 64 KB.)
constexpr int kStateStage = 32 * 64;
__device__ __forceinline__ uint32_t stage_at(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }
template <int D2>
__device__ __forceinline__ void read_rows(const float* s, unsigned char* stage, int row0, int j0, int lane, float (&v)[32]) {
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = *reinterpret_cast<const float4*>(s + (size_t)(row0 + 8 * (i & 3) + (lane >> 2)) * D2 + j0 + 16 * (i >> 2) + 4 * (lane & 3));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(stage + stage_at(8 * i + (lane >> 2), lane & 3)) = x[4 * half + i];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(stage + stage_at(lane, c));
            const int j = 16 * half + 4 * c;
            v[j] = y.x; v[j + 1] = y.y; v[j + 2] = y.z; v[j + 3] = y.w;
        }
    }
}
template <int D2>
__device__ __forceinline__ void write_rows(float* s, unsigned char* stage, int row0, int j0, int lane, const float (&v)[32]) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = 16 * half + 4 * c;
            *reinterpret_cast<float4*>(stage + stage_at(lane, c)) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(s + (size_t)(row0 + 8 * i + (lane >> 2)) * D2 + j0 + 16 * half + 4 * (lane & 3)) =
                *reinterpret_cast<const float4*>(stage + stage_at(8 * i + (lane >> 2), lane & 3));
    }
}

// A state handed from one block to a later one: each warp counts itself in once its
// part is written; every warp of the reader waits for all of them.  A block that has
// given up says so in the same word, and the blocks after it pass that on without a
// wait of their own: else a chain could hold the GPU for one bounded wait a segment.
constexpr int kLinFailed = 1 << 30;
__device__ __forceinline__ void raise_flag(int* flag) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        __threadfence();
        atomicAdd(flag, 1);
    }
}
__device__ __forceinline__ bool wait_flag(const int* flag, int count, LinWait* w) {
    const long long t0 = clock64();
    int seen;
    do {
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(seen) : "l"(flag) : "memory");
        if (seen >= kLinFailed) seen = -1;
        if (seen < count) {
            if (seen < 0 || *(volatile int*)&w->abort || clock64() - t0 > w->cap) {
                *(volatile int*)&w->abort = 1;
                break;
            }
            __nanosleep(200);
        }
    } while (seen < count);
    return __all_sync(0xffffffffu, seen >= count);
}

// ------------------------------------------------------------- chunk kernel --
constexpr int kLinStep = 32;        // tokens of one step of the update
static_assert(C / kLinStep == 4, "the chunk kernel names its steps");

template <int D1, int D2>
struct LinSmem {
    static constexpr uint32_t AT = (D1 / 64) * kTile, CT = (D2 / 64) * kTile;
    static constexpr uint32_t A = 0;
    static constexpr uint32_t B = A + AT;                        // b of two chunks
    static constexpr uint32_t CC = B + 2 * AT;                   // c of two chunks; y leaves through its own chunk's
    // Two places that Z's operand and the weighted c share in turn: bf16 Z, D2 / 64 tiles
    // of D1 rows a part, or the weighted c of one step, three parts.  The second place
    // holds step 0, then Z's second part, then step 2; the first Z's first part, then
    // steps 1 and 3.
    static constexpr uint32_t CWB = 3 * (D2 / 64) * kLinStep * 128;
    static constexpr uint32_t ZB = (D2 / 64) * D1 * 128 > CWB ? (D2 / 64) * D1 * 128 : CWB;
    static constexpr uint32_t Z = CC + 2 * CT;
    static constexpr uint32_t CW = Z + ZB;
    static constexpr uint32_t END = CW + ZB;
    static_assert(END + 1024 + 1200 <= 232448, "shared memory");
    static_assert(ZB >= D1 / 16 * 2048, "a state's way through Z's place");
};

constexpr int kLinThreads = 19 * 32;

template <int D1, int D2>
__device__ __forceinline__ void linear_tc_body(const LinTcParams& prm, int ri, int x)
{
    using Sm = LinSmem<D1, D2>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t full_a, az_done, full_b[2], empty_b[2], full_c[2], empty_c[2], p_done, p_ready,
        y_done, y_free, y_staged[2], cw_ready[2], cw_free[2], upd_done, z_ready, zh_done, zl_ready, drained;
    __shared__ uint32_t s_tmem;
    __shared__ LinWait s_wait;
    __shared__ float pw[C + 1], pw_rest[2];     // powers; second parts of those of a whole chunk and of the short one
    // weights of a 32 x 32 block of P, at [31 + row - column] for one on the diagonal (0 on the side that does not
    // count) and [31 - column], times a factor of the row, for another
    __shared__ float diag[64], edge[32];

    const LinArgs& args = prm.a;
    const LinRole& role = args.role[ri];
    const int H = args.H, h = x % H, sidx = x / H;
    if (sidx >= args.map.segments()) return;
    const LinMap::Seg g = args.map.locate(sidx);
    const bool rev = role.reverse;
    const int nch = (g.len + C - 1) / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t zsize = (size_t)D1 * D2, user = ((size_t)g.seq * H + h) * zsize;
    const int parts = role.parts;
    int* const flag = args.chained ? args.flags + ((size_t)sidx * H + h) * args.roles + ri : nullptr;
    // in registers: the asm statements below make the compiler read memory again
    const float c_inter = role.c_inter, c_intra = role.c_intra, c_upd = role.c_upd;
    __nv_bfloat16* const yout = static_cast<__nv_bfloat16*>(role.y);

    if (tid == 0) {
        s_wait.abort = 0;
        s_wait.cap = args.wait_cap > 0 ? args.wait_cap : kWaitCycles;
        mbar_init(&full_a, 1);
        mbar_init(&az_done, 1);
        mbar_init(&p_done, 1);
        mbar_init(&p_ready, 256);
        mbar_init(&y_done, 1);
        mbar_init(&y_free, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full_b[i], 1);
            mbar_init(&empty_b[i], 1);
            mbar_init(&full_c[i], 1);
            mbar_init(&empty_c[i], 1);
            mbar_init(&y_staged[i], 256);
            mbar_init(&cw_ready[i], 256);
            mbar_init(&cw_free[i], 1);
        }
        mbar_init(&upd_done, 1);
        mbar_init(&z_ready, 256);
        mbar_init(&zh_done, 1);
        mbar_init(&zl_ready, 256);
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (tid == 17 * 32) {
        tma_prefetch_desc(&prm.map[role.b]);
        tma_prefetch_desc(&prm.map[role.c]);
        tma_prefetch_desc(&prm.map[role.a]);
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    {
        const double l = lin_log_decay(args.log_decay, h);
        if (tid <= C) pw[tid] = lin_pow(l, tid);
        else if (tid >= 256 && tid < 258) pw_rest[tid - 256] = lin_pow2(l, tid == 256 ? C : g.len % C).y;
        else if (tid >= 160 && tid < 192) edge[tid - 160] = lin_pow(l, rev ? 191 - tid : tid - 160);
        else if (tid >= 192 && tid < 255) {
            const int n = rev ? 31 - (tid - 192) : tid - 192 - 31;
            diag[tid - 192] = n >= 0 ? lin_pow(l, n) : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t ZREG = tmem, UACC = tmem + 128, PACC = tmem + 256, YACC = tmem + 384;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const int quad = warp & 3, row = quad * 32 + lane;
    const int sub = (warp >> 2) & 1;            // the two warps of a group that share 32 TMEM lanes split the columns
    auto chunk_of = [&](int n) { return rev ? nch - 1 - n : n; };
    // b and c of chunk n are use n / 2 of their buffer n % 2
    auto buf_b = [&](int n) { return sm + Sm::B + (n & 1) * Sm::AT; };
    auto buf_c = [&](int n) { return sm + Sm::CC + (n & 1) * Sm::CT; };

    if (warp == 17) {                                   // ---- TMA loads
        if (lane == 0) {
            tma_prefetch_desc(&prm.ymap[ri]);
            int nb = 0, nc = 0, na = 0;
            for (int n = 0; n < nch; ++n) {             // in the order in which the buffers become free
                const int tok = g.begin + chunk_of(n) * C, i = n & 1;
                const uint32_t before = ((n >> 1) - 1) & 1;
                if (n > 1 && !lin_wait(&empty_b[i], before, &s_wait)) break;
                load_tile<D1>(buf_b(n), &prm.map[role.b], &full_b[i], h, tok);
                ++nb;
                if (n > 1 && !lin_wait(&empty_c[i], before, &s_wait)) break;
                load_tile<D2>(buf_c(n), &prm.map[role.c], &full_c[i], h, tok);
                ++nc;
                if (n > 0 && !lin_wait(&az_done, (n - 1) & 1, &s_wait)) break;
                // the test hook's missing copy
                if (args.wait_cap > 0 && (args.chained ? g.index == 0 : blockIdx.x == 0) && n == min(2, nch - 1)) continue;
                load_tile<D1>(sm + Sm::A, &prm.map[role.a], &full_a, h, tok);
                ++na;
            }
            // every copy issued has landed before the CTA's memory goes away
            if (na) (void)mbar_wait_cycles(&full_a, (na - 1) & 1, kWaitCycles);
            for (int n = max(nb - 2, 0); n < nb; ++n) (void)mbar_wait_cycles(&full_b[n & 1], (n >> 1) & 1, kWaitCycles);
            for (int n = max(nc - 2, 0); n < nc; ++n) (void)mbar_wait_cycles(&full_c[n & 1], (n >> 1) & 1, kWaitCycles);
        }
    } else if (warp == 18) {                            // ---- y out, from c's buffer
        if (lane == 0) {
            for (int n = 0; n < nch; ++n) {
                if (!lin_wait(&y_staged[n & 1], (n >> 1) & 1, &s_wait)) break;
                const int ch = chunk_of(n);
                if (g.len - ch * C >= C) {              // a short chunk's rows have been written one by one
#pragma unroll
                    for (int t = 0; t < D2 / 64; ++t)
                        tma_store_3d(&prm.ymap[ri], buf_c(n) + t * kTile, 64 * t, h, g.begin + ch * C);
                    bulk_store_commit();
                    bulk_store_wait_read();
                }
                mbar_arrive(&empty_c[n & 1]);
            }
            bulk_store_wait_all();
        }
    } else if (warp == 16) {                            // ---- MMA issue
        // the whole warp goes through the loop together; one lane issues
        // descriptors: K-major a, b; MN-major b (the update's A), Z, c, weighted c in its two places
        const uint64_t a_k = smem_desc(smem_u32(sm + Sm::A), 16, 1024, kLayoutSW128);
        const uint64_t z_mn = smem_desc(smem_u32(sm + Sm::Z), D1 * 128, 1024, kLayoutSW128);
        const uint64_t zl_mn = smem_desc(smem_u32(sm + Sm::CW), D1 * 128, 1024, kLayoutSW128);
        const uint64_t w_mn0 = smem_desc(smem_u32(sm + Sm::CW), kLinStep * 128, 1024, kLayoutSW128);
        const uint64_t w_mn1 = smem_desc(smem_u32(sm + Sm::Z), kLinStep * 128, 1024, kLayoutSW128);
        const uint64_t b_k0 = smem_desc(smem_u32(sm + Sm::B), 16, 1024, kLayoutSW128);
        const uint64_t b_mn0 = smem_desc(smem_u32(sm + Sm::B), kTile, 1024, kLayoutSW128);
        const uint64_t c_mn0 = smem_desc(smem_u32(sm + Sm::CC), kTile, 1024, kLayoutSW128);
        constexpr uint32_t id_p = instr_desc(kFmtBF16, 128, 128);
        constexpr uint32_t id_y = instr_desc(kFmtBF16, 128, D2, false, true);
        for (int n = 0; n < nch; ++n) {
            const uint32_t ph = n & 1, prev = (n - 1) & 1;
            const uint64_t b_k = desc_at(b_k0, (n & 1) * Sm::AT), b_mn = desc_at(b_mn0, (n & 1) * Sm::AT);
            const uint64_t c_mn = desc_at(c_mn0, (n & 1) * Sm::CT);
            // P = a b^T, over the previous chunk's weighted P once y has been formed from it
            if (!lin_wait_warp(&full_a, ph, &s_wait) || !lin_wait_warp(&full_b[n & 1], (n >> 1) & 1, &s_wait)) break;
            if (n > 0 && !lin_wait_warp(&y_done, prev, &s_wait)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D1 / 16; ++k) {
                    const uint32_t off = (k >> 2) * kTile + (k & 3) * 32;
                    mma_f16(PACC, desc_at(a_k, off), desc_at(b_k, off), id_p, k != 0);
                }
                mma_commit(&p_done);
            }
            // U = b^T (weighted c) in four steps, as their operands come; between them y = a Z and,
            // on top of its weighted rows, y += P c
            auto update = [&](int i) {
                const bool ok = lin_wait_warp(&cw_ready[i & 1], i >> 1, &s_wait);
                tc_fence_after();
                if (ok && elect_one()) {
                    issue_update<D2, kLinStep>(UACC, b_mn, i & 1 ? w_mn1 : w_mn0, kLinStep * i, parts, i == 0);
                    mma_commit(&cw_free[i & 1]);
                }
                return ok;
            };
            if (!lin_wait_warp(&z_ready, ph, &s_wait) || !update(0)) break;
            if (n > 0 && !lin_wait_warp(&y_free, prev, &s_wait)) break;
            tc_fence_after();
            // y = a Z: Z's first part, then its second, which comes where step 0 was
            auto read_z = [&](uint64_t z, bool first) {
#pragma unroll
                for (int k = 0; k < D1 / 16; ++k)
                    mma_f16(YACC, desc_at(a_k, (k >> 2) * kTile + (k & 3) * 32), desc_at(z, k * 2048), id_y, !(first && k == 0));
            };
            if (elect_one()) {
                read_z(z_mn, true);
                mma_commit(&zh_done);
            }
            if (!lin_wait_warp(&zl_ready, ph, &s_wait)) break;
            tc_fence_after();
            if (elect_one()) {
                read_z(zl_mn, false);
                mma_commit(&az_done);
            }
            if (!update(1) || !update(2) || !lin_wait_warp(&p_ready, ph, &s_wait)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)             // both parts of P (8 columns of 16 each)
#pragma unroll
                    for (int q = 1; q >= 0; --q)
                        mma_f16_ts(YACC, PACC + k * 16 + q * 8, desc_at(c_mn, k * 2048), id_y, true);
                mma_commit(&y_done);
            }
            if (!update(3)) break;
            if (elect_one()) {
                mma_commit(&upd_done);
                mma_commit(&empty_b[n & 1]);
            }
        }
        if (elect_one()) mma_commit(&drained);
        (void)mbar_wait_cycles(&drained, 0, kWaitCycles);
    } else if (warp < 8) {                              // ---- P, then y
        for (int n = 0; n < nch; ++n) {
            const int ch = chunk_of(n), L = min(C, g.len - ch * C), tok = g.begin + ch * C;
            if (!lin_wait_warp(&p_done, n & 1, &s_wait)) break;
            tc_fence_after();
#pragma unroll 1
            for (int b = sub; b < 4; b += 2) {
                const uint32_t at = PACC + lane_base + 32 * b;
                uint32_t pk[32];
                if (rev ? b >= quad : b <= quad) {      // these rows see this block of columns
                    float v[32];
                    tmem_ld32_sync(at, v);
                    // columns past L hold other tokens' products, and on the diagonal's other side one may be infinite
                    if (L < C || b == quad) {
                        uint32_t keep = L >= 32 * b + 32 ? ~0u : L > 32 * b ? (1u << (L - 32 * b)) - 1 : 0u;
                        if (b == quad) keep &= rev ? ~0u << lane : ~0u >> (31 - lane);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(keep >> j & 1)) v[j] = 0.f;
                    }
                    // off the diagonal |r - i| = (distance to the block's near edge) + (distance within it): both factors <= 1
                    const bool on = b == quad;
                    const float f = c_intra * (on ? 1.f : pw[rev ? 32 * b - row : row - (32 * b + 31)]);
                    const float* w = on ? diag + 31 + lane : edge + 31;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = mul2(make_float2(v[2 * j], v[2 * j + 1]), mul2(make_float2(f, f), make_float2(w[-2 * j], w[-2 * j - 1])));
                        const uint32_t hi = pack_bf16(x.x, x.y);
                        const float2 y = rest_of(x, hi);
                        pk[(j >> 3) * 16 + (j & 7)] = hi;           // per 16 columns: 8 of the first part, 8 of the second
                        pk[(j >> 3) * 16 + 8 + (j & 7)] = pack_bf16(y.x, y.y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = 0;
                }
                tmem_st32(at, pk);
            }
            // y's rows of a Z get their weight, P c goes on top
            if (!lin_wait_warp(&az_done, n & 1, &s_wait)) break;
            tc_fence_after();
            const float wz = c_inter * pw[row < L ? (rev ? L - 1 - row : row + 1) : 0];
#pragma unroll 1
            for (int j0 = 32 * sub; j0 < D2; j0 += 64) {
                float v[32];
                uint32_t d[32];
                tmem_ld32_sync(YACC + lane_base + j0, v);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 x = mul2(make_float2(wz, wz), make_float2(v[j], v[j + 1]));
                    d[j] = __float_as_uint(x.x);
                    d[j + 1] = __float_as_uint(x.y);
                }
                tmem_st32(YACC + lane_base + j0, d);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_ready);

            // the update's last step, while P c runs
            if (!lin_wait_warp(&full_c[n & 1], (n >> 1) & 1, &s_wait) || !lin_wait_warp(&cw_free[1], 0, &s_wait)) break;
            weight_c<D2, kLinStep>(buf_c(n), sm + Sm::Z, 3 * kLinStep, parts, L, pw, c_upd, rev, tid);
            fence_proxy_async_smem();
            mbar_arrive(&cw_ready[1]);

            // y, through c's place: P c has been formed, and all eight warps have weighted their c
            if (!lin_wait_warp(&y_done, n & 1, &s_wait) || !lin_wait_warp(&cw_ready[1], 1, &s_wait)) break;
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 32 * sub; j0 < D2; j0 += 64) {
                float v[32];
                tmem_ld32_sync(YACC + lane_base + j0, v);
                uint4 y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                      pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
                if (L == C) {       // out by TMA as whole rows
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(buf_c(n) + (j0 >> 6) * kTile + sw128_offset(row, 64 * sub + 16 * e)) = y[e];
                } else if (row < L) {   // a short chunk: a tile would reach into the next sequence
                    uint4* dst = reinterpret_cast<uint4*>(yout + ((size_t)(tok + row) * H + h) * D2 + j0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[e] = y[e];
                }
            }
            tc_fence_before();
            mbar_arrive(&y_free);
            fence_proxy_async_smem();
            mbar_arrive(&y_staged[n & 1]);
        }
    } else {                                            // ---- Z, then the weighted c
        const int t = tid - 256;
        bool ok = true;
        const bool mine = D1 == 128 || quad < 2;        // warps with rows of Z
        unsigned char* const stage = sm + Sm::Z + kStateStage * (D1 == 128 ? warp - 8 : 2 * sub + (quad & 1));
        if (mine) {
            const bool scanned = args.scanned && g.count > 1;
            const int before = sidx + (rev ? 1 : -1);           // the segment processed before this one
            const bool chained = args.chained && g.index != (rev ? g.count - 1 : 0);
            if (chained) {
                ok = wait_flag(args.flags + ((size_t)before * H + h) * args.roles + ri, D1 / 16, &s_wait);
                if (!ok && lane == 0) atomicOr(flag, kLinFailed);
            }
            const float* own = chained ? role.seg + ((size_t)before * H + h) * zsize
                             : scanned ? role.seg + ((size_t)sidx * H + h) * zsize : nullptr;
            const float* given = role.s_in ? role.s_in + user : nullptr;
            const double l = lin_log_decay(args.log_decay, h);
#pragma unroll 1
            for (int j0 = 32 * sub; j0 < D2; j0 += 64) {
                float v[32];
                if (own || (given && role.transposed)) {
                    read_columns<D1>(own ? own : given, row, j0, v);
                } else if (given) {
                    read_rows<D2>(given, stage, 32 * quad, j0, lane, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                }
                if (!scanned && !args.chained)
                    lin_enter(args.map, g, sidx, rev, l, [&](int slot, float2 w) {
                        float u[32];
                        read_columns<D1>(role.seg + ((size_t)slot * H + h) * zsize, row, j0, u);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = decay_add(w, v[j], u[j]);
                    });
                tmem_st32_sync(ZREG + lane_base + j0, v);
            }
        }
        named_bar_sync(1, 256);     // Z's operand goes where the states went through (all these warps come here)
        for (int n = 0; ok && n < nch; ++n) {
            const int L = min(C, g.len - chunk_of(n) * C), len_before = n > 0 ? min(C, g.len - chunk_of(n - 1) * C) : 0;
            ok = lin_wait_warp(&full_b[n & 1], (n >> 1) & 1, &s_wait) && lin_wait_warp(&full_c[n & 1], (n >> 1) & 1, &s_wait);
            if (!ok) break;
            if (L < C) {        // P's MMA may still read b: its columns past L are dropped when P is weighted
                clear_rows(buf_b(n), D1, L, t, 256);
                clear_rows(buf_c(n), D2, L, t, 256);
                fence_proxy_async_smem();
            }
#pragma unroll 1
            for (int i = 0; i < 3; ++i) {
                // the step's place is free: of the step or the part of Z before
                if (i == 0) ok = n == 0 || lin_wait_warp(&cw_free[0], 1, &s_wait);
                else ok = lin_wait_warp(i == 1 ? &zh_done : &az_done, n & 1, &s_wait);
                if (!ok) break;
                weight_c<D2, kLinStep>(buf_c(n), sm + (i & 1 ? Sm::Z : Sm::CW), kLinStep * i, parts, L, pw, c_upd, rev, t);
                fence_proxy_async_smem();
                mbar_arrive(&cw_ready[i & 1]);
                if (i > 0) continue;

                // Z, while the others wait for it: step 0 was ahead, during the previous chunk's update
                if (n > 0) ok = lin_wait_warp(&upd_done, (n - 1) & 1, &s_wait);
                if (!ok) break;
                tc_fence_after();
                if (mine) {                             // Z <- lambda^L Z + U of the previous chunk; its operand's first part
                    const float2 gam = n > 0 ? make_float2(pw[len_before], pw_rest[len_before < C]) : make_float2(1.f, 0.f);
#pragma unroll 1
                    for (int j0 = 32 * sub; j0 < D2; j0 += 64) {
                        float v[32], u[32];
                        tmem_ld32x2_sync(ZREG + lane_base + j0, UACC + lane_base + j0, v, u);
                        if (n > 0) {
                            uint32_t d[32];
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const float2 x = decay_add(gam, make_float2(v[j], v[j + 1]), make_float2(u[j], u[j + 1]));
                                v[j] = x.x; v[j + 1] = x.y;
                                d[j] = __float_as_uint(x.x);
                                d[j + 1] = __float_as_uint(x.y);
                            }
                            tmem_st32(ZREG + lane_base + j0, d);
                        }
#pragma unroll
                        for (int j8 = 0; j8 < 4; ++j8)
                            *reinterpret_cast<uint4*>(sm + Sm::Z + (j0 >> 6) * (D1 * 128) + sw128_offset(row, 64 * sub + 16 * j8)) =
                                make_uint4(pack_bf16(v[8 * j8], v[8 * j8 + 1]), pack_bf16(v[8 * j8 + 2], v[8 * j8 + 3]),
                                           pack_bf16(v[8 * j8 + 4], v[8 * j8 + 5]), pack_bf16(v[8 * j8 + 6], v[8 * j8 + 7]));
                    }
                    tmem_wait_st();
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&z_ready);

                ok = lin_wait_warp(&cw_free[0], 0, &s_wait);
                if (!ok) break;
                if (mine) {                             // what the first part has left of Z
#pragma unroll 1
                    for (int j0 = 32 * sub; j0 < D2; j0 += 64) {
                        float v[32];
                        uint32_t p[16];
                        tmem_ld32_sync(ZREG + lane_base + j0, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 x = rest_of(make_float2(v[2 * j], v[2 * j + 1]), pack_bf16(v[2 * j], v[2 * j + 1]));
                            p[j] = pack_bf16(x.x, x.y);
                        }
#pragma unroll
                        for (int j8 = 0; j8 < 4; ++j8)
                            *reinterpret_cast<uint4*>(sm + Sm::CW + (j0 >> 6) * (D1 * 128) + sw128_offset(row, 64 * sub + 16 * j8)) =
                                make_uint4(p[4 * j8], p[4 * j8 + 1], p[4 * j8 + 2], p[4 * j8 + 3]);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&zl_ready);
            }
        }
        if (ok && nch > 0) ok = lin_wait_warp(&upd_done, (nch - 1) & 1, &s_wait);
        const bool last = g.index == (rev ? 0 : g.count - 1), hand = args.chained && !last;
        if (ok && mine && (hand || (last && role.s_out))) {
            tc_fence_after();
            float* to = hand ? role.seg + ((size_t)sidx * H + h) * zsize : role.s_out + user;
            const int len = nch > 0 ? min(C, g.len - chunk_of(nch - 1) * C) : 0;
            const float2 gam = make_float2(pw[len], len ? pw_rest[len < C] : 0.f);
#pragma unroll 1
            for (int j0 = 32 * sub; j0 < D2; j0 += 64) {
                float v[32];
                tmem_ld32_sync(ZREG + lane_base + j0, v);
                if (nch > 0) {
                    float u[32];
                    tmem_ld32_sync(UACC + lane_base + j0, u);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = decay_add(gam, v[j], u[j]);
                }
                if (hand || role.transposed) write_columns<D1>(to, row, j0, v);
                else write_rows<D2>(to, stage, 32 * quad, j0, lane, v);
            }
            if (hand) raise_flag(flag);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && s_wait.abort) {
        if (args.hdr) flag_error(args.hdr, kStatusTimeout);
        if (flag) atomicOr(flag, kLinFailed);
    }
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// One launch for all roles: those over (DK, DV) and those over (DV, DK).
template <int DK, int DV>
__global__ void __launch_bounds__(kLinThreads, 1)
linear_tc_kernel(const __grid_constant__ LinTcParams prm)
{
    const LinArgs& a = prm.a;
    if (!lin_begin(a)) return;
    int ri = blockIdx.x % a.roles, x = blockIdx.x / a.roles;
    if (a.chained) {
        // Work is claimed in order, all first segments before all second ones: the state a
        // segment waits for comes from work that was claimed before and is running or done,
        // in whatever order the blocks have started.
        __shared__ int claimed;
        if (threadIdx.x == 0) claimed = atomicAdd(&a.hdr->next_pair, 1);
        __syncthreads();
        const int chains = a.map.N * a.H * a.roles, j = claimed / chains, c = claimed - j * chains;
        ri = c % a.roles;
        const int nh = c / a.roles, n = nh / a.H, h = nh - n * a.H;
        x = (n * a.map.num_seg + (a.role[ri].reverse ? a.map.num_seg - 1 - j : j)) * a.H + h;
    }
    if (DK == DV || !a.role[ri].transposed) linear_tc_body<DK, DV>(prm, ri, x);
    else linear_tc_body<DV, DK>(prm, ri, x);
}

// ----------------------------------------------------------- segment's sum --
// Z of one segment (or a piece of it) from zero: sum_i lambda^{tokens from i to its end}
// b_i c_i^T.  The weights count to that end, so nothing is rescaled.  Each
// chunk's sum is formed in TMEM (two of them, in turn) and added in registers, 32
// elements a thread: the tensor core's cut-off sums would pile up over a long
// segment.  Half a chunk of c is weighted, by sixteen warps, while the other half is
// multiplied.  2.0 us a chunk, half of the chunk kernel's: the weights (three parts of
// 128 x D2) are what it waits for.
constexpr int kLinSumThreads = 18 * 32;

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
__device__ __forceinline__ void linear_sum_tc_body(const LinTcParams& prm, int ri)
{
    using Sm = LinSumSmem<D1, D2>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t full[2], empty[2], cw_ready[2], cw_free[2], upd_done, drained;
    __shared__ uint32_t s_tmem;
    __shared__ LinWait s_wait;
    __shared__ float pw[C + 1];

    const LinArgs& args = prm.a;
    const LinRole& role = args.role[ri];
    const int x = blockIdx.x / args.roles;
    const int H = args.H, h = x % H, slot = x / H;
    if (slot >= args.map.segments() * args.map.pieces) return;
    const LinMap::Seg g = args.map.locate_piece(slot);
    const bool rev = role.reverse;
    if (g.index == (rev ? 0 : g.count - 1)) return;     // processed last: its sum enters no other segment
    if (g.len <= 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = role.parts;
    const float c_upd = role.c_upd;
    const double l = lin_log_decay(args.log_decay, h);
    const int chunks = (g.len + C - 1) / C, skip = lin_skip(l, g.len, C, chunks, rev), nch = chunks - skip;

    if (tid == 0) {
        s_wait.abort = 0;
        s_wait.cap = args.wait_cap > 0 ? args.wait_cap : kWaitCycles;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], 1);
            mbar_init(&cw_ready[i], 512);
            mbar_init(&cw_free[i], 1);
        }
        mbar_init(&upd_done, 1);
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, 256);
        tmem_relinquish();
    }
    if (tid <= C) pw[tid] = lin_pow(l, tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto chunk_of = [&](int n) { return rev ? nch - 1 - n : skip + n; };

    if (warp == 17) {                                   // ---- TMA loads
        if (lane == 0) {
            int n = 0;
            for (; n < nch; ++n) {
                const int tok = g.begin + chunk_of(n) * C, st = n & 1;
                if (n > 1 && !lin_wait(&empty[st], ((n >> 1) - 1) & 1, &s_wait)) break;
                load_tile<D1>(sm + st * Sm::STAGE, &prm.map[role.b], &full[st], h, tok);
                load_tile<D2>(sm + st * Sm::STAGE + Sm::BT, &prm.map[role.c], &full[st], h, tok);
            }
            for (int i = 0; i < 2; ++i) {
                const int count = (n - i + 1) >> 1;     // loads into stage i
                if (count > 0) (void)mbar_wait_cycles(&full[i], (count - 1) & 1, kWaitCycles);
            }
        }
    } else if (warp == 16) {                            // ---- MMA issue
        const uint64_t b_mn0 = smem_desc(smem_u32(sm), kTile, 1024, kLayoutSW128);
        const uint64_t w_mn0 = smem_desc(smem_u32(sm + Sm::CW), 64 * 128, 1024, kLayoutSW128);
        bool ok = true;
        for (int n = 0; ok && n < nch; ++n) {
            const uint64_t b_mn = desc_at(b_mn0, (n & 1) * Sm::STAGE);
            ok = lin_wait_warp(&full[n & 1], (n >> 1) & 1, &s_wait);
#pragma unroll 1
            for (int half = 0; ok && half < 2; ++half) {
                ok = lin_wait_warp(&cw_ready[half], n & 1, &s_wait);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_update<D2, 64>(tmem + 128 * (n & 1), b_mn, desc_at(w_mn0, half * Sm::CWH), 64 * half, parts, half == 0);
                    mma_commit(&cw_free[half]);
                    if (half == 1) {
                        mma_commit(&upd_done);
                        mma_commit(&empty[n & 1]);
                    }
                }
            }
        }
        if (elect_one()) mma_commit(&drained);
        (void)mbar_wait_cycles(&drained, 0, kWaitCycles);
    } else {                                            // ---- weighted c, the sum
        const int quad = warp & 3, sub = warp >> 2, row = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
        constexpr int COLS = D2 / 4;                    // columns COLS sub .. of this thread's row
        float z[COLS];
#pragma unroll
        for (int j = 0; j < COLS; ++j) z[j] = 0.f;
        auto add = [&](int n) {                         // Z += chunk n's sum
            if (!lin_wait_warp(&upd_done, n & 1, &s_wait)) return false;
            tc_fence_after();
            if (D1 == 128 || quad < 2) {
#pragma unroll
                for (int j0 = 0; j0 < COLS; j0 += 16) {
                    float v[16];
                    tmem_ld16_sync(tmem + 128 * (n & 1) + lane_base + COLS * sub + j0, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) z[j0 + j] += v[j];
                }
            }
            tc_fence_before();
            return true;
        };
        bool ok = true;
        for (int n = 0; ok && n < nch; ++n) {
            const int ch = chunk_of(n), L = min(C, g.len - ch * C);
            const int after = rev ? ch * C : g.len - ch * C - L;    // tokens of the segment still to come
            unsigned char* bt = sm + (n & 1) * Sm::STAGE;
            const float cw = c_upd * lin_pow(l, after);
            ok = lin_wait_warp(&full[n & 1], (n >> 1) & 1, &s_wait);
            if (!ok) break;
            if (L < C) {
                clear_rows(bt, D1, L, tid, 512);
                fence_proxy_async_smem();
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                // the last chunk's sum before this chunk's second half, without which the barrier cannot go on
                if (n > 0) ok = lin_wait_warp(&cw_free[half], (n - 1) & 1, &s_wait) && (half == 0 || add(n - 1));
                if (!ok) break;
                weight_c<D2, 64>(bt + Sm::BT, sm + Sm::CW + half * Sm::CWH, 64 * half, parts, L, pw, cw, rev, tid);
                fence_proxy_async_smem();
                mbar_arrive(&cw_ready[half]);
            }
        }
        if (ok) ok = add(nch - 1);
        if (ok && (D1 == 128 || quad < 2)) {
            float* to = role.seg + ((size_t)slot * H + h) * D1 * D2 + (size_t)COLS * sub * D1 + row;
#pragma unroll
            for (int j = 0; j < COLS; ++j) to[(size_t)j * D1] = z[j];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && s_wait.abort && args.hdr) flag_error(args.hdr, kStatusTimeout);
    if (warp == 0) tmem_dealloc(tmem, 256);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kLinSumThreads, 1)
linear_sum_tc_kernel(const __grid_constant__ LinTcParams prm)
{
    if (!lin_begin(prm.a)) return;
    const int ri = blockIdx.x % prm.a.roles;
    if (DK == DV || !prm.a.role[ri].transposed) linear_sum_tc_body<DK, DV>(prm, ri);
    else linear_sum_tc_body<DV, DK>(prm, ri);
}

template <int DK, int DV>
cudaError_t launch_tc_t(const LinTcParams& p, bool states_only) {
    const LinArgs& a = p.a;
    auto kern = states_only ? linear_sum_tc_kernel<DK, DV> : linear_tc_kernel<DK, DV>;
    const uint32_t sum = std::max(LinSumSmem<DK, DV>::END, LinSumSmem<DV, DK>::END);
    const uint32_t chunk = std::max(LinSmem<DK, DV>::END, LinSmem<DV, DK>::END);
    const int smem = (int)(states_only ? sum : chunk) + 1024;
    static std::atomic<uint64_t> done[2];
    void* args[] = {const_cast<LinTcParams*>(&p)};
    return lin_launch(reinterpret_cast<const void*>(kern), (size_t)a.max_segments * (states_only ? a.map.pieces : 1) * a.H * a.roles,
                      states_only ? kLinSumThreads : kLinThreads, smem, args, a.follows, a.stream, done[states_only]);
}

}  // namespace

cudaError_t launch_linear_tc(const LinArgs& a, bool states_only) {
    LinTcParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    auto fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    // [tokens, H, d] in boxes of 64 channels x 1 head x 128 tokens
    auto encode = [&](CUtensorMap* m, const void* base, int d) {
        const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)a.H, (cuuint64_t)a.tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)a.H * d * 2};
        const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)C}, estr[3] = {1u, 1u, 1u};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (a.tokens > 0) {
        for (int i = 0; i < 4; ++i)
            if (a.x[i] && !encode(&p.map[i], a.x[i], a.dim[i])) return cudaErrorInvalidValue;
        for (int i = 0; !states_only && i < a.roles; ++i)
            if (!encode(&p.ymap[i], a.role[i].y, a.dim[a.role[i].c])) return cudaErrorInvalidValue;
    }
    if (a.dk == 128 && a.dv == 128) return launch_tc_t<128, 128>(p, states_only);
    if (a.dk == 128 && a.dv == 64) return launch_tc_t<128, 64>(p, states_only);
    if (a.dk == 64 && a.dv == 128) return launch_tc_t<64, 128>(p, states_only);
    if (a.dk == 64 && a.dv == 64) return launch_tc_t<64, 64>(p, states_only);
    return cudaErrorInvalidValue;
}

}  // namespace kda
