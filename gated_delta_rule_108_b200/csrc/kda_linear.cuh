// kda_linear.cuh -- definitions shared by the files of the linear attention with
// one fixed decay per head: how its forward and its three gradients map onto one
// recurrence, how sequences are cut into segments, and the launchers.
//
// With lambda = e^l per head, scale s = dk^{-1/2} and states of dk x dv:
//
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = s S_t^T q_t                    (forward)
//   dq_t = s S_t d_o_t                                                       (first to last token)
//   G_t = lambda G_{t+1} + s q_t d_o_t^T, dk_t = G_t v_t, dv_t = G_t^T k_t   (last to first token)
//
// where G_T also holds the cotangent of the final state.  Every line has the form
//
//   Z_t = lambda Z_{t-1} + c_upd b_t c_t^T,   y_t = (read weight) Z_t^T a_t
//
// in its own direction, with (a, b, c, y) = (q, k, v, o), (d_o, v, k, dq),
// (v, d_o, q, dk), (k, q, d_o, dv) and Z = S, S^T, G^T, G.  LinRole names one line.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_common.cuh"

namespace kda {

constexpr int kLinChunk = 128;    // tokens per chunk: the rows of one tensor-core tile
constexpr int kLinMaxRoles = 3;
// Segments per sequence up to which no scan is launched: each CTA adds up the sums before
// it itself.  Without and with the scan: two segments (B=4, T=4096, H=16) 121 and 130 us,
// four (T=4096, H=32) 75 and 78 us, eight (T=8192, H=16) 79 and 75 us, eleven (B=2,
// T=8192, H=20) 195 and 181 us, sixteen (T=4096, H=8) 48.5 and 33.1 us.
constexpr int kLinDirect = 8;

struct LinRole {
    int a, b, c;            // LinArgs::x indices of the query-, key- and value-like inputs
    void* y;                // output [tokens, H, D2], input dtype
    const float* s_in;      // state before the first processed token, nullable (zeros)
    float* s_out;           // state after the last one, nullable
    float* seg;             // [segments][pieces][H][D1 * D2]: each segment's own sum; after the scan its entering state;
                            // rows of Z with fp32 inputs, columns ([D2][D1]) with bf16
    bool transposed;        // Z is the transpose of the user's [dk, dv] states
    bool reverse;           // from the last token to the first
    float c_inter, c_intra; // y_t = c_inter lambda^.. Z_0^T a_t + c_intra sum_i lambda^.. <a_t, b_i> c_i
    float c_upd;
    int parts;              // bf16 parts of the weighted c; the role decides, so that no output depends on another being asked for
};

// Where the segments lie.  Sequences are B rows of T tokens, or packed by cu.
// A segment is a run of seg_tok tokens of one sequence (its last one may be
// short; a sequence without tokens has one empty segment).  With one segment per
// sequence a single pass over the tokens does all; otherwise a pass over keys and
// values first sums every segment's own contribution to the state, and a scan
// turns those into the states that enter each segment, so that all segments run
// at the same time.  With few segments (kLinDirect) each CTA forms its entering state
// from the sums of the segments before it, and there is no scan; then a segment may be
// summed in pieces, where the segments alone would leave SMs without work in that pass.
// Or the segments of a sequence run one after another, each starting from the state
// that the one before has left in memory (LinArgs::chained): nothing is summed twice,
// and chains that do not divide evenly among the SMs still do.
// Packed sequences: tab = [seg_tok][first segment of the r-th sequence, r = 0..N]
// [r-th sequence], longest first, so that long segments start first.
struct LinMap {
    const int32_t* cu;
    const int32_t* tab;
    int N, T;               // T: tokens per sequence, or in all when packed
    int seg_tok, num_seg;   // not packed: tokens per segment, segments per sequence
    int pieces;             // sums per segment, 1 where a scan follows

    struct Seg {
        int seq, begin, len;      // sequence, first token in the flat token order, tokens
        int index, count;         // which segment of how many of its sequence
        int size, tail;           // tokens of each of them, and of the last one
    };
    __device__ __forceinline__ int piece_tok(int size) const {   // tokens of a piece, whole chunks
        return pieces == 1 ? size : ((size + kLinChunk - 1) / kLinChunk + pieces - 1) / pieces * kLinChunk;
    }
    __device__ __forceinline__ int segments() const { return cu ? tab[1 + N] : N * num_seg; }
    __device__ __forceinline__ void range(int r, int& seq, int& first, int& count) const {   // r-th sequence's segments
        if (!cu) {
            seq = r; first = r * num_seg; count = num_seg;
            return;
        }
        seq = tab[2 + N + r]; first = tab[1 + r]; count = tab[2 + r] - first;
    }
    __device__ __forceinline__ Seg locate(int s) const {
        Seg g;
        int first, seq_begin, seq_len, size;
        if (!cu) {
            g.seq = s / num_seg; first = g.seq * num_seg;
            g.count = num_seg;
            seq_begin = g.seq * T; seq_len = T; size = seg_tok;
        } else {
            int lo = 0, hi = N - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tab[1 + mid] <= s) lo = mid; else hi = mid - 1;
            }
            range(lo, g.seq, first, g.count);
            seq_begin = cu[g.seq]; seq_len = cu[g.seq + 1] - seq_begin; size = tab[0];
        }
        g.index = s - first;
        const int off = g.index * size;          // < seq_len + size, see the host's check of T
        g.begin = seq_begin + off;
        g.len = min(size, seq_len - off);
        g.size = size;
        g.tail = seq_len - (g.count - 1) * size;
        return g;
    }
    // Segment s / pieces cut down to its piece s % pieces (len <= 0: an empty one).
    __device__ __forceinline__ Seg locate_piece(int s) const {
        Seg g = locate(s / pieces);
        const int tok = piece_tok(g.size), off = s % pieces * tok;
        g.begin += off;
        g.len = min(tok, g.len - off);
        return g;
    }
};

struct LinArgs {
    const void* x[4];             // inputs the roles name: q, k, v, d_o
    int dim[4];                   // channels of each
    const float* log_decay;       // [H], nullable (no decay)
    int H, dk, dv;
    int64_t tokens;               // in all
    bool bf16;
    LinMap map;
    int max_segments;             // host bound on map.segments()
    bool scanned;                 // sequences are cut, and the scan has turned sums into entering states
    bool chained;                 // segments take their entering state from the one before
    int* flags;                   // chained: [segments][H][roles] warps that have left their part of the state; a bit where it will not come
    int roles, slices;            // slices: column slices of the CUDA-core kernel, of the widest role
    LinRole role[kLinMaxRoles];
    WsHeader* hdr;                // null where a call needs no more workspace than this and the caller gave none
    long long wait_cap;           // test hook: cycles after which a wait gives up, one copy left out (0: neither)
    bool reset;                   // the launch starts the call: block 0 clears the status
    bool follows;                 // another kernel of the call comes before this launch
    cudaStream_t stream;
};

// What every kernel of a call begins with, before it reads or writes anything that
// another kernel of the call touches: true where the call goes on.  The
// segment table's kernel has left the status of a packed batch; otherwise the first
// launch clears it (block 0 is among the first to run, and another block records an
// error only after a wait of a second).
__device__ __forceinline__ bool lin_begin(const LinArgs& a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");    // the kernel of this call before this one has ended
    if (a.map.cu) return a.hdr->status == kStatusOk;
    if (a.reset && a.hdr && blockIdx.x == 0 && threadIdx.x == 0) {
        a.hdr->status = kStatusOk;
        a.hdr->runtime_err = 0;
    }
    return true;
}

// Powers of a head's decay: e^(l n), from a 64-bit exponent; l is kept finite so
// that l n is 0 at n = 0 also for l = -inf (a state forgotten at every token).
__device__ __forceinline__ double lin_log_decay(const float* log_decay, int h) {
    if (!log_decay) return 0.0;
    const float l = log_decay[h];
    return l < -1e30f ? -1e30 : (double)l;
}
__device__ __forceinline__ float lin_pow(double l, int n) { return (float)exp(l * (double)n); }
// The same in two fp32 parts.  A state that decays chunk after chunk takes the power's
// rounding each time, always the same one: 65,536 tokens at l = -1e-6 leave 6e-6 of it
// with one part, and nothing with two.
__device__ __forceinline__ float2 lin_pow2(double l, int n) {
    const double e = exp(l * (double)n);
    return make_float2((float)e, (float)(e - (double)(float)e));
}
// (w in two parts) * z + u
__device__ __forceinline__ float decay_add(float2 w, float z, float u) { return fmaf(w.x, z, fmaf(w.y, z, u)); }
__device__ __forceinline__ float2 decay_add(float2 w, float2 z, float2 u) {
    return fma2(make_float2(w.x, w.x), z, fma2(make_float2(w.y, w.y), z, u));
}

// The sums before segment g of a sequence, in processing order: `fold(slot, w)` is to
// make E = w E + (the sum in that slot), w in two parts, E beginning as the initial state.
template <class Fold>
__device__ __forceinline__ void lin_enter(const LinMap& map, const LinMap::Seg& g, int sidx, bool rev, double l, Fold fold) {
    const int first = sidx - g.index, n = rev ? g.count - 1 - g.index : g.index, tok = map.piece_tok(g.size);
    int w_len = 0;
    float2 w = make_float2(1.f, 0.f);
    for (int i = 0; i < n * map.pieces; ++i) {
        const int seg = rev ? g.count - 1 - i / map.pieces : i / map.pieces;
        const int piece = rev ? map.pieces - 1 - i % map.pieces : i % map.pieces;
        const int len = min(tok, (seg == g.count - 1 ? g.tail : g.size) - piece * tok);
        if (len <= 0) continue;
        if (len != w_len) w = lin_pow2(l, w_len = len);
        fold((first + seg) * map.pieces + piece, w);
    }
}

// How many of a segment's chunks, in processing order, add nothing to the state that
// leaves it: those after which so many tokens follow that the decay over them is zero
// in fp32 (e^-104 is below half the smallest number).
__device__ __forceinline__ int lin_skip(double l, int len, int chunk, int chunks, bool rev) {
    if (l > -1e-7) return 0;                       // no decay that 2^30 tokens could bring to zero
    const double reach = 104.0 / -l;               // tokens
    if (!(reach < (double)len)) return 0;         // a NaN among the decays skips nothing
    return rev ? max(chunks - 1 - (int)(reach / chunk), 0) : max((len - (int)reach - 1) / chunk, 0);
}

// Launches a kernel with more shared memory than every kernel may have.  It is allowed
// that on the current device once (`done` holds a bit for each device, above 64 every
// call asks), and again if this launch itself is refused, as after a reset of the
// device; an error that an earlier call has left says nothing about this one.  With
// `follows` the blocks may start while the kernel before, of the same call, ends; they
// wait for it in lin_begin.  T=2048, H=8: 26.8 us without, 26.0 with; five packed
// sequences 30.8 and 30.0.
inline cudaError_t lin_launch(const void* kernel, size_t grid, int threads, int smem_bytes, void** args,
                              bool follows, cudaStream_t stream, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute after{};
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem_bytes;
    c.stream = stream;
    c.attrs = &after;
    c.numAttrs = follows ? 1 : 0;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) {
        e = cudaLaunchKernelExC(&c, kernel, args);
        if (e != cudaErrorInvalidValue) return e;
        cudaGetLastError();
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
    return cudaLaunchKernelExC(&c, kernel, args);
}

cudaError_t launch_linear_prep(const LinArgs& a, int32_t* tab, int seg_tok, int balance_tokens);
cudaError_t launch_linear_scan(const LinArgs& a);
cudaError_t launch_linear_simt(const LinArgs& a, bool states_only);
cudaError_t launch_linear_tc(const LinArgs& a, bool states_only);

struct LinStepArgs {
    const void* q; const void* k; const void* v;
    const float* log_decay;       // [H], nullable
    float* state; void* o;
    int B, H, dk, dv;
    bool bf16;
    float scale;
    cudaStream_t stream;
};
cudaError_t launch_linear_step(const LinStepArgs& a);

}  // namespace kda
