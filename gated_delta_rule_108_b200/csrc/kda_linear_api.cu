// kda_linear_api.cu -- the C entry points of the linear attention with one fixed
// decay per head (declared in include/kda.h): argument checks, the plan of
// segments, the workspace, the launches.
#include <algorithm>
#include <cmath>

#include "../../include/kda.h"
#include "kda_linear.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

thread_local long long g_drop_cap = 0;   // armed by kda_linear_debug_drop_copy (one call)

constexpr int kSms = 148;   // the plan and the workspace size are those of one B200

template <typename... A>
kda_status fail(kda_status st, const char* fmt, A... args) {
    return (kda_status)set_error(st, fmt, args...);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported_dim(int d) { return d == 64 || d == 128; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// How long the segments of a sequence of `chunks` chunks are, when `chains` CTAs work
// on each segment number, and in how many pieces each is summed: the cheapest by the
// count of waves over the SMs.  In units of one chunk of the chunk kernel (8,050 cycles at
// dk = dv = 128), as measured: a chunk of the summing pass 0.5, a CTA 1.5 to start and
// end (1 there), its launch 2.  Pieces only where no scan follows.  B=4, T=4096, H=16 (64
// chains of 32 chunks, two segments): 120 us in one piece, 109 in two.  The same units
// serve fp32 and d = 64: of 28 forwards and gradients of either type (1,021 to 32,768
// tokens, 4 to 64 heads and sequences, d 64 and 128), each with 1 to 32 segments, 24 came
// within 3 % of the best with the plan's choice, uncut or not (fp32, T=4096, H=8: 969 us
// uncut, 178 in the plan's eight; B=4, T=4096, H=16: 973 uncut as planned, 1,156 in two),
// and the worst at 1.18 times (fp32, d = 64, B=2, T=8192, H=20: 519 us in three, 438 in twelve).
int plan_segment_chunks(int64_t chains, int64_t chunks, double& best, int& pieces) {
    int64_t best_len = std::max<int64_t>(chunks, 1);
    best = 0;
    pieces = 1;
    for (int64_t s = 1; s <= std::min<int64_t>(chunks, 96); ++s) {
        const int64_t len = (chunks + s - 1) / s, n = (chunks + len - 1) / len;
        const double waves = std::ceil((double)(chains * n) / kSms);
        for (int r = 1; r == 1 || (r <= len && n > 1 && (n - 1) * r < kLinDirect); ++r) {
            const double sums = std::ceil((double)(chains * (n - 1) * r) / kSms);
            const double cost = waves * (len + 1.5) + (n > 1 ? sums * (0.5 * std::ceil((double)len / r) + 1.0) + 2.0 : 0.0);
            if ((s == 1 && r == 1) || cost < best) {
                best = cost;
                best_len = len;
                pieces = r;
            }
        }
    }
    return (int)best_len;
}

// The same where segments follow one another: n of them take n turns at least; 2.5 for
// a segment's start and end with the state handed on, 1 for clearing the flags.  The
// gradients at B=4, T=4096, H=16 (192 chains of 32 chunks): 283 us uncut, 229 in two,
// 222 in three, 250 in four segments.
int plan_chained_chunks(int64_t chains, int64_t chunks, double& best) {
    int64_t best_len = 0;
    for (int64_t s = 2; s <= std::min<int64_t>(chunks, 16); ++s) {
        const int64_t len = (chunks + s - 1) / s, n = (chunks + len - 1) / len;
        const double turns = std::max(std::ceil((double)(chains * n) / kSms), (double)n);
        const double cost = turns * (len + 2.5) + 1.0;
        if (best_len == 0 || cost < best) {
            best = cost;
            best_len = len;
        }
    }
    return (int)best_len;
}

struct Plan {
    int N, seg_tok, num_seg, pieces, max_segments, balance_tokens;
    bool split, chained;
    size_t tab_off, seg_off, seg_bytes, total;   // seg_bytes: one role's segment states
    size_t flag_bytes;                           // chained: the flags, where packed batches have their table
};

bool make_plan(int B, int T, int H, int dk, int dv, int num_seqs, bool varlen, kda_dtype dtype, int roles, Plan& p) {
    if (B < 0 || T < 0 || H <= 0 || !supported_dim(dk) || !supported_dim(dv)) return false;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return false;
    if (varlen && (B != 1 || num_seqs < 0)) return false;
    if ((int64_t)B * T >= (int64_t)1 << 30 || H > 65535 || (varlen ? num_seqs : B) >= 1 << 24) return false;
    p.N = varlen ? num_seqs : B;
    // CTAs per segment and head: the CUDA-core kernel takes 64 value columns each
    const int64_t per_head = (int64_t)roles * (dtype == KDA_BF16 ? 1 : std::max(dk, dv) / 64);
    const int64_t chunks = ((int64_t)T + kLinChunk - 1) / kLinChunk;
    const int64_t chains = per_head * H * (varlen ? 1 : std::max(B, 1));
    double cost = 0, cost_chained = 0;
    int len = plan_segment_chunks(chains, chunks, cost, p.pieces);
    const int len_chained = (varlen || dtype != KDA_BF16) ? 0 : plan_chained_chunks(chains, chunks, cost_chained);
    p.chained = len_chained > 0 && cost_chained < 0.95 * cost;
    if (p.chained) len = len_chained;
    p.seg_tok = std::max(len, 1) * kLinChunk;
    p.num_seg = std::max<int>(1, (int)((chunks + len - 1) / std::max(len, 1)));
    p.split = p.num_seg > 1 && !p.chained;
    // a sequence of a packed batch may have one segment more than the plan counts
    if (!p.split || p.num_seg * p.pieces > kLinDirect) p.pieces = 1;
    // packed: every sequence may end in a short segment; unsplit when the longest is
    // within 1.75 times one SM's share.  H=16, cut and not: longest at 1.2 shares (of
    // 65,536 tokens in 15 sequences) 437 and 320 us, at 1.6 428 and 408, at 3 488 and 732
    const int64_t most = varlen ? (int64_t)p.N + T / p.seg_tok : (int64_t)p.N * p.num_seg;
    if (most * p.pieces * H * per_head >= (int64_t)1 << 31) return false;
    p.max_segments = (int)most;
    p.balance_tokens = (int)std::min<int64_t>((int64_t)1 << 30, (int64_t)(1.75 * (double)T * H * per_head / kSms));
    if (!p.split) p.balance_tokens = 1 << 30;
    p.tab_off = kHeaderBytes;
    p.flag_bytes = p.chained ? sizeof(int) * (size_t)p.max_segments * H * roles : 0;
    p.seg_off = round_up(p.tab_off + (varlen ? sizeof(int32_t) * (2 * (size_t)p.N + 2) : p.flag_bytes), 256);
    p.seg_bytes = p.split || p.chained ? sizeof(float) * (size_t)p.max_segments * p.pieces * H * dk * dv : 0;
    p.total = round_up(p.seg_off + p.seg_bytes * roles, 256);
    return true;
}

kda_status check_sizes(int B, int T, int H, int dk, int dv, int num_seqs, bool varlen, kda_dtype dtype, int roles, Plan& p) {
    if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (B < 0 || T < 0 || H <= 0) return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%d T=%d H=%d", B, T, H);
    if (dk <= 0 || dv <= 0) return fail(KDA_ERR_INVALID_ARG, "bad head sizes dk=%d dv=%d", dk, dv);
    if (!supported_dim(dk) || !supported_dim(dv))
        return fail(KDA_ERR_UNSUPPORTED, "head sizes dk=%d dv=%d not in {64, 128}", dk, dv);
    if (varlen && B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1 (got B=%d)", B);
    if (varlen && num_seqs < 0) return fail(KDA_ERR_INVALID_ARG, "num_seqs=%d < 0", num_seqs);
    if (!make_plan(B, T, H, dk, dv, num_seqs, varlen, dtype, roles, p))
        return fail(KDA_ERR_UNSUPPORTED, "B=%d T=%d H=%d num_seqs=%d is too large", B, T, H, num_seqs);
    return KDA_OK;
}

kda_status check_workspace(void* workspace, size_t bytes, size_t need) {
    if (!workspace && need <= (size_t)kHeaderBytes) return KDA_OK;   // nothing but the status would be in it
    if (!workspace) return fail(KDA_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (bytes < need) return fail(KDA_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", bytes, need);
    return KDA_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const char *x = (const char*)a, *y = (const char*)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}

struct Span { const void* p; size_t bytes; };

// True where one of the `n_out` tensors overlaps another or one of the `n_in`.
bool any_overlap(const Span* out, int n_out, const Span* in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    }
    return false;
}

LinArgs common_args(const Plan& p, const float* log_decay, const int32_t* cu, int B, int T, int H, int dk, int dv,
                    kda_dtype dtype, void* workspace, void* stream) {
    LinArgs a{};
    char* ws = static_cast<char*>(workspace);
    a.log_decay = log_decay;
    a.H = H; a.dk = dk; a.dv = dv;
    a.tokens = (int64_t)B * T;
    a.bf16 = dtype == KDA_BF16;
    a.map.cu = cu;
    a.map.tab = cu ? reinterpret_cast<int32_t*>(ws + p.tab_off) : nullptr;
    a.map.N = p.N; a.map.T = T; a.map.seg_tok = p.seg_tok; a.map.num_seg = p.num_seg; a.map.pieces = 1;
    a.max_segments = p.max_segments;
    a.hdr = static_cast<WsHeader*>(workspace);
    a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

// The launches of a call: the segment table of a packed batch, the segments' sums
// and their scan where sequences are cut, the chunk kernel.
cudaError_t run_roles(const LinArgs& a, const Plan& p, char* ws) {
    LinArgs all = a;
    for (int i = 0; i < all.roles; ++i)
        all.role[i].seg = p.split || p.chained ? reinterpret_cast<float*>(ws + p.seg_off + p.seg_bytes * i) : nullptr;
    cudaError_t e = cudaSuccess;
    if (all.map.cu) e = launch_linear_prep(all, const_cast<int32_t*>(all.map.tab), p.seg_tok, p.balance_tokens);
    else if (p.max_segments == 0 && all.hdr) e = cudaMemsetAsync(all.hdr, 0, sizeof(WsHeader), all.stream);
    if (p.max_segments == 0) return e;
    if (p.chained) {
        all.chained = true;
        all.flags = reinterpret_cast<int*>(ws + p.tab_off);
        e = cudaMemsetAsync(ws, 0, p.tab_off + p.flag_bytes, all.stream);   // status, claims and flags
        return e == cudaSuccess ? launch_linear_tc(all, false) : e;
    }
    auto pass = [&](bool states_only) { return all.bf16 ? launch_linear_tc(all, states_only) : launch_linear_simt(all, states_only); };
    all.reset = true;
    all.follows = all.map.cu != nullptr;
    if (p.split && e == cudaSuccess) {
        // the most segments a sequence may have; and a state updated in place is read by the
        // scan, before the chunk kernel's last segments overwrite it
        all.scanned = (all.map.cu ? all.map.T / p.seg_tok + 1 : p.num_seg) > kLinDirect;
        for (int i = 0; i < all.roles; ++i) all.scanned |= all.role[i].s_in && all.role[i].s_in == all.role[i].s_out;
        if (!all.scanned) all.map.pieces = p.pieces;
        e = pass(true);
        all.reset = false;
        all.follows = true;
        if (e == cudaSuccess && all.scanned) e = launch_linear_scan(all);
    }
    return e == cudaSuccess ? pass(false) : e;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_linear_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int num_seqs, int varlen, kda_dtype dtype) {
    Plan p;
    return make_plan(B, T, H, dk, dv, num_seqs, varlen != 0, dtype, 1, p) ? p.total : 0;
}

size_t kda_linear_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, int num_seqs, int varlen, kda_dtype dtype) {
    Plan p;
    return make_plan(B, T, H, dk, dv, num_seqs, varlen != 0, dtype, 3, p) ? p.total : 0;
}

kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                                const float* initial_state, const int32_t* cu_seqlens, int B, int T, int H, int dk,
                                int dv, int num_seqs, kda_dtype dtype, void* o, float* final_state, void* workspace,
                                size_t workspace_bytes, void* stream) {
    Plan p;
    kda_status st = check_sizes(B, T, H, dk, dv, num_seqs, cu_seqlens != nullptr, dtype, 1, p);
    if (st != KDA_OK) return st;
    if ((int64_t)B * T > 0) {
        if (!q || !k || !v || !o) return fail(KDA_ERR_INVALID_ARG, "null input/output pointer");
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
            return fail(KDA_ERR_INVALID_ARG, "q/k/v/o must be 16-byte aligned");
    }
    const size_t es = dtype == KDA_BF16 ? 2 : 4, kbytes = (size_t)B * T * H * dk * es, vbytes = (size_t)B * T * H * dv * es;
    if (!aligned16(initial_state)) return fail(KDA_ERR_INVALID_ARG, "initial_state misaligned");
    if (!aligned16(final_state)) return fail(KDA_ERR_INVALID_ARG, "final_state misaligned");
    const size_t state_bytes = (size_t)p.N * H * dk * dv * sizeof(float);
    st = check_workspace(workspace, workspace_bytes, p.total);
    if (st != KDA_OK) return st;
    // a state may be updated in place, but not be moved by less than its size
    const Span out[] = {{o, vbytes}, {final_state, state_bytes}, {workspace, p.total}};
    const Span in[] = {{q, kbytes}, {k, kbytes}, {v, vbytes}, {initial_state != final_state ? initial_state : nullptr, state_bytes},
                       {log_decay, sizeof(float) * (size_t)H}, {cu_seqlens, sizeof(int32_t) * ((size_t)p.N + 1)}};
    if (any_overlap(out, 3, in, 6))
        return fail(KDA_ERR_INVALID_ARG, "an output or the workspace overlaps an input, another output or the workspace");

    LinArgs a = common_args(p, log_decay, cu_seqlens, B, T, H, dk, dv, dtype, workspace, stream);
    const void* x[4] = {q, k, v, nullptr};
    const int dims[4] = {dk, dk, dv, dv};
    for (int i = 0; i < 4; ++i) { a.x[i] = x[i]; a.dim[i] = dims[i]; }
    const float s = 1.0f / sqrtf((float)dk);
    a.roles = 1;
    if (a.bf16) {
        a.wait_cap = g_drop_cap;
        g_drop_cap = 0;
    }
    a.role[0] = {0, 1, 2, o, initial_state, final_state, nullptr, false, false, s, s, 1.f, 3};
    const cudaError_t e = run_roles(a, p, static_cast<char*>(workspace));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "kda_linear_chunk_fwd launch failed: %s", cudaGetErrorString(e));
    return fail(KDA_OK, "");
}

kda_status kda_linear_debug_drop_copy(long long wait_cycles) {
    if (wait_cycles < 0) return fail(KDA_ERR_INVALID_ARG, "wait_cycles=%lld < 0", wait_cycles);
    g_drop_cap = wait_cycles;
    return fail(KDA_OK, "");
}

kda_status kda_linear_chunk_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                                const float* initial_state, const int32_t* cu_seqlens, const void* d_o,
                                const float* d_final_state, int B, int T, int H, int dk, int dv, int num_seqs,
                                kda_dtype dtype, void* dq, void* dk_out, void* dv_out, float* d_initial_state,
                                void* workspace, size_t workspace_bytes, void* stream) {
    Plan p;
    kda_status st = check_sizes(B, T, H, dk, dv, num_seqs, cu_seqlens != nullptr, dtype, 3, p);
    if (st != KDA_OK) return st;
    if ((int64_t)B * T > 0) {
        if (!q || !k || !v || !d_o || !dq || !dk_out || !dv_out) return fail(KDA_ERR_INVALID_ARG, "null input/output pointer");
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(d_o) || !aligned16(dq) || !aligned16(dk_out) ||
            !aligned16(dv_out))
            return fail(KDA_ERR_INVALID_ARG, "q/k/v/d_o/dq/dk/dv must be 16-byte aligned");
    }
    const size_t es = dtype == KDA_BF16 ? 2 : 4, kbytes = (size_t)B * T * H * dk * es, vbytes = (size_t)B * T * H * dv * es;
    if (!aligned16(initial_state)) return fail(KDA_ERR_INVALID_ARG, "initial_state misaligned");
    if (!aligned16(d_final_state)) return fail(KDA_ERR_INVALID_ARG, "d_final_state misaligned");
    if (!aligned16(d_initial_state)) return fail(KDA_ERR_INVALID_ARG, "d_initial_state misaligned");
    const size_t state_bytes = (size_t)p.N * H * dk * dv * sizeof(float);
    st = check_workspace(workspace, workspace_bytes, p.total);
    if (st != KDA_OK) return st;
    const Span out[] = {{dq, kbytes}, {dk_out, kbytes}, {dv_out, vbytes}, {d_initial_state, state_bytes}, {workspace, p.total}};
    const Span in[] = {{q, kbytes}, {k, kbytes}, {v, vbytes}, {d_o, vbytes}, {initial_state, state_bytes}, {d_final_state, state_bytes},
                       {log_decay, sizeof(float) * (size_t)H}, {cu_seqlens, sizeof(int32_t) * ((size_t)p.N + 1)}};
    if (any_overlap(out, 5, in, 8))
        return fail(KDA_ERR_INVALID_ARG, "a gradient or the workspace overlaps an input, another gradient or the workspace");

    LinArgs a = common_args(p, log_decay, cu_seqlens, B, T, H, dk, dv, dtype, workspace, stream);
    const void* x[4] = {q, k, v, d_o};
    const int dims[4] = {dk, dk, dv, dv};
    for (int i = 0; i < 4; ++i) { a.x[i] = x[i]; a.dim[i] = dims[i]; }
    const float s = 1.0f / sqrtf((float)dk);
    a.roles = 3;
    a.role[0] = {3, 2, 1, dq, initial_state, nullptr, nullptr, true, false, s, s, 1.f, 2};
    a.role[1] = {2, 3, 0, dk_out, d_final_state, nullptr, nullptr, true, true, 1.f, s, s, 2};
    a.role[2] = {1, 0, 3, dv_out, d_final_state, d_initial_state, nullptr, false, true, 1.f, s, s, 3};
    const cudaError_t e = run_roles(a, p, static_cast<char*>(workspace));
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "kda_linear_chunk_bwd launch failed: %s", cudaGetErrorString(e));
    return fail(KDA_OK, "");
}

kda_status kda_linear_recurrent_step(const void* q, const void* k, const void* v, const float* log_decay,
                                     float* state_inout, int B, int H, int dk, int dv, kda_dtype dtype, void* o,
                                     void* stream) {
    if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (B < 0 || H <= 0 || dk <= 0 || dv <= 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%d H=%d dk=%d dv=%d", B, H, dk, dv);
    if (!supported_dim(dk) || !supported_dim(dv))
        return fail(KDA_ERR_UNSUPPORTED, "head sizes dk=%d dv=%d not in {64, 128}", dk, dv);
    if ((int64_t)B * H >= (int64_t)1 << 28) return fail(KDA_ERR_UNSUPPORTED, "state too large");
    if (B > 0) {
        if (!q || !k || !v || !state_inout || !o) return fail(KDA_ERR_INVALID_ARG, "null pointer");
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_inout) || !aligned16(o))
            return fail(KDA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
        const size_t es = dtype == KDA_BF16 ? 2 : 4, kbytes = (size_t)B * H * dk * es, vbytes = (size_t)B * H * dv * es;
        const Span out[] = {{o, vbytes}, {state_inout, (size_t)B * H * dk * dv * sizeof(float)}};
        const Span in[] = {{q, kbytes}, {k, kbytes}, {v, vbytes}, {log_decay, sizeof(float) * (size_t)H}};
        if (any_overlap(out, 2, in, 4)) return fail(KDA_ERR_INVALID_ARG, "o or the state overlaps another tensor");
    }
    LinStepArgs a{};
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.state = state_inout; a.o = o;
    a.B = B; a.H = H; a.dk = dk; a.dv = dv;
    a.bf16 = dtype == KDA_BF16;
    a.scale = 1.0f / sqrtf((float)dk);
    a.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_linear_step(a);
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "kda_linear_recurrent_step launch failed: %s", cudaGetErrorString(e));
    return fail(KDA_OK, "");
}

}  // extern "C"
