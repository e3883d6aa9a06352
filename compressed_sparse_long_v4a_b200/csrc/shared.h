// shared.h -- what the kernels over a v4a_shared_cache have in common.
#pragma once

#include "common.cuh"

namespace v4a {

struct SharedArgs {
    const void* q;        // [B][n_q][H][d]
    const void* prefix;   // [n_prefix][d]
    const void* own;      // [B][own_rows][d]
    const void* ring;     // [B][ring_rows][d]
    const int32_t* own_count;
    const int32_t* own_entry;
    const int64_t* ctx_lens;
    void* out;            // [B][n_q][H][d]
    float* lse;           // [B][n_q][H] or null (attention: written; weights: read)
    const float* weights_in;
    float* weights_out;   // [B][own_rows]
    float decay;
    int* dev_status;
    const float* sink;
    v4a_dtype dtype, out_dtype;
    int batch, n_q, heads, d, m, window, own_rows, ring_rows, rope_dims;
    float rope_base;
    long long n_prefix, ctx_len;
};

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

// length of sequence b; a length outside 0 .. ctx_len counts as 0
__device__ __forceinline__ long long seq_len(const SharedArgs& a, int b) {
    if (!a.ctx_lens) return a.ctx_len;
    const long long n = a.ctx_lens[b];
    return n < 0 || n > a.ctx_len ? 0 : n;
}
// slots of sequence b that hold something
__device__ __forceinline__ int own_slots(const SharedArgs& a, int b) {
    if (!a.own_count) return a.own_rows;
    const int n = a.own_count[b];
    return n < 0 ? 0 : n > a.own_rows ? a.own_rows : n;
}
// the number of entries that a query at position t sees; 0 for one that has no candidates at all (before
// position 0, or not behind the whole prefix)
__device__ __forceinline__ long long seen_entries(const SharedArgs& a, long long t) {
    if (t < 0) return 0;
    const long long n = n_visible(t, a.m);
    return n < a.n_prefix ? 0 : n;
}
__device__ __forceinline__ bool has_candidates(const SharedArgs& a, long long t) {
    return t >= 0 && n_visible(t, a.m) >= a.n_prefix;
}
// whether a query that sees `seen` entries sees own slot i (i < own_slots) of sequence b
__device__ __forceinline__ bool slot_seen(const SharedArgs& a, int b, int i, long long seen) {
    const long long e = a.own_entry ? (long long)a.own_entry[(long long)b * a.own_rows + i] : a.n_prefix + i;
    return e >= 0 && e < seen;
}
// report what is wrong with sequence b's length or count (one thread per sequence calls this)
__device__ __forceinline__ void report_sequence(const SharedArgs& a, int b) {
    if (!a.dev_status) return;
    bool bad = false;
    long long n = a.ctx_len;
    if (a.ctx_lens) {
        n = a.ctx_lens[b];
        bad = n < 0 || n > a.ctx_len;
    }
    if (!bad && n > 0) {
        const long long t0 = n - a.n_q < 0 ? 0 : n - a.n_q;  // its first query at a position of its own
        bad = n_visible(t0, a.m) < a.n_prefix;
    }
    if (a.own_count) bad |= a.own_count[b] < 0 || a.own_count[b] > a.own_rows;
    if (bad) atomicExch(a.dev_status, (int)V4A_ERR_DEVICE_FAULT);
}

// ---- attend_shared_tc.cu (tcgen05 path: bf16, d = 512) ------------------
bool shared_tc_shape_ok(const SharedArgs& a);
size_t shared_tc_workspace_bytes(const SharedArgs& a);
cudaError_t launch_shared_tc(const SharedArgs& a, void* ws, cudaStream_t stream);

// ---- attend_weights_tc.cu (tcgen05 path: bf16) ---------------------------
cudaError_t launch_weights_tc(const SharedArgs& a, cudaStream_t stream);

}  // namespace v4a
