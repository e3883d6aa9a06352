// attend_shared.cu -- HCA attention over a prefix that a batch shares, entries of each sequence's own and the
// window, and the weights that the own entries receive: entry points, and the CUDA-core kernels
// (fp32; attention also bf16 with d < 512).
//
//     out = sum_r p_r v_r,  p = softmax_r(q . v_r / sqrt(d)),  lse = log sum_r e^{q . v_r / sqrt(d)}
//
// over the prefix, the own entries that the query sees, and the window.  Every query of the batch sees
// the whole prefix, so for it the queries and heads of all sequences are just rows of one matrix: they are
// taken in groups that ignore where one sequence ends, and a prefix row that has been loaded serves a
// whole group.  The own entries and the window go by query.  The two kinds of work are cut into pieces
// along the keys, each with its running maximum m, sum l and unnormalised output, and joined at the
// end: out = sum_i e^{m_i - m} o_i / sum_i e^{m_i - m} l_i.
//
// CUDA-core kernels: a block takes 16 rows (4 per warp) and tiles of 32 keys staged as fp32 in shared
// memory (fp32 by asynchronous copies, all of a tile in flight).  For the scores a lane is a key; for the output it is a
// slice of d, and each probability is broadcast from the lane that has it.  4 rows per warp mean 16 FMAs per
// 16-byte read of a key, which the FMA pipes bound in long calls; short ones are bound by their two launches.  Products and
// sums in fp32 throughout.  3 sequences of 16 heads, d = 128, over 1,000 entries: 9.3 us (split 5.9, join 3.6, or 5.1 if
// no piece's output is loaded before the weights are known); the weights of 500 slots 4.5 us.
#include "common.cuh"
#include "internal.h"
#include "shared.h"
#include "tc_pair.cuh"
#include "tensor_map.h"
#include "turns.h"

#include <type_traits>

namespace v4a {
namespace {

constexpr int kRowsB = 16;    // rows per block
constexpr int kKeys = 32;     // keys per tile
constexpr int kThreads = 128;
constexpr int kRw = 4;        // rows per warp

struct SimtPlan {
    int groups;            // row groups of the prefix part
    int splits;            // its pieces per group
    int head_tiles;        // row groups per query of the own part
    int own_splits;        // its pieces
    int own_keys;          // own_rows + window
    long long rows;        // batch * n_q * heads
};

template <typename T, int D>
struct __align__(16) Tile {
    float k[kKeys][D + 4];
    float q[kRowsB][D];
    const T* src[kKeys];  // null: a key that no row sees
};

// Rows of D elements as fp32 in shared memory, by a block of N threads: row i from src(i) (null: zeros).  The copies of
// all rows are in flight together (fp32: asynchronous; the caller waits for them).
template <typename T, int D, int N, int STRIDE, typename F>
__device__ __forceinline__ void stage_rows(float (*dst)[STRIDE], int rows, const T* any, F src) {
    if constexpr (sizeof(T) == 4) {
        constexpr int kC = D / 4;
#pragma unroll 4
        for (int i = threadIdx.x; i < rows * kC; i += N) {
            const int r = i / kC, c = i % kC * 4;
            const T* p = src(r);
            tc::cp_async_16_or_zero(&dst[r][c], p ? p + c : any, p != nullptr);
        }
    } else {
        constexpr int kC = D / 8, kU = 4;
        for (int i0 = threadIdx.x; i0 < rows * kC; i0 += kU * N) {
            float f[kU][8];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = i0 + u * N;
                const T* p = i < rows * kC ? src(i / kC) : nullptr;
#pragma unroll
                for (int e = 0; e < 8; ++e) f[u][e] = 0.f;
                if (p) Vec8<T>::load_nc(p + i % kC * 8, f[u]);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = i0 + u * N;
                if (i < rows * kC) Vec8<float>::store(&dst[i / kC][i % kC * 8], f[u]);
            }
        }
    }
}

// this lane's key against the warp's four rows
template <int D>
__device__ __forceinline__ void dots(const float* key, const float (*q)[D], float (&s)[kRw]) {
#pragma unroll
    for (int r = 0; r < kRw; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        const float4 k = *reinterpret_cast<const float4*>(key + c);
#pragma unroll
        for (int r = 0; r < kRw; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(&q[r][c]);
            s[r] = fmaf(x.x, k.x, s[r]);
            s[r] = fmaf(x.y, k.y, s[r]);
            s[r] = fmaf(x.z, k.z, s[r]);
            s[r] = fmaf(x.w, k.w, s[r]);
        }
    }
}

// One piece: 16 rows against a range of keys.  Blocks below groups * splits take prefix pieces, the others
// own-and-window pieces.  A piece's rows go to part_ml / part_o [piece][16] (see piece_of).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) shared_split_kernel(SharedArgs a, SimtPlan p, float2* part_ml, float* part_o) {
    griddep_wait();  // everything before this kernel on the stream has finished
    griddep_launch_dependents();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Tile<T, D>& sm = *reinterpret_cast<Tile<T, D>*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long piece = blockIdx.x;
    const long long n_pre = (long long)p.groups * p.splits;
    const bool pre = piece < n_pre;
    long long row0, k0, k1, t = 0, seen = 0;
    int n_rows, b = 0, count = 0;
    if (pre) {
        const long long g = piece / p.splits;
        const int sp = (int)(piece % p.splits);
        row0 = g * kRowsB;
        n_rows = (int)(p.rows - row0 < kRowsB ? p.rows - row0 : kRowsB);
        const long long per = (a.n_prefix + p.splits - 1) / p.splits;
        k0 = sp * per;
        k1 = k0 + per < a.n_prefix ? k0 + per : a.n_prefix;
    } else {
        long long i = piece - n_pre;
        const int sp = (int)(i % p.own_splits);
        i /= p.own_splits;
        const int ht = (int)(i % p.head_tiles);
        const long long query = i / p.head_tiles;
        b = (int)(query / a.n_q);
        row0 = query * a.heads + ht * kRowsB;
        n_rows = a.heads - ht * kRowsB < kRowsB ? a.heads - ht * kRowsB : kRowsB;
        t = seq_len(a, b) - a.n_q + query % a.n_q;
        seen = seen_entries(a, t);
        count = own_slots(a, b);
        const int per = (p.own_keys + p.own_splits - 1) / p.own_splits;
        k0 = (long long)sp * per;
        k1 = k0 + per < p.own_keys ? k0 + per : p.own_keys;
        if (!has_candidates(a, t)) k1 = k0;
    }
    const T* const q = static_cast<const T*>(a.q);
    stage_rows<T, D, kThreads>(sm.q, kRowsB, q, [&](int r) { return r < n_rows ? q + (row0 + r) * D : nullptr; });
    constexpr int kE = D / 32;  // output elements per lane and row, in groups of 4 (2 for D = 64)
    constexpr int kV = kE < 4 ? kE : 4;
    float o[kRw][kE], m_run[kRw], l_run[kRw];
#pragma unroll
    for (int r = 0; r < kRw; ++r) {
        m_run[r] = -INFINITY;
        l_run[r] = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) o[r][e] = 0.f;
    }
    const float scale = kLog2eF / sqrtf((float)D);
    for (long long base = k0; base < k1; base += kKeys) {
        __syncthreads();
        if (threadIdx.x < kKeys) {
            const long long c = base + threadIdx.x;
            const T* src = nullptr;
            if (c < k1) {
                if (pre) {
                    src = static_cast<const T*>(a.prefix) + c * D;
                } else if (c < a.own_rows) {
                    if (c < count && slot_seen(a, b, (int)c, seen)) src = static_cast<const T*>(a.own) + ((long long)b * a.own_rows + c) * D;
                } else {
                    const long long pos = t - a.window + 1 + (c - a.own_rows);
                    if (pos >= 0) src = static_cast<const T*>(a.ring) + ((long long)b * a.ring_rows + pos % a.ring_rows) * D;
                }
            }
            sm.src[threadIdx.x] = src;
        }
        __syncthreads();
        stage_rows<T, D, kThreads>(sm.k, kKeys, q, [&](int r) { return sm.src[r]; });
        tc::cp_async_commit();
        tc::cp_async_wait<0>();
        __syncthreads();
        float s[kRw];
        dots<D>(sm.k[lane], &sm.q[warp * kRw], s);
        const bool ok = sm.src[lane] != nullptr;
#pragma unroll
        for (int r = 0; r < kRw; ++r) {
            const float x = ok ? s[r] * scale : -INFINITY;
            const float mt = group_max<32>(x), m_new = fmaxf(m_run[r], mt);
            const float msub = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = exp2f(m_run[r] - msub);
            s[r] = exp2f(x - msub);
            l_run[r] = l_run[r] * alpha + s[r];  // each lane's own share of the row sum
            m_run[r] = m_new;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[r][e] *= alpha;
        }
        for (int j = 0; j < kKeys; ++j) {
            float v[kE], pj[kRw];
#pragma unroll
            for (int g = 0; g < kE / kV; ++g) {
                const float* vp = &sm.k[j][g * 32 * kV + lane * kV];
#pragma unroll
                for (int e = 0; e < kV; ++e) v[g * kV + e] = vp[e];
            }
#pragma unroll
            for (int r = 0; r < kRw; ++r) pj[r] = __shfl_sync(0xffffffffu, s[r], j);
#pragma unroll
            for (int r = 0; r < kRw; ++r)
#pragma unroll
                for (int e = 0; e < kE; ++e) o[r][e] = fmaf(pj[r], v[e], o[r][e]);
        }
    }
    tc::cp_async_commit();  // of a piece without keys
    tc::cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < kRw; ++r) {
        const float l = group_sum<32>(l_run[r]);
        const long long pr = piece * kRowsB + warp * kRw + r;
        if (lane == 0) part_ml[pr] = make_float2(isnan(l) ? NAN : m_run[r], l);  // a NaN logit poisons its row
        float* op = part_o + pr * D;
#pragma unroll
        for (int g = 0; g < kE / kV; ++g)
#pragma unroll
            for (int e = 0; e < kV; ++e) op[g * 32 * kV + lane * kV + e] = o[r][g * kV + e];
    }
}

// One block per row (query, head) joins its pieces: their maxima and sums a thread each, then a warp takes every
// fourth piece, a lane four neighbouring dims of each 128, with several pieces in flight.
constexpr int kMaxPieces = 2 * 1024;

__device__ __forceinline__ float block_reduce(float x, float* red, bool max) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = !max ? x + y : isnan(x) || isnan(y) ? NAN : fmaxf(x, y);
    }
    __syncthreads();
    if (lane == 0) red[warp] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) x = !max ? x + red[w] : isnan(x) || isnan(red[w]) ? NAN : fmaxf(x, red[w]);
    return x;
}

__global__ void __launch_bounds__(kThreads) shared_join_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ SimtPlan p,
                                                               const __grid_constant__ Turns turns, const float2* part_ml, const float* part_o) {
    const bool f32 = a.out_dtype == V4A_F32;
    griddep_wait();
    // bf16 rows may be the first query of an attention kernel, which reads it before it waits for this grid: it is let
    // in when they have reached L2
    if (f32) griddep_launch_dependents();
    __shared__ float w[kMaxPieces];  // weight of every piece
    __shared__ __align__(16) float sum[kThreads / 32][512];
    __shared__ float red[kThreads / 32];
    const long long row = blockIdx.x;
    const int d = a.d, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long query = row / a.heads;
    const int h = (int)(row % a.heads), b = (int)(query / a.n_q);
    const long long t = seq_len(a, b) - a.n_q + query % a.n_q;
    const bool live = has_candidates(a, t);
    const int n_pre = p.groups ? p.splits : 0, n = live ? n_pre + p.own_splits : 0;
    // row of piece i in part_ml / part_o
    const long long row_pre = (row / kRowsB) * p.splits * kRowsB + row % kRowsB;
    const long long row_own = ((long long)p.groups * p.splits + (query * p.head_tiles + h / kRowsB) * p.own_splits) * kRowsB + h % kRowsB;
    auto piece_row = [&](int i) -> long long { return i < n_pre ? row_pre + (long long)i * kRowsB : row_own + (long long)(i - n_pre) * kRowsB; };
    if (threadIdx.x == 0 && h == 0 && query % a.n_q == 0) report_sequence(a, b);
    // the first pieces' outputs are on their way while the weights are worked out
    constexpr int kAhead = 10;  // of each warp, in registers
    float4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = warp + k * (kThreads / 32);
        ahead[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n && lane * 4 < d) ahead[k] = __ldcg(reinterpret_cast<const float4*>(part_o + piece_row(i) * d + lane * 4));
    }
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const float x = part_ml[piece_row(i)].x;
        m = isnan(x) || isnan(m) ? NAN : fmaxf(m, x);
    }
    m = block_reduce(m, red, true);
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const float2 ml = part_ml[piece_row(i)];
        w[i] = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);  // of an empty piece: 0
        if (ml.x != -INFINITY) l += w[i] * ml.y;
    }
    l = block_reduce(l, red, false);  // behind its barriers every weight is written
    float keep = 1.f;
    if (a.sink && m != -INFINITY) {
        const float s = a.sink[h] * kLog2eF;
        if (s > m && s < INFINITY) {  // the sink outweighs every key: it becomes the reference
            keep = exp2f(m - s);
            l *= keep;
            m = s;
        }
        l += exp2f(s - m);
    }
    const float inv = l > 0.f ? keep / l : (l == 0.f ? 0.f : l);  // NaN stays
    if (threadIdx.x == 0 && a.lse) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2F : (l == 0.f ? -INFINITY : l);
    for (int e = lane * 4; e < d; e += 128) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        int from = warp;
        if (e == lane * 4) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = warp + k * (kThreads / 32);
                const float wi = i < n ? w[i] : 0.f;
                o.x = fmaf(wi, ahead[k].x, o.x);
                o.y = fmaf(wi, ahead[k].y, o.y);
                o.z = fmaf(wi, ahead[k].z, o.z);
                o.w = fmaf(wi, ahead[k].w, o.w);
            }
            from += kAhead * (kThreads / 32);
        }
#pragma unroll 4
        for (int i = from; i < n; i += kThreads / 32) {
            const float wi = w[i];
            const float4 v = __ldcg(reinterpret_cast<const float4*>(part_o + piece_row(i) * d + e));
            o.x = fmaf(wi, v.x, o.x);
            o.y = fmaf(wi, v.y, o.y);
            o.z = fmaf(wi, v.z, o.z);
            o.w = fmaf(wi, v.w, o.w);
        }
        *reinterpret_cast<float4*>(&sum[warp][e]) = o;
    }
    __syncthreads();
    const int r0 = d - a.rope_dims;
    for (int e = threadIdx.x * 2; e < d; e += 2 * kThreads) {
        float x = ((sum[0][e] + sum[1][e]) + (sum[2][e] + sum[3][e])) * inv;
        float y = ((sum[0][e + 1] + sum[1][e + 1]) + (sum[2][e + 1] + sum[3][e + 1])) * inv;
        if (a.rope_dims > 0 && e >= r0 && live) {
            const float2 r = turn((double)t, turns.hi[(e - r0) >> 1], turns.lo[(e - r0) >> 1]);
            const float u = x;
            x = fmaf(u, r.x, y * r.y);  // back by the position
            y = fmaf(y, r.x, -u * r.y);
        }
        if (a.out_dtype == V4A_F32) {
            *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * d + e) = make_float2(x, y);
        } else {
            *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + row * d + e) = __floats2bfloat162_rn(x, y);
        }
    }
    if (!f32) __threadfence();
}

// Weights, fp32: a block takes 32 own slots of one sequence and runs over the sequence's rows (query, head), 32 at
// a time.  A warp's lane is a slot; the eight warps' sums are added in a fixed order.
constexpr int kWThreads = 256;
constexpr int kWRows = kWThreads / 32 * kRw;

template <int D>
struct __align__(16) WeightTile {
    float k[kKeys][D + 4];
    float q[kWRows][D];
    float lse[kWRows];      // -inf: no candidates, or no such row
    long long seen[kWRows];
    float sums[kWThreads / 32][kKeys];
};

template <int D>
__global__ void __launch_bounds__(kWThreads) weights_kernel(SharedArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    WeightTile<D>& sm = *reinterpret_cast<WeightTile<D>*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, i0 = blockIdx.x * kKeys, count = own_slots(a, b);
    if (blockIdx.x == 0 && threadIdx.x == 0) report_sequence(a, b);
    if (i0 >= count) return;
    const float* const q = static_cast<const float*>(a.q);
    const float* const own = static_cast<const float*>(a.own) + ((long long)b * a.own_rows + i0) * D;
    const int n = a.n_q * a.heads;
    const long long row0 = (long long)b * n;
    stage_rows<float, D, kWThreads>(sm.k, kKeys, q, [&](int r) { return i0 + r < count ? own + (long long)r * D : nullptr; });
    const int slot = i0 + lane;
    const long long at = (long long)b * a.own_rows + slot;
    long long e = -1;  // this lane's entry
    float before = 0.f;
    if (slot < count) {
        e = a.own_entry ? (long long)a.own_entry[at] : a.n_prefix + slot;
        if (warp == 0 && a.decay != 0.f) before = a.weights_in[at];
    }
    const long long len = seq_len(a, b);
    const float scale = 1.f / sqrtf((float)D);
    float got = 0.f;
    for (int base = 0; base < n; base += kWRows) {
        __syncthreads();
        stage_rows<float, D, kWThreads>(sm.q, kWRows, q, [&](int r) { return base + r < n ? q + (row0 + base + r) * D : nullptr; });
        if (threadIdx.x < kWRows) {
            const int i = base + threadIdx.x;
            sm.lse[threadIdx.x] = i < n ? a.lse[row0 + i] : -INFINITY;
            sm.seen[threadIdx.x] = i < n ? seen_entries(a, len - a.n_q + i / a.heads) : 0;
        }
        tc::cp_async_commit();
        tc::cp_async_wait<0>();
        __syncthreads();
        float s[kRw];
        dots<D>(sm.k[lane], &sm.q[warp * kRw], s);
#pragma unroll
        for (int r = 0; r < kRw; ++r) {
            const float lse = sm.lse[warp * kRw + r];
            // lse off the logit in one rounding, before the exponent's log2 e (lse log2 e, rounded, costs |lse| 2^-24 of the weight)
            if (e >= 0 && e < sm.seen[warp * kRw + r] && lse != -INFINITY) got += exp2f(fmaf(s[r], scale, -lse) * kLog2eF);
        }
    }
    sm.sums[warp][lane] = got;
    __syncthreads();
    if (warp == 0 && slot < count) {
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWThreads / 32; ++w) total += sm.sums[w][lane];
        a.weights_out[at] = a.decay == 0.f ? total : fmaf(a.decay, before, total);
    }
}

SimtPlan simt_plan(const SharedArgs& a) {
    SimtPlan p;
    p.rows = (long long)a.batch * a.n_q * a.heads;
    p.groups = a.n_prefix > 0 ? (int)((p.rows + kRowsB - 1) / kRowsB) : 0;
    p.head_tiles = (a.heads + kRowsB - 1) / kRowsB;
    p.own_keys = a.own_rows + a.window;
    const long long queries = (long long)a.batch * a.n_q;
    auto cut = [](long long pieces, long long keys) {  // enough blocks for the SMs, 32 keys each at least
        long long want = pieces > 0 ? (4LL * kNumSMs + pieces - 1) / pieces : 1, most = (keys + kKeys - 1) / kKeys;
        if (want > most) want = most;
        return (int)(want < 1 ? 1 : want > 1024 ? 1024 : want);
    };
    p.splits = p.groups ? cut(p.groups, a.n_prefix) : 0;
    p.own_splits = p.own_keys > 0 ? cut(queries * p.head_tiles, p.own_keys) : 0;
    return p;
}

long long simt_pieces(const SharedArgs& a, const SimtPlan& p) {
    return (long long)p.groups * p.splits + (long long)a.batch * a.n_q * p.head_tiles * p.own_splits;
}

size_t simt_bytes(const SharedArgs& a) {
    const long long n = simt_pieces(a, simt_plan(a)) * kRowsB;
    return align256(n * sizeof(float2)) + n * a.d * sizeof(float);
}

template <typename T, int D>
cudaError_t simt_attend(const SharedArgs& a, void* ws, cudaStream_t st) {
    const SimtPlan p = simt_plan(a);
    const long long pieces = simt_pieces(a, p);
    float2* ml = static_cast<float2*>(ws);
    float* po = reinterpret_cast<float*>(static_cast<char*>(ws) + align256(pieces * kRowsB * sizeof(float2)));
    auto* kernel = shared_split_kernel<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Tile<T, D>));
    if (e == cudaSuccess && pieces > 0)
        e = launch_pdl(kernel, dim3((unsigned)pieces), dim3(kThreads), sizeof(Tile<T, D>), st, a, p, ml, po);
    if (e == cudaSuccess)
    {
        Turns turns;
        if (a.rope_dims > 0) make_turns(a.rope_dims, a.rope_base, &turns);
        e = launch_pdl(shared_join_kernel, dim3((unsigned)p.rows), dim3(kThreads), 0, st, a, p, turns, (const float2*)ml, (const float*)po);
    }
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D>
cudaError_t simt_weights(const SharedArgs& a, cudaStream_t st) {
    auto* kernel = weights_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(WeightTile<D>));
    if (e == cudaSuccess)
        e = launch_pdl(kernel, dim3((unsigned)((a.own_rows + kKeys - 1) / kKeys), (unsigned)a.batch), dim3(kWThreads),
                       sizeof(WeightTile<D>), st, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename F>
cudaError_t by_shape(const SharedArgs& a, F f) {
    const bool f32 = a.dtype == V4A_F32;
    switch (a.d) {
    case 64: return f32 ? f(0.f, std::integral_constant<int, 64>()) : f(__nv_bfloat16(), std::integral_constant<int, 64>());
    case 128: return f32 ? f(0.f, std::integral_constant<int, 128>()) : f(__nv_bfloat16(), std::integral_constant<int, 128>());
    case 256: return f32 ? f(0.f, std::integral_constant<int, 256>()) : f(__nv_bfloat16(), std::integral_constant<int, 256>());
    default: return f(0.f, std::integral_constant<int, 512>());  // bf16: the tensor-core kernels
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int kMaxRows = 0x3fffffff;  // of the prefix, of a sequence's slots, of the window
bool dims_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }

// the checks that both calls share; fills everything but the outputs
v4a_status shared_args(const char* what, const void* q, const v4a_shared_cache* c, v4a_dtype dtype, int* dev_status,
                       const v4a_shape* s, SharedArgs* a) {
    if (!s || !c) return report(V4A_ERR_INVALID_ARG, "%s: shape or cache is NULL", what);
    if (s->batch < 0 || s->n_q < 1 || s->m < 1 || s->ctx_len < 1 || s->n_q > s->ctx_len)
        return report(V4A_ERR_INVALID_ARG, "%s: need batch >= 0, m >= 1, 1 <= n_q <= ctx_len", what);
    if ((long long)s->batch * s->n_q > 65535) return report(V4A_ERR_UNSUPPORTED, "%s: batch * n_q must be <= 65535", what);
    if (s->heads < 1 || s->heads > 1024) return report(V4A_ERR_INVALID_ARG, "%s: heads must be in 1..1024", what);
    if (!dims_ok(s->d))
        return report(V4A_ERR_UNSUPPORTED, "%s: d must be 64, 128, 256 or 512", what);
    if (dtype != V4A_F32 && dtype != V4A_BF16) return report(V4A_ERR_UNSUPPORTED, "%s: dtype must be F32 or BF16", what);
    if (c->n_prefix < 0 || c->n_prefix > s->ctx_len / s->m || c->n_prefix > kMaxRows)
        return report(V4A_ERR_INVALID_ARG, "%s: n_prefix must be in 0..ctx_len / m", what);
    if (c->own_rows < 0 || c->own_rows > kMaxRows) return report(V4A_ERR_INVALID_ARG, "%s: own_rows out of range", what);
    if (s->window < 0 || s->window > kMaxRows) return report(V4A_ERR_INVALID_ARG, "%s: window must be >= 0", what);
    if (c->n_prefix + (long long)s->batch * ((long long)c->own_rows + s->window + s->n_q) >= 1LL << 31)
        return report(V4A_ERR_UNSUPPORTED, "%s: n_prefix + batch * (own_rows + window + n_q) must be < 2^31", what);
    if (s->batch > 0 && (!q || (c->own_rows > 0 && !c->own))) return report(V4A_ERR_INVALID_ARG, "%s: q and own are required", what);
    if (!aligned(q, 16) || !aligned(c->own, 16) || !aligned(c->prefix, 16) || !aligned(c->ring, 16))
        return report(V4A_ERR_INVALID_ARG, "%s: q, prefix, own and ring must be 16-byte aligned", what);
    if (!aligned(c->own_count, 4) || !aligned(c->own_entry, 4) || !aligned(c->ctx_lens, 8) || !aligned(dev_status, 4))
        return report(V4A_ERR_INVALID_ARG, "%s: own_count, own_entry, ctx_lens or dev_status misaligned", what);
    *a = SharedArgs{};
    a->q = q;
    a->prefix = c->prefix;
    a->own = c->own;
    a->ring = c->ring;
    a->own_count = c->own_count;
    a->own_entry = c->own_entry;
    a->ctx_lens = c->ctx_lens;
    a->dev_status = dev_status;
    a->dtype = dtype;
    a->batch = s->batch;
    a->n_q = s->n_q;
    a->heads = s->heads;
    a->d = s->d;
    a->m = s->m;
    a->own_rows = c->own_rows;
    a->ring_rows = c->ring_rows;
    a->n_prefix = c->n_prefix;
    a->ctx_len = s->ctx_len;
    return V4A_OK;
}

v4a_status from_cuda(cudaError_t e, const char* what) {
    return e == cudaSuccess ? V4A_OK : report(V4A_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace v4a

extern "C" {

v4a_status v4a_hca_attend_shared(const void* q, const v4a_shared_cache* cache, void* out, v4a_dtype out_dtype,
                                 float* lse, v4a_dtype dtype, void* workspace, size_t workspace_bytes,
                                 int* dev_status, const v4a_attend_ext* ext, const v4a_shape* shape, void* stream) {
    using namespace v4a;
    const char* what = "v4a_hca_attend_shared";
    SharedArgs a;
    const v4a_status st = shared_args(what, q, cache, dtype, dev_status, shape, &a);
    if (st != V4A_OK) return st;
    a.window = shape->window;
    if (a.batch == 0) return V4A_OK;
    if (!out) return report(V4A_ERR_INVALID_ARG, "%s: out is required", what);
    if (a.n_prefix > 0 && !a.prefix) return report(V4A_ERR_INVALID_ARG, "%s: prefix is required", what);
    if (out_dtype != V4A_F32 && !(out_dtype == V4A_BF16 && dtype == V4A_BF16))
        return report(V4A_ERR_UNSUPPORTED, "%s: out_dtype must be F32, or BF16 with BF16 inputs", what);
    if (!aligned(out, 16) || !aligned(lse, 4)) return report(V4A_ERR_INVALID_ARG, "%s: out (16 bytes) or lse (4 bytes) misaligned", what);
    if (a.window > 0 && (!a.ring || a.ring_rows < 1 || (long long)a.ring_rows < (long long)a.window + a.n_q - 1))
        return report(V4A_ERR_INVALID_ARG, "%s: the ring of %d rows cannot hold the window (%d + %d - 1)", what,
                      a.ring ? a.ring_rows : 0, a.window, a.n_q);
    if (ext) {
        if (ext->rope_dims < 0 || ext->rope_dims > a.d || (ext->rope_dims & 1))
            return report(V4A_ERR_INVALID_ARG, "%s: rope_dims must be even and in 0..d", what);
        if (ext->rope_dims > 0 && !(ext->rope_base > 0.f)) return report(V4A_ERR_INVALID_ARG, "%s: rope_base must be > 0", what);
        if (!aligned(ext->sink, 4)) return report(V4A_ERR_INVALID_ARG, "%s: sink must be 4-byte aligned", what);
        a.sink = ext->sink;
        a.rope_dims = ext->rope_dims;
        a.rope_base = ext->rope_base;
    }
    a.out = out;
    a.out_dtype = out_dtype;
    a.lse = lse;
    const size_t need = v4a_shared_workspace_size(shape, a.n_prefix, a.own_rows, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return report(V4A_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    if (!aligned(workspace, 256)) return report(V4A_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (const cudaError_t e = bind_context(); e != cudaSuccess) return from_cuda(e, what);
    cudaStream_t s = (cudaStream_t)stream;
    if (dev_status) {
        const cudaError_t e = launch_zero_words(reinterpret_cast<uint32_t*>(dev_status), 1, s);
        if (e != cudaSuccess) return from_cuda(e, "dev_status reset");
    }
    if (shared_tc_shape_ok(a)) return from_cuda(launch_shared_tc(a, workspace, s), what);
    return from_cuda(by_shape(a, [&](auto t, auto d) { return simt_attend<decltype(t), decltype(d)::value>(a, workspace, s); }), what);
}

size_t v4a_shared_workspace_size(const v4a_shape* shape, long long n_prefix, int own_rows, v4a_dtype dtype) {
    using namespace v4a;
    if (!shape || shape->batch < 1 || shape->n_q < 1 || (long long)shape->batch * shape->n_q > 65535 || shape->heads < 1 ||
        shape->heads > 1024 || !dims_ok(shape->d) || (dtype != V4A_F32 && dtype != V4A_BF16) || n_prefix < 0 || n_prefix > kMaxRows ||
        own_rows < 0 || own_rows > kMaxRows || shape->window < 0 || shape->window > kMaxRows ||
        n_prefix + (long long)shape->batch * ((long long)own_rows + shape->window + shape->n_q) >= 1LL << 31)
        return 0;
    SharedArgs a = {};
    a.batch = shape->batch;
    a.n_q = shape->n_q;
    a.heads = shape->heads;
    a.d = shape->d;
    a.window = shape->window;
    a.own_rows = own_rows;
    a.n_prefix = n_prefix;
    a.dtype = dtype;
    return shared_tc_shape_ok(a) ? shared_tc_workspace_bytes(a) : simt_bytes(a);
}

v4a_status v4a_attend_weights(const void* q, const v4a_shared_cache* cache, const float* lse, const float* weights_in,
                              float* weights_out, float decay, v4a_dtype dtype, int* dev_status, const v4a_shape* shape,
                              void* stream) {
    using namespace v4a;
    const char* what = "v4a_attend_weights";
    SharedArgs a;
    const v4a_status st = shared_args(what, q, cache, dtype, dev_status, shape, &a);
    if (st != V4A_OK) return st;
    if (!(decay >= 0.f) || isinf(decay)) return report(V4A_ERR_INVALID_ARG, "%s: decay must be finite and >= 0", what);
    if (a.batch == 0) return V4A_OK;
    if (!lse || (a.own_rows > 0 && (!weights_out || (decay != 0.f && !weights_in))))
        return report(V4A_ERR_INVALID_ARG, "%s: lse, weights_out and (with decay > 0) weights_in are required", what);
    if (!aligned(lse, 4) || !aligned(weights_in, 4) || !aligned(weights_out, 4))
        return report(V4A_ERR_INVALID_ARG, "%s: lse or weights misaligned", what);
    const uintptr_t w_in = reinterpret_cast<uintptr_t>(weights_in), w_out = reinterpret_cast<uintptr_t>(weights_out);
    const uintptr_t w_bytes = (uintptr_t)a.batch * a.own_rows * 4;
    if (decay != 0.f && w_in != w_out && w_in < w_out + w_bytes && w_out < w_in + w_bytes)
        return report(V4A_ERR_INVALID_ARG, "%s: weights_in and weights_out overlap without being the same", what);
    a.lse = const_cast<float*>(lse);  // read only
    a.weights_in = weights_in;
    a.weights_out = weights_out;
    a.decay = decay;
    if (const cudaError_t e = bind_context(); e != cudaSuccess) return from_cuda(e, what);
    cudaStream_t s = (cudaStream_t)stream;
    if (dev_status) {
        const cudaError_t e = launch_zero_words(reinterpret_cast<uint32_t*>(dev_status), 1, s);
        if (e != cudaSuccess) return from_cuda(e, "dev_status reset");
    }
    if (a.own_rows == 0) return V4A_OK;
    if (a.dtype == V4A_BF16) return from_cuda(launch_weights_tc(a, s), what);
    switch (a.d) {
    case 64: return from_cuda(simt_weights<64>(a, s), what);
    case 128: return from_cuda(simt_weights<128>(a, s), what);
    case 256: return from_cuda(simt_weights<256>(a, s), what);
    default: return from_cuda(simt_weights<512>(a, s), what);
    }
}

}  // extern "C"
