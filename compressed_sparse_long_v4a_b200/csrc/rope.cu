// rope.cu -- rotary positions: y = s R(+-p f_k) x on R of a row's d dims.
//
// Pair k of a row at position p turns by the angle p f_k, f_k = base^(-2k/R) (scaled for long contexts
// on the host).  What is read and written once bounds it: 2 d elements per row (2 R in place), against
// 3 flops per rotated element.  An item is 8 elements of a row (16 bytes of bf16).  A thread keeps one
// column of items and runs down the heads of its token, so the column's angles stay in registers (of adjacent pairs), the
// copied columns pass through as they are, and no index is worked out per item.  A block takes one
// token, or several where their rows are few: its (cos, sin) are made once in shared memory while
// the first rows are on their way, and that has to pay.  Then the rows of all its tokens are one run, and
// the angles are read again for every row.  Measured: 4,096 tokens of 64 x 512 bf16 89.6 us, 6.1 TB/s, 93% of the measured copy
// bandwidth (an index per item and a barrier per token took 267 us); 16,000 tokens of (8 + 1) x 512 and 4 x 128 65 us, 5.1 TB/s
// (a token per block: 102 us), half pairs 69 us; 1,554 of 17 x 128 fp32, half pairs, 7.6 us; a decode step of four tokens 3.1 us on the
// device.  4,096 tokens of 65 x 512 bf16: 88 us, half pairs 118; in place 21 and 18; in rows of 513 (any alignment, an element
// at a time) 322 us, in place 42.  With few tokens (a decode step) a token's heads are cut over blocks.
#include "common.cuh"
#include "internal.h"
#include "turns.h"

namespace v4a {
namespace {

constexpr int kMaxStreams = 8;
constexpr int kThreads = 256;
constexpr int kTable = 2 * kThreads;  // angles of a block's tokens at most
constexpr int kMaxTok = 64;           // its tokens at most

struct RopeStream {
    const void* x;
    void* out;
    int heads, off;
    int rot, row_items;  // items of a row: rotated ones first, then the copied ones
    // vectors: tokens per block (several where their rows are few), heads side by side in it, and the blocks that a
    // token's heads and columns are cut over; any alignment: blocks per token (h_parts)
    int tokens, h_par, h_parts, c_parts;
    unsigned block0;     // its first block
    long long xb, xt, xh, ob, ot, oh;
};

struct RopeArgs {
    RopeStream s[kMaxStreams];
    Turns f;
    int n, n_tok, pairs, half, inverse;
    unsigned all_tok;        // batch * n_tok
    float scale;
    const int64_t* positions;
    long long pos_stride, pos0, pos_step;
};

// a parameter by its address: the lanes of a warp read neighbouring ones, which constant memory serialises
template <typename X>
__device__ __forceinline__ X by_address(const X* p) {
    asm("" : "+l"(p));
    return *p;
}

// (cos, sin) of n tokens from `tok` on: cs[i * pairs + k], one per thread
__device__ __forceinline__ void make_table(const RopeArgs& a, unsigned tok, int n, float2* cs) {
    for (int i = threadIdx.x; i < n * a.pairs; i += kThreads) {
        const int k = i % a.pairs;
        const unsigned at = tok + i / a.pairs, b = at / (unsigned)a.n_tok, t = at % (unsigned)a.n_tok;
        const long long p = a.positions ? a.positions[b * a.pos_stride + t] : a.pos0 + t * a.pos_step;
        const float2 v = turn((double)p, by_address(&a.f.hi[k]), by_address(&a.f.lo[k]));
        cs[i] = make_float2(v.x * a.scale, (a.inverse ? -v.y : v.y) * a.scale);
    }
    __syncthreads();
}

__device__ __forceinline__ const RopeStream& which_stream(const RopeArgs& a) {
    int k = 0;
    while (k + 1 < a.n && blockIdx.x >= a.s[k + 1].block0) ++k;
    return a.s[k];
}

// 8 elements as they lie in memory
template <typename T>
struct Item {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { Vec8<T>::load(reinterpret_cast<const T*>(w), f); }
    __device__ __forceinline__ void set(const float (&f)[8]) { Vec8<T>::store(reinterpret_cast<T*>(w), f); }
};

// the pairs of a rotated item (u, and in the half layout v) turned by w
template <typename T, bool HALF>
__device__ __forceinline__ void rotate(Item<T>& u, Item<T>& v, const float2* w) {
    float x[8], y[8];
    u.get(x);
    if (HALF) {
        v.get(y);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float p = x[k], q = y[k];
            x[k] = p * w[k].x - q * w[k].y;
            y[k] = q * w[k].x + p * w[k].y;
        }
        v.set(y);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float p = x[2 * k], q = x[2 * k + 1];
            x[2 * k] = p * w[k].x - q * w[k].y;
            x[2 * k + 1] = q * w[k].x + p * w[k].y;
        }
    }
    u.set(x);
}

// Rows, offsets and strides in multiples of 8 elements: an item is one 8-element chunk, or, in the half
// layout, the two chunks that a rotated item pairs up.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 5) rope_vec_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float2 cs[kTable];
    __shared__ long long from[2][kMaxTok];  // where the tokens begin in x and out
    griddep_wait();  // everything before this kernel on the stream has finished
    const RopeStream& s = which_stream(a);
    constexpr int kU = sizeof(T) == 2 ? 2 : 1;  // rows in flight (twice as many with 4 blocks per SM: 4.2 instead of 4.7 TB/s)
    constexpr int kA = HALF ? 8 : 4;            // pairs of an item
    const int parts = s.h_parts * s.c_parts;
    const unsigned local = blockIdx.x - s.block0, group = local / (unsigned)parts;
    const unsigned tok0 = group * (unsigned)s.tokens;
    const int n_tok = (int)min((unsigned)s.tokens, a.all_tok - tok0);
    Item<T> u[kU], v[kU];
    float2 w[kA];
    auto angles = [&](int at) {
#pragma unroll
        for (int k = 0; k < kA; k += 2) {
            const float4 x = *reinterpret_cast<const float4*>(&cs[at + k]);
            w[k] = make_float2(x.x, x.y);
            w[k + 1] = make_float2(x.z, x.w);
        }
    };
    auto element = [&](int c) {  // where item c of a row begins
        const int e = 8 * (c < s.rot ? c : c - s.rot);
        return c < s.rot ? e + s.off : e >= s.off ? e + 2 * a.pairs : e;
    };
    if (s.tokens > 1) {
        // several tokens: this thread's column c, and its first row of (token, head)
        if ((int)threadIdx.x < n_tok) {
            const unsigned tok = tok0 + threadIdx.x, b = tok / (unsigned)a.n_tok, t = tok % (unsigned)a.n_tok;
            from[0][threadIdx.x] = b * s.xb + t * s.xt;
            from[1][threadIdx.x] = b * s.ob + t * s.ot;
        }
        __syncthreads();
        const int r = (int)threadIdx.x / s.row_items, c = (int)threadIdx.x - r * s.row_items, rows = n_tok * s.heads;
        const float per_head = 1.f / s.heads;
        const bool rotated = c < s.rot;
        const int e = element(c);
        int row = r < s.h_par ? r : rows;
        const T* const xp = static_cast<const T*>(s.x) + e;
        T* const op = static_cast<T*>(s.out) + e;
        auto token = [&](int at) { return (int)((at + 0.5f) * per_head); };  // exact: rows are few
        auto load = [&]() {
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                const int at = row + j * s.h_par, i = token(at);
                if (at >= rows) continue;
                const T* p = xp + (from[0][i] + (at - i * s.heads) * s.xh);
                u[j].load(p);
                if (HALF && rotated) v[j].load(p + a.pairs);
            }
        };
        load();  // on its way while the angles are worked out
        make_table(a, tok0, n_tok, cs);
        while (row < rows) {
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                const int at = row + j * s.h_par, i = token(at);
                if (at >= rows) continue;
                T* p = op + (from[1][i] + (at - i * s.heads) * s.oh);
                if (rotated) {
                    angles(i * a.pairs + kA * c);
                    rotate<T, HALF>(u[j], v[j], w);
                    if (HALF) v[j].store(p + a.pairs);
                }
                u[j].store(p);
            }
            row += kU * s.h_par;
            load();
        }
    } else {
        // one token: this thread's column c, and its first head
        const int part = (int)(local % (unsigned)parts);
        int c, h;
        bool on;
        if (s.c_parts > 1) {
            c = part % s.c_parts * kThreads + threadIdx.x;
            h = part / s.c_parts;
            on = c < s.row_items;
        } else {
            const int r = (int)threadIdx.x / s.row_items;
            c = (int)threadIdx.x - r * s.row_items;
            h = part * s.h_par + r;
            on = r < s.h_par;
        }
        if (!on) h = s.heads;
        const int step = s.h_par * s.h_parts;
        const unsigned b = tok0 / (unsigned)a.n_tok, t = tok0 % (unsigned)a.n_tok;
        const bool rotated = c < s.rot;
        const int e = element(c);
        const T* xp = static_cast<const T*>(s.x) + b * s.xb + t * s.xt + e;
        T* op = static_cast<T*>(s.out) + b * s.ob + t * s.ot + e;
        auto load = [&]() {
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                const int hj = h + j * step;
                if (hj >= s.heads) continue;
                u[j].load(xp + hj * s.xh);
                if (HALF && rotated) v[j].load(xp + hj * s.xh + a.pairs);
            }
        };
        load();
        make_table(a, tok0, 1, cs);
        if (!HALF && on && rotated) angles(kA * c);
        while (h < s.heads) {
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                const int hj = h + j * step;
                if (hj >= s.heads) continue;
                if (HALF && rotated) angles(kA * c);  // 16 registers that spilled when held: 137 instead of 116 us
                if (rotated) rotate<T, HALF>(u[j], v[j], w);
                u[j].store(op + hj * s.oh);
                if (HALF && rotated) v[j].store(op + hj * s.oh + a.pairs);
            }
            h += kU * step;
            load();
        }
    }
    // The attention kernels read their first query before they wait for this grid (they may, once all its
    // blocks have ended): the rows have reached L2 by then.  For the same reason there is no early
    // griddep_launch_dependents here.
    __threadfence();
}

// any alignment: an item is a pair, or one copied element
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 cs[kMaxPairs];
    griddep_wait();
    const RopeStream& s = which_stream(a);
    const unsigned local = blockIdx.x - s.block0, tok = local / (unsigned)s.h_parts;
    const int part = (int)(local % (unsigned)s.h_parts);
    const unsigned b = tok / (unsigned)a.n_tok, t = tok % (unsigned)a.n_tok;
    const T* xt = static_cast<const T*>(s.x) + b * s.xb + t * s.xt;
    T* ot = static_cast<T*>(s.out) + b * s.ob + t * s.ot;
    make_table(a, tok, 1, cs);
    const unsigned items = (unsigned)s.heads * s.row_items;
    const unsigned per = (items + s.h_parts - 1) / s.h_parts;
    const unsigned i0 = part * per, i1 = min(items, i0 + per);
    for (unsigned i = i0 + threadIdx.x; i < i1; i += kThreads) {
        const unsigned h = i / (unsigned)s.row_items, c = i % (unsigned)s.row_items;
        const T* xp = xt + h * s.xh;
        T* op = ot + h * s.oh;
        if ((int)c < s.rot) {
            const int e0 = s.off + (a.half ? c : 2 * c), e1 = a.half ? e0 + a.pairs : e0 + 1;
            const float2 w = cs[c];
            const float x = (float)xp[e0], y = (float)xp[e1];
            op[e0] = (T)(x * w.x - y * w.y);
            op[e1] = (T)(y * w.x + x * w.y);
        } else {
            int e = c - s.rot;
            if (e >= s.off) e += 2 * a.pairs;
            op[e] = xp[e];
        }
    }
    __threadfence();
}

// whether the rows of out, [n0][n1][n2][d] with these strides, are all apart
bool rows_apart(long long d, long long n0, long long s0, long long n1, long long s1, long long n2, long long s2) {
    long long n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (s[j] > s[j + 1]) {
                long long x = s[j]; s[j] = s[j + 1]; s[j + 1] = x;
                x = n[j]; n[j] = n[j + 1]; n[j + 1] = x;
            }
    long long reach = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < reach) return false;
        reach += (n[i] - 1) * s[i];
    }
    return true;
}

// What a stream's rows touch on one side: n[0] x n[1] x n[2] pieces of `bytes` from `at` on, s bytes apart.
struct Extent {
    uintptr_t at;
    long long bytes, n[3], s[3];
    long long reach() const { return (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + (n[2] - 1) * s[2] + bytes; }
};

// Whether whole numbers v[i] in lo[i] .. hi[i], i >= k, make delta + sum v[i] s[i] lie in low .. high.  The strides
// descend, and where each is at least what the smaller ones reach together, as in rows that lie apart, a level has three
// values to try at most.  `budget` bounds the search for others: when it is used up, the answer is yes.
bool meets(long long delta, long long low, long long high, const long long* s, const long long* lo, const long long* hi, int n, int k, int& budget) {
    if (k == n) return low <= delta && delta <= high;
    if (--budget < 0) return true;
    long long least = 0, most = 0;  // of the smaller strides' sum
    for (int i = k + 1; i < n; ++i) {
        least += lo[i] * s[i];
        most += hi[i] * s[i];
    }
    auto floor_div = [](long long a, long long b) { return a / b - (a % b < 0); };
    long long v0 = -floor_div(-(low - delta - most), s[k]), v1 = floor_div(high - delta - least, s[k]);
    v0 = v0 > lo[k] ? v0 : lo[k];
    v1 = v1 < hi[k] ? v1 : hi[k];
    for (long long v = v0; v <= v1; ++v)
        if (meets(delta + v * s[k], low, high, s, lo, hi, n, k + 1, budget)) return true;
    return false;
}

// whether two streams' rows share a byte; rows of one may lie between those of the other (heads of one projection)
bool overlap(const Extent& a, const Extent& b) {
    if (a.at + (uintptr_t)a.reach() <= b.at || b.at + (uintptr_t)b.reach() <= a.at) return false;
    // row j of b begins at b.at - a.at + sum j s_b - sum i s_a behind row i of a; equal strides are one number j - i
    long long s[6], lo[6], hi[6];
    int n = 0;
    auto add = [&](long long stride, long long from, long long to) {
        if (stride == 0 || from == to) return;
        int k = 0;
        while (k < n && s[k] > stride) ++k;
        if (k < n && s[k] == stride) {
            lo[k] += from;
            hi[k] += to;
            return;
        }
        for (int i = n++; i > k; --i) s[i] = s[i - 1], lo[i] = lo[i - 1], hi[i] = hi[i - 1];
        s[k] = stride, lo[k] = from, hi[k] = to;
    };
    for (int i = 0; i < 3; ++i) {
        add(a.s[i], -(a.n[i] - 1), 0);
        add(b.s[i], 0, b.n[i] - 1);
    }
    int budget = 10000;
    return meets((long long)(b.at - a.at), 1 - b.bytes, a.bytes - 1, s, lo, hi, n, 0, budget);
}

}  // namespace
}  // namespace v4a

extern "C" v4a_status v4a_rope(const v4a_rope_io* io, int n_streams, int batch, long long n_tok,
                               const int64_t* positions, long long pos_stride, long long pos0, long long pos_step,
                               const v4a_rope_params* params, void* stream) {
    using namespace v4a;
    if (n_streams < 0 || n_streams > kMaxStreams) return report(V4A_ERR_INVALID_ARG, "v4a_rope: 0 .. 8 streams");
    if (batch < 0 || n_tok < 0) return report(V4A_ERR_INVALID_ARG, "v4a_rope: need batch >= 0, n_tok >= 0");
    if (!params) return report(V4A_ERR_INVALID_ARG, "v4a_rope: params is NULL");
    const v4a_rope_params& p = *params;
    if (p.rope_dims < 2 || p.rope_dims > 2 * kMaxPairs || (p.rope_dims & 1))
        return report(V4A_ERR_INVALID_ARG, "v4a_rope: rope_dims must be even and in 2..512");
    if (!(p.base > 0) || !(p.factor > 0) || !isfinite(p.base) || !isfinite(p.factor) || !isfinite(p.out_scale))
        return report(V4A_ERR_INVALID_ARG, "v4a_rope: base and factor must be > 0, out_scale finite");
    if (p.orig_ctx < 0 || (p.orig_ctx > 0 && !(p.beta_fast > p.beta_slow && isfinite(p.beta_fast) && isfinite(p.beta_slow))))
        return report(V4A_ERR_INVALID_ARG, "v4a_rope: need orig_ctx >= 0 and, with it, finite beta_fast > beta_slow");
    if (n_streams == 0 || batch == 0 || n_tok == 0) return V4A_OK;
    if (!io) return report(V4A_ERR_INVALID_ARG, "v4a_rope: io is NULL");
    if (n_tok > 0x7fffffffLL || (long long)batch * n_tok > 0x7fffffffLL)
        return report(V4A_ERR_UNSUPPORTED, "v4a_rope: batch * n_tok must be < 2^31");
    if (positions && (reinterpret_cast<uintptr_t>(positions) % 8 || pos_stride < 0))
        return report(V4A_ERR_INVALID_ARG, "v4a_rope: positions misaligned or pos_stride < 0");

    RopeArgs a;
    Extent read[kMaxStreams], written[kMaxStreams];
    bool vec = true;
    for (int i = 0; i < n_streams; ++i) {
        v4a_rope_io r = io[i];
        if (batch == 1) r.x_batch_stride = r.out_batch_stride = 0;  // strides that nothing steps over
        if (n_tok == 1) r.x_tok_stride = r.out_tok_stride = 0;
        if (r.heads == 1) r.x_head_stride = r.out_head_stride = 0;
        if (r.dtype != V4A_F32 && r.dtype != V4A_BF16)
            return report(V4A_ERR_UNSUPPORTED, "v4a_rope: stream %d: dtype must be F32 or BF16", i);
        if (r.dtype != io[0].dtype)
            return report(V4A_ERR_UNSUPPORTED, "v4a_rope: the streams of a call share a dtype");
        const long long es = r.dtype == V4A_F32 ? 4 : 2;
        if (!r.x || !r.out || r.heads < 1 || r.d < p.rope_dims || r.rope_offset < 0 ||
            r.rope_offset > r.d - p.rope_dims || reinterpret_cast<uintptr_t>(r.x) % es ||
            reinterpret_cast<uintptr_t>(r.out) % es)
            return report(V4A_ERR_INVALID_ARG, "v4a_rope: stream %d: pointers, heads, d or rope_offset", i);
        if ((long long)r.heads * r.d > (1LL << 30)) return report(V4A_ERR_UNSUPPORTED, "v4a_rope: stream %d: heads * d too large", i);
        if (r.x_batch_stride < 0 || r.x_tok_stride < 0 || r.x_head_stride < 0 || r.out_batch_stride < 0 ||
            r.out_tok_stride < 0 || r.out_head_stride < 0)
            return report(V4A_ERR_INVALID_ARG, "v4a_rope: stream %d: negative stride", i);
        const long long counts[3] = {batch, n_tok, r.heads}, strides[2][3] = {{r.x_batch_stride, r.x_tok_stride, r.x_head_stride},
                                                                               {r.out_batch_stride, r.out_tok_stride, r.out_head_stride}};
        for (const auto& side : strides)
            for (int k = 0; k < 3; ++k)
                if (counts[k] > 1 && side[k] > (1LL << 48) / (counts[k] - 1))
                    return report(V4A_ERR_INVALID_ARG, "v4a_rope: stream %d: stride out of range", i);
        if (!rows_apart(r.d, batch, r.out_batch_stride, n_tok, r.out_tok_stride, r.heads, r.out_head_stride))
            return report(V4A_ERR_INVALID_ARG, "v4a_rope: stream %d: rows of out overlap", i);
        const bool in_place = r.x == r.out;
        if (in_place && (r.x_batch_stride != r.out_batch_stride || r.x_tok_stride != r.out_tok_stride ||
                         r.x_head_stride != r.out_head_stride))
            return report(V4A_ERR_INVALID_ARG, "v4a_rope: stream %d: in place needs equal strides", i);
        // what is read and written; in place that is the rotated dims alone
        const long long first = in_place ? r.rope_offset * es : 0, touched = (in_place ? p.rope_dims : r.d) * es;
        read[i] = {reinterpret_cast<uintptr_t>(r.x) + first, touched, {batch, n_tok, r.heads},
                   {r.x_batch_stride * es, r.x_tok_stride * es, r.x_head_stride * es}};
        written[i] = {reinterpret_cast<uintptr_t>(r.out) + first, touched, {batch, n_tok, r.heads},
                      {r.out_batch_stride * es, r.out_tok_stride * es, r.out_head_stride * es}};
        if (!in_place && overlap(read[i], written[i]))
            return report(V4A_ERR_INVALID_ARG, "v4a_rope: stream %d: x and out overlap without being the same", i);
        for (int j = 0; j < i; ++j)
            if (overlap(written[i], written[j]) || overlap(written[i], read[j]) || overlap(read[i], written[j]))
                return report(V4A_ERR_INVALID_ARG, "v4a_rope: streams %d and %d overlap", j, i);
        RopeStream& s = a.s[i];
        s.x = r.x;
        s.out = r.out;
        s.heads = r.heads;
        s.off = r.rope_offset;
        s.xb = r.x_batch_stride;
        s.xt = r.x_tok_stride;
        s.xh = r.x_head_stride;
        s.ob = r.out_batch_stride;
        s.ot = r.out_tok_stride;
        s.oh = r.out_head_stride;
        s.row_items = in_place ? 0 : r.d - p.rope_dims;  // copied elements; made items below
        vec = vec && r.d % 8 == 0 && r.rope_offset % 8 == 0 && reinterpret_cast<uintptr_t>(r.x) % 16 == 0 &&
              reinterpret_cast<uintptr_t>(r.out) % 16 == 0 && (s.xb | s.xt | s.xh | s.ob | s.ot | s.oh) % 8 == 0;
    }
    vec = vec && p.rope_dims % (p.half ? 16 : 8) == 0;
    a.n = n_streams;
    a.n_tok = (int)n_tok;
    a.pairs = p.rope_dims / 2;
    a.half = p.half ? 1 : 0;
    a.inverse = p.inverse ? 1 : 0;
    a.scale = (float)p.out_scale;
    a.positions = positions;
    a.pos_stride = pos_stride;
    a.pos0 = pos0;
    a.pos_step = pos_step;
    make_turns(p.rope_dims, p.base, &a.f, p.factor, p.orig_ctx, p.beta_fast, p.beta_slow);
    const long long tokens = (long long)batch * n_tok;
    a.all_tok = (unsigned)tokens;
    const long long want = (8LL * kNumSMs + tokens - 1) / tokens;  // blocks per token that fill the SMs
    // items per thread that make a block worth its angles, and blocks per SM that are worth more than that (4 and 6:
    // 16,000 tokens of half pairs 76 us where 8 and 4 take 69, 1,554 tokens of fp32 9.0 instead of 7.6 us, as 8 and 6 do)
    constexpr int kWork = 8, kFill = 4;
    long long blocks = 0;
    for (int i = 0; i < n_streams; ++i) {
        RopeStream& s = a.s[i];
        s.rot = vec ? p.rope_dims / (p.half ? 16 : 8) : a.pairs;
        s.row_items = s.rot + (vec ? s.row_items / 8 : s.row_items);
        s.tokens = s.h_par = s.c_parts = 1;
        long long most;  // blocks that a token's heads can be cut over
        if (!vec) {
            most = ((long long)s.heads * s.row_items + kThreads - 1) / kThreads;
        } else if (s.row_items > kThreads) {
            s.c_parts = (s.row_items + kThreads - 1) / kThreads;
            most = s.heads;
        } else {
            const long long per_tok = (long long)s.heads * s.row_items;
            // as many tokens as give each thread kWork items, while enough blocks remain to fill the SMs
            long long most_tok = kWork * kThreads / per_tok, even = (tokens + kFill * kNumSMs - 1) / (kFill * kNumSMs), room = kThreads / per_tok;
            if (most_tok > even) most_tok = even > room ? even : room;
            if (most_tok > kTable / a.pairs) most_tok = kTable / a.pairs;
            if (most_tok > kMaxTok) most_tok = kMaxTok;
            if (most_tok > tokens) most_tok = tokens;
            s.tokens = most_tok > 1 ? (int)most_tok : 1;
            s.h_par = kThreads / s.row_items;
            if (s.h_par > s.heads * s.tokens) s.h_par = s.heads * s.tokens;
            most = s.tokens > 1 ? 1 : (s.heads + s.h_par - 1) / s.h_par;
        }
        s.h_parts = (int)(want < most ? want : most);
        if (s.h_parts > 65535) s.h_parts = 65535;
        s.block0 = (unsigned)blocks;
        blocks += (tokens + s.tokens - 1) / s.tokens * s.h_parts * s.c_parts;
    }
    if (blocks > 0x7fffffffLL) return report(V4A_ERR_UNSUPPORTED, "v4a_rope: too many rows for one call");
    const dim3 grid((unsigned)blocks);
    const bool f32 = io[0].dtype == V4A_F32;
    auto* kernel = !vec     ? (f32 ? rope_any_kernel<float> : rope_any_kernel<__nv_bfloat16>)
                   : p.half ? (f32 ? rope_vec_kernel<float, true> : rope_vec_kernel<__nv_bfloat16, true>)
                            : (f32 ? rope_vec_kernel<float, false> : rope_vec_kernel<__nv_bfloat16, false>);
    cudaError_t e = launch_pdl(kernel, grid, dim3(kThreads), 0, (cudaStream_t)stream, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? V4A_OK : report(V4A_ERR_CUDA, "v4a_rope: %s", cudaGetErrorString(e));
}
