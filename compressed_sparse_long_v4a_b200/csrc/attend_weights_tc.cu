// attend_weights_tc.cu -- tensor-core (tcgen05 / TMEM / TMA) form of v4a_attend_weights (bf16):
//
//     out[b][i] = decay * in[b][i] + sum_{j, h} exp(q[b][j][h] . own[b][i] / sqrt(d) - lse[b][j][h])
//
// The own rows are read once, 2 d bytes each, against 2 d n_q heads flops: at 64 heads HBM bounds it.  The
// scores come transposed, S^T = K Q^T (M = 128 slots, N = the sequence's rows of q), so a thread has one
// slot and all its columns: the sum over heads needs no exchange and has a fixed order.
//
// An item is one or two tiles of 128 slots of a sequence, taken in slabs of 64 dims: a stage holds the tiles'
// slab and that of up to 256 rows of q.  The queries come from L2 again for every item; with two
// tiles that is a quarter of the loads at 64 heads, and it leaves all of shared memory to the ring.
// Items that hold something are shared out evenly: every block adds up the counts first.
//
// 32 sequences of 8,192 slots and 64 heads: 47-49 us, 5.6-5.8 TB/s, 86-88% of the measured copy bandwidth.
//
// Warps: 0 loads, 1 issues the MMAs, 2-9 (four per tile) take exponentials and sums, while the next item's
// products run into the other half of tensor memory (up to 128 columns).  Every wait is bounded; on a
// time-out the block records a device fault and writes NaN for its items.
#include "common.cuh"
#include "internal.h"
#include "shared.h"
#include "tc_pair.cuh"
#include "tensor_map.h"

namespace v4a {
namespace {

constexpr int kTile = 128;          // slots
constexpr uint32_t kTileBytes = kTile * 128;
constexpr int kMaxCols = 256;
constexpr int kMaxStages = 6;
constexpr int kThreads = 10 * 32;
constexpr uint32_t kRing = 200 * 1024;  // bytes of the ring at most

struct WeightArgs {
    SharedArgs a;
    int per_seq, chunks;      // rows of q per sequence, in chunks of up to 256
    int cols, slabs, tiles;   // columns of an MMA (a multiple of 16), d / 64, tiles per item
    int stages, bufs;
    float scale;              // 1 / sqrt(d)
};

struct __align__(16) Shared {
    float2 col[kMaxCols];     // of a column: -lse, and the entries that its query sees (as int bits); read in pairs
    uint64_t full[kMaxStages], empty[kMaxStages], d_full[2], d_free[2], drain;
    long long warp_sum[kThreads / 32];
    long long left;
    int b0, i0, abort_flag;
    uint32_t tmem_base;
};

static_assert(offsetof(Shared, col) % 16 == 0, "pairs of columns are read as float4");

__device__ __forceinline__ int items_of(const WeightArgs& c, int b) {
    const int per = kTile * c.tiles;
    return (own_slots(c.a, b) + per - 1) / per;
}

struct Walk {
    int b, i, n;
    long long left;
    __device__ Walk(const WeightArgs& c, const Shared& sm) : b(sm.b0), i(sm.i0), n(0), left(sm.left) {
        if (left > 0) n = items_of(c, b);
    }
    __device__ bool next(const WeightArgs& c, int& item) {
        if (left == 0) return false;
        --left;
        while (i >= n) {
            ++b;
            i = 0;
            n = items_of(c, b);
        }
        item = i++;
        return true;
    }
};

// this block's equal share of the items
__device__ void find_share(const WeightArgs& c, Shared& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, batch = c.a.batch;
    const int per = (batch + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, batch), b1 = min(b0 + per, batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        mine += items_of(c, b);
        if (blockIdx.x == 0) report_sequence(c.a, b);
    }
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) sm.warp_sum[warp] = sum;
    if (threadIdx.x == 0) sm.left = 0;
    __syncthreads();
    long long total = 0, before = sum - mine;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sm.warp_sum[w];
        total += sm.warp_sum[w];
    }
    const long long f0 = (long long)blockIdx.x * total / gridDim.x, f1 = (long long)(blockIdx.x + 1) * total / gridDim.x;
    if (f0 < f1 && f0 >= before && f0 < before + mine) {
        int b = b0;
        long long at = f0 - before;
        for (int n; at >= (n = items_of(c, b)); ++b) at -= n;
        sm.b0 = b;
        sm.i0 = (int)at;
        sm.left = f1 - f0;
    }
    __syncthreads();
}

__device__ void fault(const WeightArgs& c, Shared& sm) {
    *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
    if (c.a.dev_status) atomicExch(c.a.dev_status, (int)V4A_ERR_DEVICE_FAULT);
}
__device__ __forceinline__ bool aborted(Shared& sm) { return *reinterpret_cast<volatile int*>(&sm.abort_flag) != 0; }
__device__ __forceinline__ uint64_t dadd(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// tiles of the item that hold anything
__device__ __forceinline__ int live_tiles(const WeightArgs& c, int b, int item) {
    const int n = own_slots(c.a, b) - item * kTile * c.tiles;
    return c.tiles == 2 && n > kTile ? 2 : 1;
}

__device__ void load(const WeightArgs& c, Shared& sm, uint8_t* ring, const CUtensorMap* own_map, const CUtensorMap* q_map) {
    const uint64_t again = tc::l2_evict_normal(), stream = tc::l2_stream_policy(c.chunks);
    const uint32_t q_bytes = c.cols * 128, stage = c.tiles * kTileBytes + q_bytes;
    Walk walk(c, sm);
    int j = 0, item;
    bool ok = true;
    while (ok && walk.next(c, item)) {
        const int live = live_tiles(c, walk.b, item);
        for (int ch = 0; ok && ch < c.chunks; ++ch) {
            for (int s = 0; s < c.slabs; ++s, ++j) {
                const int st = j % c.stages;
                if (aborted(sm) || (j >= c.stages && !tc::mbar_wait(&sm.empty[st], (j / c.stages - 1) & 1))) { ok = false; break; }
                uint8_t* dst = ring + st * stage;
                tc::mbar_arrive_expect_tx(&sm.full[st], live * kTileBytes + q_bytes);
                for (int t = 0; t < live; ++t)
                    tc::tma_load_4d(dst + t * kTileBytes, own_map, 0, (item * c.tiles + t) * kTile, s, walk.b, &sm.full[st], stream);
                tc::tma_load_4d(dst + c.tiles * kTileBytes, q_map, 0, walk.b * c.per_seq + ch * kMaxCols, s, 0, &sm.full[st], again);
            }
        }
    }
    // nothing is in flight when the block ends
    for (int k = j < c.stages ? 0 : j - c.stages; k < j; ++k) ok = tc::mbar_wait(&sm.full[k % c.stages], (k / c.stages) & 1) && ok;
    if (!ok) fault(c, sm);
}

__device__ void issue(const WeightArgs& c, Shared& sm, uint8_t* ring, uint32_t tmem) {
    const uint32_t stage = c.tiles * kTileBytes + c.cols * 128;
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(c.cols >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
    Walk walk(c, sm);
    int j = 0, it = 0, item;
    bool ok = true;
    while (ok && walk.next(c, item)) {
        const int live = live_tiles(c, walk.b, item);
        for (int ch = 0; ok && ch < c.chunks; ++ch, ++it) {
            const int buf = it % c.bufs;
            const uint32_t d = tmem + buf * 256;
            ok = !aborted(sm) && (it < c.bufs || tc::mbar_wait(&sm.d_free[buf], (it / c.bufs - 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
            for (int s = 0; ok && s < c.slabs; ++s, ++j) {
                const int st = j % c.stages;
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.full[st], (j / c.stages) & 1));
                if (!ok) break;
                tc::tc_fence_after();
                const uint64_t k0 = tc::sw128_desc(tc::smem_u32(ring + st * stage), 16, 1024);
                const uint64_t q0 = dadd(k0, c.tiles * kTileBytes);
                for (int t = 0; t < live; ++t)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::mma_f16(d + t * c.cols, dadd(k0, t * kTileBytes + kk * 32), dadd(q0, kk * 32), idesc, (s | kk) ? 1u : 0u);
                tc::mma_commit(&sm.empty[st]);
            }
            if (ok) tc::mma_commit(&sm.d_full[buf]);
        }
    }
    if (!ok) fault(c, sm);
    tc::mma_commit(&sm.drain);
    tc::mbar_wait(&sm.drain, 0);
}

// This thread's slot against N columns.  lse is subtracted from the logit in one rounding, before the factor log2 e of the
// exponent: rounded as lse log2 e it would cost a weight |lse| 2^-24 of its value.
template <int N>
__device__ __forceinline__ void add_columns(const float2* col, const uint32_t (&s)[N], float scale, int e, float (&acc)[4]) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const float4 z = *reinterpret_cast<const float4*>(col + k);
        const float p0 = exp2f(fmaf(__uint_as_float(s[k]), scale, z.x) * kLog2eF), p1 = exp2f(fmaf(__uint_as_float(s[k + 1]), scale, z.z) * kLog2eF);
        acc[k & 3] += e < __float_as_int(z.y) ? p0 : 0.f;
        acc[(k + 1) & 3] += e < __float_as_int(z.w) ? p1 : 0.f;
    }
}

__device__ void sum_up(const WeightArgs& c, Shared& sm, uint32_t tmem) {
    const SharedArgs& a = c.a;
    const int warp = (threadIdx.x >> 5) - 2, tile = warp >> 2, sub = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int t256 = threadIdx.x - 64;
    const uint32_t lanes = tmem + ((uint32_t)(32 * sub) << 16) + tile * c.cols;
    Walk walk(c, sm);
    int it = 0, item, have = -1;  // sequence and chunk of the columns in shared memory
    bool ok = true;
    while (walk.next(c, item)) {
        const int b = walk.b, slot = (item * c.tiles + tile) * kTile + 32 * sub + lane;
        const bool held = tile < c.tiles && slot < own_slots(a, b);
        const long long at = (long long)b * a.own_rows + slot;
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, before = 0.f;
        int e = 0x7fffffff;  // seen by no query
        if (held) {
            e = a.own_entry ? a.own_entry[at] : (int)(a.n_prefix + slot);
            if (e < 0) e = 0x7fffffff;
            if (a.decay != 0.f) before = a.weights_in[at];
        }
        const bool used = tile < live_tiles(c, b, item);
        for (int ch = 0; ch < c.chunks; ++ch, ++it) {
            const int buf = it % c.bufs;
            if (c.chunks > 1 || have != b) {
                tc::named_barrier(1, 256);  // nobody reads the columns of the item before
                const int row = ch * kMaxCols + t256;
                float2 z = make_float2(0.f, __int_as_float(0));
                if (row < c.per_seq) {
                    const float lse = a.lse[(long long)b * c.per_seq + row];
                    const long long seen = seen_entries(a, seq_len(a, b) - a.n_q + row / a.heads);
                    if (lse != -INFINITY)
                        z = make_float2(-lse, __int_as_float(seen < 0x7fffffff ? (int)seen : 0x7fffffff));
                }
                sm.col[t256] = z;
                tc::named_barrier(1, 256);
                have = b;
            }
            ok = ok && !aborted(sm) && tc::mbar_wait(&sm.d_full[buf], (it / c.bufs) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && used) {
                tc::tc_fence_after();
                int c0 = 0;
                for (; c0 + 32 <= c.cols; c0 += 32) {
                    uint32_t s[32];
                    tc::tmem_ld_x32(lanes + buf * 256 + c0, s);
                    tc::tmem_ld_wait();
                    add_columns<32>(sm.col + c0, s, c.scale, e, acc);
                }
                if (c0 < c.cols) {
                    uint32_t s[16];
                    tc::tmem_ld_x16(lanes + buf * 256 + c0, s);
                    tc::tmem_ld_wait();
                    add_columns<16>(sm.col + c0, s, c.scale, e, acc);
                }
                tc::tc_fence_before();
            }
            __syncwarp();
            if (lane == 0 && ok) tc::mbar_arrive(&sm.d_free[buf]);
        }
        if (held) {
            const float total = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            a.weights_out[at] = !ok ? NAN : a.decay == 0.f ? total : fmaf(a.decay, before, total);
        }
    }
    if (!ok) fault(c, sm);
}

__global__ void __launch_bounds__(kThreads, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap own_map, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ WeightArgs c) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sm;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            tc::mbar_init(&sm.full[i], 1);
            tc::mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sm.d_full[i], 1);
            tc::mbar_init(&sm.d_free[i], 8);
        }
        tc::mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) tc::tmem_alloc(&sm.tmem_base, 512);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    griddep_wait();  // everything before this kernel on the stream has finished
    griddep_launch_dependents();
    find_share(c, sm);
    const uint32_t tmem = sm.tmem_base;
    if (warp == 0) {
        if (lane == 0) load(c, sm, ring, &own_map, &q_map);
    } else if (warp == 1) {
        issue(c, sm, ring, tmem);
    } else {
        sum_up(c, sm, tmem);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_weights_tc(const SharedArgs& a, cudaStream_t st) {
    WeightArgs c;
    c.a = a;
    c.per_seq = a.n_q * a.heads;
    c.chunks = (c.per_seq + kMaxCols - 1) / kMaxCols;
    c.cols = c.per_seq < kMaxCols ? (c.per_seq + 15) / 16 * 16 : kMaxCols;
    c.slabs = a.d / 64;
    c.bufs = c.cols <= kMaxCols / 2 ? 2 : 1;
    c.scale = 1.f / sqrtf((float)a.d);
    const long long tiles = (long long)a.batch * ((a.own_rows + kTile - 1) / kTile);
    c.tiles = tiles > 2 * kNumSMs ? 2 : 1;  // few tiles: one per item, so that more blocks have one
    const uint32_t stage = c.tiles * kTileBytes + c.cols * 128;
    c.stages = (int)(kRing / stage) < kMaxStages ? (int)(kRing / stage) : kMaxStages;
    const size_t smem = (size_t)c.stages * stage + 1024;
    CUtensorMap own_map, q_map;
    if (!make_slab_map(&own_map, a.own, a.batch, a.own_rows, a.d, kTile, 1) ||
        !make_slab_map(&q_map, a.q, 1, (long long)a.batch * c.per_seq, a.d, c.cols, 1))
        return cudaErrorNotSupported;
    const long long items = (tiles + c.tiles - 1) / c.tiles;
    // the most of any call: host threads share the attribute, and another one may set it before this launch
    cudaError_t e = cudaFuncSetAttribute(weights_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 1024);
    if (e == cudaSuccess)
        e = launch_pdl(weights_tc_kernel, dim3((unsigned)(items < kNumSMs ? items : kNumSMs)), dim3(kThreads), smem, st, own_map,
                       q_map, c);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace v4a
