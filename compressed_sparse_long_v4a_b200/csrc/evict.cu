// evict.cu -- eviction from a cache by accumulated attention weight.
//
// Of a sequence's n slots the `budget` heaviest stay (the first and last ones always), moved to the front
// in order.  The rows that stay are read and written once: that copy bounds the call.  Choosing them is
// a radix select over order-preserving 32-bit keys of the weights, by a block per sequence, or a cluster
// of up to 8 where a block's threads would have more than 8 keys each (what a cluster adds is a barrier and reads of
// the other blocks' counts per pass).  The keys are loaded once and stay in shared memory: three histogram passes of 11, 11 and
// 10 bits, the counts of a cluster's blocks added up through distributed shared memory, then one ordered
// pass that places the slots by ballots.  evict_rows_kernel then moves the rows, a warp per row, four rows
// in flight.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

#include <cstddef>

namespace cg = cooperative_groups;

namespace v4a {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;

struct EvictArgs {
    const float* weights;
    const int32_t* own_count;
    const int32_t* own_entry;
    float* weights_out;
    int32_t* entry_out;
    int32_t* kept;
    int32_t* count_out;
    int* dev_status;
    int own_rows, out_rows, budget, first, recent, first_entry;
};

struct __align__(16) EvictSmem {
    uint32_t hist[3][kBins];  // this block's counts, by pass
    uint32_t total[2];        // this block's slots above the threshold, and at it
    uint32_t pick[2];         // chosen digit, how many of it are still wanted
    uint32_t warp[32];
};

static_assert(offsetof(EvictSmem, hist) % 8 == 0 && offsetof(EvictSmem, total) % 8 == 0, "read in pairs by other blocks");

// exclusive prefix sum over the block's threads; *sum: the block's total
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_s, uint32_t* sum) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_s[w] = x;
    __syncthreads();
    if (w == 0) {
        uint32_t y = warp_s[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        warp_s[lane] = y;
    }
    __syncthreads();
    const uint32_t before = w ? warp_s[w - 1] : 0u;
    *sum = warp_s[31];
    __syncthreads();
    return before + x - v;
}

// STORED: the keys stay in (dynamic) shared memory, `rounds` per thread; else they are made again in every pass.
// Slots ascend over blocks, then warps, then a warp's rounds, then lanes.  The loops are rolled: the code runs cold,
// and fetching unrolled copies took most of the time (8 keys a thread in registers: 17 us instead of 7).
template <bool STORED>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    __shared__ EvictSmem sm;
    extern __shared__ uint32_t stored[];
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
    griddep_wait();  // everything before this kernel on the stream has finished
    griddep_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto sync_all = [&] {
        if (csize > 1) cluster.sync();
        else __syncthreads();
    };
    const int b = blockIdx.x / csize;
    unsigned n = (unsigned)a.own_rows;
    if (a.own_count) {
        const int c = a.own_count[b], in = c < 0 ? 0 : c > a.own_rows ? a.own_rows : c;
        if (c != in && a.dev_status && threadIdx.x == 0 && crank == 0) atomicExch(a.dev_status, (int)V4A_ERR_DEVICE_FAULT);
        n = (unsigned)in;
    }
    const unsigned want = n < (unsigned)a.budget ? n : (unsigned)a.budget;
    const bool all = want == n;
    const float* w = a.weights + (long long)b * a.own_rows;
    const unsigned width = (unsigned)csize * kThreads;
    const int rounds = (int)((n + width - 1) / width);
    const unsigned base = ((unsigned)crank * kThreads + warp * 32) * rounds + lane;
    const unsigned first = (unsigned)a.first, free_slots = n > (unsigned)a.first + a.recent ? n - a.first - a.recent : 0;
    auto make_key = [&](unsigned i) -> uint32_t {
        if (i - first >= free_slots) return 0xffffffffu;  // always kept
        const float x = w[i];
        return isnan(x) ? 0u : float_to_ordered(x);  // -inf: 0x007fffff, +inf: 0xff800000
    };
    if (STORED && !all) {
#pragma unroll 8
        for (int j = 0; j < rounds; ++j)
            if (base + 32 * j < n) stored[j * kThreads + threadIdx.x] = make_key(base + 32 * j);
    }
    auto key = [&](int j) -> uint32_t { return STORED ? stored[j * kThreads + threadIdx.x] : make_key(base + 32 * j); };
    // radix select of the want-th largest key; digits of 11, 11 and 10 bits
    uint32_t prefix = 0, need = want;
    if (!all) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1024u : 2048u;
            const uint32_t above = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
            uint32_t* hist = sm.hist[pass];
            if (pass == 0) __syncthreads();  // the counts are zero
#pragma unroll 1
            for (int j = 0; j < rounds; ++j) {
                const bool in = base + 32 * j < n;
                const uint32_t k = in ? key(j) : 0u;
                const bool mine = in && ((k ^ prefix) & above) == 0;
                const uint32_t m = __ballot_sync(0xffffffffu, mine);
                if (m == 0) continue;
                // equal weights are common, and 32 additions to one counter slow
                const uint32_t d = (k >> shift) & (digits - 1), d0 = __shfl_sync(0xffffffffu, d, __ffs(m) - 1);
                if (__all_sync(0xffffffffu, !mine || d == d0)) {
                    if (lane == 0) atomicAdd(&hist[d0], (uint32_t)__popc(m));
                } else if (mine) {
                    atomicAdd(&hist[d], 1u);
                }
            }
            sync_all();
            // this thread's two bins, the highest digits first
            uint32_t c[2] = {0, 0};
            const uint32_t d0 = digits - 1 - 2 * threadIdx.x;
            if (2 * threadIdx.x < digits) {
                if (csize == 1) {
                    c[0] = hist[d0];
                    c[1] = hist[d0 - 1];
                } else {
#pragma unroll 4
                    for (int r = 0; r < csize; ++r) {
                        const uint2 h = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(hist, r) + d0 - 1);
                        c[0] += h.y;
                        c[1] += h.x;
                    }
                }
            }
            uint32_t sum;
            const uint32_t before = block_scan(c[0] + c[1], sm.warp, &sum);
            if (before < need && need <= before + c[0] + c[1]) {
                const bool second = need > before + c[0];
                sm.pick[0] = second ? d0 - 1 : d0;
                sm.pick[1] = need - before - (second ? c[0] : 0u);
            }
            __syncthreads();
            prefix |= sm.pick[0] << shift;
            need = sm.pick[1];
        }
    }
    // Slots above the threshold stay, and the first `need` of those at it; with all of them, every slot counts as above.
    uint32_t gt = 0, eq = 0;
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        if (base + 32 * j >= n) continue;
        const uint32_t k = all ? 0u : key(j);
        gt += all || k > prefix;
        eq += !all && k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);  // of this warp
    eq = __reduce_add_sync(0xffffffffu, eq);
    uint32_t sum_gt, sum_eq;
    uint32_t at_gt = block_scan(lane == 0 ? gt : 0u, sm.warp, &sum_gt), at_eq = block_scan(lane == 0 ? eq : 0u, sm.warp, &sum_eq);
    at_gt = __shfl_sync(0xffffffffu, at_gt, 0);
    at_eq = __shfl_sync(0xffffffffu, at_eq, 0);
    if (csize > 1) {
        if (threadIdx.x == 0) {
            sm.total[0] = sum_gt;
            sm.total[1] = sum_eq;
        }
        cluster.sync();
        for (int r = 0; r < crank; ++r) {
            const uint2 t = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(sm.total, r));
            at_gt += t.x;
            at_eq += t.y;
        }
    }
    int32_t* kept = a.kept + (long long)b * a.budget;
    const long long orow = (long long)b * a.out_rows;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 2
    for (int j = 0; j < rounds; ++j) {
        const unsigned i = base + 32 * j;
        const bool in = i < n;
        const uint32_t k = in && !all ? key(j) : 0u;
        const bool is_gt = in && (all || k > prefix), is_eq = in && !all && k == prefix;
        const uint32_t m_gt = __ballot_sync(0xffffffffu, is_gt), m_eq = __ballot_sync(0xffffffffu, is_eq);
        const uint32_t g = at_gt + __popc(m_gt & below), r = at_eq + __popc(m_eq & below);
        at_gt += __popc(m_gt);
        at_eq += __popc(m_eq);
        if (is_gt || (is_eq && r < need)) {
            const uint32_t pos = g + (r < need ? r : need);  // the slots kept before this one
            kept[pos] = (int32_t)i;
            a.weights_out[orow + pos] = w[i];
            if (a.entry_out)
                a.entry_out[orow + pos] = a.own_entry ? a.own_entry[(long long)b * a.own_rows + i] : a.first_entry + (int)i;
        }
    }
    // pad the list
    for (long long i = (long long)want + crank * kThreads + threadIdx.x; i < a.budget; i += (long long)csize * kThreads) kept[i] = -1;
    if (crank == 0 && threadIdx.x == 0) a.count_out[b] = (int32_t)want;
    if (csize > 1) cluster.sync();  // no block leaves while another may read its shared memory
}

// One warp per four output rows of a sequence: 16-byte chunks, up to two per lane and row in flight.
__global__ void __launch_bounds__(256) evict_rows_kernel(const uint4* own, uint4* own_out, const int32_t* kept,
                                                         int own_rows, int out_rows, int budget, int chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const long long p0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
    if (p0 >= budget) return;
    int slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = p0 + i < budget ? kept[(long long)b * budget + p0 + i] : -1;
    const uint4* src = own + (long long)b * own_rows * chunks;
    uint4* dst = own_out + ((long long)b * out_rows + p0) * chunks;
    for (int c = lane; c < chunks; c += 64) {
        uint4 v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (slot[i] >= 0 && c + 32 * j < chunks) v[i][j] = __ldcs(src + (long long)slot[i] * chunks + c + 32 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (slot[i] >= 0 && c + 32 * j < chunks) __stcs(dst + (long long)i * chunks + c + 32 * j, v[i][j]);
    }
}

bool overlap(const void* p, size_t n, const void* q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && n && m && a < b + m && b < a + n;
}

}  // namespace
}  // namespace v4a

extern "C" v4a_status v4a_evict(const v4a_evict_io* io, int batch, int budget, int keep_first, int keep_recent,
                                int* dev_status, void* stream) {
    using namespace v4a;
    if (!io) return report(V4A_ERR_INVALID_ARG, "v4a_evict: io is NULL");
    if (batch < 0 || batch > 65535) return report(V4A_ERR_INVALID_ARG, "v4a_evict: batch must be in 0..65535");
    if (budget < 1 || keep_first < 0 || keep_recent < 0 || (long long)keep_first + keep_recent > budget)
        return report(V4A_ERR_INVALID_ARG, "v4a_evict: need budget >= 1 and keep_first + keep_recent <= budget");
    if (io->dtype != V4A_F32 && io->dtype != V4A_BF16) return report(V4A_ERR_UNSUPPORTED, "v4a_evict: dtype must be F32 or BF16");
    const size_t es = io->dtype == V4A_F32 ? 4 : 2;
    if (io->own_rows < 0 || io->d < 1 || io->d > 65536 || (io->d * es) % 16 || io->out_rows < budget)
        return report(V4A_ERR_INVALID_ARG, "v4a_evict: own_rows, d (rows in multiples of 16 bytes) or out_rows < budget");
    if (dev_status && reinterpret_cast<uintptr_t>(dev_status) % 4) return report(V4A_ERR_INVALID_ARG, "v4a_evict: dev_status misaligned");
    if (batch == 0) return V4A_OK;
    if ((io->own_rows > 0 && (!io->own || !io->weights)) || !io->own_out || !io->weights_out || !io->kept || !io->count_out)
        return report(V4A_ERR_INVALID_ARG, "v4a_evict: own, weights, own_out, weights_out, kept and count_out are required");
    const size_t row = io->d * es, n_in = (size_t)batch * io->own_rows, n_out = (size_t)batch * io->out_rows;
    for (const void* p : {io->own, (const void*)io->own_out})
        if (reinterpret_cast<uintptr_t>(p) % 16) return report(V4A_ERR_INVALID_ARG, "v4a_evict: own and own_out must be 16-byte aligned");
    const struct { const void* p; size_t n; } in[4] = {{io->own, n_in * row}, {io->weights, n_in * 4},
        {io->own_entry, n_in * 4}, {io->own_count, (size_t)batch * 4}},
        out[5] = {{io->own_out, n_out * row}, {io->weights_out, n_out * 4}, {io->entry_out, n_out * 4},
                  {io->kept, (size_t)batch * budget * 4}, {io->count_out, (size_t)batch * 4}};
    for (int i = 0; i < 4; ++i)
        if (reinterpret_cast<uintptr_t>(in[i].p) % 4) return report(V4A_ERR_INVALID_ARG, "v4a_evict: an input is misaligned");
    for (int i = 0; i < 5; ++i) {
        if (reinterpret_cast<uintptr_t>(out[i].p) % 4) return report(V4A_ERR_INVALID_ARG, "v4a_evict: an output is misaligned");
        for (int j = 0; j < 4; ++j)
            if (overlap(in[j].p, in[j].n, out[i].p, out[i].n)) return report(V4A_ERR_INVALID_ARG, "v4a_evict: an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[j].p, out[j].n, out[i].p, out[i].n)) return report(V4A_ERR_INVALID_ARG, "v4a_evict: two outputs overlap");
    }
    cudaStream_t st = (cudaStream_t)stream;
    if (dev_status) {
        cudaError_t e = launch_zero_words(reinterpret_cast<uint32_t*>(dev_status), 1, st);
        if (e != cudaSuccess) return report(V4A_ERR_CUDA, "v4a_evict: %s", cudaGetErrorString(e));
    }
    EvictArgs a;
    a.weights = io->weights;
    a.own_count = io->own_count;
    a.own_entry = io->own_entry;
    a.weights_out = io->weights_out;
    a.entry_out = io->entry_out;
    a.kept = io->kept;
    a.count_out = io->count_out;
    a.dev_status = dev_status;
    a.own_rows = io->own_rows;
    a.out_rows = io->out_rows;
    a.budget = budget;
    a.first = keep_first;
    a.recent = keep_recent;
    a.first_entry = io->first_entry;
    // a cluster of up to 8 blocks (the portable size) per sequence: as many as leave each thread at most 8 keys
    int cs = 1;
    while (cs < 8 && (long long)cs * kThreads * 8 < io->own_rows) cs *= 2;
    const long long per = ((long long)io->own_rows + cs * kThreads - 1) / (cs * kThreads);
    const bool keep = per <= 48;  // 4 KB each
    auto* kernel = keep ? evict_select_kernel<true> : evict_select_kernel<false>;
    const size_t smem = keep ? (size_t)per * kThreads * 4 : 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_pdl_cluster(kernel, dim3((unsigned)(batch * cs)), dim3(kThreads), smem, st, cs, a);
    if (e == cudaSuccess && io->own_rows > 0)
        e = launch_pdl(evict_rows_kernel, dim3((unsigned)((budget + 31) / 32), (unsigned)batch), dim3(256), 0, st,
                       static_cast<const uint4*>(io->own), static_cast<uint4*>(io->own_out), (const int32_t*)io->kept,
                       io->own_rows, io->out_rows, budget, (int)(row / 16));
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? V4A_OK : report(V4A_ERR_CUDA, "v4a_evict: %s", cudaGetErrorString(e));
}
