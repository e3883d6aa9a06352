// evict.cu -- eviction from a cache by accumulated attention weight.
//
// Of a sequence's n slots the `budget` heaviest stay (the first and last ones always), moved to the front
// in order.  The rows that stay are read and written once: that copy bounds the call.  Choosing them is a
// radix select over order-preserving 32-bit keys of the weights, by a block per sequence, or a cluster of
// up to 16 where a block's threads would have more than 8 weights each.  Their keys stay in shared memory.
// Histogram passes of 11, 11 and 10 bits (a cluster's counts are added up through distributed shared memory) narrow the
// threshold's digits; as soon as at most 256 candidates share them, which one or two passes usually
// achieve, the candidates are listed and ranked against each other.  That gives the last
// slot kept, (key, slot), and one ordered pass places what comes before it by ballots.  The loops are rolled: the
// code runs cold, and fetching unrolled copies costs more than they save.  evict_rows_kernel then moves
// the rows, a warp per row, four rows in flight.  Measured: 32 caches of 8,192 rows cut to half 54 us, of which the copy takes
// 41.6 (6.4 TB/s, 98% of the measured copy bandwidth) and the choice 12.7; one cache of 262,144 cut to a quarter 45 us
// (copy 22, choice 23: the passes of 16 blocks and nine cluster barriers).
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

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

constexpr int kList = 256;  // four threads rank each
constexpr int kMaxStored = 44;  // keys per thread that stay in shared memory, 4 KB a block each

struct __align__(16) EvictSmem {
    uint32_t hist[3][kBins];  // this block's counts, by pass
    uint32_t sums[3][kBins / 2];  // a cluster's counts of this block's share of the bins
    uint2 list[kList];        // block 0 of the cluster: candidates, (key, slot)
    uint2 last;               // ... the last slot kept, (key, slot)
    uint32_t listed;          // ... how many candidates
    uint32_t total;           // this block's kept slots, or its candidates
    uint32_t pick[3];         // the threshold's digit, how many of those who have it are wanted, and how many have it
    uint32_t warp[32];
};

static_assert(sizeof(EvictSmem) + kMaxStored * kThreads * 4 <= 232448, "shared memory");
static_assert(offsetof(EvictSmem, hist) % 8 == 0 && offsetof(EvictSmem, sums) % 8 == 0 && offsetof(EvictSmem, list) % 8 == 0 && offsetof(EvictSmem, last) % 8 == 0, "read in pairs");

// Exclusive prefix sum of a number per warp (the same in all its lanes) over the block's warps; *sum: the block's total.  One
// barrier; the next call's writes to warp_s come behind another one.
__device__ __forceinline__ uint32_t warps_before(uint32_t v, uint32_t* warp_s, uint32_t* sum) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0) warp_s[w] = v;
    __syncthreads();
    const uint32_t x = warp_s[lane];
    *sum = __reduce_add_sync(0xffffffffu, x);
    return __reduce_add_sync(0xffffffffu, lane < w ? x : 0u);
}

// STORED: the keys stay in (dynamic) shared memory, `rounds` per thread; else they are made again in every pass.
// Slots ascend over blocks, then warps, then a warp's rounds, then lanes; slots beyond the count have key 0, the lowest,
// and come behind the real ones that have it (NaN), so they need no exception.
template <bool STORED>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    __shared__ EvictSmem sm;
    extern __shared__ uint32_t stored[];
    constexpr uint32_t kAll = 0xffffffffu;
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
    if (threadIdx.x == 0) sm.listed = 0;
    griddep_wait();  // everything before this kernel on the stream has finished
    griddep_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto sync_all = [&] {
        if (csize > 1) cluster.sync();
        else __syncthreads();
    };
    EvictSmem& lead = csize > 1 ? *cluster.map_shared_rank(&sm, 0) : sm;
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
    uint32_t* const mine_stored = stored + threadIdx.x;  // a thread reads what it copied itself
    if (STORED && !all) {
#pragma unroll 1
        for (int j = 0; j < rounds; ++j)
            if (base + 32 * j < n) tc::cp_async_4(mine_stored + j * kThreads, w + base + 32 * j);
        tc::cp_async_commit();
        tc::cp_async_wait<0>();
    }
    const unsigned first = (unsigned)a.first, free_slots = n > (unsigned)a.first + a.recent ? n - a.first - a.recent : 0;
    auto make_key = [&](unsigned i, float x) -> uint32_t {
        uint32_t k = isnan(x) ? 0u : float_to_ordered(x);  // -inf: 0x007fffff, +inf: 0xff800000
        if (i - first >= free_slots) k = 0xffffffffu;      // always kept
        return i < n ? k : 0u;
    };
    auto key = [&](int j) -> uint32_t {
        if (STORED) return mine_stored[j * kThreads];
        const unsigned i = base + 32 * j;
        return make_key(i, i < n ? w[i] : 0.f);
    };
    // the last slot kept: larger keys and, among equal ones, lower slots come before it
    uint32_t last_key = 0u, last_slot = 0xffffffffu;
    if (!all) {
        uint32_t prefix = 0, need = want, found = 0;
        int shift = 32, pass = 0;
        do {
            const int bits = pass == 2 ? 10 : 11;
            const uint32_t digits = 1u << bits;
            const int above = shift;  // digits already known
            shift -= bits;
            uint32_t* hist = sm.hist[pass];
            if (pass == 0) {
                __syncthreads();  // the counts are zero
#pragma unroll 2
                for (int j = 0; j < rounds; ++j) {
                    uint32_t k;
                    if (STORED) {
                        const unsigned i = base + 32 * j;
                        k = make_key(i, __uint_as_float(mine_stored[j * kThreads]));
                        mine_stored[j * kThreads] = k;
                    } else {
                        k = key(j);
                    }
                    // equal weights are common, and 32 additions to one counter slow
                    const uint32_t d = k >> 21;
                    if (__all_sync(kAll, d == __shfl_sync(kAll, d, 0))) {
                        if (lane == 0) atomicAdd(&hist[d], 32u);
                    } else {
                        atomicAdd(&hist[d], 1u);
                    }
                }
            } else {
#pragma unroll 2
                for (int j = 0; j < rounds; ++j) {
                    const uint32_t k = key(j);
                    const bool mine = (k >> above) == (prefix >> above);
                    const uint32_t m = __ballot_sync(kAll, mine);
                    if (m == 0) continue;
                    const uint32_t d = (k >> shift) & (digits - 1), d0 = __shfl_sync(kAll, d, __ffs(m) - 1);
                    if (__all_sync(kAll, !mine || d == d0)) {
                        if (lane == 0) atomicAdd(&hist[d0], (uint32_t)__popc(m));
                    } else if (mine) {
                        atomicAdd(&hist[d], 1u);
                    }
                }
            }
            sync_all();
            // Two bins per thread, the highest digits first.  In a cluster every block adds up its share of the bins first, so that
            // each count crosses once.
            uint32_t c0 = 0, c1 = 0;
            const uint32_t d0 = digits - 1 - 2 * threadIdx.x;
            if (csize > 1) {
                const uint32_t share = digits / csize;
                if (threadIdx.x < share) {
                    uint32_t h[16], c = 0;  // all on their way together
#pragma unroll
                    for (int r = 0; r < 16; ++r) h[r] = r < csize ? cluster.map_shared_rank(hist, r)[crank * share + threadIdx.x] : 0u;
#pragma unroll
                    for (int r = 0; r < 16; ++r) c += h[r];
                    sm.sums[pass][threadIdx.x] = c;
                }
                cluster.sync();
                if (2 * threadIdx.x < digits) {
                    const uint32_t* from = cluster.map_shared_rank(&sm.sums[pass][0], (int)(d0 / share));
                    const uint2 h = *reinterpret_cast<const uint2*>(from + (d0 - 1) % share);
                    c0 = h.y;
                    c1 = h.x;
                }
            } else if (2 * threadIdx.x < digits) {
                const uint2 h = *reinterpret_cast<const uint2*>(hist + d0 - 1);
                c0 = h.y;
                c1 = h.x;
            }
            uint32_t run = c0 + c1, sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kAll, run, o);
                if (lane >= o) run += y;
            }
            const uint32_t before = warps_before(__shfl_sync(kAll, run, 31), sm.warp, &sum) + run - c0 - c1;
            if (before < need && need <= before + c0 + c1) {
                const bool second = need > before + c0;
                sm.pick[0] = second ? d0 - 1 : d0;
                sm.pick[1] = need - before - (second ? c0 : 0u);
                sm.pick[2] = second ? c1 : c0;
            }
            __syncthreads();
            prefix |= sm.pick[0] << shift;
            need = sm.pick[1];
            found = sm.pick[2];
            ++pass;
        } while (found > kList && need < found && shift > 0);
        auto candidate = [&](int j) { return (key(j) >> shift) == (prefix >> shift); };
        if (need == found) {  // all of them stay
            last_key = prefix;
        } else if (found <= kList) {
#pragma unroll 1
            for (int j = 0; j < rounds; ++j) {
                const bool mine = candidate(j);
                const uint32_t m = __ballot_sync(kAll, mine);
                if (m == 0) continue;
                uint32_t at = 0;
                if (lane == 0) at = atomicAdd(&lead.listed, (uint32_t)__popc(m));
                at = __shfl_sync(kAll, at, 0) + __popc(m & ((1u << lane) - 1u));
                if (mine) lead.list[at] = make_uint2(key(j), base + 32 * j);
            }
            sync_all();
            if (crank == 0) {
                const uint32_t at = threadIdx.x >> 2;
                const uint2 me = sm.list[at < found ? at : 0];
                uint32_t rank = 0;
#pragma unroll 4
                for (uint32_t i = threadIdx.x & 3; i < found; i += 4) {
                    const uint2 o = sm.list[i];
                    rank += o.x > me.x || (o.x == me.x && o.y < me.y);
                }
                rank += __shfl_xor_sync(kAll, rank, 1);
                rank += __shfl_xor_sync(kAll, rank, 2);
                if (at < found && rank == need - 1) sm.last = me;
            }
            sync_all();
            last_key = lead.last.x;
            last_slot = lead.last.y;
        } else {  // more equal keys than the list holds: the need-th of them in the order of the slots
            uint32_t mine = 0, sum;
#pragma unroll 1
            for (int j = 0; j < rounds; ++j) mine += candidate(j);
            mine = __reduce_add_sync(kAll, mine);
            uint32_t at = warps_before(mine, sm.warp, &sum);
            if (threadIdx.x == 0) sm.total = sum;
            sync_all();
            for (int r = 0; r < crank; ++r) at += *cluster.map_shared_rank(&sm.total, r);
            if (at < need && need <= at + mine) {
#pragma unroll 1
                for (int j = 0; j < rounds; ++j) {
                    const uint32_t m = __ballot_sync(kAll, candidate(j));
                    if (((m >> lane) & 1) && at + __popc(m & ((1u << lane) - 1u)) == need - 1) lead.last = make_uint2(prefix, base + 32 * j);
                    at += __popc(m);
                }
            }
            sync_all();
            last_key = prefix;
            last_slot = lead.last.y;
        }
    }
    auto stays = [&](int j) {
        const unsigned i = base + 32 * j;
        if (all) return i < n;
        const uint32_t k = key(j);
        return k > last_key || (k == last_key && i <= last_slot);
    };
    uint32_t mine = 0, sum;
#pragma unroll 2
    for (int j = 0; j < rounds; ++j) mine += stays(j);
    __syncthreads();  // sm.warp was read
    uint32_t at = warps_before(__reduce_add_sync(kAll, mine), sm.warp, &sum);
    if (csize > 1) {
        cluster.sync();  // sm.total was read
        if (threadIdx.x == 0) sm.total = sum;
        cluster.sync();
        for (int r = 0; r < crank; ++r) at += *cluster.map_shared_rank(&sm.total, r);
    }
    int32_t* kept = a.kept + (long long)b * a.budget;
    const long long orow = (long long)b * a.out_rows;
    float* weights_out = a.weights_out + orow;
    int32_t* entry_out = a.entry_out ? a.entry_out + orow : nullptr;
    const int32_t* own_entry = a.own_entry ? a.own_entry + (long long)b * a.own_rows : nullptr;
#pragma unroll 2
    for (int j = 0; j < rounds; ++j) {
        const bool s = stays(j);
        const uint32_t m = __ballot_sync(kAll, s), pos = at + __popc(m & ((1u << lane) - 1u));
        at += __popc(m);
        if (s) {
            const unsigned i = base + 32 * j;
            kept[pos] = (int32_t)i;
            weights_out[pos] = w[i];
            if (entry_out) entry_out[pos] = own_entry ? own_entry[i] : a.first_entry + (int)i;
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
    // no early griddep_launch_dependents: blocks of the next kernel that wait here take room from the copies in flight
    // (32 caches of 8,192 rows: 41 us without, 51 with)
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
    if (io->entry_out && !io->own_entry && (long long)io->first_entry + io->own_rows - 1 > 0x7fffffffLL)
        return report(V4A_ERR_INVALID_ARG, "v4a_evict: first_entry + own_rows passes 2^31");
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
    // a cluster per sequence, as many blocks as leave each thread at most 8 weights: up to 8, which every device
    // schedules, or 16 where this one does
    int cs = 1;
    while (cs < 16 && (long long)cs * kThreads * 8 < io->own_rows) cs *= 2;
    cudaError_t e = cudaSuccess;
    auto launch = [&](int blocks) {
        const long long per = ((long long)io->own_rows + blocks * kThreads - 1) / (blocks * kThreads);
        const bool keep = per <= kMaxStored;
        auto* kernel = keep ? evict_select_kernel<true> : evict_select_kernel<false>;
        const size_t smem = keep ? (size_t)per * kThreads * 4 : 0;
        // the most of any call: host threads share the attribute, and another one may set it before this launch
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, keep ? kMaxStored * kThreads * 4 : 0);
        if (e == cudaSuccess && blocks > 8) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)blocks);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)blocks;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int fit = 0;
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
            if (e != cudaSuccess || fit < 1) {
                cudaGetLastError();
                return false;
            }
        }
        if (e == cudaSuccess) e = launch_pdl_cluster(kernel, dim3((unsigned)(batch * blocks)), dim3(kThreads), smem, st, blocks, a);
        return true;
    };
    if (!launch(cs)) launch(8);
    if (e == cudaSuccess && io->own_rows > 0)
        e = launch_pdl(evict_rows_kernel, dim3(((unsigned)budget + 31u) / 32u, (unsigned)batch), dim3(256), 0, st,
                       static_cast<const uint4*>(io->own), static_cast<uint4*>(io->own_out), (const int32_t*)io->kept,
                       io->own_rows, io->out_rows, budget, (int)(row / 16));
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? V4A_OK : report(V4A_ERR_CUDA, "v4a_evict: %s", cudaGetErrorString(e));
}
