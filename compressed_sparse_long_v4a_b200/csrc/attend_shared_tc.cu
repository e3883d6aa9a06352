// attend_shared_tc.cu -- tensor-core (tcgen05 / TMEM / TMA) HCA attention over a prefix that a batch shares
// (bf16, d = 512, any number of heads).
//
//     out = sum_r p_r v_r,  p = softmax_r(q . v_r / sqrt(d)),  lse = log sum_r e^{q . v_r / sqrt(d)}
//
// Every query of the batch sees the whole prefix, so the rows (sequence, query, head) of all sequences are
// one matrix, taken in groups of 128 that ignore where a sequence ends.  A group's keys come in boxes of 64:
// the prefix, then the own slots and the window of each sequence that has rows in the group; rows of
// other sequences are masked there.  The boxes of all groups form one flat sequence, cut into equal ranges;
// two boxes that hold anything, of whatever kind, make a tile of 128 keys.
//
// A range goes to a CTA pair (two SMs, cta_group::2), each CTA holding 64 of the 128 rows.  Per tile
//     S  = Q K^T   M = 128 rows x N = 128 keys x K = 512   (each CTA brings a box of 64 of the keys)
//     P  = softmax(S), four threads per row, lazily rescaled maximum
//     O += P V     M = 128 x N = 2 x 256 dims x K = 128 keys (each CTA brings half of the dims)
// With 64 rows of 512 dims a CTA's O is half of tensor memory, and 64 rows at the full rate of the tensor
// cores need the pair (measured per MMA of K = 16: pair M = 128, N = 128: 32 cycles, N = 256: 66; one CTA, M = 64,
// N = 64: 38, N = 128: 64).  Shared memory feeds both operands: with N = 64 it, not the tensor core, bounds S
// (26 cycles instead of 16), hence tiles of 128 keys in two stages rather than 64 in four.
// Since S wants all dims of half of the keys and O half of the dims of all keys, a stage of 64 KB is used
// twice: it is loaded with this CTA's 64 keys ("X"), and once S is done the slabs of dims that O does not need
// here make room for the other 64 keys of those that it does ("Z").  So a tile costs 96 KB of loads per CTA
// and 64 KB of shared memory, and two stages fit beside the 64 KB of queries.
//
// Slabs are 64 dims (128 bytes) wide; slab s of the CTA's own keys lies at 8192 s.  CTA 0 has the even slabs
// of O, CTA 1 the odd ones: block u (16384 u) becomes the 128 keys of slab 2 u + rank.
//
// What bounds it: two stages, each turned over in a chain of 6,400 cycles (load, S, softmax, O), are a tile in 3,200, of which
// the tensor cores are busy 2,100; by the counters nothing is saturated (tensor pipe 43%, L1 38%, DRAM 5%).  By count a
// tile moves 340 KB through a CTA's shared memory (operands of the MMAs, loads, P), which at 128 bytes a cycle would
// bound it at 2,650, and 96 KB into it from L2, 30 of the 45 bytes a cycle that loads alone reach.  Tiles of 64 keys in
// four stages took 2,300 cycles per 64 keys and of 96 in three 1,750, against 1,610.  A piece costs another ~6,000 cycles
// (128 KB of O per CTA at 32 bytes a cycle).  32 sequences of 64 heads over 8,192 shared entries: 51 us (42 + 9 for the join),
// 0.68 PFLOP/s, 42% of the measured bf16 peak.
//
// The ranges are cut by what the caches have room for, since the host does not know the counts: where they hold less, the
// pairs with the prefix have more to do than the others.  The same with 64 own slots filled per sequence: 45 us in caches of 64,
// 51 in 1,024, 67 in 4,096, 91 in 8,192.
//
// Masked places may hold anything.  A NaN or infinity in a row of K = V makes the raw S of every row of the
// matrix non-finite at that key, so the softmax threads see it, also for rows that do not see the
// key; such a tile's V is scrubbed of non-finite values before the product (0 x NaN would spoil the rows of
// other sequences).  Rows that do see the key have a NaN in P, or weight 0 for a logit of -inf.
//
// Warps: 0 loads Q and X, 10 loads Z, 1 and 11 of CTA 0 issue the MMAs, 1 of CTA 1 reports that Z is there, 2-9 run the
// softmax and write pieces.
// Every wait is bounded; on a time-out both CTAs record a device fault, their pieces become NaN and they
// wind down.  Pieces (m, l, O) are merged by shared_tc_join_kernel: out = sum_i e^{m_i - m} o_i / l.
#include "common.cuh"
#include "internal.h"
#include "shared.h"
#include "tc_pair.cuh"
#include "tensor_map.h"
#include "turns.h"

namespace v4a {
namespace {

constexpr int kD = 512;
constexpr int kRows = 128;          // rows of a group
constexpr int kHalf = 64;           // ... of one CTA
constexpr int kBox = 64;            // keys of a box, which one load brings
constexpr int kKeys = 2 * kBox;     // keys of a tile: a box per CTA
constexpr int kStages = 2;          // and S buffers
constexpr int kPairs = kNumSMs / 2;
constexpr uint32_t kXBytes = kBox * kD * 2, kZBytes = kXBytes / 2, kQBytes = kHalf * kD * 2;
constexpr uint32_t kSlab = kBox * 128;  // 64 dims of a CTA's keys
constexpr uint32_t kColS = 256, kColsS = 64, kTmemCols = 512;  // O: columns 0-255
constexpr int kThreads = 12 * 32;
constexpr float kSlack = 8.0f;           // keep a stale running max until the true one exceeds it by 2^8
constexpr uint32_t kIdescQK = tc::idesc_f16(128, kKeys, 0, 0), kIdescPV = tc::idesc_f16(128, 256, 0, 1);

enum Kind { kPrefix, kOwn, kWindow };
// first, last: of its piece; end: last of the range; none: the range holds nothing; plain: of the prefix alone; same: a
// full tile of the prefix behind another one
enum : int { kFirst = 1, kLast = 2, kEnd = 4, kNone = 8, kPlain = 16, kSame = 32 };

struct Box {
    int kind, b;         // b: the sequence (own, window)
    int y, n;            // first row of its 64 in prefix / own / ring, rows that count
    long long p0;        // what row y holds: own slot, or position
};
struct __align__(16) Tile {
    int flags, group;
    Box box[2];          // of CTA 0, which are keys 0-63, and of CTA 1
};

struct __align__(1024) Smem {
    uint8_t q[kQBytes];
    uint8_t kv[kStages][kXBytes];
    uint8_t p[2][kHalf * 128];  // by half of the keys
    Tile tile[kStages];  // what each stage holds
    float mx[4][kHalf];  // row maxima of a tile's quarters
    float ls[4][kHalf];
    // x_full, z_ready, p_full and q_full count in CTA 0 only
    uint64_t told[kStages], x_full[kStages][2], z_full[kStages], z_ready[kStages], kv_empty[kStages][2], s_full[kStages];
    uint64_t p_full, p_free;
    uint64_t q_full, q_empty, drain;
    int abort_flag;
    uint32_t tmem_base;
};

struct Range {
    int g, i, n;   // a pair's first box: its group and its place in it; how many boxes
    int last;      // group of the last one
};

constexpr int kSpans = 256;

struct PairArgs {
    SharedArgs a;
    float2* part_ml;       // [pieces][128] (m in base-2 logits, l); piece = pair + group
    float4* part_o;        // [pieces][128 quads of dims][128 rows]
    long long total;       // boxes of all groups
    unsigned rows, per_seq, lcm;  // batch * n_q * heads; n_q * heads; least common multiple of that and 128
    int groups, pairs;
    int pre_tail;          // keys of the prefix's last box
    int pre, own, win;     // boxes: prefix; own and window of a sequence (win: one more than the window fills, for a
                           // ring that wraps inside it)
    float scale_log2;
    uint32_t polls;        // of a wait, before it gives up
    int withhold;          // test hook (v4a_test_attend_fault): the tile of every pair whose loads are left out, or -1
    Range range[kPairs];
    struct { unsigned char first, n; } span[kSpans];  // the pairs that have boxes of a group, for the first groups
};

// Boxes of the groups before g (host).  A group has `pre` boxes and own + win for every sequence with rows in it: one
// more than the sequences that begin inside it, behind its first row.
long long boxes_before(const PairArgs& c, int g) {
    if (g == 0) return 0;
    const unsigned long long e = (unsigned long long)g * kRows;
    const unsigned last = (unsigned)(e < c.rows ? e : c.rows) - 1;
    const long long seqs = g + (long long)(last / c.per_seq) - (long long)(last / c.lcm);
    return (long long)g * c.pre + seqs * (c.own + c.win);
}

// The pairs that have boxes of group g: from the last one that begins no later than its first box to the last that begins
// no later than its last.
__host__ __device__ inline void find_pairs(const PairArgs& c, int g, int* first, int* n) {
    int p0 = 0, p1 = 0;
    for (int k = 64; k > 0; k >>= 1) {
        if (p0 + k < c.pairs && (c.range[p0 + k].g < g || (c.range[p0 + k].g == g && c.range[p0 + k].i == 0))) p0 += k;
        if (p1 + k < c.pairs && c.range[p1 + k].g <= g) p1 += k;
    }
    *first = p0;
    *n = c.pairs > 0 ? p1 - p0 + 1 : 0;
}

// walks the boxes of a range that hold anything
struct Walk {
    int left, g, i, per;        // boxes to go; group, box in it, its boxes
    int s, w;                   // sequence and its box
    bool entered;               // the sequence's numbers are read
    int count, row0, n_a, n_w;  // own slots; window: ring row of position lo, positions before the ring's end, all
    long long lo;

    __device__ void enter_group(const PairArgs& c) {
        const unsigned r0 = (unsigned)g * kRows, r1 = min(r0 + kRows, c.rows) - 1;
        s = (int)(r0 / c.per_seq);
        per = c.pre + ((int)(r1 / c.per_seq) - s + 1) * (c.own + c.win);
        entered = false;
        w = 0;
    }
    __device__ void enter_sequence(const PairArgs& c) {
        const long long len = seq_len(c.a, s);
        count = len > 0 ? own_slots(c.a, s) : 0;
        lo = len - c.a.n_q - c.a.window + 1;
        lo = lo < 0 ? 0 : lo;
        n_w = c.a.window > 0 && len > 0 ? (int)(len - lo) : 0;
        row0 = n_w > 0 ? (int)(lo % c.a.ring_rows) : 0;
        n_a = n_w < c.a.ring_rows - row0 ? n_w : c.a.ring_rows - row0;
    }
    __device__ Walk(const PairArgs& c, int pair) {
        const Range r = c.range[pair];
        left = r.n;
        g = r.g;
        i = r.i;
        enter_group(c);
        if (i >= c.pre) {
            const int k = i - c.pre;
            s += k / (c.own + c.win);
            w = k % (c.own + c.win);
        }
    }
    __device__ bool next(const PairArgs& c, Box& t, int& group) {
        while (left > 0) {
            if (i == per) {
                ++g;
                i = 0;
                enter_group(c);
            }
            --left;
            group = g;
            if (i < c.pre) {
                t.kind = kPrefix;
                t.y = i * kBox;
                t.n = i + 1 == c.pre ? c.pre_tail : kBox;
                t.b = 0;
                t.p0 = t.y;
                ++i;
            } else {
                if (!entered) enter_sequence(c);
                entered = true;
                t.b = s;
                if (w < c.own) {
                    t.kind = kOwn;
                    t.y = w * kBox;
                    t.p0 = t.y;
                    t.n = min(count - t.y, kBox);
                } else {
                    int at = (w - c.own) * kBox;
                    const int a_rows = (n_a + kBox - 1) / kBox * kBox;
                    t.kind = kWindow;
                    if (at < a_rows) {
                        t.y = row0 + at;
                        t.p0 = lo + at;
                        t.n = min(n_a - at, kBox);
                    } else {
                        at -= a_rows;
                        t.y = at;
                        t.p0 = lo + n_a + at;
                        t.n = min(n_w - n_a - at, kBox);
                    }
                }
                ++i;
                if (++w == c.own + c.win) {
                    w = 0;
                    ++s;
                    entered = false;
                }
            }
            if (t.n > 0) return true;
        }
        return false;
    }
};

__device__ void fault(Smem& sm, const PairArgs& c, uint32_t rank) {
    *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
    tc::peer_store(tc::peer_addr(&sm.abort_flag, rank ^ 1), 1);
    if (c.a.dev_status) atomicExch(c.a.dev_status, (int)V4A_ERR_DEVICE_FAULT);
}
__device__ __forceinline__ bool aborted(Smem& sm) { return *reinterpret_cast<volatile int*>(&sm.abort_flag) != 0; }

// ---------------------------------------------------------------------
// warp 0, one lane: finds the tiles, tells the other warps of this CTA about them, and loads the queries and this CTA's
// 64 keys.  Both CTAs' copies complete on CTA 0's barriers, which expect the bytes of both.
// ---------------------------------------------------------------------
struct Maps {
    CUtensorMap x[3], z[3], q;  // by Kind: 64 rows x 4 slabs; 64 rows x 1 slab
};

__device__ void load_x(Smem& sm, const PairArgs& c, const Maps& maps, int pair, uint32_t rank) {
    const uint64_t again = tc::l2_evict_normal(), once = tc::l2_stream_policy((int)((c.per_seq + kRows - 1) / kRows));
    const uint32_t x_full = tc::peer_addr(&sm.x_full[0][0], 0), q_full = tc::peer_addr(&sm.q_full, 0);
    Walk walk(c, pair);
    Tile t;
    Box nxt;  // the box behind the tile's
    int piece = 0, group = -1, nxt_group = 0;
    bool ok = true, more = true, plain = false;
    auto load = [&](int st, int h) {
        const Box& x = t.box[rank];
        tc::tma_load_4d_pair(sm.kv[st] + 4 * kSlab * h, &maps.x[x.kind], 0, x.y, 4 * h, x.b, x_full + 16 * st + 8 * h,
                             x.kind == kPrefix ? again : once);
    };
    auto load_q = [&] {
        tc::tma_load_4d_pair(sm.q, &maps.q, 0, t.group * kRows + (int)rank * kHalf, 0, 0, q_full, again);
    };
    auto set_flags = [&] {  // with the box behind the tile known
        const bool first = t.group != group, all = t.box[0].kind == kPrefix && t.box[1].kind == kPrefix;
        const bool full = all && t.box[0].n == kBox && t.box[1].n == kBox;
        t.flags = (first ? kFirst : 0) | (!more ? kLast | kEnd : nxt_group != t.group ? kLast : 0) | (all ? kPlain : 0) |
                  (full && plain && !first ? kSame : 0);
        group = t.group;
        plain = full;
    };
    auto next_tile = [&] {  // two boxes of one group, or the last one and an empty one (rows beyond every array: zeros)
        t.group = nxt_group;
        t.box[0] = t.box[1] = nxt;
        t.box[1].n = 0;
        t.box[1].y = 0x3fffffff;
        more = walk.next(c, nxt, nxt_group);
        if (more && nxt_group == t.group) {
            t.box[1] = nxt;
            more = walk.next(c, nxt, nxt_group);
        }
        set_flags();
    };
    // What can be done before the kernel before this one has finished: a tile of the prefix depends on sizes alone.  Its
    // loads are the first thing then (the barriers complete only once their bytes are announced below).
    const bool early = c.range[pair].i + 1 < c.pre && c.range[pair].n > 1;
    tc::prefetch_map(&maps.q);
    tc::prefetch_map(&maps.x[kPrefix]);
    tc::prefetch_map(&maps.z[kPrefix]);
    if (early) {
        walk.next(c, t.box[0], t.group);
        walk.next(c, t.box[1], t.group);
    }
    griddep_wait();
    if (early) {
        load_q();
        if (c.withhold != 0) {
            load(0, 0);
            load(0, 1);
        }
        more = walk.next(c, nxt, nxt_group);
        set_flags();
    } else if (walk.next(c, nxt, nxt_group)) {
        next_tile();
    } else {
        t.flags = kNone;
        sm.tile[0].flags = kNone;
        tc::mbar_arrive(&sm.told[0]);
        if (rank == 0) tc::mbar_arrive(&sm.x_full[0][0]);
    }
    for (int j = 0; !(t.flags & kNone); ++j) {
        const int st = j % kStages;
        if (aborted(sm)) ok = false;
        if (ok && (t.flags & kFirst)) {
            if (piece > 0) ok = tc::mbar_wait(&sm.q_empty, (piece - 1) & 1, c.polls);
            if (ok && rank == 0) tc::mbar_arrive_expect_tx(&sm.q_full, 2 * kQBytes);
            if (ok && (j > 0 || !early)) load_q();
            ++piece;
        }
        // slabs 0-3, then 4-7: O is done with them one after the other
        for (int h = 0; ok && h < 2; ++h) {
            if (j >= kStages) ok = tc::mbar_wait(&sm.kv_empty[st][h], (j / kStages - 1) & 1, c.polls);
            if (!ok) break;
            if (h == 0) {
                sm.tile[st] = t;
                tc::mbar_arrive(&sm.told[st]);
            }
            if (j == c.withhold) continue;
            if (rank == 0) tc::mbar_arrive_expect_tx(&sm.x_full[st][h], kXBytes);
            if (j > 0 || !early) load(st, h);
        }
        if (!ok || (t.flags & kEnd)) break;
        next_tile();
    }
    if (!ok) {  // what was asked for lands long before this ends
        fault(sm, c, rank);
        for (int i = 0; i < 2000; ++i) __nanosleep(1000);
    }
}

// warp 10, one lane: the other CTA's 64 keys of this CTA's slabs, once S has been computed
__device__ void load_z(Smem& sm, const PairArgs& c, const Maps& maps, uint32_t rank) {
    const uint64_t again = tc::l2_evict_normal();
    const uint32_t other = rank ^ 1;
    for (int j = 0;; ++j) {
        const int st = j % kStages;
        const uint32_t phase = (j / kStages) & 1;
        if (aborted(sm) || !tc::mbar_wait(&sm.told[st], phase, c.polls)) { fault(sm, c, rank); return; }
        const int flags = sm.tile[st].flags;
        if (flags & kNone) return;
        const Box z = sm.tile[st].box[other];
        if (!tc::mbar_wait(&sm.s_full[st], phase, c.polls)) { fault(sm, c, rank); return; }
        tc::mbar_arrive_expect_tx(&sm.z_full[st], kZBytes);
#pragma unroll 1
        for (int u = 0; u < 4; ++u)
            tc::tma_load_4d(sm.kv[st] + kSlab * (2 * u + other), &maps.z[z.kind], 0, z.y, 2 * u + (int)rank, z.b, &sm.z_full[st], again);
        if (flags & kEnd) return;
    }
}

// warp 1 of CTA 1, one lane: tells CTA 0 that Z has landed here
__device__ void pass_on_z(Smem& sm, const PairArgs& c) {
    const uint32_t ready = tc::peer_addr(&sm.z_ready[0], 0);
    for (int j = 0;; ++j) {
        const int st = j % kStages;
        const uint32_t phase = (j / kStages) & 1;
        if (aborted(sm) || !tc::mbar_wait(&sm.told[st], phase, c.polls)) { fault(sm, c, 1); return; }
        const int flags = sm.tile[st].flags;
        if (flags & kNone) return;
        if (!tc::mbar_wait(&sm.z_full[st], phase, c.polls)) { fault(sm, c, 1); return; }
        tc::fence_proxy_async();
        tc::peer_arrive(ready + 8 * st);
        if (flags & kEnd) return;
    }
}

// ---------------------------------------------------------------------
// CTA 0, warps 1 and 11: every MMA of the pair, S and O by a warp each, so that the waits of one are filled by the
// other's products.  The code is kept small: these loops run between those of the softmax, and a line of
// instructions fetched again costs more than an MMA (all 40 of a tile unrolled, a copy per stage, took 75 cycles
// each to issue, rolled 44; the smaller ones execute in 26).
// ---------------------------------------------------------------------
// Descriptors: the address, in 16-byte units, is in the low word and the rest of the high one the same for all.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint32_t polls) {
    for (uint32_t i = 0; i < polls; ++i)
        if (__any_sync(kAll, tc::mbar_try_cluster(bar, parity))) return true;
    return false;
}

// S = Q K^T: A = Q (64 rows per CTA), B = 64 keys per CTA.  One S buffer per stage: a stage that is free again means
// that its S was read.
__device__ void issue_s(Smem& sm, const PairArgs& c, uint32_t tmem) {
    const uint32_t a0 = (uint32_t)tc::sw128_desc(tc::smem_u32(sm.q), 16, 1024), b0 = (uint32_t)tc::sw128_desc(tc::smem_u32(sm.kv), 16, 1024);
    int pieces = 0;
    bool ok = wait_cluster(&sm.x_full[0][0], 0, c.polls);
    int flags = ok ? sm.tile[0].flags : kNone;
    for (int j = 0; ok && !(flags & kNone); ++j) {
        const int st = j % kStages, st1 = (j + 1) % kStages;
        const uint32_t phase1 = (uint32_t)((j + 1) / kStages) & 1;
        if (flags & kFirst) ok = wait_cluster(&sm.q_full, pieces++ & 1, c.polls);
        if (!ok) break;
        tc::tc_fence_after();
        uint32_t a = a0, b = b0 + st * (kXBytes >> 4);
        const uint32_t d = tmem + kColS + kColsS * st;
#pragma unroll 1
        for (int s = 0; s < 8; ++s) {
            if (s == 4 && !wait_cluster(&sm.x_full[st][1], (uint32_t)(j / kStages) & 1, c.polls)) ok = false;
            if (s == 4) tc::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc::mma_f16_pair(d, a + 2 * kk, b + 2 * kk, kDescHigh, kIdescQK, (uint32_t)(s | kk));
            a += kSlab >> 4;  // a slab of 64 rows of Q is as large
            b += kSlab >> 4;
        }
        if (!ok) break;
        tc::mma_commit_pair(&sm.s_full[st]);
        if (flags & kLast) tc::mma_commit_pair(&sm.q_empty);
        if (flags & kEnd) break;
        ok = wait_cluster(&sm.x_full[st1][0], phase1, c.polls);
        flags = sm.tile[st1].flags;
    }
    if (!ok) fault(sm, c, 0);
    tc::mma_commit_pair(&sm.drain);
}
// O += P V: A = P (64 rows of 128 bytes per CTA and half of the keys), B = 16 keys x 128 dims (2 blocks, 16 KB apart) per
// CTA
__device__ void issue_o(Smem& sm, const PairArgs& c, uint32_t tmem) {
    const uint32_t a0 = (uint32_t)tc::sw128_desc(tc::smem_u32(sm.p), 16, 1024), b0 = (uint32_t)tc::sw128_desc(tc::smem_u32(sm.kv), 2 * kSlab, 1024);
    bool ok = true;
    for (int j = 0;; ++j) {
        const int st = j % kStages;
        const uint32_t phase = (uint32_t)(j / kStages) & 1;
        ok = wait_cluster(&sm.told[st], phase, c.polls);
        if (!ok) break;
        const int flags = sm.tile[st].flags;
        if (flags & kNone) break;
        ok = wait_cluster(&sm.z_full[st], phase, c.polls) && wait_cluster(&sm.z_ready[st], phase, c.polls) && wait_cluster(&sm.p_full, (uint32_t)j & 1, c.polls);
        if (!ok) break;
        tc::tc_fence_after();
        uint32_t b = b0 + st * (kXBytes >> 4);
        const uint32_t add = flags & kFirst ? 0 : 1;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // 256 dims
            uint32_t a = a0;
#pragma unroll 1
            for (int kk = 0; kk < kKeys / 16; kk += 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_f16_pair(tmem + 128 * h, a + 2 * k, b + (2048 >> 4) * k, kDescHigh, kIdescPV, (uint32_t)(kk | k) | add);
                a += kHalf * 128 >> 4;
                b += 4 * 2048 >> 4;
            }
            b += 2 * kSlab >> 4;
            tc::mma_commit_pair(&sm.kv_empty[st][h]);
        }
        tc::mma_commit_pair(&sm.p_free);
        if (flags & kEnd) break;
    }
    if (!ok) fault(sm, c, 0);
    tc::mma_commit_pair(&sm.drain);
}

// ---------------------------------------------------------------------
// warps 2-9: softmax, rescaling, pieces
// ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t low_bits(long long n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// zero what is not finite in 8 bf16
__device__ __forceinline__ uint32_t scrub(uint32_t x) {
    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
    return x;
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp; results below the normal range become 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ void softmax(Smem& sm, const PairArgs& c, uint32_t tmem, int pair, uint32_t rank) {
    const SharedArgs& a = c.a;
    // TMEM lanes 32 sub ..: rows 32 (sub & 1) .., of a tile's keys (and of O's slabs) half sub >> 1; the second
    // four warps take the second 32 of those keys.  So four threads share a row, each a quarter of the keys.
    const int sub = (threadIdx.x >> 5) & 3, wg = (threadIdx.x - 64) >> 7;
    const int lane = threadIdx.x & 31, half = sub >> 1, r = 32 * (sub & 1) + lane, quarter = 2 * half + wg;
    const uint32_t lanes = tmem + ((uint32_t)(32 * sub) << 16);
    const uint32_t p_full = tc::peer_addr(&sm.p_full, 0);
    uint8_t* const prow = sm.p[half] + (r >> 3) * 1024 + (r & 7) * 128;
    const int first_group = c.range[pair].g, last_group = c.range[pair].last;
    auto ml = [&](int group) -> float2& { return c.part_ml[(pair + (long long)group) * kRows + rank * kHalf + r]; };
    int next_group = first_group;
    float m_run = -INFINITY, l_run = 0.f;
    // this row's query
    int b = 0;
    long long pos = 0, seen = 0;
    bool alive = false, ok = true;
    uint32_t mask = 0;  // of this thread's 32 keys
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(kAll, ok && tc::mbar_test(bar, parity))) return true;
        if (ok) ok = tc::mbar_wait(bar, parity, c.polls);
        ok = __all_sync(kAll, ok);
        return ok;
    };
    // a time-out makes `ok` false, which the barrier of the (next) tile tells all eight warps: they leave together
    for (int j = 0;; ++j) {
        const int st = j % kStages;
        const uint32_t phase = (j / kStages) & 1;
        int flags = kSame | kPlain, group = first_group;
        if (wait(&sm.told[st], phase)) {
            flags = sm.tile[st].flags;
            group = sm.tile[st].group;
        }
        if (flags & kNone) break;
        if (flags & kFirst) {
            m_run = -INFINITY;
            l_run = 0.f;
            const unsigned row = (unsigned)group * kRows + rank * kHalf + r;
            alive = row < c.rows;
            if (alive) {
                const unsigned query = row / (unsigned)a.heads;
                b = (int)(query / (unsigned)a.n_q);
                pos = seq_len(a, b) - a.n_q + (int)(query % (unsigned)a.n_q);
                alive = has_candidates(a, pos);
                seen = seen_entries(a, pos);
            }
        }
        if (!(flags & kSame)) {
            const Box t = sm.tile[st].box[half];
            mask = alive ? ~0u : 0u;
            const int key0 = 32 * wg, n = t.n - key0;
            if (t.kind == kPrefix) {
                mask &= low_bits(n);
            } else if (t.kind == kOwn) {
                const bool mine = alive && b == t.b;
                if (a.own_entry) {
                    int e = -1;
                    if (lane < n) e = a.own_entry[(long long)t.b * a.own_rows + t.p0 + key0 + lane];
                    mask = 0;
#pragma unroll 4
                    for (int k = 0; k < 32; ++k) {
                        const int ek = __shfl_sync(kAll, e, k);
                        mask |= (uint32_t)(ek >= 0 && ek < seen) << k;
                    }
                    if (!mine) mask = 0;
                } else {
                    const long long lim = seen - a.n_prefix - t.p0 - key0;
                    mask = mine ? mask & low_bits(lim < n ? lim : n) : 0u;
                }
            } else {
                const long long from = pos - a.window + 1 - t.p0 - key0, to = pos + 1 - t.p0 - key0;
                mask = alive && b == t.b ? mask & low_bits(to < n ? to : n) & ~low_bits(from) : 0u;
            }
        }
        float x[32];
        if (wait(&sm.s_full[st], phase)) {
            tc::tc_fence_after();
            uint32_t u[32];
            tc::tmem_ld_x32(lanes + kColS + kColsS * st + 32 * wg, u);
            tc::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(u[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = 0.f;
        }
        bool odd = false;  // a key of this tile is not finite
        if (!(flags & kPlain)) {
            float d = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k) d = fmaf(x[k], 0.f, d);
            odd = !(d == 0.f);
        }
        if (mask != ~0u) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = (mask >> k) & 1 ? x[k] : -INFINITY;
        }
        float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k < 32; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], x[k]);
        float mt = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * c.scale_log2;  // of NaN alone: NaN
        // The weights are taken against the maximum so far.  Where that was too low for some row, the four threads of each row agree on
        // a new one and take them again: at the start of a piece, hardly ever later.
        uint32_t pk[16];
        float ls[2] = {0.f, 0.f}, alpha = 1.f;
        bool leave = false, settled = false;
        const bool fresh = flags & kFirst;  // nothing to take them against yet
#pragma unroll 1
        for (;;) {
            if (!fresh || settled) {
                const float sub_m = m_run == -INFINITY ? 0.f : m_run;  // nothing seen so far: every x is -inf
                ls[0] = ls[1] = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float p0 = exp2_fast(fmaf(x[2 * k], c.scale_log2, -sub_m)), p1 = exp2_fast(fmaf(x[2 * k + 1], c.scale_log2, -sub_m));
                    ls[k & 1] += p0 + p1;  // the sum is of the unrounded weights
                    // To V's type, which the tensor cores multiply it with: off by up to 2^-8 of itself, also for fp32 outputs (two
                    // bf16 parts would double the products of O).  The outputs' error against 64 bits is 1.8e-3 to 2.0e-3 with it,
                    // relative, as bf16 outputs, 1.65e-3 without.
                    const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
                    pk[k] = *reinterpret_cast<const uint32_t*>(&pb);
                }
            }
            if (settled || !tc::named_barrier_or(1, 256, fresh || mt > m_run + kSlack || odd || !ok)) break;
            settled = true;
            sm.mx[quarter][r] = mt;
            leave = tc::named_barrier_or(1, 256, !ok);
            if (leave) break;
            odd = tc::named_barrier_or(1, 256, odd);
            mt = fmaxf(fmaxf(sm.mx[0][r], sm.mx[1][r]), fmaxf(sm.mx[2][r], sm.mx[3][r]));
            if (mt > m_run + kSlack) {
                if (m_run != -INFINITY) alpha = exp2f(m_run - mt);
                m_run = mt;
            }
        }
        if (leave) {
            ok = false;
            break;
        }
        l_run = l_run * alpha + (ls[0] + ls[1]);
        // P and O are free once the product of the tile before is done
        const bool free = j == 0 || wait(&sm.p_free, (j - 1) & 1);
        if (__any_sync(kAll, alpha != 1.f) && free) {
            // O follows the maximum: 128 columns of this warp's lanes
            tc::tc_fence_after();
#pragma unroll 1
            for (int q = 4 * wg; q < 4 * wg + 4; ++q) {
                uint32_t o[32];
                tc::tmem_ld_x32(lanes + 32 * q, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tc::tmem_st_x32(lanes + 32 * q, o);
            }
            tc::tmem_st_wait();
        }
        if (free) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(prow + (((4 * wg + k) ^ (r & 7)) << 4)) =
                    make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
        if (odd && wait(&sm.z_full[st], phase)) {
            // both halves of V are here: scrub it
            uint4* v = reinterpret_cast<uint4*>(sm.kv[st]);
            for (int k = threadIdx.x - 64; k < (int)(kXBytes / 16); k += 256) {
                const uint4 w = v[k];
                v[k] = make_uint4(scrub(w.x), scrub(w.y), scrub(w.z), scrub(w.w));
            }
        }
        tc::fence_proxy_async();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) tc::peer_arrive(p_full);

        if (flags & kLast) {
            // write the piece
            for (; next_group < group; ++next_group)  // groups of the range without a box that holds anything
                if (quarter == 0) ml(next_group) = make_float2(-INFINITY, 0.f);
            ++next_group;
            sm.ls[quarter][r] = l_run;
            tc::named_barrier(1, 256);
            if (quarter == 0) {
                const float l = (l_run + sm.ls[1][r]) + (sm.ls[2][r] + sm.ls[3][r]);
                ml(group) = make_float2(isnan(l) ? NAN : m_run, l);
            }
            if (wait(&sm.p_free, j & 1)) {
                tc::tc_fence_after();
                const bool has = m_run != -INFINITY;  // the join does not read the others
                float4* po = c.part_o + (pair + (long long)group) * (kRows * kD / 4) + rank * kHalf + r;
#pragma unroll 1
                for (int q = 4 * wg; q < 4 * wg + 4; ++q) {
                    uint32_t o[32];
                    tc::tmem_ld_x32(lanes + 32 * q, o);
                    tc::tmem_ld_wait();
                    // columns 64 i .. of O are slab 2 i + half: 16 quads of dims
                    float4* pq = po + (long long)((q & ~1) + half) * 16 * kRows + (q & 1) * 8 * kRows;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (has) pq[k * kRows] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                    __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                }
                tc::tc_fence_before();
            }
        }
        if (flags & kEnd) break;
    }
    for (; next_group <= last_group; ++next_group)
        if (quarter == 0) ml(next_group) = make_float2(-INFINITY, 0.f);
    if (!ok || aborted(sm)) {
        fault(sm, c, rank);
        for (int g = first_group; g <= last_group; ++g)
            if (quarter == 0) ml(g) = make_float2(NAN, NAN);
    }
}

__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PairArgs c) {
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&sm.told[i], 1);
            for (int h = 0; h < 2; ++h) {
                tc::mbar_init(&sm.x_full[i][h], 1);
                tc::mbar_init(&sm.kv_empty[i][h], 1);
            }
            tc::mbar_init(&sm.z_full[i], 1);
            tc::mbar_init(&sm.z_ready[i], 1);
            tc::mbar_init(&sm.s_full[i], 1);
        }
        tc::mbar_init(&sm.p_full, 16);  // the softmax warps of both CTAs
        tc::mbar_init(&sm.p_free, 1);
        tc::mbar_init(&sm.q_full, 1);
        tc::mbar_init(&sm.q_empty, 1);
        tc::mbar_init(&sm.drain, 2);  // both warps that issue
        sm.abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) tc::tmem_alloc_pair(&sm.tmem_base, kTmemCols);
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    if (warp > 0) griddep_wait();  // everything before this kernel on the stream has finished (warp 0: see load_x)
    const uint32_t tmem = sm.tmem_base;
    if (warp == 0) {
        if (lane == 0) load_x(sm, c, maps, pair, rank);
    } else if (warp == 10) {
        if (lane == 0) load_z(sm, c, maps, rank);
    } else if (warp == 1) {
        if (rank == 0) issue_s(sm, c, tmem);
        else if (lane == 0) pass_on_z(sm, c);
    } else if (warp == 11) {
        if (rank == 0) issue_o(sm, c, tmem);
    } else {
        softmax(sm, c, tmem, pair, rank);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();  // neither CTA leaves, or frees tensor memory, while the other uses it
    if (warp == 1) {
        tc::mbar_wait(&sm.drain, 0);  // every MMA issued has completed
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// Joins the pieces.  A block takes 32 rows (a lane each) and 16 dims (4 per warp): a warp's load of a
// piece is 512 contiguous bytes.  The output leaves through shared memory, 32 or 64 bytes per row.
__global__ void __launch_bounds__(128) shared_tc_join_kernel(const __grid_constant__ PairArgs c, const __grid_constant__ Turns turns) {
    const bool f32 = c.a.out_dtype == V4A_F32;
    griddep_wait();
    // The attention kernels read their first query before they wait for the grid before them; bf16 rows may be it, so the
    // next kernel is let in when they have reached L2 (0.8 to 2 us a call more than letting it in here)
    if (f32) griddep_launch_dependents();
    __shared__ float tile[32][20];
    const SharedArgs& a = c.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned row = blockIdx.x * 32 + lane;
    const int g = (int)(blockIdx.x / (kRows / 32)), rg = (int)(row % kRows);
    const int quad = blockIdx.y * 4 + warp, dim = quad * 4;
    bool live = false;
    long long pos = 0;
    int h = 0;
    if (row < c.rows) {
        const unsigned query = row / (unsigned)a.heads;
        h = (int)(row % (unsigned)a.heads);
        const int b = (int)(query / (unsigned)a.n_q);
        pos = seq_len(a, b) - a.n_q + (int)(query % (unsigned)a.n_q);
        live = has_candidates(a, pos);
        if (blockIdx.y == 0 && warp == 0 && h == 0 && query % (unsigned)a.n_q == 0) report_sequence(a, b);
    }
    // pieces of this group: pairs p0 .. p0 + n - 1
    int p0 = 0, n = 0;
    if (g < kSpans) {
        p0 = c.span[g].first;
        n = c.span[g].n;
    } else {
        find_pairs(c, g, &p0, &n);
    }
    const float2* ml = c.part_ml + (long long)(p0 + g) * kRows + rg;
    const float4* po = c.part_o + (long long)(p0 + g) * (kRows * kD / 4) + quad * kRows + rg;
    // kU pieces are on their way together, their maxima and sums beside them
    constexpr int kU = 8;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0; live && i0 < n; i0 += kU) {
        float4 v[kU];
        float2 x[kU];
        float top = m;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            x[u] = make_float2(-INFINITY, 0.f);
            if (i0 + u < n) {
                x[u] = __ldcg(ml + (long long)(i0 + u) * kRows);
                v[u] = __ldcg(po + (long long)(i0 + u) * (kRows * kD / 4));  // of a piece without tiles: not used
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) top = isnan(x[u].x) || isnan(top) ? NAN : fmaxf(top, x[u].x);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - top);
        l *= keep;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (x[u].x == -INFINITY) continue;
            const float w = exp2f(x[u].x - top);
            l = fmaf(w, x[u].y, l);
            o.x = fmaf(w, v[u].x, o.x);
            o.y = fmaf(w, v[u].y, o.y);
            o.z = fmaf(w, v[u].z, o.z);
            o.w = fmaf(w, v[u].w, o.w);
        }
        m = top;
    }
    if (m != -INFINITY && a.sink) {
        const float s = a.sink[h] * kLog2eF;
        if (s > m && s < INFINITY) {  // the sink outweighs every key: it becomes the reference
            const float keep = exp2f(m - s);
            l *= keep;
            o.x *= keep;
            o.y *= keep;
            o.z *= keep;
            o.w *= keep;
            m = s;
        }
        l += exp2f(s - m);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
    if (a.lse && blockIdx.y == 0 && warp == 0 && row < c.rows)
        a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2F : (l == 0.f ? -INFINITY : l);
    o.x *= inv;
    o.y *= inv;
    o.z *= inv;
    o.w *= inv;
    const int k0 = (dim - (kD - a.rope_dims)) >> 1;  // rotated back by the query's position
    if (live && a.rope_dims > 0 && k0 >= -1) {
        if (k0 >= 0) {
            const float2 w = turn((double)pos, turns.hi[k0], turns.lo[k0]);
            const float u = o.x;
            o.x = fmaf(u, w.x, o.y * w.y);
            o.y = fmaf(o.y, w.x, -u * w.y);
        }
        const float2 w = turn((double)pos, turns.hi[k0 + 1], turns.lo[k0 + 1]);
        const float u = o.z;
        o.z = fmaf(u, w.x, o.w * w.y);
        o.w = fmaf(o.w, w.x, -u * w.y);
    }
    *reinterpret_cast<float4*>(&tile[lane][4 * warp]) = o;
    __syncthreads();
    const int tr = threadIdx.x >> 2, part = threadIdx.x & 3;  // 4 threads per row
    const long long orow = (long long)blockIdx.x * 32 + tr;
    if (orow >= c.rows) return;
    const float4 v = *reinterpret_cast<const float4*>(&tile[tr][4 * part]);
    const long long at = orow * kD + blockIdx.y * 16 + 4 * part;
    if (a.out_dtype == V4A_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
    } else {
        const __nv_bfloat162 p[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = *reinterpret_cast<const uint2*>(p);
        __threadfence();
    }
}

// everything of the arguments that the sizes alone decide
void plan(const SharedArgs& a, PairArgs* c) {
    c->a = a;
    c->rows = (unsigned)((long long)a.batch * a.n_q * a.heads);
    c->per_seq = (unsigned)(a.n_q * a.heads);
    unsigned x = c->per_seq, y = kRows;
    while (y) { const unsigned z = x % y; x = y; y = z; }
    const unsigned long long lcm = (unsigned long long)(c->per_seq / x) * kRows;
    c->lcm = lcm < 0xffffffffULL ? (unsigned)lcm : 0xffffffffu;  // beyond every row: divides to 0 either way
    c->groups = (int)((c->rows + kRows - 1) / kRows);
    c->pre = (int)((a.n_prefix + kBox - 1) / kBox);
    c->pre_tail = (int)(a.n_prefix - (long long)(c->pre - 1) * kBox);
    c->own = (a.own_rows + kBox - 1) / kBox;
    c->win = a.window > 0 ? (int)(((long long)a.window + a.n_q - 1 + kBox - 1) / kBox) + 1 : 0;
    c->total = boxes_before(*c, c->groups);
    c->pairs = (c->total + 1) / 2 < kPairs ? (int)((c->total + 1) / 2) : kPairs;
    c->scale_log2 = kLog2eF / sqrtf((float)kD);
    c->withhold = g_test_fault.withhold;
    c->polls = c->withhold >= 0 ? g_test_fault.wait_polls : tc::kWaitPolls;
    // Equal shares of the work: the boxes, and kPiece for every piece (queries loaded, O written).  With many groups
    // a pair has many pieces anyway, and the boxes alone are shared out.
    constexpr int kPiece = 4;
    const int extra = c->groups <= 8 * kPairs ? kPiece : 0;
    const long long cost = c->total + (long long)extra * (c->groups + c->pairs - 1);
    long long f = 0;
    int g = 0, pairs = 0;
    for (int p = 0; p < c->pairs && f < c->total; ++p) {
        // up to where the work so far is p + 1 shares
        long long f1 = f, budget = (p + 1) * cost / c->pairs - (f + (long long)extra * (g + p));
        int h = g;
        if (extra == 0) {
            f1 = (p + 1) * c->total / c->pairs;
        } else {
            for (budget -= extra; budget > 0 && f1 < c->total;) {
                const long long end = boxes_before(*c, h + 1), n = end - f1 < budget ? end - f1 : budget;
                f1 += n;
                budget -= n;
                if (f1 == end) {
                    ++h;
                    budget -= extra;
                }
            }
            if (p == c->pairs - 1) f1 = c->total;
        }
        // whole tiles of a group
        for (h = g; h + 1 < c->groups && boxes_before(*c, h + 1) <= f1;) ++h;
        if (f1 < c->total && ((f1 - boxes_before(*c, h)) & 1)) --f1;
        if (f1 <= f) f1 = f + 2 < boxes_before(*c, g + 1) ? f + 2 : boxes_before(*c, g + 1);
        while (g + 1 < c->groups && boxes_before(*c, g + 1) <= f) ++g;
        Range& r = c->range[p];
        r.g = g;
        r.i = (int)(f - boxes_before(*c, g));
        r.n = (int)(f1 - f);
        if (p > 0) c->range[p - 1].last = r.i > 0 ? g : g - 1;
        r.last = c->groups - 1;
        f = f1;
        while (g + 1 < c->groups && boxes_before(*c, g + 1) <= f) ++g;
        pairs = p + 1;
    }
    c->pairs = pairs;
    for (int k = 0; k < c->groups && k < kSpans; ++k) {
        int first, n;
        find_pairs(*c, k, &first, &n);
        c->span[k].first = (unsigned char)first;
        c->span[k].n = (unsigned char)n;
    }
}
long long pieces(const PairArgs& c) { return c.total > 0 ? (long long)c.groups + c.pairs - 1 : 0; }

}  // namespace

bool shared_tc_shape_ok(const SharedArgs& a) {
    return a.dtype == V4A_BF16 && a.d == kD;
}

size_t shared_tc_workspace_bytes(const SharedArgs& a) {
    PairArgs c;
    plan(a, &c);
    return align256(pieces(c) * kRows * sizeof(float2)) + pieces(c) * kRows * kD * sizeof(float);
}

cudaError_t launch_shared_tc(const SharedArgs& a, void* ws, cudaStream_t st) {
    PairArgs c;
    plan(a, &c);
    c.part_ml = static_cast<float2*>(ws);
    c.part_o = reinterpret_cast<float4*>(static_cast<char*>(ws) + align256(pieces(c) * kRows * sizeof(float2)));
    Maps maps;
    if (c.total > 0) {
        const struct { const void* p; long long n, rows; } in[3] = {
            {a.prefix, 1, a.n_prefix}, {a.own, a.batch, a.own_rows}, {a.window > 0 ? a.ring : nullptr, a.batch, a.ring_rows}};
        bool ok = make_slab_map(&maps.q, a.q, 1, c.rows, kD, kHalf, 8);
        for (int k = 0; k < 3; ++k) {
            const bool have = in[k].p && in[k].rows > 0;  // without: no tile asks for it
            ok = ok && make_slab_map(&maps.x[k], have ? in[k].p : a.q, have ? in[k].n : 1, have ? in[k].rows : c.rows, kD, kBox, 4) &&
                 make_slab_map(&maps.z[k], have ? in[k].p : a.q, have ? in[k].n : 1, have ? in[k].rows : c.rows, kD, kBox, 1);
        }
        if (!ok) return cudaErrorNotSupported;
        const size_t smem = sizeof(Smem) + 1024;
        static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory");
        cudaError_t e = cudaFuncSetAttribute(shared_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = launch_pdl_cluster(shared_tc_kernel, dim3(2 * c.pairs), dim3(kThreads), smem, st, 2, maps, c);
        if (e != cudaSuccess) return e;
    }
    Turns turns;
    if (a.rope_dims > 0) make_turns(a.rope_dims, a.rope_base, &turns);
    cudaError_t e = launch_pdl(shared_tc_join_kernel, dim3((c.rows + 31) / 32, kD / 16), dim3(128), 0, st, c, turns);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace v4a
