// logprobs.cu -- log probabilities of given tokens with the row's entropy and
// its k likeliest entries, and their gradient, sm_103a.
//
// Forward.  A row is read once.  Every thread keeps the running sums of a
// softmax over its entries (ws_logits.cuh) in registers and notes the maximum
// of what it read; the sums then meet in a fixed order: warp, block, cluster.
// The k likeliest entries come from the same read: the noted maxima are
// delegates, a bisection over their order bits finds a threshold that k of
// them reach and few more, and only the entries behind those are looked at
// again.  Entries that reach the threshold become candidates, ranked
// as 64-bit keys (value, then lower index; ws_select.cuh).  Ties are what
// makes a threshold let too many through (rows that a mask leaves little of,
// constant rows): the delegates then do not part, and the first k entries
// equal to the threshold are taken in index order instead.
//
// Rows of at most 256 vectors (16 bytes each): logprobs_short_kernel, a warp a
// row with the row in registers, and no barrier at all.
// Longer ones, where there are enough of them or they are of middle length:
// logprobs_rows_kernel, a warp or a block of four a row, which stream it
// through registers.
// Few long rows: logprobs_kernel, a thread-block cluster of up to 16 blocks a
// row, eight warps a block, each with a ring of chunks in shared memory,
// filled by bulk copies that its lane 0 issues, so that nothing is shared
// until the run has been summed.  All of a block's warps then select, from
// shared memory where the run still lies there, and the blocks' sums and
// sorted lists meet in every block's shared memory.
//
// Backward.  One pass: p from the forward's maximum and sum, and the gradient
// of each entry, read and written as 16-byte vectors.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "ws_internal.cuh"
#include "ws_logits.cuh"
#include "ws_ptx.cuh"
#include "ws_select.cuh"

namespace ws {
namespace {

constexpr int kThreads = 256;                 // streaming threads of a block; of a backward block
constexpr int kWarps = kThreads / 32;
constexpr int kMaxStages = 8;                 // chunks of a warp's ring, at most
constexpr int kMaxima = 8;                    // maxima a thread notes a row, each of a group of its chunks
constexpr int kMaxCluster = 16;
constexpr int kClusterSizes = 5;              // 1, 2, 4, 8, 16 blocks
constexpr int kMaxK = 32;
constexpr int kShortRow = 256;                // vectors of a row that a warp holds
constexpr int kWarpRow = 4096;                // ... that a warp streams
constexpr int kNoted = kWarpRow / 256;        // maxima a lane notes of them
constexpr int kListCap = 384;                 // candidate keys
constexpr int kLook = 4;                      // vectors that a selecting lane has in flight
constexpr int kStash = 32 * kLook;            // vectors of candidates
constexpr int kWarpStash = kStash / kWarps;   // ... of each of a block's warps
constexpr int kWork = 64;                     // threads to look at
constexpr int kItems = 512;                   // groups of vectors to look at
constexpr int kLooked = 128;                  // ... that collect() looks at in one go
constexpr int kTies = 96;                     // delegates that may reach a threshold which ties keep from rising
constexpr int kRankMax = 128;                 // candidates ranked by counting; more are cut to k first
constexpr int kSpare = 6;                     // delegates above k that are not worth another bisection step
constexpr int kRaise = 5;                     // most steps of the block's bisection

struct LogprobsParams {
    const void* x;
    long long stride;       // elements between rows
    long long rows, cols;
    const void* tokens;
    int tok64;
    int k;
    int cluster_log2;       // blocks a row: 1 << cluster_log2
    int stages;             // chunks of a warp's ring
    int resident;           // one row a block, and it fits the rings
    int group;              // chunks that a noted maximum covers
    float c;                // log2(e) / temperature
    float temperature;
    float above;            // see clamp_above
    float* logprob;
    float* entropy;
    float* lse;
    float* stats;           // [rows][2]: maximum, ln of the sum relative to it
    float* top_logprob;
    int* top_idx;
    uint32_t* err;
    unsigned long long wait_ns;   // the limit of a wait for a copy
    int withhold;                 // a self-test: the last warp of odd rows' last block, and of even rows' every block, fetches nothing
};

// What a row's results are made of.
struct RowResult {
    float m, ln_s;   // ln_s: ln of the sum relative to m; 0 for a row in which nothing is left
    bool bad;        // a +inf entry
};

__device__ __forceinline__ RowResult row_result(const SoftSums& a) {
    RowResult r;
    r.m = a.m;
    r.ln_s = a.m > -INFINITY ? logf(a.s) : 0.f;
    r.bad = a.m == INFINITY;
    return r;
}

__device__ __forceinline__ float entry_logprob(const RowResult& r, float x, float temperature) {
    if (r.bad) return NAN;
    if (!(x > -INFINITY)) return -INFINITY;
    return half_gap(x, r.m) / (0.5f * temperature) - r.ln_s;
}

// One thread writes what a row has one of.
__device__ __forceinline__ void write_row(const LogprobsParams& p, long long row, const SoftSums& total, const RowResult& r,
                                          long long token, float x_tok) {
    if (p.lse) p.lse[row] = r.bad ? INFINITY : r.m / p.temperature + r.ln_s;
    if (p.stats) {
        p.stats[2 * row] = r.m;
        p.stats[2 * row + 1] = r.bad ? NAN : r.ln_s;
    }
    if (p.entropy) p.entropy[row] = r.bad ? NAN : r.m > -INFINITY ? r.ln_s - total.t / (total.s * p.temperature) : 0.f;
    if (p.logprob) {
        float lp = token < 0 ? 0.f : entry_logprob(r, x_tok, p.temperature);
        if (token >= p.cols) {
            lp = NAN;
            atomicOr(p.err, (uint32_t)kDevErrBadIndex);
        }
        p.logprob[row] = lp;
    }
}

__device__ __forceinline__ void write_top(const LogprobsParams& p, long long row, const RowResult& r, int at,
                                          unsigned long long key) {
    p.top_logprob[row * p.k + at] = entry_logprob(r, order_value((uint32_t)(key >> 32)), p.temperature);
    p.top_idx[row * p.k + at] = (int)key_index(key);
}

// Entry `at` of a row whose copies did not come in time, where no key is left for it.
__device__ __forceinline__ void write_lost(const LogprobsParams& p, long long row, int at) {
    p.top_logprob[row * p.k + at] = NAN;
    p.top_idx[row * p.k + at] = -1;
}

// The largest entry of a vector (NaN gives way).
template <class E>
__device__ __forceinline__ float vector_max(const uint4& q) {
    return E::max_of(E::max_word(E::max_word(E::kNegInf, E::max_word(q.x, q.y)), E::max_word(q.z, q.w)));
}

// ------------------------------------------------------- selection by a warp
// It runs once at the end of a row, while other rows' warps stream, so what
// counts is the length of its chain of instructions and the
// size of its code (straight-line code runs at the rate of the instruction
// cache's misses): short loops in which every lane has an item, lists
// compacted by ballots, no shared-memory atomics.

struct SelectList {
    unsigned long long keys[kListCap];
    uint4 stash[kStash];        // vectors that reach the floor, and their index in the row
    int stash_at[kStash];
    unsigned short work[kWork]; // logprobs_kernel: threads whose entries are looked at
    int items[kItems];          // the first vectors behind the notes that are looked at
    unsigned cnt;
};

__device__ __forceinline__ unsigned lanes_below() { return (1u << (threadIdx.x & 31)) - 1u; }

// Cuts a list to its k largest keys; returns the k-th.
__device__ __noinline__ unsigned long long cut_list(SelectList& list, int k) {
    const int lane = threadIdx.x & 31;
    const int n = (int)list.cnt;
    unsigned long long kth = 0;   // the largest with at least k keys at or above it: the k-th largest
    for (int b = 63; b >= 0; --b) {
        const unsigned long long t = kth | 1ull << b;
        unsigned c = 0;
        for (int i = lane; i < n; i += 32) c += list.keys[i] >= t ? 1u : 0u;
        if ((int)__reduce_add_sync(kFull, c) >= k) kth = t;
    }
    int at = 0;
    for (int base = 0; base < n; base += 32) {
        const int i = base + lane;
        const unsigned long long key = i < n ? list.keys[i] : 0ull;
        const unsigned keep = __ballot_sync(kFull, i < n && key >= kth);
        if (keep >> lane & 1u) list.keys[at + __popc(keep & lanes_below())] = key;
        at += __popc(keep);
        __syncwarp();
    }
    if (lane == 0) list.cnt = (unsigned)k;
    __syncwarp();
    return kth;
}

// Appends the first `left` of a warp's entries whose order bits are t to a
// list of n keys, in index order (the lanes' vectors v follow one another);
// returns how many it took.
template <class E>
__device__ __noinline__ int take_equal(SelectList& list, int n, bool use, const uint4 q, int v, int lead, int cols, uint32_t t,
                                       int left) {
    float f[E::kPer];
    E::unpack(q, f);
    const int e0 = v * E::kPer - lead;
    unsigned eq = 0;
#pragma unroll
    for (int i = 0; i < E::kPer; ++i)
        if (use && order_bits(f[i]) == t && e0 + i >= 0 && e0 + i < cols) eq |= 1u << i;
    const int mine = __popc(eq);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, o);
        if ((threadIdx.x & 31) >= o) incl += u;
    }
    int at = incl - mine;
    for (; eq && at < left; eq &= eq - 1, ++at) list.keys[n + at] = make_key(t, (uint32_t)(e0 + __ffs(eq) - 1));
    return min(__shfl_sync(kFull, incl, 31), left);
}

// How a warp selects: every entry that reaches `floor` (a value; NaN fails
// it) goes to the list; when that is full it is cut to the k largest so far,
// which raises the floor.  cnt and stashed are the lists' lengths, the same
// in every lane.
template <class E>
struct WarpSelect {
    SelectList& list;
    int k;
    int cols;
    float floor;
    int cnt, stashed;

    __device__ __forceinline__ WarpSelect(SelectList& l, int k_, int cols_)
        : list(l), k(k_), cols(cols_), floor(0.f), cnt(0), stashed(0) {}

    // A threshold on the delegates' order bits (0: none).  True: what reaches
    // t is wanted; at most `most` delegates do.  False: the delegates do not
    // part at t (or fewer than k lie above -inf): wanted are the entries above
    // t, and the first k equal to it.
    template <int kN>
    __device__ __forceinline__ bool threshold(const uint32_t (&d)[kN], uint32_t& t, int most) const {
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) mine = max(mine, d[i]);
        uint32_t hi = __reduce_max_sync(kFull, mine) + 1u;   // reached by none
        t = max(__reduce_min_sync(kFull, mine), kOrderNegInf + 1u);   // every lane has one there, where all are above -inf
        uint32_t at = t;
        int reach = 0;
        while (true) {
            unsigned c = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i) c += d[i] >= at ? 1u : 0u;
            const int n = (int)__reduce_add_sync(kFull, c);
            if (n >= k) {
                t = at;
                reach = n;
                if (n <= k + kSpare) return true;
            } else {
                hi = at;
                if (reach == 0) {   // nothing is known to be reached by k yet: the lowest
                    if (at == kOrderNegInf + 1u) break;
                    at = kOrderNegInf + 1u;
                    continue;
                }
            }
            if (hi - t <= 1u) return reach <= most;   // some ties
            at = t + (hi - t) / 2;
        }
        t = kOrderNegInf;
        return false;
    }

    __device__ __forceinline__ void from(uint32_t t) { floor = order_value(t); }

    // The row's first k entries equal to t, in index order.
    __device__ __forceinline__ void take_ties(const RowBlocks<E>& rb, uint32_t t) {
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int v0 = 0; v0 < rb.nvec && cnt < k; v0 += 32 * kLook) {
            uint4 q[kLook];
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const int v = v0 + i * 32 + lane;
                q[i] = v < rb.nvec ? __ldg(rb.base + v) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const int v = v0 + i * 32 + lane;
                if (cnt < k) cnt += take_equal<E>(list, cnt, v < rb.nvec, q[i], v, rb.lead, cols, t, k - cnt);
            }
        }
    }

    __device__ __forceinline__ void cut() {
        if (cnt <= k) return;
        if ((threadIdx.x & 31) == 0) list.cnt = (unsigned)cnt;
        __syncwarp();
        const unsigned long long kth = cut_list(list, k);
        cnt = k;
        floor = fmaxf(floor, order_value((uint32_t)(kth >> 32)));
    }

    // One vector a lane (those with `use`), vector v of the row: those that
    // reach the floor are stashed.  At most 32 more than before.
    __device__ __forceinline__ void stash(bool use, const uint4& q, int v) {
        const bool pass = use && vector_max<E>(q) >= floor;
        const unsigned who = __ballot_sync(kFull, pass);
        if (pass) {
            const int at = stashed + __popc(who & lanes_below());
            list.stash[at] = q;
            list.stash_at[at] = v;
        }
        stashed += __popc(who);
    }

    // The stashed vectors' entries that reach the floor, to the list: a
    // vector a lane, its entries' places from a scan of their numbers.
    __device__ __forceinline__ void drain(int lead) {
        __syncwarp();
#pragma unroll 1
        for (int base = 0; base < stashed; base += 32) {
            const int i = base + (int)(threadIdx.x & 31);
            float f[E::kPer];
            unsigned want = 0;
            int e0 = 0;
            if (i < stashed) {
                E::unpack(list.stash[i], f);
                e0 = list.stash_at[i] * E::kPer - lead;
#pragma unroll
                for (int j = 0; j < E::kPer; ++j)
                    if (f[j] >= floor && e0 + j >= 0 && e0 + j < cols) want |= 1u << j;
            }
            int incl = __popc(want);
            const int mine = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, incl, o);
                if ((threadIdx.x & 31) >= o) incl += u;
            }
            const int total = __shfl_sync(kFull, incl, 31);   // at most 32 * kPer
            if (cnt + total > kListCap) cut();
            unsigned long long* to = list.keys + cnt + incl - mine;
#pragma unroll
            for (int j = 0; j < E::kPer; ++j)
                if (want >> j & 1u) *to++ = make_key(order_bits(f[j]), (uint32_t)(e0 + j));
            cnt += total;
        }
        stashed = 0;
        __syncwarp();
    }

    // Calls emit(rank, key) for the k largest keys.
    template <class Emit>
    __device__ __forceinline__ void ranked(Emit emit) {
        if (cnt > kRankMax) cut();
        __syncwarp();
#pragma unroll 1
        for (int i = threadIdx.x & 31; i < cnt; i += 32) {
            const unsigned long long key = list.keys[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < cnt; ++j) rank += list.keys[j] > key ? 1 : 0;
            if (rank < k) emit(rank, key);
        }
    }
};

// ------------------------------------------------------------- short rows

// A warp a row of at most 32 * kV vectors, held in registers: vector j of a
// lane is vector j * 32 + lane of the row.  The lane's vectors' maxima are
// the delegates.  One row is a chain of load, sums and selection: 3.5 us for
// [1,1000] f32 top 5; [4096,1000] f32 takes 9.5 us (1.7 TB/s, bound by the
// selection's instructions), by blocks of nine warps 41 us.
template <class E, bool kTop, int kV>
__global__ void __launch_bounds__(128) logprobs_short_kernel(const __grid_constant__ LogprobsParams p) {
    using S = typename E::Storage;
    __shared__ SelectList lists[kTop ? 4 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    launch_dependents();
    const long long row = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
    if (row >= p.rows) return;
    const S* xr = static_cast<const S*>(p.x) + row * p.stride;
    const RowBlocks<E> rb(xr, p.cols);
    const int nvec = rb.nvec;
    uint4 q[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = j * 32 + lane;
        q[j] = v < nvec ? load_stream(rb.base + v) : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
    }
    long long token = -1;
    float x_tok = 0.f;
    if (p.logprob) {
        token = load_index(p.tokens, row, p.tok64);
        if (token >= 0 && token < p.cols) x_tok = E::load(xr + token);
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = j * 32 + lane;
        mask_ends<E>(q[j], v, rb, p.cols);
    }
    RunningSums a;
    a.clear();
    add_vectors<E, kV, true>(a, q, p.c, p.above);
    const SoftSums total = warp_sums(a.sums(), p.c);
    const RowResult r = row_result(total);
    if (lane == 0) write_row(p, row, total, r, token, x_tok);
    if constexpr (kTop) {
        uint32_t d[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) d[j] = j * 32 + lane < nvec ? order_bits(vector_max<E>(q[j])) : 0u;
        WarpSelect<E> w(lists[warp], p.k, (int)p.cols);
        uint32_t t;
        if (!w.threshold(d, t, kStash)) {
            w.take_ties(rb, t);
            ++t;
        }
        w.from(t);
        // the stash holds the vectors of all delegates that reach t
#pragma unroll
        for (int j = 0; j < kV; ++j) w.stash(d[j] >= t, q[j], j * 32 + lane);
        w.drain(rb.lead);
        w.ranked([&](int at, unsigned long long key) { write_top(p, row, r, at, key); });
    }
}

// kR warps a row (1, or a block's 4), which take steps of 256 vectors in
// turn, the next step's in flight in registers.  A lane notes the maximum of
// each of its steps' vectors, or (kGroups) of p.group steps'; the notes that
// reach the threshold are read again.  The delegates that decide it are the
// notes, or, with four warps, every thread's largest.
//
// Sixteen warps an SM keep 64 KB in flight, and a row's warps that select
// leave the memory to the others.  Bound by memory where rows are long and
// many ([4096,131072] bf16 without top entries 153 us, 7.0 TB/s; with eight
// 175 us, 6.2 TB/s), by the instructions of loads and selection where they
// are short ([2000,8192] bf16 top 8, a warp a row: 12.6 us).  Nine warps a
// block with bulk-copy rings, one of them selecting, walking over the rows,
// took 195 and 173 us for the former, 30.5 us for the latter.
template <class E, bool kTop, int kR, bool kGroups>
__global__ void __launch_bounds__(128, 4) logprobs_rows_kernel(const __grid_constant__ LogprobsParams p) {
    using S = typename E::Storage;
    constexpr int kV = 8, kStep = 32 * kV, kN = kNoted;
    __shared__ SelectList lists[kTop ? 4 : 1];
    __shared__ SoftSums part[4];
    __shared__ uint32_t largest[4][32];
    __shared__ int counts[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    launch_dependents();
    const int sub = kR == 1 ? 0 : warp;   // of the row's warps
    const long long row = kR == 1 ? (long long)blockIdx.x * 4 + warp : (long long)blockIdx.x;
    if (row >= p.rows) return;
    const S* xr = static_cast<const S*>(p.x) + row * p.stride;
    const RowBlocks<E> rb(xr, p.cols);
    const int nvec = rb.nvec, group = kGroups ? p.group : 1;
    auto load = [&](uint4 (&q)[kV], int v0) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int v = v0 + j * 32 + lane;
            q[j] = v < nvec ? load_stream(rb.base + v) : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
        }
    };
    uint4 q[kV], next[kV];
    load(next, sub * kStep);
    long long token = -1;
    float x_tok = 0.f;
    if (p.logprob && sub == 0) {
        token = load_index(p.tokens, row, p.tok64);
        if (token >= 0 && token < p.cols) x_tok = E::load(xr + token);
    }
    RunningSums a;
    a.clear();
    uint32_t d[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) d[i] = 0u;
    float top = -INFINITY;
    int note = 0, left = group;
#pragma unroll 1
    for (int v0 = sub * kStep; v0 < nvec; v0 += kR * kStep) {
#pragma unroll
        for (int j = 0; j < kV; ++j) q[j] = next[j];
        if (v0 + kR * kStep < nvec) load(next, v0 + kR * kStep);
        if (v0 == 0 || v0 + kStep >= nvec) {
#pragma unroll
            for (int j = 0; j < kV; ++j) mask_ends<E>(q[j], v0 + j * 32 + lane, rb, p.cols);
        }
        // a step's sums by themselves: an entry is one of 32 that follow one
        // another, a step one of few, however long the row
        RunningSums mine;
        mine.clear();
        mine.m = a.m;
        const float of_step = add_vectors<E, kV, true>(mine, q, p.c, p.above);
        a.add(mine, p.c);
        if constexpr (kTop) {
            top = kGroups ? fmaxf(top, of_step) : of_step;
            // order bits 0: no entry
            const uint32_t bits = top > -INFINITY || v0 + lane < nvec ? order_bits(top) : 0u;
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (i == note) d[i] = bits;
            if (!kGroups || --left == 0) {
                ++note;
                left = group;
                top = -INFINITY;
            }
        }
    }
    SoftSums total = warp_sums(a.sums(), p.c);
    uint32_t mine = 0u;
    if constexpr (kR > 1) {
        if (lane == 0) part[warp] = total;
        if constexpr (kTop) {
#pragma unroll
            for (int i = 0; i < kN; ++i) mine = max(mine, d[i]);
            largest[warp][lane] = mine;
        }
        __syncthreads();
        if (!kTop && warp > 0) return;
        total = lane_sums(part, kR, p.c);
    }
    const RowResult r = row_result(total);
    if (sub == 0 && lane == 0) write_row(p, row, total, r, token, x_tok);
    if constexpr (kTop) {
        SelectList& list = lists[warp];
        WarpSelect<E> w(list, p.k, (int)p.cols);
        uint32_t t;
        bool parted;
        if constexpr (kR == 1) {
            parted = w.threshold(d, t, kTies);
        } else {
            uint32_t all[kR];
#pragma unroll
            for (int i = 0; i < kR; ++i) all[i] = largest[i][lane];
            parted = w.threshold(all, t, kTies);   // the same in every warp
        }
        if (!parted) {
            if (sub == 0) w.take_ties(rb, t);
            ++t;
        }
        w.from(t);
        int items = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const bool reaches = d[i] >= t;
            const unsigned who = __ballot_sync(kFull, reaches);
            if (reaches) list.items[items + __popc(who & lanes_below())] = (i * group * kR + sub) * kStep + lane;
            items += __popc(who);
        }
        __syncwarp();
        // the listed notes' vectors, four a lane in flight
        const int per = kV * group;   // of a note
#pragma unroll 1
        for (int first = 0; first < items * per; first += 32 * kLook) {
            uint4 again[kLook];
            int at[kLook];
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const int n = first + i * 32 + lane, item = n / per, of = n - item * per;
                at[i] = n < items * per ? list.items[item] + of / kV * (kR * kStep) + of % kV * 32 : nvec;
                again[i] = at[i] < nvec ? __ldg(rb.base + at[i]) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kLook; ++i) w.stash(at[i] < nvec, again[i], at[i]);
            w.drain(rb.lead);
        }
        if constexpr (kR == 1) {
            w.ranked([&](int at, unsigned long long key) { write_top(p, row, r, at, key); });
        } else {
            // each warp ranks its keys among all
            if (w.cnt > kRankMax / 2) w.cut();
            __syncwarp();
            if (lane == 0) counts[warp] = w.cnt;
            __syncthreads();
#pragma unroll 1
            for (int i = lane; i < w.cnt; i += 32) {
                const unsigned long long key = list.keys[i];
                int rank = 0;
#pragma unroll 1
                for (int o = 0; o < kR; ++o) {
                    const int n = counts[o];
#pragma unroll 4
                    for (int j = 0; j < n; ++j) rank += lists[o].keys[j] > key ? 1 : 0;
                }
                if (rank < p.k) write_top(p, row, r, rank, key);
            }
        }
    }
}

static_assert(kMaxK + kSpare <= kStash, "the short rows' stash");
static_assert(kTies <= kItems && kNoted * 32 <= kItems, "the notes that reach a threshold");
static_assert(kMaxK + 32 * 8 <= kListCap, "a cut list takes 32 vectors' entries");

// --------------------------------------------------------------- long rows

struct __align__(16) Shared {
    uint64_t bar[kWarps][kMaxStages];             // a chunk of a warp's ring has landed
    float m[kThreads], sum[kThreads], tilt[kThreads];   // the threads' sums; m are the delegates
    SoftSums cpart[kMaxCluster];                  // every block's sums (of the block itself without a cluster)
    SelectList list;
    uint32_t warp_t[kWarps], warp_max[kWarps];    // the warps' thresholds and largest delegates
    uint32_t threshold;                           // a bisected one
    int rank[32];                                 // the ranks of the block's keys in the row
    long long token;
    float x_tok;
    int late;                                     // a bounded wait ran out: everything ends
};

// A row's noted maxima (the upper halves of their order bits), eight a thread.
struct Noted {
    uint4 of[kThreads];
};
static_assert(kMaxima * 2 == sizeof(uint4), "a thread's noted maxima fill a vector");

// A cluster's blocks' sorted keys, 0 past them.
struct Lists {
    unsigned long long of[kMaxCluster][32];
};

// A block's run of a row, for the selection.  Positions count vectors from
// the chunk boundary in memory (2 KB with kU = 4) at or below the run's start,
// as chunks do.  Copies that cross such boundaries are slow: where blocks took
// a row each, 3648 rows of 65536 float32 entries were read in 157 us with every
// row on one, in 219 us with 32 entries of padding a row and chunks from the
// rows' starts on, and in 164 us so; 16 bytes off, bf16, in 118 us and 83 us.
struct Run {
    const uint4* vectors;   // position 0: global, or the rings while the run is resident there
    int off;                // the first position that holds a vector
    int n;                  // positions up to the run's end
    int v0;                 // index in the row of the vector at position 0
    int lead;               // see RowBlocks
    int group;              // chunks that a noted maximum covers
};

// A run's chunks are dealt to the warps in turn.  How many a warp has:
__device__ __forceinline__ int chunks_of(int nv, int chunk, int warp) {
    return max(0, ((nv + chunk - 1) / chunk - warp + kWarps - 1) / kWarps);
}

// Bit g: the maximum of group g of a thread's chunks reaches order bits t.
__device__ __forceinline__ unsigned groups_reaching(const Noted& noted, const Run& run, int chunk, int thread, uint32_t t) {
    const uint4 q = noted.of[thread];
    const uint32_t h[4] = {q.x, q.y, q.z, q.w}, t2 = (t >> 16) * 0x10001u;
    unsigned g = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = __vcmpgeu2(h[i], t2);
        g |= (r & 1u) << (2 * i) | (r >> 31) << (2 * i + 1);
    }
    // only the groups that its warp's chunks fill
    int filled = 0;
    for (int c = chunks_of(run.n, chunk, thread >> 5); c > 0; c -= run.group) ++filled;
    return g & ((1u << filled) - 1u);
}

// The threads' maxima as delegates, eight a lane: delegate i of a lane is
// thread i * 32 + lane of the block.
__device__ __forceinline__ void load_delegates(const float* m, int nv, int chunk, uint32_t (&d)[kWarps]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) d[i] = i * chunk + lane < nv ? order_bits(m[i * 32 + lane]) : 0u;
}

// One warp lists a run's candidates: at least the k largest keys (all of
// them where the run has fewer).  Returns how many.
template <class E, int kU>
__device__ __noinline__ int collect(SelectList& list, int k, int cols, const Run run, const float* m, const Noted& noted) {
    constexpr int kChunk = 32 * kU;
    const int lane = threadIdx.x & 31;
    WarpSelect<E> w(list, k, cols);
    uint32_t d[kWarps], t;
    load_delegates(m, run.n, kChunk, d);
    if (!w.threshold(d, t, kWork)) {
        int g = 0, g_left = run.group * kWarps;
#pragma unroll 1
        for (int c = 0; c * kChunk < run.n && w.cnt < k; ++c) {
            const bool any = __any_sync(kFull, groups_reaching(noted, run, kChunk, c % kWarps * 32 + lane, t) >> g & 1u);
            if (--g_left == 0) {
                ++g;
                g_left = run.group * kWarps;
            }
#pragma unroll 1
            for (int j = 0; j < kU && any && w.cnt < k; ++j) {
                const int at = c * kChunk + j * 32 + lane;
                uint4 q = make_uint4(0, 0, 0, 0);
                const bool has = at >= run.off && at < run.n;
                if (has) q = run.vectors[at];
                w.cnt += take_equal<E>(list, w.cnt, has, q, run.v0 + at, run.lead, cols, t, k - w.cnt);
            }
        }
        ++t;
    }
    w.from(t);
    // the threads whose delegates reach t
    int threads = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const unsigned who = __ballot_sync(kFull, d[i] >= t);
        if (d[i] >= t) list.work[threads + __popc(who & lanes_below())] = (unsigned short)(i * 32 + lane);
        threads += __popc(who);
    }
    __syncwarp();
    // A thread a lane: the first vectors of its groups that reach t are
    // listed; when the list is full or complete their chunks' vectors are
    // looked at, four a lane in flight, and those that reach the floor
    // stashed; the stash is drained before it could overflow.
    int items = 0, base = 0, thread = 0;
    unsigned groups = 0;
    while (true) {
        while (items <= kLooked - 32) {
            const unsigned who = __ballot_sync(kFull, groups != 0);
            if (who == 0) {
                if (base >= threads) break;
                const bool has = base + lane < threads;
                thread = has ? list.work[base + lane] : 0;
                groups = has ? groups_reaching(noted, run, kChunk, thread, t) : 0u;
                base += 32;
                continue;
            }
            if (groups) {
                const int g = __ffs(groups) - 1;
                groups &= groups - 1;
                list.items[items + __popc(who & lanes_below())] =
                    (g * run.group * kWarps + (thread >> 5)) * kChunk + (thread & 31);
            }
            items += __popc(who);
        }
        if (items == 0) break;
        __syncwarp();
        const int vectors = items * run.group * kU;
        const float per_item = 1.0f / (float)items;
#pragma unroll 1
        for (int first = 0; first < vectors; first += 32 * kLook) {
            uint4 q[kLook];
            int at[kLook];
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                // all items' first chunks, then their second ones, ... (the quotient
                // is exact: with 128 items at most for chunks' counts up to 2^15 a
                // group, that is rows of 2^31 entries in four blocks)
                const int n = first + i * 32 + lane;
                const int cc = (int)(((float)(n / kU) + 0.5f) * per_item), item = n / kU - cc * items;
                at[i] = n < vectors ? list.items[item] + cc * kWarps * kChunk + n % kU * 32 : run.n;
                q[i] = make_uint4(0, 0, 0, 0);
                if (at[i] < run.off) at[i] = run.n;
                if (at[i] < run.n) q[i] = run.vectors[at[i]];
            }
#pragma unroll
            for (int i = 0; i < kLook; ++i) w.stash(at[i] < run.n, q[i], run.v0 + at[i]);
            w.drain(run.lead);
        }
        items = 0;
        __syncwarp();
    }
    return w.cnt;
}

// A block's sums from its threads', by one warp in a fixed order: eight
// threads' a lane, then the lanes'.
__device__ __forceinline__ SoftSums block_sums(const float* m, const float* s, const float* t, float c) {
    const int lane = threadIdx.x & 31;
    SoftSums total{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total.m = fmaxf(total.m, m[i * 32 + lane]);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        SoftSums part{m[i * 32 + lane], s[i * 32 + lane], t[i * 32 + lane]};
        rebase(part, total.m, c);
        total.s += part.s;
        total.t += part.t;
    }
    return warp_sums(total, c);
}

// kU: vectors of a chunk that a lane reads.
//
// A chain of launch, copies, cluster barrier, selection and merge bounds it:
// 6.7 us for [1,131072] bf16 top 20, 9.8 us for [32,131072] f32 top 32, of
// which the copies' 16.8 MB are some 4.  Runs stay in the rings where they
// fit (up to 128 KB), for the second look.
template <class E, bool kTop, int kU>
__global__ void __launch_bounds__(kThreads + 32, 3) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
    using S = typename E::Storage;
    constexpr int kPer = E::kPer;
    constexpr int kChunk = 32 * kU;               // vectors of a warp's chunk
    __shared__ Shared s;
    extern __shared__ __align__(128) unsigned char dsmem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int stages = p.stages;
    // the rings: stage i of a warp at ring + i * kWarps * kChunk
    uint4* ring = reinterpret_cast<uint4*>(dsmem) + warp * kChunk;
    Noted* noted = reinterpret_cast<Noted*>(dsmem + (size_t)stages * kWarps * kChunk * 16);
    unsigned long long (*lists)[32] = reinterpret_cast<Lists*>(noted + 1)->of;
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < stages; ++i) mbar_init(&s.bar[w][i], 1);
        s.late = 0;
        fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    launch_dependents();
    const int C = 1 << p.cluster_log2;
    if ((int)cluster_nctarank() != C) {
        if (tid == 0) atomicOr(p.err, (uint32_t)kDevErrBadLaunch);
        return;
    }
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    if (C > 1) cluster_arrive_relaxed();   // this block has started: it may be written to
    const long long row = blockIdx.x >> p.cluster_log2;
    const S* xr = static_cast<const S*>(p.x) + row * p.stride;
    const RowBlocks<E> rb(xr, p.cols);
    // the block's run of the row's vectors, [v0, v1), and the one at the chunk
    // boundary at or below v0
    const int per = (rb.nvec + C - 1) >> p.cluster_log2;
    const int v0 = min(rank * per, rb.nvec), v1 = min(v0 + per, rb.nvec);
    const int start = v0 - (int)((reinterpret_cast<uintptr_t>(rb.base + v0) >> 4) & (kChunk - 1));
    volatile int* late = &s.late;

    if (warp < kWarps) {
        // ------------------------------------------------ a streaming warp
        uint32_t phase = 0;     // bit i: parity of stage i's next completion
        uint32_t pending = 0;   // bit i: a copy into stage i has not been waited for
        constexpr int kStride = kWarps * kChunk;   // from one chunk of the warp to its next
        int next = start + warp * kChunk;          // the next chunk to fetch
        if (p.withhold && warp == kWarps - 1 && (rank == C - 1 || row % 2 == 0)) next = v1;
        auto fetch = [&](int st) {                 // into stage st, if anything is left
            if (next >= v1) return;
            pending |= 1u << st;
            if (lane == 0) {
                const int from = max(next, v0);
                const uint32_t bytes = (uint32_t)max(0, min(next + kChunk, v1) - from) * 16u;
                if (bytes > 0) {
                    mbar_arrive_expect_tx(&s.bar[warp][st], bytes);
                    bulk_g2s(ring + st * kStride + (from - next), rb.base + from, bytes, &s.bar[warp][st]);
                } else {
                    mbar_arrive(&s.bar[warp][st]);   // an empty run may have a first chunk
                }
            }
            next += kStride;
        };
        for (int i = 0; i < stages; ++i) fetch(i);
        int stage = 0;
        bool ok = true;
        int note = tid * kMaxima;
        RunningSums a;
        a.clear();
        float gm = -INFINITY;
        int g_left = p.group;
        for (int vb = start + warp * kChunk; vb < v1; vb += kStride) {
            const int st = stage;
            if (!__all_sync(kFull, mbar_wait_bounded(&s.bar[warp][st], (phase >> st) & 1u, p.wait_ns))) {
                ok = false;
                break;
            }
            phase ^= 1u << st;
            pending &= ~(1u << st);
            stage = st + 1 == stages ? 0 : st + 1;
            const uint4* src = ring + st * kStride;
            const int left = v1 - vb;
            uint4 q[kU];
#pragma unroll
            for (int j = 0; j < kU; ++j) q[j] = src[j * 32 + lane];
            if (vb <= v0 || left <= kChunk) {
                // outside the run, and foreign entries in the row's first and last vector
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    const int v = vb + j * 32 + lane;
                    if (v < v0 || v >= v1) q[j] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
                    else mask_ends<E>(q[j], v, rb, p.cols);
                }
            }
            if (!p.resident) {
                __syncwarp();   // every lane has read the stage
                fetch(st);
            }
            const float bm = add_vectors<E, kU, true>(a, q, p.c, p.above);
            if (kTop) {
                gm = fmaxf(gm, bm);
                if (--g_left == 0 || left <= kStride) {
                    reinterpret_cast<uint16_t*>(noted)[note++] = (uint16_t)(order_bits(gm) >> 16);
                    gm = -INFINITY;
                    g_left = p.group;
                }
            }
        }
        const SoftSums sums = a.sums();
        s.m[tid] = sums.m;
        s.sum[tid] = sums.s;
        s.tilt[tid] = sums.t;
        if (!ok) {
            // A copy did not come in time.  The copies in flight are waited
            // for before the block's memory is given up.
            *late = 1;
            if (lane == 0) atomicOr(p.err, (uint32_t)kDevErrBulkCopyTimeout);
            for (int i = 0; i < stages; ++i)
                if (pending >> i & 1u) mbar_wait_bounded(&s.bar[warp][i], (phase >> i) & 1u, kWaitLimitNs);
        }
    } else if (rank == 0 && p.logprob && lane == 0) {
        const long long token = load_index(p.tokens, row, p.tok64);
        s.token = token;
        s.x_tok = token >= 0 && token < p.cols ? E::load(xr + token) : 0.f;
    }
    const Run run{p.resident ? reinterpret_cast<const uint4*>(dsmem) : rb.base + start, v0 - start, v1 - start, start, rb.lead,
                  p.group};
    const int nv = run.n;
    const int lost = __syncthreads_or(*late);
    if (C > 1) cluster_wait();   // every block has started
    if (warp == kWarps) {
        SoftSums total = block_sums(s.m, s.sum, s.tilt, p.c);
        if (lost) total.m = INFINITY;   // the row's results become NaN
        if (C == 1) {
            if (lane == 0) s.cpart[0] = total;
        } else if (lane < C) {
            const uint32_t dst = cluster_map(&s.cpart[rank], (uint32_t)lane);
            st_cluster_u32(dst, __float_as_uint(total.m));
            st_cluster_u32(dst + 4, __float_as_uint(total.s));
            st_cluster_u32(dst + 8, __float_as_uint(total.t));
        }
    }
    if constexpr (kTop) {
        // The threshold: every streaming warp's kw-th largest delegate, and
        // the least of them; k delegates reach it where enough warps have kw
        // above -inf.  It is raised by a few steps of a bisection, which the
        // block counts together.  (Runs that a mask leaves some warps nothing
        // of take one warp's bisection from -inf on.)
        const float mine = s.m[min(tid, kThreads - 1)];
        const bool holds = warp < kWarps && warp * kChunk + lane < nv;
        if (warp < kWarps) {
            const int kw = (p.k + kWarps - 1) / kWarps;
            uint32_t d = holds && mine > -INFINITY ? order_bits(mine) : 0u, t = 0;
            for (int i = 0; i < kw; ++i) {
                t = __reduce_max_sync(kFull, d);
                if (i == 0 && lane == 0) s.warp_max[warp] = t;
                const unsigned who = __ballot_sync(kFull, d == t);
                if (lane == __ffs(who) - 1) d = 0;
            }
            if (lane == 0) s.warp_t[warp] = t;
        } else {
            if (lane == 0) s.list.cnt = 0u;
            s.rank[lane] = 0;
        }
        __syncthreads();
        uint32_t t = 0xffffffffu, hi = 0;
        int vouching = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const uint32_t w = s.warp_t[i];
            hi = max(hi, s.warp_max[i] + 1u);
            if (w != 0u) {
                t = min(t, w);
                vouching += (p.k + kWarps - 1) / kWarps;
            }
        }
        if (vouching < p.k) {
            if (warp == kWarps) {
                const WarpSelect<E> w(s.list, p.k, (int)p.cols);
                uint32_t d[kWarps];
                load_delegates(s.m, nv, kChunk, d);
                const bool parted = w.threshold(d, t, kWork);
                if (lane == 0) s.threshold = parted ? t : 0u;
            }
            __syncthreads();
            t = s.threshold;
        } else {
            const uint32_t mine_bits = holds ? order_bits(mine) : 0u;
            int reach = __syncthreads_count(mine_bits >= t);
            for (int i = 0; i < kRaise && reach > p.k + 2 * kSpare && hi - t > 1u; ++i) {
                const uint32_t mid = t + (hi - t) / 2;
                const int c = __syncthreads_count(mine_bits >= mid);
                if (c >= p.k) {
                    t = mid;
                    reach = c;
                } else {
                    hi = mid;
                }
            }
        }
        if (lost) t = 0u;   // 0: the warp's selection is needed
        // each warp looks at its threads' vectors whose delegate reaches the
        // threshold: those vectors that do are stashed, and their entries
        // listed in one go
        if (t != 0u && warp < kWarps) {
            const float floor = order_value(t);
            unsigned groups = holds && mine >= floor ? groups_reaching(*noted, run, kChunk, tid, t) : 0u;
            int stashed = 0;
            while (__any_sync(kFull, groups != 0)) {
                const int first = (__ffs(groups) - 1) * p.group;   // (not used where there is none)
                const bool some = groups != 0;
                groups &= groups - 1;
#pragma unroll 1
                for (int c = first; c < first + p.group; ++c) {
                    const int at = (c * kWarps + warp) * kChunk + lane;
#pragma unroll 1
                    for (int j = 0; j < kU; ++j) {
                        const int to = at + j * 32;
                        uint4 q = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
                        if (some && to >= run.off && to < nv) q = run.vectors[to];
                        const bool pass = vector_max<E>(q) >= floor;
                        const unsigned who = __ballot_sync(kFull, pass);
                        const int place = stashed + __popc(who & lanes_below());
                        if (pass && place < kWarpStash) {
                            s.list.stash[warp * kWarpStash + place] = q;
                            s.list.stash_at[warp * kWarpStash + place] = start + to;
                        }
                        stashed += __popc(who);
                    }
                }
            }
            __syncwarp();
            float f[kPer];
            unsigned want = 0;
            int e0 = 0;
            if (lane < min(stashed, kWarpStash)) {
                E::unpack(s.list.stash[warp * kWarpStash + lane], f);
                e0 = s.list.stash_at[warp * kWarpStash + lane] * kPer - rb.lead;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (f[j] >= floor && e0 + j >= 0 && e0 + j < p.cols) want |= 1u << j;
            }
            const int n = __popc(want);
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += u;
            }
            int total = __shfl_sync(kFull, incl, 31), base = 0;
            if (stashed > kWarpStash) total = kListCap + 1;   // by the warp's selection then
            if (lane == 0) base = (int)atomicAdd(&s.list.cnt, (unsigned)total);
            base = __shfl_sync(kFull, base, 0);
            if (base + total <= kListCap) {
                unsigned long long* to = s.list.keys + base + incl - n;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (want >> j & 1u) *to++ = make_key(order_bits(f[j]), (uint32_t)(e0 + j));
            }
        }
        __syncthreads();
        if (t == 0u || s.list.cnt > (unsigned)kThreads) {
            // ties, or more than a few candidates: by one warp, whatever the entries
            if (warp == kWarps && !lost) {
                WarpSelect<E> w(s.list, p.k, (int)p.cols);
                w.cnt = collect<E, kU>(s.list, p.k, (int)p.cols, run, s.m, *noted);
                if (w.cnt > kRankMax) w.cut();
                __syncwarp();
                if (lane == 0) s.list.cnt = (unsigned)w.cnt;
            }
            __syncthreads();
        }
        const int cnt = lost ? 0 : (int)s.list.cnt;
        // ranked by their numbers of larger keys, a thread a candidate
        unsigned long long key = 0ull;
        int at = p.k;
        if (tid < cnt) {
            key = s.list.keys[tid];
            at = 0;
#pragma unroll 4
            for (int j = 0; j < cnt; ++j) at += s.list.keys[j] > key ? 1 : 0;
        }
        if (C == 1) {
            if (at < p.k) write_top(p, row, row_result(s.cpart[0]), at, key);
        } else {
            // to every block of the cluster
            if (at < p.k)
                for (int i = 0; i < C; ++i) st_cluster_u64(cluster_map(&lists[rank][at], (uint32_t)i), key);
            const int have = min(cnt, p.k);
            for (int i = tid; i < 32 * C; i += kThreads + 32)
                if ((i & 31) >= have) st_cluster_u64(cluster_map(&lists[rank][i & 31], (uint32_t)(i >> 5)), 0ull);
            for (int i = C * 32 + tid; i < kMaxCluster * 32; i += kThreads + 32) lists[i >> 5][i & 31] = 0ull;
        }
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    }
    __syncthreads();
    if constexpr (kTop) {
        if (C > 1 && warp < kWarps) {
            // each block ranks its own keys among all, each warp in two lists
            const unsigned long long key = lists[rank][lane];
            const int larger = rank_in_lists<1>(lists + warp, key) + (C > kWarps ? rank_in_lists<1>(lists + warp + kWarps, key) : 0);
            if (larger > 0) atomicAdd(&s.rank[lane], larger);
        }
    }
    RowResult r{};
    if (warp == kWarps && (rank == 0 || (kTop && C > 1))) {
        const SoftSums total = lane_sums(s.cpart, C, p.c);
        r = row_result(total);
        if (rank == 0 && lane == 0) write_row(p, row, total, r, s.token, s.x_tok);
        if (kTop && rank == 0 && r.bad) {   // blocks that lost their runs have no keys
            int keys = C == 1 && !s.late ? p.k : 0;
            for (int i = 0; C > 1 && i < C; ++i) keys += __popc(__ballot_sync(kFull, lists[i][lane] != 0ull));
            if (lane >= keys && lane < p.k) write_lost(p, row, lane);
        }
    }
    if constexpr (kTop) {
        if (C > 1) {
            __syncthreads();
            if (warp == kWarps) {
                const unsigned long long key = lists[rank][lane];
                if (key != 0ull && s.rank[lane] < p.k) write_top(p, row, r, s.rank[lane], key);
            }
        }
    }
}

// ---------------------------------------------------------------- backward


struct BackwardParams {
    const void* x;
    void* grad;
    long long stride, grad_stride;
    long long cols;
    const void* tokens;
    int tok64;
    int segments;           // blocks a row
    float c;                // log2(e) / temperature
    float inv_t;            // 1 / temperature
    float above;            // see clamp_above
    const float* stats;
    const float* entropy;
    const float* grad_logprob;
    const float* grad_entropy;
    uint32_t* err;
};

// A row's gradient.  With d = x - m, ln p = d / T - ln_s and
//   out = p (-g_lp - g_H (ln p + H)) / T = 2^(d c - l) (d a + b),
// and `at` added at the token; d is held at -1e18, where p is 0.
struct RowGradient {
    float m, l, a, b, at;
    long long token;   // negative: none
};

__device__ __forceinline__ RowGradient row_gradient(const BackwardParams& p, long long row) {
    RowGradient g;
    g.token = p.grad_logprob ? load_index(p.tokens, row, p.tok64) : -1;
    g.m = p.stats[2 * row];
    const float ln_s = p.stats[2 * row + 1];
    const float g_lp = g.token >= 0 ? p.grad_logprob[row] : 0.f;
    const float g_h = p.grad_entropy ? p.grad_entropy[row] * p.inv_t : 0.f;
    const float h = p.grad_entropy ? p.entropy[row] : 0.f;
    g.at = g_lp * p.inv_t;
    g.l = ln_s * 1.4426950408889634f;
    g.a = -g_h * p.inv_t;
    g.b = -g.at - g_h * (h - ln_s);
    if (g.token >= p.cols) {
        atomicOr(p.err, (uint32_t)kDevErrBadIndex);
        g.b = NAN;
    } else if (g.m == -INFINITY) {   // nothing left in the row
        g.m = g.l = g.a = g.b = g.at = 0.f;
    } else if (!(g.m < INFINITY)) {
        g.b = NAN;
    }
    return g;
}

// A block a segment of 256 kU vectors, kU a thread in flight while the row's
// numbers are read: nothing is shared and nothing waited for, so that memory
// bounds it.  [4096,131072] bf16 takes 314 us, 6.8 TB/s read and written (1.01
// of a copy's), [500,20001] f32 14.0 us (5.7), of which the launch's ramp is
// some 2; [8,1000] 1.5 us.
// kU and kBlocks: eight vectors a thread and four blocks an SM for the 16-bit
// types (314 us; four and five 325, two and eight 331), four and six for
// float32 ([2048,131072] 305 us, eight and four 310), whose vectors hold half
// the entries; two and eight where rows are short ([4096,1000] f32 8.2 us,
// four and six 9.5).
template <class E, int kU, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) logprobs_backward_kernel(const __grid_constant__ BackwardParams p) {
    using S = typename E::Storage;
    constexpr int kPer = E::kPer;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    launch_dependents();
    const unsigned row = blockIdx.x / (unsigned)p.segments;
    const int seg = (int)(blockIdx.x - row * (unsigned)p.segments);
    const S* xr = static_cast<const S*>(p.x) + row * p.stride;
    S* gr = static_cast<S*>(p.grad) + row * p.grad_stride;
    const RowBlocks<E> rb(xr, p.cols);
    const RowBlocks<E> gb(gr, p.cols);
    const int v0 = seg * kThreads * kU, v1 = min(v0 + kThreads * kU, rb.nvec);
    const uint4* src = rb.base + v0 + tid;
    uint4 q[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
        if (v0 + j * kThreads + tid < v1) q[j] = __ldcs(src + j * kThreads);
    const RowGradient g = row_gradient(p, row);
    const f32x2 m2 = pack2(-g.m, -g.m), c2 = pack2(p.c, p.c), l2 = pack2(-g.l, -g.l), a2 = pack2(g.a, g.a),
                b2 = pack2(g.b, g.b);
    const bool words = kPer == 8 && g.m > p.above && g.m < INFINITY;   // see add_vectors
    const int shift = (rb.lead - gb.lead + kPer) % kPer;
    const int token_v = g.token >= 0 && g.token < p.cols ? (int)((g.token + rb.lead) / kPer) : -1;
    const int a = max(0, v0 * kPer - rb.lead), b = (int)min(p.cols, (long long)v1 * kPer - rb.lead);   // the block's entries
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        const int v = v0 + j * kThreads + tid;
        if (__all_sync(kFull, v >= v1)) break;
        float out[kPer];
        auto pair = [&](f32x2 d, int i) {
            float e0, e1;
            unpack2(fma2(d, c2, l2), e0, e1);
            unpack2(mul2(pack2(exp2_fast(e0), exp2_fast(e1)), fma2(d, a2, b2)), out[i], out[i + 1]);
        };
        if (words) {
            if constexpr (kPer == 8) {
                const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) pair(add2(E::widen(E::max_word(w[i], E::kLow)), m2), 2 * i);
            }
        } else {
            float f[kPer];
            E::unpack(q[j], f);
#pragma unroll
            for (int i = 0; i < kPer; i += 2) pair(pack2(fmaxf(f[i] - g.m, -1.0e18f), fmaxf(f[i + 1] - g.m, -1.0e18f)), i);
        }
        if (v == token_v) {
            const int at = (int)g.token + rb.lead - v * kPer;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i == at) out[i] += g.at;
        }
        const uint4 r = E::pack(out);
        if (shift == 0) {
            if (v < v1) store_vector<E>(gr, gb, v, a, b, r);
        } else {
            store_shifted<E>(gr, r, v * kPer - rb.lead, a, b, shift);
        }
    }
}

ws_status validate_desc(const ws_logprobs_desc* d) {
    if (!d) return fail(WS_ERR_INVALID_ARGUMENT, "desc is NULL");
    WS_TRY(validate_logits(d->rows, d->cols, d->row_stride, d->dtype, d->index_type, d->temperature));
    if (d->k < 0 || d->k > kMaxK) return fail(WS_ERR_INVALID_ARGUMENT, "k %d outside 0..%d", d->k, kMaxK);
    if (d->k > d->cols) return fail(WS_ERR_INVALID_ARGUMENT, "k %d > cols %lld", d->k, (long long)d->cols);
    return WS_OK;
}

// The most 16-byte blocks a row of any alignment takes.
long long max_vectors(int64_t cols, int per) { return (cols + 2 * per - 2) / per; }

// How a forward call is cut.
struct ForwardPlan {
    enum Kind { kShort, kWarp, kBlock, kCluster } kind;
    int cluster_log2;    // blocks a row
    int unroll;     // vectors a lane reads at a time (short rows: holds)
    int stages, resident;
    int group;      // see LogprobsParams
};

// Chunks of a warp's ring: as many as let three, two and one blocks share an
// SM.
constexpr int kRings = 3;
constexpr int kRingStages[kRings] = {3, 5, kMaxStages};

// Clusters of 2^i blocks that the device holds at once with rings of that many
// chunks (0: it cannot place one; 16 blocks are a size that it need not
// support).
using Resident = AskedOnce<kRings, kClusterSizes>;

ForwardPlan plan_forward(long long rows, long long nvec, int sm_count, const Resident& resident) {
    ForwardPlan f{};
    if (nvec <= kShortRow) {
        f.kind = ForwardPlan::kShort;
        f.unroll = nvec <= 64 ? 2 : 8;   // [2000,200] f32: 4.2 us with two, 6.7 with eight
        return f;
    }
    // Many rows of middle length by a warp each: [2000,8192] bf16 top 8 takes
    // 12.6 us so and 21.9 by a block each, [1000,32000] f16 19.3 and 19.7,
    // [500,8192] 7.2 and 6.6; [4000,50257] f16 81 and 92, [2000,50257] 47 and
    // 50, [1000,65536] bf16 33 and 29.
    const bool warps = nvec <= kWarpRow ? rows >= 5LL * sm_count : nvec <= 2 * kWarpRow && rows >= 12LL * sm_count;
    // Rows enough for every SM, and few ones of middle length, by a block each:
    // [300,131072] 19.2 us so and 30.1 by blocks of logprobs_kernel, [100,32000]
    // 6.7 and 9.0, [1,8192] 4.6 and 5.3, but [100,131072] 15.2 and 13.9 in
    // clusters, [1,16384] f32 5.8 and 5.6.
    if (warps || nvec <= kWarpRow || rows > sm_count) {
        f.kind = warps ? ForwardPlan::kWarp : ForwardPlan::kBlock;
        const int steps = (warps ? 1 : 4) * 256;   // vectors that the row's warps read at a time
        f.group = (int)((nvec + steps * kNoted - 1) / (steps * kNoted));
        return f;
    }
    // More blocks a row while all of them are resident at once, and each has
    // a vector a thread, or eight where they fill the SMs more than twice:
    // [100,131072] bf16 top 8 takes 13.9 us on 400 blocks and 17.4 on 200.
    // Where not all find room [64,131072] takes 16.6 us (512 blocks) against
    // 10.4 (256).
    f.kind = ForwardPlan::kCluster;
    int cluster = 1;
    while (cluster < kMaxCluster && rows <= resident.of[0][f.cluster_log2 + 1] &&
           nvec / (2 * cluster) >= (rows * cluster <= sm_count ? 1 : 8) * kThreads) {
        cluster *= 2;
        ++f.cluster_log2;
    }
    const long long per = (nvec + cluster - 1) / cluster;
    // chunks as large as give every warp one: runs of 256 vectors (8 rows of
    // 1024 over four blocks each) took 5.3 us with one vector a lane and 6.5
    // with four; [32,131072] f32 10.1 with four, 14.7 with two, 17.6 with one
    f.unroll = per >= 4 * kThreads ? 4 : per >= 2 * kThreads ? 2 : 1;
    const long long chunks = (per + 32 * f.unroll - 1 + kThreads * f.unroll - 1) / (kThreads * f.unroll);   // of a warp, at most
    // The longest rings with which all blocks are still resident: with five
    // chunks a warp [152,131072] f32 top 8 takes 24.8 us and [32,131072] top 32
    // 9.8, with three 30.7 and 13.0; [8,1000000] f32 takes 18.4 us with three,
    // and 30.7 with eight, of which not all find room.
    int ring = 0;
    while (ring + 1 < kRings && rows <= resident.of[ring + 1][f.cluster_log2]) ++ring;
    f.stages = (int)std::min<long long>(chunks, kRingStages[ring]);
    f.resident = f.stages >= chunks;
    f.group = (int)((chunks + kMaxima - 1) / kMaxima);
    return f;
}

// Rings of that many stages of chunks, and the noted maxima.
constexpr size_t dynamic_memory(int stages, int unroll, bool top) {
    return (size_t)stages * kThreads * unroll * 16 + (top ? sizeof(Noted) + sizeof(Lists) : 0);
}

template <class E, bool kTop, int kU>
cudaError_t set_attributes(int dev) {
    static std::atomic<bool> set[64];
    if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const auto kernel = logprobs_kernel<E, kTop, kU>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    (int)dynamic_memory(kMaxStages, 4, true));
    if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
    return e;
}

// What the device holds at once; asked once per device.
Resident resident_clusters(int dev) {
    static std::mutex mu;
    static Resident known[64];
    std::lock_guard<std::mutex> lock(mu);
    Resident& of = known[dev];
    of.ask(
        [&] {
            const bool ok = set_attributes<ElemF16, true, 4>(dev) == cudaSuccess;
            if (!ok) (void)cudaGetLastError();
            return ok;
        },
        [&](int ring, int size, int* n) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(1u << size);
            cfg.blockDim = dim3(kThreads + 32);
            cfg.dynamicSmemBytes = dynamic_memory(kRingStages[ring], 4, true);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << size;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            const bool ok = cudaOccupancyMaxActiveClusters(n, logprobs_kernel<ElemF16, true, 4>, &cfg) == cudaSuccess;
            if (!ok) (void)cudaGetLastError();
            return ok;
        });
    return of;
}

template <class E, bool kTop, int kU>
cudaError_t launch_long(const LogprobsParams& p, const ForwardPlan& f, int dev, cudaStream_t stream) {
    const cudaError_t e = set_attributes<E, kTop, kU>(dev);
    if (e != cudaSuccess) return e;
    return launch_clusters(logprobs_kernel<E, kTop, kU>, dim3((unsigned)(p.rows << f.cluster_log2)), kThreads + 32,
                           1 << f.cluster_log2, dynamic_memory(f.stages, kU, kTop), stream, p);
}

template <class E, bool kTop, int kV>
cudaError_t launch_short(const LogprobsParams& p, int sm_count, cudaStream_t stream) {
    // one warp a block while the rows alone do not fill the SMs, four after:
    // [4096,1000] f32 top 5 takes 9.5 us with four and 13.2 with one
    const int warps = p.rows <= 4LL * sm_count ? 1 : 4;
    return launch_pdl(logprobs_short_kernel<E, kTop, kV>, dim3((unsigned)((p.rows + warps - 1) / warps)), dim3(32 * warps),
                      0, stream, p);
}

template <class E, bool kTop, int kR>
cudaError_t launch_noted(const LogprobsParams& p, const ForwardPlan& f, dim3 grid, cudaStream_t stream) {
    if constexpr (kTop)
        if (f.group > 1) return launch_pdl(logprobs_rows_kernel<E, true, kR, true>, grid, dim3(128), 0, stream, p);
    return launch_pdl(logprobs_rows_kernel<E, kTop, kR, false>, grid, dim3(128), 0, stream, p);
}

template <class E, bool kTop>
cudaError_t launch_forward(const LogprobsParams& p, const ForwardPlan& f, int dev, int sm_count, cudaStream_t stream) {
    if (f.kind == ForwardPlan::kShort)
        return f.unroll == 2 ? launch_short<E, kTop, 2>(p, sm_count, stream) : launch_short<E, kTop, 8>(p, sm_count, stream);
    if (f.kind == ForwardPlan::kWarp)
        return launch_noted<E, kTop, 1>(p, f, dim3((unsigned)((p.rows + 3) / 4)), stream);
    if (f.kind == ForwardPlan::kBlock) return launch_noted<E, kTop, 4>(p, f, dim3((unsigned)p.rows), stream);
    switch (f.unroll) {
        case 1: return launch_long<E, kTop, 1>(p, f, dev, stream);
        case 2: return launch_long<E, kTop, 2>(p, f, dev, stream);
        default: return launch_long<E, kTop, 4>(p, f, dev, stream);
    }
}

// The forward call; selftest_us: the limit of ws_logprobs_selftest_wait_timeout, else 0.
ws_status enqueue_logprobs(const ws_logprobs_desc* desc, const void* logits, const void* tokens, float* logprob,
                           float* entropy, float* lse, float* stats, float* top_logprob, int32_t* top_idx,
                           uint32_t selftest_us, cudaStream_t stream) {
    clear_error();
    WS_TRY(validate_desc(desc));
    const size_t size = elem_size(desc->dtype);
    WS_TRY(check_pointer(logits, size, "logits"));
    if (logprob && !tokens) return fail(WS_ERR_INVALID_ARGUMENT, "logprob without tokens");
    if (tokens) WS_TRY(check_pointer(tokens, desc->index_type == WS_INDEX_I64 ? 8 : 4, "tokens"));
    if (desc->k > 0) {
        WS_TRY(check_pointer(top_logprob, 4, "top_logprob"));
        WS_TRY(check_pointer(top_idx, 4, "top_idx"));
    } else if (top_logprob || top_idx) {
        return fail(WS_ERR_INVALID_ARGUMENT, "top_logprob or top_idx with k 0");
    }
    if (logprob) WS_TRY(check_pointer(logprob, 4, "logprob"));
    if (entropy) WS_TRY(check_pointer(entropy, 4, "entropy"));
    if (lse) WS_TRY(check_pointer(lse, 4, "lse"));
    if (stats) WS_TRY(check_pointer(stats, 4, "stats"));
    if (!logprob && !entropy && !lse && !stats && desc->k == 0) return fail(WS_ERR_INVALID_ARGUMENT, "no output asked for");

    int dev;
    const DeviceInfo* info;
    WS_TRY(current_device_info(&dev, &info));
    const int per = (int)(16 / size);
    const bool aligned = (uintptr_t)logits % 16 == 0 && (desc->rows == 1 || desc->row_stride % per == 0);
    const long long nvec = aligned ? (desc->cols + per - 1) / per : max_vectors(desc->cols, per);
    const ForwardPlan f = plan_forward(desc->rows, nvec, info->sm_count, resident_clusters(dev));
    if (selftest_us && f.kind != ForwardPlan::kCluster)
        return fail(WS_ERR_UNSUPPORTED, "these rows are read without bounded waits");
    LogprobsParams p{};
    p.x = logits;
    p.stride = desc->row_stride;
    p.rows = desc->rows;
    p.cols = desc->cols;
    p.tokens = tokens;
    p.tok64 = desc->index_type == WS_INDEX_I64;
    p.k = desc->k;
    p.cluster_log2 = f.cluster_log2;
    p.stages = f.stages;
    p.resident = f.resident;
    p.group = f.group;
    p.c = log2e_over(desc->temperature);
    p.temperature = desc->temperature;
    p.above = clamp_above(desc->dtype, desc->temperature);
    p.logprob = logprob;
    p.entropy = entropy;
    p.lse = lse;
    p.stats = stats;
    p.top_logprob = top_logprob;
    p.top_idx = top_idx;
    p.err = device_error_word();
    p.wait_ns = selftest_us ? 1000ull * selftest_us : kWaitLimitNs;
    p.withhold = selftest_us != 0;
    if (desc->rows > 2147483647LL) return fail(WS_ERR_UNSUPPORTED, "too many rows");
    cudaError_t e;
    const bool top = desc->k > 0;
    if (desc->dtype == WS_DTYPE_F32)
        e = top ? launch_forward<ElemF32, true>(p, f, dev, info->sm_count, stream)
                : launch_forward<ElemF32, false>(p, f, dev, info->sm_count, stream);
    else if (desc->dtype == WS_DTYPE_F16)
        e = top ? launch_forward<ElemF16, true>(p, f, dev, info->sm_count, stream)
                : launch_forward<ElemF16, false>(p, f, dev, info->sm_count, stream);
    else
        e = top ? launch_forward<ElemBF16, true>(p, f, dev, info->sm_count, stream)
                : launch_forward<ElemBF16, false>(p, f, dev, info->sm_count, stream);
    if (e != cudaSuccess) return cuda_fail(e, "log-probability launch");
    return WS_OK;
}

}  // namespace
}  // namespace ws

extern "C" {

ws_status ws_logprobs_validate(const ws_logprobs_desc* desc) {
    ws::clear_error();
    return ws::validate_desc(desc);
}

ws_status ws_logprobs(const ws_logprobs_desc* desc, const void* logits, const void* tokens, float* logprob,
                      float* entropy, float* lse, float* stats, float* top_logprob, int32_t* top_idx,
                      cudaStream_t stream) {
    return ws::enqueue_logprobs(desc, logits, tokens, logprob, entropy, lse, stats, top_logprob, top_idx, 0, stream);
}

ws_status ws_logprobs_selftest_wait_timeout(const ws_logprobs_desc* desc, const void* logits, const void* tokens,
                                            float* logprob, float* entropy, float* lse, float* stats,
                                            float* top_logprob, int32_t* top_idx, uint32_t limit_us,
                                            cudaStream_t stream) {
    ws::clear_error();
    if (limit_us < 1 || limit_us > 1000000)
        return ws::fail(WS_ERR_INVALID_ARGUMENT, "limit_us %u outside 1..1000000", limit_us);
    return ws::enqueue_logprobs(desc, logits, tokens, logprob, entropy, lse, stats, top_logprob, top_idx, limit_us, stream);
}

ws_status ws_logprobs_backward(const ws_logprobs_desc* desc, const void* logits, const void* tokens,
                               const float* stats, const float* entropy, const float* grad_logprob,
                               const float* grad_entropy, void* grad_logits, int64_t grad_stride,
                               cudaStream_t stream) {
    using namespace ws;
    clear_error();
    WS_TRY(validate_desc(desc));
    const size_t size = elem_size(desc->dtype);
    WS_TRY(check_pointer(logits, size, "logits"));
    WS_TRY(check_pointer(grad_logits, size, "grad_logits"));
    WS_TRY(check_pointer(stats, 4, "stats"));
    if (grad_stride < desc->cols)
        return fail(WS_ERR_INVALID_ARGUMENT, "grad_stride %lld < cols %lld", (long long)grad_stride, (long long)desc->cols);
    if (desc->rows > (1LL << 40) / grad_stride) return fail(WS_ERR_INVALID_ARGUMENT, "rows * grad_stride too large");
    WS_TRY(check_gradient(logits, desc->row_stride, grad_logits, grad_stride, desc->rows, desc->cols, size));
    if (grad_logprob) {
        WS_TRY(check_pointer(grad_logprob, 4, "grad_logprob"));
        WS_TRY(check_pointer(tokens, desc->index_type == WS_INDEX_I64 ? 8 : 4, "tokens"));
    }
    if (grad_entropy) {
        WS_TRY(check_pointer(grad_entropy, 4, "grad_entropy"));
        WS_TRY(check_pointer(entropy, 4, "entropy"));
    }
    if (!grad_logprob && !grad_entropy) return fail(WS_ERR_INVALID_ARGUMENT, "neither grad_logprob nor grad_entropy");

    BackwardParams p{};
    p.x = logits;
    p.grad = grad_logits;
    p.stride = desc->row_stride;
    p.grad_stride = grad_stride;
    p.cols = desc->cols;
    p.tokens = tokens;
    p.tok64 = desc->index_type == WS_INDEX_I64;
    const long long nvec = max_vectors(desc->cols, (int)(16 / size));
    const int unroll = nvec <= 512 ? 2 : size == 2 ? 8 : 4;   // see the kernel
    p.segments = (int)((nvec + kThreads * unroll - 1) / (kThreads * unroll));
    p.c = log2e_over(desc->temperature);
    p.inv_t = 1.0f / desc->temperature;
    p.above = clamp_above(desc->dtype, desc->temperature);
    p.stats = stats;
    p.entropy = entropy;
    p.grad_logprob = grad_logprob;
    p.grad_entropy = grad_entropy;
    int dev;
    const DeviceInfo* info;
    WS_TRY(current_device_info(&dev, &info));
    p.err = device_error_word();
    if (desc->rows * p.segments > 2147483647LL) return fail(WS_ERR_UNSUPPORTED, "too many blocks");
    const dim3 grid((unsigned)(desc->rows * p.segments));
    cudaError_t e;
    if (desc->dtype == WS_DTYPE_F32)
        e = unroll == 2 ? launch_pdl(logprobs_backward_kernel<ElemF32, 2, 8>, grid, dim3(kThreads), 0, stream, p)
                        : launch_pdl(logprobs_backward_kernel<ElemF32, 4, 6>, grid, dim3(kThreads), 0, stream, p);
    else if (desc->dtype == WS_DTYPE_F16)
        e = unroll == 2 ? launch_pdl(logprobs_backward_kernel<ElemF16, 2, 8>, grid, dim3(kThreads), 0, stream, p)
                        : launch_pdl(logprobs_backward_kernel<ElemF16, 8, 4>, grid, dim3(kThreads), 0, stream, p);
    else
        e = unroll == 2 ? launch_pdl(logprobs_backward_kernel<ElemBF16, 2, 8>, grid, dim3(kThreads), 0, stream, p)
                        : launch_pdl(logprobs_backward_kernel<ElemBF16, 8, 4>, grid, dim3(kThreads), 0, stream, p);
    if (e != cudaSuccess) return cuda_fail(e, "log-probability gradient launch");
    return WS_OK;
}

}  // extern "C"
