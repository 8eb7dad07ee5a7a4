// distill.cu -- divergence from a teacher's top entries to the student's
// softmax, with the gradient of the student's logits, sm_103a.
//
// Rows of at most 256 vectors (16 bytes each): distill_short_kernel, a warp a
// row.  Longer ones: distill_kernel.
//
// A row is held by a thread-block cluster, each block taking one contiguous
// run of the row's 16-byte vectors: the logits are read once, what has to be
// known of the whole row meets through distributed shared memory, and the
// gradient is computed from what is on chip and written once.  (Loss and
// gradient in two passes over global memory would read the logits twice.)
//
// A cluster walks over many rows.  In each block
//  - the streaming warps take the run from shared memory, keep 2^((x - m) c)
//    of every entry in registers (m: the thread's largest) and send their
//    sums to every block; when the row's totals are known the gradient is one
//    product an entry, rounded and stored.  A buffer is free once its entries
//    are in registers;
//  - one warp patches the runs that have landed and has the next ones copied
//    in (two buffers);
//  - one warp derives the teacher's mass, from every block's sums the row's
//    totals, the same in every block, and its loss.  (Every streaming warp
//    deriving the totals for itself took [2048,131072] bf16 to 305 us.)
//
// Patching: the entries at the teacher's columns are read, sent to every
// block of the cluster and set to -inf in shared memory.  What is summed is
// the student's mass off the teacher's columns, without the cancellation of
// 1 - sum p; the gradient at them takes the place of the 0 that results
// there.  All sums are added in a fixed order.
//
// The blocks tell one another by asynchronous stores that count their bytes
// on the receiver's barrier.  (A store and a release at cluster scope waits
// for the thread's gradient stores to reach L2: [2048,131072] bf16 took 372 us
// that way against 312 us.)
// A row that the clusters cannot hold (beyond 1 MB) is processed in tiles by
// distill_tiled_kernel, and read again for the gradient.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "ws_internal.cuh"
#include "ws_logits.cuh"
#include "ws_ptx.cuh"
#include "ws_select.cuh"

namespace ws {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kMaxCluster = 16;
constexpr int kMaxK = 256;             // one teacher entry a thread
constexpr float kTailMin = 1.0f / 1048576.0f;
constexpr float kLog2e = 1.4426950408889634f;

static_assert(kMaxK <= kThreads, "a thread holds at most one teacher entry");

struct DistillParams {
    const void* x;
    void* grad;             // NULL: the loss alone
    long long stride, grad_stride;
    long long rows, cols;
    const void* ids;
    int id64;
    int k;
    int tail;               // WS_DISTILL_TAIL
    int cluster;            // blocks a row
    int per;                // vectors of a block's run, at most
    int tile;               // vectors of the tiled kernel's buffer
    const float* teacher;
    const float* weight;
    float* loss;
    float c;                // log2(e) / temperature
    float inv_t;            // 1 / temperature
    float above;            // see clamp_above
    uint32_t* err;
};

// A row's entries, in every block.
struct RowExchange {
    float x[kMaxK];                 // the student's logits at the entries
    float lq[kMaxK];                // the teacher's log probabilities, -inf: no entry
};

struct __align__(16) TiledShared {
    RowExchange row;
    float m, m_off, scale, on, wt;  // of the row's totals
    SoftSums part[kWarps];          // the warps' sums
    float2 block[8];                // every block's maximum and sum
    float q[kMaxK];                 // the teacher's probabilities
    uint64_t bar;                   // a tile's copy has landed
    int bad;                        // a column past the row's end
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The teacher's probabilities of a row's entries into q_of (and, renormalised,
// their logarithms into r.lq); returns their sum.  One warp.
__device__ __forceinline__ float teacher_mass(const DistillParams& p, RowExchange& r, float* q_of) {
    const int lane = threadIdx.x & 31;
    float shift = 0.f;
    if (!p.tail) {
        float top = -INFINITY, sum = 0.f;
        for (int k = lane; k < p.k; k += 32) top = fmaxf(top, r.lq[k]);
        top = warp_max(top);
        if (top > -INFINITY) {
            for (int k = lane; k < p.k; k += 32) sum += exp2_fast((r.lq[k] - top) * kLog2e);
            shift = top + logf(warp_sum(sum));
        }
    }
    float mass = 0.f;
    for (int k = lane; k < p.k; k += 32) {
        const float lq = r.lq[k] - shift;
        const float q = lq > -INFINITY ? expf(lq) : 0.f;
        r.lq[k] = lq;
        q_of[k] = q;
        mass += q;
    }
    return warp_sum(mass);
}

// What the teacher alone gives of a row.
struct RowTeacher {
    float rest;      // the mass off its entries
    float whole;     // the mass in all: 1 but for rounding, 0 without entries where they are renormalised
    float wt;        // the row's weight / temperature
};

__device__ __forceinline__ RowTeacher row_teacher(const DistillParams& p, float mass, float weight) {
    RowTeacher t;
    t.rest = p.tail ? fmaxf(1.f - mass, 0.f) : 0.f;
    if (t.rest < kTailMin) t.rest = 0.f;
    t.whole = p.tail ? mass + t.rest : mass > 0.f ? 1.f : 0.f;
    t.wt = weight * p.inv_t;
    return t;
}

// What a row's loss and gradient are made of, in every lane of a warp.
//
// The sums off the teacher's columns stay relative to the largest logit there:
// a student that is sure of the teacher's columns has a mass off them that no
// float32 holds (2^-126 is a gap of 87 temperatures), but the tail's share
// of the gradient is the teacher's remaining mass spread by what each entry is
// of that mass, and the loss takes its logarithm.
struct RowTotals {
    float m;         // the largest logit
    float m_off;     // ... off the teacher's columns
    float off;       // the sum off them, relative to m_off
    float per_off;   // 2^((m_off - m) c): off is off * per_off relative to m
    float total;     // the sum over all, relative to m
    float scale;     // an entry off the teacher's columns: scale 2^((x - m_off) c)
    float on;        // an entry on them: on 2^((x - m) c) - wt q
    float wt;
};

// From n partial sums off the teacher's columns (maximum, sum) and the
// entries.  What the streaming warps wait for, so the chain is short: four
// partial sums a lane at once, one reduction of the maxima, one of the sums.
__device__ __forceinline__ RowTotals row_totals(const DistillParams& p, const RowExchange& r, const float2* part, int n,
                                                const RowTeacher& teacher) {
    const int lane = threadIdx.x & 31;
    RowTotals t;
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lane + 32 * i < n ? part[lane + 32 * i] : make_float2(-INFINITY, 0.f);
    const float x = lane < p.k ? r.x[lane] : -INFINITY;
    float m_off = fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x)), m_on = x;
    for (int i = lane + 128; i < n; i += 32) m_off = fmaxf(m_off, part[i].x);
    for (int k = lane + 32; k < p.k; k += 32) m_on = fmaxf(m_on, r.x[k]);
    t.m_off = order_value(__reduce_max_sync(0xffffffffu, order_bits(m_off)));
    t.m = fmaxf(t.m_off, order_value(__reduce_max_sync(0xffffffffu, order_bits(m_on))));
    float off = 0.f, on = exp2_fast(below(x, t.m) * p.c);
#pragma unroll
    for (int i = 0; i < 4; ++i) off += v[i].y * exp2_fast(below(v[i].x, t.m_off) * p.c);
    for (int i = lane + 128; i < n; i += 32) off += part[i].y * exp2_fast(below(part[i].x, t.m_off) * p.c);
    for (int k = lane + 32; k < p.k; k += 32) on += exp2_fast(below(r.x[k], t.m) * p.c);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        off += __shfl_xor_sync(0xffffffffu, off, o);
        on += __shfl_xor_sync(0xffffffffu, on, o);
    }
    t.off = off;
    t.per_off = exp2_fast(below(t.m_off, t.m) * p.c);
    t.total = off * t.per_off + on;
    t.wt = teacher.wt;
    t.on = teacher.whole * __fdividef(t.wt, t.total);   // 2 ulp
    t.scale = t.on * t.per_off;
    // off is 1 at least where anything is left off the teacher's columns
    if (teacher.rest > 0.f && t.m_off > -INFINITY) t.scale -= t.wt * __fdividef(teacher.rest, off);
    if (t.m == -INFINITY) t.scale = t.on = t.wt = 0.f;   // the student has nothing left
    if (t.m == INFINITY) t.scale = t.on = NAN;
    return t;
}

// The gradient at an entry on the teacher's columns.
__device__ __forceinline__ float entry_gradient(const DistillParams& p, const RowTotals& t, float x, float q) {
    return exp2_fast(below(x, t.m) * p.c) * t.on - t.wt * q;
}

// The row's weighted loss.
__device__ __forceinline__ float row_loss(const DistillParams& p, const RowExchange& r, const float* q_of, const RowTotals& t,
                                          const RowTeacher& teacher, float weight) {
    const int lane = threadIdx.x & 31;
    if (t.m == -INFINITY) return 0.f;   // the student has nothing left
    if (t.m == INFINITY) return NAN;
    const float ln_s = logf(t.total), per_total = 1.f / t.total;
    float term = 0.f, more = 0.f;
    for (int k = lane; k < p.k; k += 32) {
        const float x = r.x[k], q = q_of[k];
        // the student's log probability; -inf where it is masked
        const float lp = x > -INFINITY ? half_gap(x, t.m) * (2.f * p.inv_t) - ln_s : -INFINITY;
        if (q > 0.f) term += q * (r.lq[k] - lp);
        more += exp2_fast(below(x, t.m) * p.c) * per_total - q;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        term += __shfl_xor_sync(0xffffffffu, term, o);
        more += __shfl_xor_sync(0xffffffffu, more, o);   // the student's mass on the entries less the teacher's
    }
    float loss = term;
    if (teacher.rest > 0.f) {
        if (t.m_off > -INFINITY) {
            // ln(rest / p_off) by their difference while that is the exact
            // one, else by their logarithms (p_off itself may be below 2^-126)
            const float rel = more / (t.off * t.per_off * per_total);
            loss += teacher.rest * (rel > -0.5f && rel < 1.f
                                        ? log1pf(rel)
                                        : logf(teacher.rest) - (half_gap(t.m_off, t.m) * (2.f * p.inv_t) + (logf(t.off) - ln_s)));
        } else {
            loss = INFINITY;
        }
    }
    return loss * weight;
}

// The gradient of one vector of entries.
template <class E>
__device__ __forceinline__ uint4 gradient_of(const uint4& q, float m, f32x2 c2, f32x2 scale2, bool clamp_words) {
    float out[E::kPer];
    const f32x2 m2 = pack2(-m, -m);
    auto pair = [&](f32x2 d, int i) {
        float a0, a1;
        unpack2(mul2(d, c2), a0, a1);
        unpack2(mul2(pack2(exp2_fast(a0), exp2_fast(a1)), scale2), out[i], out[i + 1]);
    };
    if constexpr (E::kPer == 8) {
        if (clamp_words) {   // see add_vectors
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) pair(add2(E::widen(E::max_word(w[i], E::kLow)), m2), 2 * i);
            return E::pack(out);
        }
    }
    float f[E::kPer];
    E::unpack(q, f);
#pragma unroll
    for (int i = 0; i < E::kPer; i += 2) pair(pack2(below(f[i], m), below(f[i + 1], m)), i);
    return E::pack(out);
}

// The gradient of the n vectors of a row from vector t0 on, which lie in buf
// patched: by the threads tid, tid + threads, ...
template <class E>
__device__ __forceinline__ void write_gradient(const DistillParams& p, typename E::Storage* gr, const RowBlocks<E>& rb,
                                               const uint4* buf, int t0, int n, float m, float scale, int tid, int threads) {
    constexpr int kPer = E::kPer;
    const RowBlocks<E> gb(gr, p.cols);
    const f32x2 c2 = pack2(p.c, p.c), scale2 = pack2(scale, scale);
    const bool clamp_words = m > p.above && m < INFINITY;
    const int a = max(0, t0 * kPer - rb.lead), b = (int)min(p.cols, (long long)(t0 + n) * kPer - rb.lead);   // entries
    const int shift = (rb.lead - gb.lead + kPer) % kPer;
    if (shift == 0) {   // vector for vector
        for (int v = tid; v < n; v += threads)
            store_vector<E>(gr, gb, t0 + v, a, b, gradient_of<E>(buf[v], m, c2, scale2, clamp_words));
        return;
    }
    // a vector of the gradient takes entries of two of the run's
    for (int v = (a + gb.lead) / kPer + tid; v < (b + gb.lead + kPer - 1) / kPer; v += threads) {
        const int from = (v * kPer - gb.lead + rb.lead - shift) / kPer - t0;   // -1 .. n - 1
        const uint4 lo = from >= 0 ? buf[from] : make_uint4(0, 0, 0, 0);
        const uint4 hi = from + 1 < n ? buf[from + 1] : make_uint4(0, 0, 0, 0);
        store_vector<E>(gr, gb, v, a, b, gradient_of<E>(shifted<E>(lo, hi, shift), m, c2, scale2, clamp_words));
    }
}

// Zeros over the entries of a row that the run [v0, v1) holds.
template <class E>
__device__ __forceinline__ void write_zeros(const DistillParams& p, typename E::Storage* gr, const RowBlocks<E>& rb, int v0, int v1,
                                            int tid, int threads) {
    constexpr int kPer = E::kPer;
    const RowBlocks<E> gb(gr, p.cols);
    const int a = max(0, v0 * kPer - rb.lead), b = (int)min(p.cols, (long long)v1 * kPer - rb.lead);
    if (a >= b) return;
    for (int v = (a + gb.lead) / kPer + tid; v < (b + gb.lead + kPer - 1) / kPer; v += threads)
        store_vector<E>(gr, gb, v, a, b, make_uint4(0, 0, 0, 0));
}

// A block's run [v0, v1) of a row's vectors.
template <class E>
__device__ __forceinline__ void run_of(const DistillParams& p, const RowBlocks<E>& rb, int rank, int& v0, int& v1) {
    const int nvec = rb.nvec;
    v0 = min(rank * p.per, nvec);
    v1 = min(v0 + p.per, nvec);
}

// Where in its 128-byte line a vector lies.  A copy into shared memory whose
// source and destination lie differently is slow (see Run in logprobs.cu).
__device__ __forceinline__ int copy_offset(const uint4* p) { return (int)(reinterpret_cast<uintptr_t>(p) >> 4) & 7; }

// Entry e of a row whose vectors from t0 on lie in buf.
template <class E>
__device__ __forceinline__ typename E::Storage* entry_in(uint4* buf, const RowBlocks<E>& rb, int t0, long long e) {
    return reinterpret_cast<typename E::Storage*>(buf) + (e + rb.lead - (long long)t0 * E::kPer);
}

// Sets the foreign entries of the row's first and last vector to -inf, where
// buf (n vectors from t0 on) holds them: by threads 0 .. kPer - 1.
template <class E>
__device__ __forceinline__ void patch_ends(const DistillParams& p, uint4* buf, const RowBlocks<E>& rb, int t0, int n, int tid) {
    if (tid >= E::kPer || n <= 0) return;
    const long long head = rb.first(0) + tid, last = rb.first(rb.nvec - 1) + tid;
    if (t0 == 0 && head < 0) *entry_in<E>(buf, rb, t0, head) = E::round(-INFINITY);
    if (t0 + n == rb.nvec && last >= p.cols) *entry_in<E>(buf, rb, t0, last) = E::round(-INFINITY);
}

// Sends the student's logit at the row's entry k to every block.
__device__ __forceinline__ void send_entry(RowExchange& ex, int k, float x, int blocks) {
    if (blocks == 1) {
        ex.x[k] = x;
        return;
    }
    for (int i = 0; i < blocks; ++i) st_cluster_u32(cluster_map(&ex.x[k], (uint32_t)i), __float_as_uint(x));
}

// A thread's vectors of a run, buf[0], buf[stride], ...: their largest entry
// m, the exponentials 2^((x - m) c) and their sum.
template <class E, int kH>
__device__ __forceinline__ float take_run(const DistillParams& p, const uint4* buf, int stride, f32x2 (&e)[kH][E::kPer / 2],
                                          float& total) {
    constexpr int kPer = E::kPer;
    uint32_t mw = E::kNegInf;
#pragma unroll
    for (int j = 0; j < kH; ++j) {
        const uint4 q = buf[j * stride];
        mw = E::max_word(E::max_word(mw, E::max_word(q.x, q.y)), E::max_word(q.z, q.w));
    }
    const float m = E::max_of(mw);
    f32x2 sum = pack2(0.f, 0.f);
    const f32x2 m2 = pack2(-m, -m), c2 = pack2(p.c, p.c);
    auto take = [&](f32x2 d, f32x2& to) {
        float a0, a1;
        unpack2(mul2(d, c2), a0, a1);
        to = pack2(exp2_fast(a0), exp2_fast(a1));
        sum = add2(sum, to);
    };
    bool words = false;
    if constexpr (kPer == 8) words = m > p.above && m < INFINITY;   // see add_vectors
    if (words) {
        if constexpr (kPer == 8) {
#pragma unroll
            for (int j = 0; j < kH; ++j) {
                const uint4 q = buf[j * stride];
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) take(add2(E::widen(E::max_word(w[h], E::kLow)), m2), e[j][h]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kH; ++j) {
            float f[kPer];
            E::unpack(buf[j * stride], f);
#pragma unroll
            for (int h = 0; h < kPer / 2; ++h) take(pack2(below(f[2 * h], m), below(f[2 * h + 1], m)), e[j][h]);
        }
    }
    float s0, s1;
    unpack2(sum, s0, s1);
    total = s0 + s1;
    return m;
}

// Stores f times the exponentials of a thread's vectors of the run of nv from
// v0 on: vectors at, at + stride, ... of it.
template <class E, int kH>
__device__ __forceinline__ void store_run(const DistillParams& p, typename E::Storage* gr, int lead, int v0, int nv, int at,
                                          int stride, const f32x2 (&e)[kH][E::kPer / 2], float f) {
    constexpr int kPer = E::kPer;
    const f32x2 f2 = pack2(f, f);
    auto vector = [&](int j) {
        float out[kPer];
#pragma unroll
        for (int h = 0; h < kPer / 2; ++h) unpack2(mul2(e[j][h], f2), out[2 * h], out[2 * h + 1]);
        return E::pack(out);
    };
    const RowBlocks<E> gb(gr, p.cols);
    const int shift = (lead - gb.lead + kPer) % kPer;
    const int a = max(0, v0 * kPer - lead), b = (int)min(p.cols, (long long)(v0 + nv) * kPer - lead);   // entries
    if (shift == 0) {
        // vector for vector, whole but at the row's ends
        uint4* out = const_cast<uint4*>(gb.base) + v0 + at;
        const int first = v0 == 0 && lead > 0 ? 1 : 0, whole = (b + lead) / kPer - v0;
#pragma unroll
        for (int j = 0; j < kH; ++j) {
            const int v = at + j * stride;
            const uint4 q = vector(j);
            if (v >= first && v < whole) out[j * stride] = q;
            else if (v < nv) store_vector<E>(gr, gb, v0 + v, a, b, q);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kH; ++j) {
            const int v = at + j * stride;
            if (__all_sync(0xffffffffu, v >= nv)) break;
            store_shifted<E>(gr, vector(j), (v0 + v) * kPer - lead, a, b, shift);
        }
    }
}

// ------------------------------------------------------------- short rows

// A warp a row of at most 32 * kH vectors.  The row lies in shared memory
// while the teacher's entries are taken out of it; after that nothing but
// shuffles.  Bound by its chain with few rows (3.7 us for [8,1000] f32, 5
// entries), by instructions with many: [20000,1000] f32 37.9 us, 4.2 TB/s.
template <class E, int kH>
__global__ void __launch_bounds__(128, 4) distill_short_kernel(const __grid_constant__ DistillParams p) {
    using S = typename E::Storage;
    struct __align__(16) RowShared {
        uint4 buf[32 * kH];
        RowExchange row;
        float q[kMaxK];
        float2 part;
    };
    __shared__ RowShared shared[4];
    const int lane = threadIdx.x & 31;
    RowShared& s = shared[threadIdx.x >> 5];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    launch_dependents();
    const long long row = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const S* xr = static_cast<const S*>(p.x) + row * p.stride;
    S* gr = p.grad ? static_cast<S*>(p.grad) + row * p.grad_stride : nullptr;
    const RowBlocks<E> rb(xr, p.cols);
    const int nvec = rb.nvec;
    const float weight = p.weight ? p.weight[row] : 1.f;
    if (weight == 0.f) {   // the row is not read
        if (lane == 0) p.loss[row] = 0.f;
        if (gr) write_zeros<E>(p, gr, rb, 0, nvec, lane, 32);
        return;
    }
    uint4 x[kH];
#pragma unroll
    for (int j = 0; j < kH; ++j) {
        const int v = j * 32 + lane;
        x[j] = v < nvec ? rb.base[v] : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
    }
    long long id = -1;
    float lq = -INFINITY;
    auto load_entry = [&](int k) {
        id = -1;
        if (k < p.k) {
            id = load_index(p.ids, row * p.k + k, p.id64);
            lq = p.teacher[row * p.k + k];
        }
    };
    load_entry(lane);
#pragma unroll
    for (int j = 0; j < kH; ++j) {
        mask_ends<E>(x[j], j * 32 + lane, rb, p.cols);
        s.buf[j * 32 + lane] = x[j];
    }
    __syncwarp();
    for (int k = lane; k - lane < p.k; k += 32) {
        if (k >= 32) load_entry(k);
        if (k < p.k) {
            const bool is = id >= 0 && id < p.cols;
            s.row.lq[k] = is ? fmaxf(lq, -INFINITY) : -INFINITY;   // NaN: no mass
            s.row.x[k] = id >= p.cols ? INFINITY : -INFINITY;      // past the end: the row's results become NaN
            if (id >= p.cols) atomicOr(p.err, (uint32_t)kDevErrBadIndex);
            if (is) {
                S* at = entry_in<E>(s.buf, rb, 0, id);
                s.row.x[k] = fmaxf(E::load(at), -INFINITY);
                *at = E::round(-INFINITY);
            }
        }
    }
    __syncwarp();
    f32x2 e[kH][E::kPer / 2];
    float sum;
    const float m = take_run<E, kH>(p, s.buf + lane, 32, e, sum);
    const float wm = order_value(__reduce_max_sync(0xffffffffu, order_bits(m)));
    const float ws = warp_sum(sum * exp2_fast(below(m, wm) * p.c));
    if (lane == 0) s.part = make_float2(wm, ws);
    const float mass = teacher_mass(p, s.row, s.q);
    __syncwarp();
    const RowTeacher teacher = row_teacher(p, mass, weight);
    const RowTotals t = row_totals(p, s.row, &s.part, 1, teacher);
    const float loss = row_loss(p, s.row, s.q, t, teacher, weight);
    if (lane == 0) p.loss[row] = loss;
    if (!gr) return;
    store_run<E, kH>(p, gr, rb.lead, 0, nvec, lane, 32, e, t.scale * exp2_fast(below(m, t.m_off) * p.c));
    __syncwarp();   // the zeros at the teacher's columns are written
    for (int k = lane; k < p.k; k += 32) {
        if (k >= 32 || p.k > 32) load_entry(k);
        if (id >= 0 && id < p.cols) gr[id] = E::round(entry_gradient(p, t, s.row.x[k], s.q[k]));
    }
}

// ------------------------------------------------------------ rows on chip

constexpr int kSlots = 4;              // rows whose exchange may be under way at once

// A live row and the block's run of it; row -1: the last one has been.
struct RowPlace {
    long long row;
    int v0, nv, lead;
    int off;        // the run begins at this vector of its buffer
};

template <int kW, int kH>
struct __align__(16) Shared {
    RowExchange row[kSlots];             // the live rows in turn
    float q[kSlots][kMaxK];              // the teacher's probabilities
    float4 totals[kSlots];               // m_off, scale, m, on of the row's totals
    float wt[kSlots];                    // ... and wt
    float2 part[kSlots][kMaxCluster * kW];   // every block's every streaming warp's maximum and sum
    int own[kSlots][kMaxK];              // the teacher's columns in this block's run: entry of the run | k << 20
    int owned[kSlots];                   // how many
    uint64_t landed[2], ready[2], taken[2];   // by buffer: the copy has landed; is patched; is in registers
    uint64_t exchanged[kSlots];          // every block's sums and entries are there
    uint64_t known[kSlots];              // the row's totals are
    uint64_t settled[kSlots];            // the loss is written: the slot has been read
    RowPlace place[kSlots];              // where the row is
};

// The rows of a cluster that take part (whose weight is not 0), in order, as
// a warp sees them: 32 rows' weights at a time.
struct LiveRows {
    const float* weight;
    int row0, step, rows;
    int base;              // of the window
    unsigned mask;         // its live rows not yet taken
    __device__ __forceinline__ unsigned window(int at) const {
        const int i = at + (int)(threadIdx.x & 31);
        return __ballot_sync(0xffffffffu, i < rows && (!weight || weight[row0 + (long long)i * step] != 0.f));
    }
    __device__ __forceinline__ LiveRows(const float* w, int r0, int st, int n)
        : weight(w), row0(r0), step(st), rows(n), base(0), mask(window(0)) {}
    // The next one, or -1.
    __device__ __forceinline__ long long next() {
        while (mask == 0) {
            if (base >= rows - 32) return -1;
            base += 32;
            mask = window(base);
        }
        const int i = base + __ffs(mask) - 1;
        mask &= mask - 1;
        return row0 + (long long)i * step;
    }
};

// kW streaming warps, kH vectors a thread.
//
// A row costs a chain: copy, sums, exchange, totals, gradient (about 3.6 us
// with 64 KB runs).  Two buffers a block let a row's copy and patching run
// under the chain of the row before, and the blocks of an SM under one
// another; registers (96 a thread, the exponentials) and shared memory bound
// how many those are.  Bound by that latency: [2048,131072] bf16 with 32
// entries and the tail class takes 192 us, 5.6 TB/s of logits and gradients
// (0.83 of a copy's), f32 410 us; [512,32000] f16 21 us, where a cluster has
// 3.4 rows.
//
// The next kernel is not launched early (griddepcontrol.launch_dependents):
// its clusters then take what is free between this one's, and [2048,131072]
// bf16 takes 272 us a call instead of 212.
template <class E, int kW, int kH>
__global__ void __launch_bounds__(32 * kW + 64, kW == 4 ? 5 : kW == 16 ? 1 : kH == 4 ? 3 : 2) distill_kernel(const __grid_constant__ DistillParams p) {
    using S = typename E::Storage;
    constexpr int kPer = E::kPer;
    constexpr int kStream = 32 * kW;
    constexpr int kRun = kStream * kH;   // vectors of a run, at most
    constexpr int kBuffer = kRun + 8;    // a run lies in its 128-byte lines as it does in memory: see copy_offset
    extern __shared__ __align__(128) unsigned char dsmem[];
    __shared__ Shared<kW, kH> s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.cluster;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.landed[i], 1);
            mbar_init(&s.ready[i], 1);
            mbar_init(&s.taken[i], kW);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.exchanged[i], C == 1 ? (uint32_t)kW : 1u);   // a cluster's by bytes: see below
            mbar_init(&s.known[i], 1);
            mbar_init(&s.settled[i], 1);
        }
        fence_mbar_init();
    }
    // what lies behind a run in its buffer is -inf throughout
    for (int i = tid; i < 2 * kBuffer; i += kStream + 64)
        reinterpret_cast<uint4*>(dsmem)[i] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
    fence_proxy_async();
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)cluster_nctarank() != C) {
        if (tid == 0) atomicOr(p.err, (uint32_t)kDevErrBadLaunch);
        return;
    }
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    if (C > 1) cluster_sync();   // every block's barriers are set up and its memory may be written to
    // this cluster's rows: row0 + i * step (below 2^31 of them, as rows * stride is at most 2^40)
    const int row0 = (int)blockIdx.x / C, step = (int)gridDim.x / C;
    const int rows = (int)((p.rows - row0 + step - 1) / step);
    auto x_of = [&](long long row) { return static_cast<const S*>(p.x) + row * p.stride; };
    auto grad_of = [&](long long row) { return static_cast<S*>(p.grad) + row * p.grad_stride; };
    auto buffer = [&](int b) { return reinterpret_cast<uint4*>(dsmem) + b * kBuffer; };
    // A bounded wait of a whole warp for the n-th use of one of `of` barriers;
    // the result is the same in every lane.  A warp whose wait has run out
    // leaves its rows: the others' waits then run out as well, and the rows
    // that were left to the cluster are not written.
    auto wait = [&](uint64_t* bar, unsigned n, unsigned of, bool cluster_scope) {
        uint64_t* at = &bar[n % of];
        const uint32_t parity = n / of & 1u;
        bool ok = cluster_scope ? mbar_wait_bounded_cluster(at, parity, 2 * kWaitLimitNs)
                                : mbar_wait_bounded(at, parity, 2 * kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (!ok && lane == 0) atomicOr(p.err, (uint32_t)kDevErrBulkCopyTimeout);
        return ok;
    };

    if (warp < kW) {
        // ------------------------------------------------ a streaming warp
        if (p.grad && p.weight)   // rows that do not take part
            for (int i = 0; i < rows; ++i) {
                const long long row = row0 + (long long)i * step;
                if (p.weight[row] != 0.f) continue;
                const RowBlocks<E> rb(x_of(row), p.cols);
                int v0, v1;
                run_of<E>(p, rb, rank, v0, v1);
                write_zeros<E>(p, grad_of(row), rb, v0, v1, tid, kStream);
            }
        for (unsigned n = 0;; ++n) {
            const unsigned slot = n % kSlots;
            if (!wait(s.ready, n, 2, false) || s.place[slot].row < 0) break;
            const int nv = s.place[slot].nv;
            const uint4* buf = buffer(n & 1) + s.place[slot].off + tid;
            f32x2 e[kH][kPer / 2];
            float sum;
            const float m = take_run<E, kH>(p, buf, kStream, e, sum);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.taken[n & 1]);
            // the warp's sum, to every block
            const float wm = order_value(__reduce_max_sync(0xffffffffu, order_bits(m)));
            const float ws = warp_sum(sum * exp2_fast(below(m, wm) * p.c));
            if (C == 1) {
                if (lane == 0) {
                    s.part[slot][warp] = make_float2(wm, ws);
                    mbar_arrive(&s.exchanged[slot]);
                }
            } else if (lane < C) {
                st_async_v2(cluster_map(&s.part[slot][rank * kW + warp], (uint32_t)lane), wm, ws,
                            cluster_map(&s.exchanged[slot], (uint32_t)lane));
            }
            __syncwarp();
            // the gradient, once the row's totals are known
            if (!wait(s.known, n, kSlots, false)) break;
            if (p.grad) {
                const int v0 = s.place[slot].v0;
                const float4 of = s.totals[slot];
                RowTotals t;
                t.m_off = of.x;
                t.scale = of.y;
                t.m = of.z;
                t.on = of.w;
                t.wt = s.wt[slot];
                S* gr = grad_of(s.place[slot].row);
                const int lead = s.place[slot].lead;
                store_run<E, kH>(p, gr, lead, v0, nv, tid, kStream, e, t.scale * exp2_fast(below(m, t.m_off) * p.c));
                // the teacher's columns among this warp's vectors, after the
                // warp's zeros there
                __syncwarp();
                for (int h = lane; h < s.owned[slot]; h += 32) {
                    const int at = s.own[slot][h] & 0xfffff, k = s.own[slot][h] >> 20;   // entry of the run
                    if (at / kPer / 32 % kW == warp)
                        gr[v0 * kPer + at - lead] = E::round(entry_gradient(p, t, s.row[slot].x[k], s.q[slot][k]));
                }
            }
        }
    } else if (warp == kW) {
        // ---------------------------------------- the warp that keeps the runs
        auto issue = [&](long long row, unsigned n) {
            if (row < 0) return;
            const RowBlocks<E> rb(x_of(row), p.cols);
            int v0, v1;
            run_of<E>(p, rb, rank, v0, v1);
            if (lane == 0) {
                if (v1 > v0) {
                    mbar_arrive_expect_tx(&s.landed[n & 1], (uint32_t)(v1 - v0) * 16u);
                    bulk_g2s(buffer(n & 1) + copy_offset(rb.base + v0), rb.base + v0, (uint32_t)(v1 - v0) * 16u, &s.landed[n & 1]);
                } else {
                    mbar_arrive(&s.landed[n & 1]);
                }
            }
        };
        LiveRows live(p.weight, row0, step, rows);
        long long row = live.next(), row1 = row < 0 ? -1 : live.next();
        issue(row, 0);
        issue(row1, 1);   // and from row 2 on when a buffer is free
        // the teacher's entries of a row, 32 at a time; the first of them a row ahead
        long long id = -1, id_next = -1;
        float lq = -INFINITY, lq_next = -INFINITY;
        auto load_entry = [&](long long r, int k, long long& to_id, float& to_lq) {
            to_id = -1;
            if (k < p.k && r >= 0) {
                to_id = load_index(p.ids, r * p.k + k, p.id64);
                to_lq = p.teacher[r * p.k + k];
            }
        };
        load_entry(row, lane, id_next, lq_next);
        bool ok = true;
        for (unsigned n = 0;; ++n) {
            id = id_next;
            lq = lq_next;
            load_entry(row1, lane, id_next, lq_next);
            const long long row2 = row1 < 0 ? -1 : live.next();
            const unsigned slot = n % kSlots;
            RowExchange& ex = s.row[slot];
            // Every block has finished with the slot: their warps sent the
            // sums of row n - 2 after they were done with row n - 4 and, as
            // below, after its loss was written.
            if (n >= 2) ok = wait(s.known, n - 2, kSlots, false) && wait(s.settled, n - 2, kSlots, false);
            if (row < 0 || !ok) {   // no more
                if (lane == 0) {
                    s.place[slot].row = -1;
                    mbar_arrive(&s.ready[n & 1]);
                }
                break;
            }
            if (!(ok = wait(s.landed, n, 2, false))) break;
            const RowBlocks<E> rb(x_of(row), p.cols);
            int v0, v1;
            run_of<E>(p, rb, rank, v0, v1);
            const int off = copy_offset(rb.base + v0);
            uint4* buf = buffer(n & 1) + off;
            patch_ends<E>(p, buf, rb, v0, v1 - v0, lane);
            // the buffer's last run may have been longer, or have lain 7 vectors further
            if (lane < 8 && v1 - v0 + lane < kRun)
                buf[v1 - v0 + lane] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
            __syncwarp();
            int entries = 0, owned = 0;   // the row's entries that are columns; those in this block's run
            for (int base = 0; base < p.k; base += 32) {
                const int k = base + lane;
                if (base > 0) load_entry(row, k, id, lq);
                const bool is = k < p.k && id >= 0 && id < p.cols;
                const int v = is ? (int)((id + rb.lead) / kPer) : -1;
                const bool mine = v >= v0 && v < v1;
                if (k < p.k) {
                    ex.lq[k] = is ? fmaxf(lq, -INFINITY) : -INFINITY;   // NaN: no mass
                    if (!is) ex.x[k] = id >= p.cols ? INFINITY : -INFINITY;   // past the end: the row's results become NaN
                    if (id >= p.cols) atomicOr(p.err, (uint32_t)kDevErrBadIndex);
                }
                const unsigned who = __ballot_sync(0xffffffffu, mine);
                if (mine) {
                    S* at = entry_in<E>(buf, rb, v0, id);
                    const float x = fmaxf(E::load(at), -INFINITY);
                    *at = E::round(-INFINITY);
                    s.own[slot][owned + __popc(who & ((1u << lane) - 1u))] =
                        (int)(at - reinterpret_cast<S*>(buf)) | k << 20;
                    if (C == 1) ex.x[k] = x;
                    for (int i = 0; C > 1 && i < C; ++i)
                        st_async_f32(cluster_map(&ex.x[k], (uint32_t)i), x, cluster_map(&s.exchanged[slot], (uint32_t)i));
                }
                owned += __popc(who);
                entries += __popc(__ballot_sync(0xffffffffu, is));
            }
            if (lane == 0) {
                s.owned[slot] = owned;
                s.place[slot] = RowPlace{row, v0, v1 - v0, rb.lead, off};
                // every block's every warp sends its sums, and each entry comes
                // from the block that holds it: so many bytes (some may have
                // landed already)
                if (C > 1) mbar_arrive_expect_tx(&s.exchanged[slot], (uint32_t)(C * kW) * 8u + (uint32_t)entries * 4u);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.ready[n & 1]);
            // the other buffer's next run, once its entries are in registers
            if (n >= 1) {
                if (!(ok = wait(s.taken, n - 1, 2, false))) break;
                fence_proxy_async();
                __syncwarp();
                issue(row1, n + 1);
            }
            row = row1;
            row1 = row2;
        }
        if (!ok)   // the copies in flight must not outlive the block (a barrier is in one phase or the other)
            for (int i = 0; i < 4; ++i) mbar_wait_bounded(&s.landed[i & 1], i >> 1, kWaitLimitNs / 8);
    } else {
        // ------------------------------------- the warp that keeps the losses
        if (rank == 0)   // rows that do not take part
            for (int i = lane; p.weight && i < rows; i += 32) {
                const long long row = row0 + (long long)i * step;
                if (p.weight[row] == 0.f) p.loss[row] = 0.f;
            }
        for (unsigned n = 0;; ++n) {
            const unsigned slot = n % kSlots;
            RowExchange& ex = s.row[slot];
            if (!wait(s.ready, n, 2, false)) break;
            const long long row = s.place[slot].row;
            if (row < 0) break;
            const float weight = p.weight ? p.weight[row] : 1.f;
            const float mass = teacher_mass(p, ex, s.q[slot]);
            const RowTeacher teacher = row_teacher(p, mass, weight);
            __syncwarp();   // every lane's q, which lane 0's arrival on `known` publishes
            if (!wait(s.exchanged, n, kSlots, true)) break;
            const RowTotals t = row_totals(p, ex, s.part[slot], C * kW, teacher);
            if (lane == 0) {
                s.totals[slot] = make_float4(t.m_off, t.scale, t.m, t.on);
                s.wt[slot] = t.wt;
                mbar_arrive(&s.known[slot]);
            }
            __syncwarp();
            const float loss = row_loss(p, ex, s.q[slot], t, teacher, weight);
            if (rank == 0 && lane == 0) p.loss[row] = loss;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.settled[slot]);
        }
    }
    if (C > 1) cluster_sync();   // no block's memory is given up while another may write to it
}

// --------------------------------------------------- rows longer than that

// One cluster of eight blocks a row, its runs in tiles: a pass for the sums,
// another for the gradient.  Phases follow one another, by all threads.  Such
// rows are longer than any vocabulary in use here; the kernel is kept simple,
// and reads them twice.
template <class E>
__global__ void __launch_bounds__(kThreads) distill_tiled_kernel(const __grid_constant__ DistillParams p) {
    using S = typename E::Storage;
    constexpr int kPer = E::kPer;
    extern __shared__ __align__(128) unsigned char dsmem[];
    uint4* buf = reinterpret_cast<uint4*>(dsmem);
    __shared__ TiledShared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        mbar_init(&s.bar, 1);
        s.bad = 0;
        fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int C = p.cluster;
    if ((int)cluster_nctarank() != C) {
        if (tid == 0) atomicOr(p.err, (uint32_t)kDevErrBadLaunch);
        return;
    }
    const int rank = (int)cluster_ctarank();
    cluster_sync();   // every block has started: its memory may be written to
    const long long row = blockIdx.x / C;
    const RowBlocks<E> rb(static_cast<const S*>(p.x) + row * p.stride, p.cols);
    S* gr = p.grad ? static_cast<S*>(p.grad) + row * p.grad_stride : nullptr;
    int v0, v1;
    run_of<E>(p, rb, rank, v0, v1);
    const float weight = p.weight ? p.weight[row] : 1.f;
    if (weight == 0.f) {   // the row is not read
        if (rank == 0 && tid == 0) p.loss[row] = 0.f;
        if (p.grad) write_zeros<E>(p, gr, rb, v0, v1, tid, kThreads);
        cluster_sync();
        return;
    }
    // Copies the tile of n vectors from t0 on and waits for it.  A copy that
    // does not land in time is waited for once more (it must not outlive the
    // block); the block then goes on without copies, its results NaN, for the
    // cluster's sake.
    uint32_t parity = 0;
    bool dead = false;
    auto fetch = [&](int t0, int n) {
        fence_proxy_async();
        __syncthreads();   // the previous tile has been read
        bool ok = true;
        if (!dead) {
            if (tid == 0) {
                mbar_arrive_expect_tx(&s.bar, (uint32_t)n * 16u);
                bulk_g2s(buf, rb.base + t0, (uint32_t)n * 16u, &s.bar);
            }
            ok = mbar_wait_bounded(&s.bar, parity, kWaitLimitNs);
            if (!ok) mbar_wait_bounded(&s.bar, parity, kWaitLimitNs);
            parity ^= 1u;
        }
        // no thread patches what another has not seen land
        if (__syncthreads_or(!ok)) {
            dead = true;
            if (tid == 0) atomicOr(p.err, (uint32_t)kDevErrBulkCopyTimeout);
        }
    };
    RowExchange& ex = s.row;
    long long id = -1;
    if (tid < p.k) {
        id = load_index(p.ids, row * p.k + tid, p.id64);
        const float l = p.teacher[row * p.k + tid];
        if (id >= p.cols) {
            id = -1;
            atomicOr(p.err, (uint32_t)kDevErrBadIndex);
            s.bad = 1;
        }
        ex.lq[tid] = id >= 0 ? fmaxf(l, -INFINITY) : -INFINITY;   // NaN: no mass
        if (id < 0) ex.x[tid] = -INFINITY;
    }
    const long long my_v = id >= 0 ? (id + rb.lead) / kPer : -1;   // the vector that holds this thread's entry
    auto patch = [&](int t0, int n, bool send) {
        if (my_v >= t0 && my_v < t0 + n) {
            S* e = entry_in<E>(buf, rb, t0, id);
            if (send) send_entry(ex, tid, fmaxf(E::load(e), -INFINITY), C);
            *e = E::round(-INFINITY);
        }
        patch_ends<E>(p, buf, rb, t0, n, tid);
        __syncthreads();
    };
    RunningSums a;
    a.clear();
    for (int t0 = v0; t0 < v1; t0 += p.tile) {
        const int n = min(p.tile, v1 - t0);
        fetch(t0, n);
        patch(t0, n, true);
        for (int v = tid; v < n; v += kThreads * kUnroll) {
            uint4 q[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                q[j] = v + j * kThreads < n ? buf[v + j * kThreads]
                                            : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
            add_vectors<E, kUnroll, false>(a, q, p.c, p.above);
        }
    }
    const SoftSums w = warp_sums(a.sums(), p.c);
    if (lane == 0) s.part[warp] = w;
    __syncthreads();
    if (warp == 0) {
        SoftSums total = lane_sums(s.part, kWarps, p.c);
        if (dead || s.bad) total.m = INFINITY;   // the row's results become NaN, in every block
        if (lane < C) {
            const uint32_t dst = cluster_map(&s.block[rank], (uint32_t)lane);
            st_cluster_u32(dst, __float_as_uint(total.m));
            st_cluster_u32(dst + 4, __float_as_uint(total.s));
        }
    }
    cluster_sync();
    if (warp == 0) {
        const float mass = teacher_mass(p, ex, s.q);
        const RowTeacher teacher = row_teacher(p, mass, weight);
        const RowTotals t = row_totals(p, ex, s.block, C, teacher);
        const float loss = row_loss(p, ex, s.q, t, teacher, weight);
        if (rank == 0 && lane == 0) p.loss[row] = loss;
        if (lane == 0) {
            s.m = t.m;
            s.m_off = t.m_off;
            s.scale = t.scale;
            s.on = t.on;
            s.wt = t.wt;
        }
    }
    __syncthreads();
    if (p.grad) {
        for (int t0 = v0; t0 < v1; t0 += p.tile) {
            const int n = min(p.tile, v1 - t0);
            fetch(t0, n);
            patch(t0, n, false);
            write_gradient<E>(p, gr, rb, buf, t0, n, s.m_off, dead ? NAN : s.scale, tid, kThreads);
        }
        __syncthreads();   // the gradient at the teacher's columns is written
        if (my_v >= v0 && my_v < v1) {
            RowTotals t{};
            t.m = s.m;
            t.on = s.on;
            t.wt = s.wt;
            gr[id] = E::round(entry_gradient(p, t, ex.x[tid], s.q[tid]));
        }
    }
}

ws_status validate_desc(const ws_distill_desc* d) {
    if (!d) return fail(WS_ERR_INVALID_ARGUMENT, "desc is NULL");
    WS_TRY(validate_logits(d->rows, d->cols, d->row_stride, d->dtype, d->index_type, d->temperature));
    if (d->grad_stride < d->cols)
        return fail(WS_ERR_INVALID_ARGUMENT, "grad_stride %lld < cols %lld", (long long)d->grad_stride, (long long)d->cols);
    if (d->rows > (1LL << 40) / d->grad_stride) return fail(WS_ERR_INVALID_ARGUMENT, "rows * grad_stride too large");
    if (d->k < 1 || d->k > kMaxK) return fail(WS_ERR_INVALID_ARGUMENT, "k %d outside 1..%d", d->k, kMaxK);
    if (d->mode != WS_DISTILL_RENORM && d->mode != WS_DISTILL_TAIL)
        return fail(WS_ERR_INVALID_ARGUMENT, "mode %d", d->mode);
    return WS_OK;
}

constexpr int kTile = 96 * 1024;      // bytes of the tiled kernel's buffer

// Two buffers of a run and 8 vectors more.
constexpr int run_memory(int warps, int held) { return 2 * (32 * warps * held + 8) * 16; }

template <class E, int kW, int kH>
cudaError_t set_attributes(int dev) {
    static std::atomic<bool> set[64];
    if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const auto kernel = distill_kernel<E, kW, kH>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         run_memory(kW, kH));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
    return e;
}

// Clusters of `cluster` blocks with `smem` bytes of runs that the
// device holds at once (0: it cannot place one).  Asked once per shape.
template <class E, int kW, int kH>
int resident_clusters(int dev, int cluster, size_t smem) {
    static std::mutex mu;
    static std::map<std::tuple<int, int, size_t>, int> known;
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(dev, cluster, smem);
    auto it = known.find(key);
    if (it != known.end()) return it->second;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(32 * kW + 64);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (set_attributes<E, kW, kH>(dev) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, distill_kernel<E, kW, kH>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();   // not kept: asked again next time
        return 0;
    }
    known.emplace(key, n);
    return n;
}

// A shape that holds a row: clusters of `cluster` blocks, each with a run of
// at most `per` vectors.
struct RowShape {
    int cluster, per;
    int resident;       // clusters that the device holds at once; 0: none
};

template <class E, int kW, int kH>
RowShape row_shape(long long nvec, int dev, int most) {
    constexpr int kRun = 32 * kW * kH;
    RowShape f{};
    if (nvec > (long long)kRun * most) return f;
    f.cluster = (int)((nvec + kRun - 1) / kRun);
    // whole 128-byte lines a run, where the rows begin on one
    f.per = (int)((nvec + 8ll * f.cluster - 1) / (8ll * f.cluster)) * 8;
    f.resident = resident_clusters<E, kW, kH>(dev, f.cluster, run_memory(kW, kH));
    return f;
}

template <class E, int kW, int kH>
cudaError_t launch_rows(DistillParams p, const RowShape& f, cudaStream_t stream) {
    p.cluster = f.cluster;
    p.per = f.per;
    const long long clusters = std::min<long long>(p.rows, f.resident);
    return launch_clusters(distill_kernel<E, kW, kH>, dim3((unsigned)(clusters * f.cluster)), 32 * kW + 64, f.cluster,
                           run_memory(kW, kH), stream, p);
}

template <class E>
cudaError_t launch_distill(DistillParams p, int dev, int sm_count, cudaStream_t stream) {
    // vectors of a row: one more where rows may start inside a vector
    const bool aligned = (uintptr_t)p.x % 16 == 0 && (p.rows == 1 || p.stride % E::kPer == 0);
    const long long nvec = aligned ? (p.cols + E::kPer - 1) / E::kPer : (p.cols + 2 * E::kPer - 2) / E::kPer;
    // [4096,1000] f32 11.8 us, 19.6 by blocks of six warps
    if (nvec <= 256 && p.rows <= 4ll * 2147483647) {
        // one warp a block while the rows alone do not fill the SMs, four after
        const int warps = p.rows <= 4ll * sm_count ? 1 : 4;
        const dim3 grid((unsigned)((p.rows + warps - 1) / warps)), block(32 * warps);
        return nvec <= 64 ? launch_pdl(distill_short_kernel<E, 2>, grid, block, 0, stream, p)
                          : launch_pdl(distill_short_kernel<E, 8>, grid, block, 0, stream, p);
    }
    if (nvec <= 512) {
        const RowShape f = row_shape<E, 4, 4>(nvec, dev, 1);
        if (f.resident > 0) return launch_rows<E, 4, 4>(p, f, stream);
    }
    // [8000,8192] bf16 62 us, 94 with eight vectors a thread, half of them empty
    if (nvec <= 1024) {
        const RowShape f = row_shape<E, 8, 4>(nvec, dev, 1);
        if (f.resident > 0) return launch_rows<E, 8, 4>(p, f, stream);
    }
    // Clusters of up to 16 blocks, a size that a device need not support: then
    // 8.  As few blocks a row as hold it (more of them while rows leave SMs
    // idle: [8,131072] bf16 7.2 us instead of 6.2).  Sixteen warps a block and
    // runs of 64 KB mean half the blocks in a row's exchange, but one block an
    // SM, whose rows' phases do not overlap: [1024,262144] bf16 takes 234 us
    // that way and 270 with eight warps, [2048,131072] 198 and 209, but
    // [301,65537] 40 and 37, [1,131072] 7.4 and 6.2.
    for (int most = 16; most >= 8; most /= 2) {
        const RowShape f = row_shape<E, 8, 8>(nvec, dev, most);
        const RowShape wide = row_shape<E, 16, 8>(nvec, dev, most);
        if (wide.resident > 0 && (f.resident == 0 || (f.cluster >= 4 && (p.rows + f.resident - 1) / f.resident >= 16)))
            return launch_rows<E, 16, 8>(p, wide, stream);
        if (f.resident > 0) return launch_rows<E, 8, 8>(p, f, stream);
    }
    // rows too long for that: in tiles, on the portable 8 blocks
    static std::atomic<bool> set[64];
    if (!set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(distill_tiled_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTile);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    p.cluster = 8;
    p.per = (int)((nvec + 7) / 8);
    p.tile = kTile / 16;
    if (p.rows > 2147483647LL / p.cluster) return cudaErrorInvalidConfiguration;
    return launch_clusters(distill_tiled_kernel<E>, dim3((unsigned)(p.rows * p.cluster)), kThreads, 8, kTile, stream, p);
}

}  // namespace
}  // namespace ws

extern "C" {

ws_status ws_distill_validate(const ws_distill_desc* desc) {
    ws::clear_error();
    return ws::validate_desc(desc);
}

ws_status ws_distill(const ws_distill_desc* desc, const void* logits, const void* teacher_idx,
                     const float* teacher_logprob, const float* weight, float* loss, void* grad_logits,
                     cudaStream_t stream) {
    using namespace ws;
    clear_error();
    WS_TRY(validate_desc(desc));
    const size_t size = elem_size(desc->dtype);
    WS_TRY(check_pointer(logits, size, "logits"));
    WS_TRY(check_pointer(teacher_idx, desc->index_type == WS_INDEX_I64 ? 8 : 4, "teacher_idx"));
    WS_TRY(check_pointer(teacher_logprob, 4, "teacher_logprob"));
    if (weight) WS_TRY(check_pointer(weight, 4, "weight"));
    WS_TRY(check_pointer(loss, 4, "loss"));
    if (grad_logits) {
        WS_TRY(check_pointer(grad_logits, size, "grad_logits"));
        WS_TRY(check_gradient(logits, desc->row_stride, grad_logits, desc->grad_stride, desc->rows, desc->cols, size));
    }

    int dev;
    const DeviceInfo* info;
    WS_TRY(current_device_info(&dev, &info));
    DistillParams p{};
    p.x = logits;
    p.grad = grad_logits;
    p.stride = desc->row_stride;
    p.grad_stride = desc->grad_stride;
    p.rows = desc->rows;
    p.cols = desc->cols;
    p.ids = teacher_idx;
    p.id64 = desc->index_type == WS_INDEX_I64;
    p.k = desc->k;
    p.tail = desc->mode == WS_DISTILL_TAIL;
    p.teacher = teacher_logprob;
    p.weight = weight;
    p.loss = loss;
    p.c = log2e_over(desc->temperature);
    p.inv_t = 1.0f / desc->temperature;
    p.above = clamp_above(desc->dtype, desc->temperature);
    p.err = device_error_word();
    cudaError_t e;
    if (desc->dtype == WS_DTYPE_F32)
        e = launch_distill<ElemF32>(p, dev, info->sm_count, stream);
    else if (desc->dtype == WS_DTYPE_F16)
        e = launch_distill<ElemF16>(p, dev, info->sm_count, stream);
    else
        e = launch_distill<ElemBF16>(p, dev, info->sm_count, stream);
    if (e != cudaSuccess) return cuda_fail(e, "distillation launch");
    return WS_OK;
}

}  // extern "C"
