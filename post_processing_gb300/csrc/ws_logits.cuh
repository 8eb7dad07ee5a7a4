// ws_logits.cuh -- what the logits kernels (logprobs.cu, distill.cu) share:
// element types, a row of logits as 16-byte vectors, and the running sums of
// a softmax.
//
// A row may start at any element, so it is read as the 16-byte blocks that
// hold its elements: `lead` entries of the first block and some of the last
// belong to its neighbours (or to the padding), are read and never used.
// Such a block holds at least one byte of the row, so no read leaves the
// memory that the row's own elements lie in.
//
// Sums of a softmax over entries x with scale c = log2(e) / temperature:
// relative to a reference m (the largest entry seen),
//   d = x - m,  e = 2^(d c),  s = sum e,  t = sum e d,
// from which the log-sum-exp is m / temperature + ln s and the entropy
// ln s - t / (s temperature).  d is taken before the scaling, so entries near
// the maximum keep their accuracy whatever the size of m, and it is held at
// -3e38 at least: a NaN or -inf entry then gives e = 0 and e d = 0.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ws_host.h"
#include "ws_internal.cuh"
#include "ws_ptx.cuh"

namespace ws {

constexpr float kLowest = -3.0e38f;

// One element type: kPer elements fill a 16-byte vector.
struct ElemF32 {
    using Storage = float;
    static constexpr int kPer = 4;
    static constexpr uint32_t kNegInf = 0xff800000u;   // a word of -inf entries
    static __device__ __forceinline__ void unpack(const uint4& q, float (&f)[4]) {
        f[0] = __uint_as_float(q.x);
        f[1] = __uint_as_float(q.y);
        f[2] = __uint_as_float(q.z);
        f[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    // the larger of two words' entries (a NaN gives way); the word's largest
    static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float max_of(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ float round(float f) { return f; }
};

struct ElemF16 {
    using Storage = __half;
    static constexpr int kPer = 8;
    static constexpr uint32_t kNegInf = 0xfc00fc00u;
    static __device__ __forceinline__ void unpack(const uint4& q, float (&f)[8]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static constexpr uint32_t kLow = 0xfbfffbffu;   // a word of entries that weigh nothing: -65504 (see clamp_above)
    static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
        const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static __device__ __forceinline__ float max_of(uint32_t w) {
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&w));
        return fmaxf(v.x, v.y);
    }
    static __device__ __forceinline__ f32x2 widen(uint32_t w) {
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&w));
        return pack2(v.x, v.y);
    }
    static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ __half round(float f) { return __float2half_rn(f); }
};

struct ElemBF16 {
    using Storage = __nv_bfloat16;
    static constexpr int kPer = 8;
    static constexpr uint32_t kNegInf = 0xff80ff80u;
    static __device__ __forceinline__ void unpack(const uint4& q, float (&f)[8]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static constexpr uint32_t kLow = 0xdd80dd80u;   // -2^60: far below any entry that counts, and finite times a coefficient
    static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static __device__ __forceinline__ float max_of(uint32_t w) {
        return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ f32x2 widen(uint32_t w) {
        return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ __nv_bfloat16 round(float f) { return __float2bfloat16_rn(f); }
};

// 2^x by the hardware's approximation (2 ulp; 2^-inf = 0).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row of `cols` elements as 16-byte blocks.
template <class E>
struct RowBlocks {
    const uint4* base;   // the block that holds the row's first element
    int lead;            // elements of that block before the row
    int nvec;            // blocks (rows have fewer than 2^31 elements)
    __device__ __forceinline__ RowBlocks(const typename E::Storage* row, long long cols) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(row);
        base = reinterpret_cast<const uint4*>(a & ~(uintptr_t)15);
        lead = (int)(a & 15) / (int)sizeof(typename E::Storage);
        nvec = (int)((unsigned)(lead + (int)cols + E::kPer - 1) / (unsigned)E::kPer);
    }
    // Index in the row of block v's first element (negative for the first
    // block of a row that starts inside it).
    __device__ __forceinline__ long long first(long long v) const { return v * E::kPer - lead; }
};

// Writes -inf over a vector's first `head` entries and those from `end` on.
template <class E>
__device__ __forceinline__ void mask_outside(uint4& q, int head, int end) {
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (E::kPer == 4) {
            if (i < head || i >= end) w[i] = E::kNegInf;
        } else {
            if (2 * i < head || 2 * i >= end) w[i] = (w[i] & 0xffff0000u) | (E::kNegInf & 0xffffu);
            if (2 * i + 1 < head || 2 * i + 1 >= end) w[i] = (w[i] & 0xffffu) | (E::kNegInf & 0xffff0000u);
        }
    }
    q = make_uint4(w[0], w[1], w[2], w[3]);
}

// ... of vector v of a row: the entries that are its neighbours'.
template <class E, class Row>
__device__ __forceinline__ void mask_ends(uint4& q, int v, const Row& rb, long long cols) {
    const int head = v == 0 ? rb.lead : 0;
    const int end = v == rb.nvec - 1 ? (int)(rb.lead + cols - (long long)v * E::kPer) : E::kPer;
    if (head > 0 || end < E::kPer) mask_outside<E>(q, head, end);
}

// Streaming 16-byte load of data that this kernel only reads.
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
    uint4 q;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "l"(p));
    return q;
}

// The sums of a softmax over some entries, relative to m.
struct SoftSums {
    float m, s, t;
};

__device__ __forceinline__ float below(float x, float m) { return fmaxf(x - m, kLowest); }

// Half of x - m for finite x and m: the difference itself passes float32's
// range for entries near both ends of it, where its quotient by a temperature
// need not.  (Halves are exact but for subnormal entries.)
__device__ __forceinline__ float half_gap(float x, float m) { return fmaf(0.5f, x, -0.5f * m); }

// The sums restated relative to m >= a.m (a.m = -inf: no entry yet).  The
// difference meets its factor first: -3e38 times 0 is 0, where s times -3e38
// overflows.
__device__ __forceinline__ void rebase(SoftSums& a, float m, float c) {
    const float delta = below(a.m, m);
    const float r = exp2_fast(delta * c);
    a.t = a.t * r + a.s * (delta * r);
    a.s *= r;
    a.m = m;
}

// The running sums of one thread, even and odd entries apart (packed
// arithmetic: two entries an instruction).
struct RunningSums {
    float m;
    f32x2 s, t;
    __device__ __forceinline__ void clear() {
        m = -INFINITY;
        s = t = pack2(0.f, 0.f);
    }
    // Restated relative to `to`, which is above m.
    template <bool kEntropy>
    __device__ __forceinline__ void raise(float to, float c) {
        const float delta = fmaxf(m - to, kLowest);
        const float r = exp2_fast(delta * c);
        const f32x2 r2 = pack2(r, r);
        if (kEntropy) {
            const float dr = delta * r;
            t = fma2(s, pack2(dr, dr), mul2(t, r2));
        }
        s = mul2(s, r2);
        m = to;
    }
    // Adds sums whose maximum is this one's or above it.
    __device__ __forceinline__ void add(const RunningSums& b, float c) {
        if (b.m > m) raise<true>(b.m, c);
        s = add2(s, b.s);
        t = add2(t, b.t);
    }
    __device__ __forceinline__ SoftSums sums() const {
        float s0, s1, t0, t1;
        unpack2(s, s0, s1);
        unpack2(t, t0, t1);
        return SoftSums{m, s0 + s1, t0 + t1};
    }
};

// Above which maximum the 16-bit types' entries may be held at E::kLow: every
// entry at it then weighs exactly 0.
inline float clamp_above(int32_t dtype, float temperature) {
    if (dtype == WS_DTYPE_F32) return INFINITY;   // not used
    return dtype == WS_DTYPE_F16 ? -65504.0f + 110.0f * temperature : -1.0e18f;
}

// Adds the entries of kN vectors.  Returns their largest (NaN gives way).
//
// Where a NaN or -inf entry is dealt with decides the cost of the loop: held
// at -3e38 after the subtraction it takes an instruction an entry; the 16-bit
// types are held at a low value before they are widened, two entries an
// instruction, while the maximum is far enough above it
// (clamp_above) that this changes nothing.
template <class E, int kN, bool kEntropy>
__device__ __forceinline__ float add_vectors(RunningSums& a, const uint4 (&q)[kN], float c, float above) {
    uint32_t mw = E::kNegInf;
#pragma unroll
    for (int j = 0; j < kN; ++j)
        mw = E::max_word(E::max_word(mw, E::max_word(q[j].x, q[j].y)), E::max_word(q[j].z, q[j].w));
    const float bm = E::max_of(mw);
    if (bm > a.m) a.raise<kEntropy>(bm, c);
    const f32x2 c2 = pack2(c, c), m2 = pack2(-a.m, -a.m);
    auto add = [&](f32x2 d) {
        float a0, a1;
        unpack2(mul2(d, c2), a0, a1);
        const f32x2 e = pack2(exp2_fast(a0), exp2_fast(a1));
        a.s = add2(a.s, e);
        if (kEntropy) a.t = fma2(e, d, a.t);
    };
    if constexpr (E::kPer == 8) {
        if (a.m > above && a.m < INFINITY) {
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) add(add2(E::widen(E::max_word(w[i], E::kLow)), m2));
            }
            return bm;
        }
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        float f[E::kPer];
        E::unpack(q[j], f);
#pragma unroll
        for (int i = 0; i < E::kPer; i += 2) add(pack2(below(f[i], a.m), below(f[i + 1], a.m)));
    }
    return bm;
}

// The warp's sums in every lane, added in a fixed order.
__device__ __forceinline__ SoftSums warp_sums(SoftSums a, float c) {
    float m = a.m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    rebase(a, m, c);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
    }
    return a;
}

// The vector of entries that starts `by` (1 .. kPer - 1) entries into lo and
// goes on in hi.
template <class E>
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int by) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int words = by * 4 / E::kPer;
    if (words & 2) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (words & 1) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (E::kPer == 8 && (by & 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Writes vector v of a gradient row's blocks: whole where its entries lie in
// [a, b), else those that do.
template <class E>
__device__ __forceinline__ void store_vector(typename E::Storage* gr, const RowBlocks<E>& gb, int v, int a, int b, const uint4& q) {
    using S = typename E::Storage;
    const int e = v * E::kPer - gb.lead;
    if (e >= a && e + E::kPer <= b) {
        const_cast<uint4*>(gb.base)[v] = q;
        return;
    }
    const S* from = reinterpret_cast<const S*>(&q);
#pragma unroll
    for (int i = 0; i < E::kPer; ++i)
        if (e + i >= a && e + i < b) gr[e + i] = from[i];
}

// Stores a warp's 32 vectors of gradients where the gradient's vectors lie
// otherwise than the run's: `by` entries of a vector belong to the vector
// before.  q holds entries e .. e + kPer of the row; entries outside [a, b)
// are not written.
template <class E>
__device__ __forceinline__ void store_shifted(typename E::Storage* gr, const uint4& q, int e, int a, int b, int by) {
    using S = typename E::Storage;
    constexpr int kPer = E::kPer;
    const int lane = threadIdx.x & 31;
    uint4 before;
    before.x = __shfl_up_sync(0xffffffffu, q.x, 1);
    before.y = __shfl_up_sync(0xffffffffu, q.y, 1);
    before.z = __shfl_up_sync(0xffffffffu, q.z, 1);
    before.w = __shfl_up_sync(0xffffffffu, q.w, 1);
    const uint4 out = shifted<E>(before, q, by);
    const int o = e - kPer + by;                // entries o .. o + kPer
    if (lane > 0 && o >= a && o + kPer <= b) {
        *reinterpret_cast<uint4*>(gr + o) = out;
    } else {
        const S* from = reinterpret_cast<const S*>(&out);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if ((lane > 0 || i >= kPer - by) && o + i >= a && o + i < b) gr[o + i] = from[i];
    }
    if (lane == 31) {   // the last vector's end begins a vector that the next warp completes
        const S* from = reinterpret_cast<const S*>(&q);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i >= by && e + i >= a && e + i < b) gr[e + i] = from[i];
    }
}

// The total of at most 32 sums in shared memory, in every lane of a warp.
__device__ __forceinline__ SoftSums lane_sums(const SoftSums* part, int n, float c) {
    const int lane = threadIdx.x & 31;
    return warp_sums(lane < n ? part[lane] : SoftSums{-INFINITY, 0.f, 0.f}, c);
}

// An index operand of either type.
__device__ __forceinline__ long long load_index(const void* p, long long i, int is64) {
    return is64 ? static_cast<const long long*>(p)[i] : (long long)static_cast<const int*>(p)[i];
}

// ---- host side: the arguments that the logits calls share ------------------

inline size_t elem_size(int32_t dtype) { return dtype == WS_DTYPE_F32 ? 4 : 2; }

inline ws_status validate_logits(int64_t rows, int64_t cols, int64_t row_stride, int32_t dtype, int32_t index_type,
                                 float temperature) {
    if (rows < 1) return fail(WS_ERR_INVALID_ARGUMENT, "rows %lld < 1", (long long)rows);
    if (cols < 1 || cols > 2147483647LL - 63)   // indices rounded up to whole vectors stay below 2^31
        return fail(WS_ERR_INVALID_ARGUMENT, "cols %lld outside 1 .. 2^31-64", (long long)cols);
    if (row_stride < cols)
        return fail(WS_ERR_INVALID_ARGUMENT, "row_stride %lld < cols %lld", (long long)row_stride, (long long)cols);
    if (rows > (1LL << 40) / row_stride) return fail(WS_ERR_INVALID_ARGUMENT, "rows * row_stride too large");
    if (dtype != WS_DTYPE_F32 && dtype != WS_DTYPE_F16 && dtype != WS_DTYPE_BF16)
        return fail(WS_ERR_INVALID_ARGUMENT, "dtype %d", dtype);
    if (index_type != WS_INDEX_I32 && index_type != WS_INDEX_I64)
        return fail(WS_ERR_INVALID_ARGUMENT, "index_type %d", index_type);
    // negated so that NaN is refused.  Within the limits log2(e) / temperature and its inverse are ordinary numbers;
    // its product with a difference of entries may overflow, to -inf and thence an exponential of 0.
    if (!(temperature >= 1.0f / 1048576.0f && temperature <= 1048576.0f))
        return fail(WS_ERR_INVALID_ARGUMENT, "temperature %g outside 2^-20 .. 2^20", (double)temperature);
    return WS_OK;
}

// A pointer to elements of `size` bytes: not NULL and aligned to them.
inline ws_status check_pointer(const void* p, size_t size, const char* name) {
    if (!p) return fail(WS_ERR_INVALID_ARGUMENT, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % size != 0)
        return fail(WS_ERR_INVALID_ARGUMENT, "%s is not aligned to its %zu-byte elements", name, size);
    return WS_OK;
}

// A gradient goes to the logits' own rows or to rows that share no element
// with them: of others, some would be written before they are read.
inline ws_status check_gradient(const void* logits, int64_t row_stride, const void* grad, int64_t grad_stride, int64_t rows,
                                int64_t cols, size_t size) {
    if (logits == grad) {
        if (rows > 1 && grad_stride != row_stride)
            return fail(WS_ERR_INVALID_ARGUMENT, "grad_logits in place with another stride");
        return WS_OK;
    }
    if (rows_overlap(logits, row_stride, grad, grad_stride, rows, cols, size))
        return fail(WS_ERR_INVALID_ARGUMENT, "grad_logits overlaps the logits");
    return WS_OK;
}

#define WS_TRY(expr)                                \
    do {                                            \
        ws_status ws_s_ = (expr);                   \
        if (ws_s_ != WS_OK) return ws_s_;           \
    } while (0)

inline float log2e_over(float temperature) { return (float)(1.4426950408889634 / (double)temperature); }

// Launches `kernel` on a grid of clusters of `cluster` blocks, as a
// programmatic dependent of the previous kernel (see launch_pdl).
template <typename Kernel, typename... Args>
cudaError_t launch_clusters(Kernel kernel, dim3 grid, int threads, int cluster, size_t smem, cudaStream_t stream,
                            Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace ws
