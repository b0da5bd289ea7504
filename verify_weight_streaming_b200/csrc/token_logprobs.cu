// token_logprobs: log probabilities of given tokens, the entropy and the most
// likely alternatives of every row of logits, in one pass over them.
//
//   lse = log sum_j exp(c x_j),  logprob(v) = c x_v - lse,
//   entropy = lse - sum_j p_j c x_j,  top-k by (value desc, index asc)
//
// HBM-bound when there are many rows, latency-bound when there are few.  A row
// is summed in up to 8 pieces of about 64 KB, how many by its bytes alone, and a
// cluster of 1 to 8 CTAs takes them: one CTA a row when the rows fill the GPU,
// more when they do not (2048 rows of 131072 bf16: 109.3 us, 90 without top-k;
// one row of 131072 fp32: 6.0 us, 3.5 without).  Threads read 16 bytes a load,
// strided by the CTA, and keep a running reference R (the largest c x log2 e so
// far), s = sum 2^d and t = sum d 2^d with d = c x log2 e - R, all in fp32: the
// exponentials are one fma and one ex2 a logit, and everything after the loop is
// a log2 of s.
// Threads, warps and pieces are joined in a fixed order that does not depend
// on how many CTAs share the row.
//
// Top-k without a second pass: a thread also keeps its largest value and the
// 16-byte vector that first had it.  The k-th largest of the 32 maxima of eight
// threads each is a value that at least k threads reach, and seldom many more;
// where ties leave too many, a bisection (a barrier with a count a step) raises
// it and then finds the vector up to which the tied value counts.  Every top-k
// element is in such a thread and reaches that (value, vector): any other has
// k better ones.  So only those threads' vectors are looked at again (about k
// of 256, from cache), and the few elements found are ranked by counting.  (Only
// the pieces of those threads that reach it: 2048 rows of 131072 bf16 152 -> 135 us at k =
// 20, but 109 -> 115 at k = 5, and one row 5.9 -> 6.8.)
// (Merging sorted lists in one warp instead cost 2.7 us a call at k = 1 and 8.7
// us at k = 32; the bisection alone 2.6 and 4.6; this 2.3 and 4.7.)
#include "topk_core.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mr {
namespace logprobs {

using namespace mr::topk;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
static_assert(kThreads == 256, "eight threads to each of 32 groups");
constexpr int kMaxK = 32;
constexpr int kMaxTokens = kThreads;
constexpr int kMaxPieces = 8;
constexpr int64_t kPieceBytes = 64 * 1024;
constexpr int kUnroll = 4;
constexpr int kCandidates = 1024;
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// Logits are taken as no less than this in the sums, so that a masked (-inf)
// one gives d 2^d = 0 and not NaN.
constexpr float kFloor = -0x1p100f;
// How far below another a reference counts as being when sums are joined: 2^-200
// is 0 already, and a masked warp's reference is 2^100 c2 below with thousands of
// logits in s, where d s would overflow and 0 times it be NaN.
constexpr float kFar = -200.0f;
// R is M c2 rounded, d = x c2 - R is not: the largest logit's d is up to half a step of R away
// from 0, in every term alike.  Below this |R| that is 64 at most, 2^d and d 2^d are far from overflow, and
// a term that underflows is 2^62 below the largest.  A row beyond it is summed again, M subtracted first
// (`rare_row`); so is one whose largest logit is near kFloor, which is far beyond, and one where some
// threads' own references lie beyond it and their sums overflowed (2^d0 = 0 then makes them NaN).
constexpr float kWide = 0x1p31f;

struct Params {
    const uint8_t *x;
    int64_t ld;         // bytes
    const int32_t *tokens;
    int64_t ldt;
    float *logprob;
    int64_t ldp;
    float *lse, *entropy;
    int32_t *top_idx;
    float *top_logprob;
    int64_t ldo;
    int n, ntok, K, pieces, cluster, deep;
    float scale;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two fp32 values in one operation (the rounding of each is fma's or add's).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// ---- 16 bytes of logits ----------------------------------------------------

// top: the largest of a vector's values (NaN ignored); unpack: the values in
// fp32, no less than kFloor (a NaN stays one).
template <int DT>
struct Type;
template <>
struct Type<MR_F32> {
    using T = uint32_t;
    static constexpr int E = 4;
    static constexpr T kMinusInf = 0xFF800000u;
    static __device__ __forceinline__ float value(T v) { return __uint_as_float(v); }
    static __device__ __forceinline__ float top(uint4 u) {
        return fmaxf(fmaxf(value(u.x), value(u.y)), fmaxf(value(u.z), value(u.w)));
    }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = max_nan(value(w[i]), kFloor);
    }
};
template <>
struct Type<MR_BF16> {
    using T = uint16_t;
    static constexpr int E = 8;
    static constexpr T kMinusInf = 0xFF80u;
    static __device__ __forceinline__ float value(T v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float top(uint4 u) {
        const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t r;  // kFloor is 0xF180 in bf16
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w[i]), "r"(0xF180F180u));
            v[2 * i] = __uint_as_float(r << 16);
            v[2 * i + 1] = __uint_as_float(r & 0xFFFF0000u);
        }
    }
};
template <>
struct Type<MR_F16> {
    using T = uint16_t;
    static constexpr int E = 8;
    static constexpr T kMinusInf = 0xFC00u;
    static __device__ __forceinline__ float value(T v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float top(uint4 u) {
        const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
        return fmaxf(value((T)m), value((T)(m >> 16)));
    }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = max_nan(value((T)w[i]), kFloor);
            v[2 * i + 1] = max_nan(value((T)(w[i] >> 16)), kFloor);
        }
    }
};

// A row as 16-byte vectors at 16-byte boundaries: vector v holds elements
// [v * E - lead, (v + 1) * E - lead) of the row, those outside [0, n) absent.
template <int DT>
struct Row {
    using T = typename Type<DT>::T;
    static constexpr int E = Type<DT>::E;
    const T *x;
    const uint4 *base;
    int lead, n, vectors, whole0, whole1;  // vectors [whole0, whole1) lie in the row
    __device__ Row(const Params &p, int64_t row) {
        const uint8_t *at = p.x + row * p.ld;
        x = reinterpret_cast<const T *>(at);
        const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 15u);
        base = reinterpret_cast<const uint4 *>(at - off);
        lead = (int)(off / sizeof(T));
        n = p.n;
        vectors = (int)(((int64_t)lead + n + E - 1) / E);
        whole0 = lead ? 1 : 0;
        whole1 = (int)(((int64_t)lead + n) / E);
    }
    __device__ __forceinline__ int64_t first(int v) const { return (int64_t)v * E - lead; }
    __device__ __forceinline__ bool whole(int v) const { return v >= whole0 && v < whole1; }
    __device__ __forceinline__ uint4 load(int v) const { return base[v]; }  // a whole vector
    // Any vector, absent elements as -inf; only what is in the row is read.
    __device__ __forceinline__ uint4 read(int v) const {
        if (whole(v)) return load(v);
        uint4 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int64_t j = first(v) + i;
            e[i] = j >= 0 && j < n ? x[j] : Type<DT>::kMinusInf;
        }
        return u;
    }
    __device__ __forceinline__ float at(int j) const { return Type<DT>::value(x[j]); }
};

// ---- sums -----------------------------------------------------------------

struct Sums {
    float R, s, t;
};

struct Best {
    float value;
    int vector;
};

// U vectors, `first` and every kThreads-th after it, into the sums and the best.
template <int DT, int U, bool TOP>
__device__ __forceinline__ void take(const uint4 (&u)[U], int first, float c, Sums &a, Best &best) {
    constexpr int E = Type<DT>::E;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const float top = Type<DT>::top(u[i]);
        if (TOP && top > best.value) {
            best.value = top;
            best.vector = first + i * kThreads;
        }
        m = fmaxf(m, top);
    }
    const float R = fmaxf(a.R, fmaxf(m, kFloor) * c), d0 = fmaxf(a.R - R, kFar), f = ex2(d0);
    a.t = f * fmaf(d0, a.s, a.t);
    a.s *= f;
    a.R = R;
    const float2 c22 = {c, c}, R2 = {-R, -R};
    float2 s = {0.0f, 0.0f}, t = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float v[E];
        Type<DT>::unpack(u[i], v);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 d = fma2({v[j], v[j + 1]}, c22, R2), e = {ex2(d.x), ex2(d.y)};
            s = add2(s, e);
            t = fma2(e, d, t);
        }
    }
    a.s += s.x + s.y;
    a.t += t.x + t.y;
}

// The sums of a warp's lanes (or of 2^n of them, the others neutral): to the
// common reference, then added in a butterfly.
__device__ __forceinline__ Sums warp_sums(Sums a) {
    float R = a.R;
#pragma unroll
    for (int d = 16; d; d >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, d));
    const float d0 = fmaxf(a.R - R, kFar), f = ex2(d0);
    float s = a.s * f, t = f * fmaf(d0, a.s, a.t);
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, d);
        t += __shfl_xor_sync(0xffffffffu, t, d);
    }
    return {R, s, t};
}

// ---- top-k of a piece -----------------------------------------------------

struct Shared {
    uint64_t list[32];
    alignas(16) uint64_t cand[kCandidates];
    alignas(16) uint64_t scratch[kWarps][64];
    uint64_t part[kWarps][32];
    alignas(16) uint32_t groups[32];  // the largest value word of every eight threads
    int who[kThreads];
    float wide[kWarps];
    int threads, count;
    // [piece][warp]; written by the cluster's CTAs into the first one's
    Sums sums[kMaxPieces * kWarps];
    uint64_t top[kMaxPieces][32];
};

// Keys of one vector's elements (0 for absent ones).
template <int DT>
__device__ __forceinline__ void vector_keys(const Row<DT> &row, int v, bool on, uint64_t (&key)[Type<DT>::E]) {
    constexpr int E = Type<DT>::E;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (on) u = row.read(v);
    const typename Type<DT>::T *e = reinterpret_cast<const typename Type<DT>::T *>(&u);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int64_t j = row.first(v) + i;
        key[i] = on && j >= 0 && j < row.n ? make_key(Type<DT>::value(e[i]), (uint32_t)j) : 0ull;
    }
}

// The K best of every element of vectors [v0, v1) as a key, one a lane of warp 0:
// for a NaN or an infinity among them, which the threads' maxima do not see, and
// for ties that leave too many candidates.
template <int DT>
__device__ __noinline__ uint64_t every_key(Shared &sh, const Row<DT> &row, int v0, int v1, int K) {
    constexpr int E = Type<DT>::E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t run = 0;
    for (int v = v0 + warp * 32; v < v1; v += kThreads) {
        uint64_t key[E];
        vector_keys<DT>(row, v + lane, v + lane < v1, key);
        run = warp_topk_merge<E>(key, run, K, lane, sh.scratch[warp]);
    }
    sh.part[warp][lane] = lane < K ? run : 0ull;
    __syncthreads();
    if (warp) return 0;
    uint64_t key[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) key[w] = sh.part[w][lane];
    return warp_topk_merge<kWarps>(key, 0ull, K, lane, sh.scratch[0]);
}

__device__ __forceinline__ uint32_t best_word(const Best &b) { return b.vector >= 0 ? order_word(b.value) : 0u; }

// The K best keys of vectors [v0, v1), one a lane of warp 0; sh.groups is
// written, sh.threads, sh.count and sh.list are zero, before a barrier.  v0 is a multiple of
// kThreads, so vector v is thread v % kThreads's.
template <int DT>
__device__ uint64_t piece_top(Shared &sh, const Row<DT> &row, int v0, int v1, int K, const Best &best, bool rare) {
    constexpr int E = Type<DT>::E;
    const int lane = threadIdx.x & 31;
    if (rare) return every_key<DT>(sh, row, v0, v1, K);
    // tau: a value at least K threads' bests reach; cut: the last vector that
    // counts with exactly that value.
    const uint32_t mine = best_word(best), group = sh.groups[lane];
    int not_less = 0, cut = 0x7FFFFFFF;
    const uint4 *q = reinterpret_cast<const uint4 *>(sh.groups);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 w = q[j];
        not_less += (w.x >= group) + (w.y >= group) + (w.z >= group) + (w.w >= group);
    }
    // (no word of a value is 0; 1: fewer than K groups have any, so all counts)
    uint32_t tau = max(1u, __reduce_max_sync(0xffffffffu, not_less >= K ? group : 0u));
    if (mine >= tau) sh.who[atomicAdd(&sh.threads, 1)] = threadIdx.x;
    __syncthreads();
    const int enough = max(2 * K, 32);
    if (sh.threads > enough) {
        int reach = sh.threads;
        uint32_t above = __reduce_max_sync(0xffffffffu, group) + 1u;
        while (reach > enough && above - tau > 1u) {
            const uint32_t mid = tau + (above - tau) / 2;
            const int n = __syncthreads_count(mine >= mid);
            if (n >= K) {
                tau = mid;
                reach = n;
            } else {
                above = mid;
            }
        }
        if (reach > enough) {
            int before = v0 - 1;
            cut = v1 - 1;
            while (cut - before > 1) {
                const int mid = before + (cut - before) / 2;
                if (__syncthreads_count(mine > tau || (mine == tau && best.vector <= mid)) >= K)
                    cut = mid;
                else
                    before = mid;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.threads = 0;
        __syncthreads();
        if (mine > tau || (mine == tau && best.vector <= cut)) sh.who[atomicAdd(&sh.threads, 1)] = threadIdx.x;
        __syncthreads();
    }
    const int rounds = (v1 - v0 + kThreads - 1) / kThreads, threads = sh.threads;
    for (int e = threadIdx.x; e < threads * rounds; e += kThreads) {
        const int v = v0 + sh.who[e / rounds] + (e % rounds) * kThreads;
        if (v >= v1) continue;
        uint64_t key[E];
        vector_keys<DT>(row, v, true, key);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint32_t w = (uint32_t)(key[i] >> 32);
            if (key[i] && (w > tau || (w == tau && v <= cut))) {
                const int at = atomicAdd(&sh.count, 1);  // in any order: keys are ranked
                if (at < kCandidates) sh.cand[at] = key[i];
            }
        }
    }
    __syncthreads();
    const int count = sh.count;
    if (count > kCandidates) return every_key<DT>(sh, row, v0, v1, K);
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t key = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < count; ++j) rank += sh.cand[j] > key ? 1 : 0;
        if (rank < K) sh.list[rank] = key;
    }
    __syncthreads();
    return sh.list[lane];
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t in_first(const void *p) {  // the same object in the cluster's first CTA
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
__device__ __forceinline__ void put(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The log probability of a logit, from the row's sums or, for a rare row, from
// its largest value M and log_sum = log sum exp(c (x - M)).
struct Result {
    bool rare;
    float c2, R, log2s;        // log2 units
    float c, M, log_sum;
    float lse, entropy;
    __device__ __forceinline__ float logprob(float x) const {
        if (!rare) {
            const float v = fmaf(x, c2, -R) - log2s;
            return v > -INFINITY ? v * kLn2 : fmaf(x, c, -lse);  // (x log2 e alone may overflow)
        }
        if (!(fabsf(lse) < INFINITY) && !(M > -INFINITY && M < INFINITY)) return fmaf(x, c, -lse);
        return (x - M) * c - log_sum;
    }
};

template <class F>
__device__ float block_fold(Shared &sh, float v, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d; d >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, d));
    __syncthreads();
    if (lane == 0) sh.wide[warp] = v;
    __syncthreads();
    v = sh.wide[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = f(v, sh.wide[w]);
    return v;
}

// A row with a NaN or an infinity, or whose largest product is beyond kWide: the formulas
// as they stand, two more passes by the cluster's first CTA.
template <int DT>
__device__ void rare_row(Shared &sh, const Row<DT> &row, float c, Result &r) {
    float M = -INFINITY;
    for (int j = threadIdx.x; j < row.n; j += kThreads) M = max_nan(M, row.at(j));
    M = block_fold(sh, M, [](float a, float b) { return max_nan(a, b); });
    r.rare = true;
    r.c = c;
    r.M = M;
    r.log_sum = 0.0f;
    r.lse = M;             // NaN, +inf or -inf
    r.entropy = NAN;
    if (!(M > -INFINITY && M < INFINITY)) return;
    float s = 0.0f, t = 0.0f;
    for (int j = threadIdx.x; j < row.n; j += kThreads) {
        const float d = (row.at(j) - M) * c, e = expf(d);
        s += e;
        if (e > 0.0f) t = fmaf(e, d, t);
    }
    auto add = [](float a, float b) { return a + b; };
    s = block_fold(sh, s, add);
    t = block_fold(sh, t, add);
    r.log_sum = logf(s);
    r.lse = fmaf(M, c, r.log_sum);
    r.entropy = r.log_sum - t / s;
}

// DEEP: the next loads are on their way while some are summed, and 4 CTAs share an
// SM; without, 5 do.
template <int DT, bool TOP, bool DEEP>
__global__ void __launch_bounds__(kThreads, DEEP ? 4 : 5) logprobs_kernel(const Params p) {
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t r = blockIdx.x / p.cluster;
    const Row<DT> row(p, r);
    // Pieces begin at multiples of kThreads vectors; this CTA's are [p0, p1).
    const int p0 = p.pieces * rank / p.cluster, p1 = p.pieces * (rank + 1) / p.cluster;
    auto begin = [&](int i) {
        return i == p.pieces ? row.vectors : (int)((int64_t)row.vectors * i / p.pieces) / kThreads * kThreads;
    };
    const int v0 = begin(p0), v1 = begin(p1);
    const float c2 = p.scale * kLog2E;
    if (p.cluster > 1) cluster_arrive();  // every CTA of the cluster runs before any writes to the first
    grid_dependency_wait();
    // After the wait: a product that reads its weight ahead may come next, and that weight from the kernel
    // before this one.  (Given at entry: 16 rows of 151667 10.2 us instead of 9.5; a chain of cast, 4-bit head of
    // 32000 x 2560 and this kernel 20.6 instead of 22.4, as the next head's weight came that much earlier.)
    grid_launch_dependents();

    // The given tokens' logits, ahead of the pass.
    float given = NAN;
    if (rank == 0 && (int)threadIdx.x < p.ntok) {
        const int32_t v = p.tokens[r * p.ldt + threadIdx.x];
        if (v >= 0 && v < p.n) given = row.at(v);
    }

    bool odd = false;  // a NaN or +inf: not seen by the maxima
    Best best = {-INFINITY, v0 + (int)threadIdx.x < v1 ? v0 + (int)threadIdx.x : -1};
    int v = v0 + threadIdx.x;
    for (int piece = p0; piece < p1; ++piece) {
        const int end = begin(piece + 1);
        Sums a = {kFloor * c2, 0.0f, 0.0f};
        constexpr int kStep = kUnroll * kThreads, kLast = (kUnroll - 1) * kThreads;
        auto fetch = [&](uint4 (&u)[kUnroll]) {
            if (v >= row.whole0 && v + kLast < row.whole1) {
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) u[i] = row.load(v + i * kThreads);
            } else {
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) u[i] = row.read(v + i * kThreads);
            }
        };
        if (!DEEP) {
            for (; v + kLast < end; v += kStep) {
                uint4 u[kUnroll];
                fetch(u);
                take<DT, kUnroll, TOP>(u, v, c2, a, best);
            }
        } else if (v + kLast < end) {
            uint4 u[kUnroll];
            fetch(u);
            for (v += kStep; v + kLast < end; v += kStep) {
                uint4 w[kUnroll];
                fetch(w);
                take<DT, kUnroll, TOP>(u, v - kStep, c2, a, best);
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) u[i] = w[i];
            }
            take<DT, kUnroll, TOP>(u, v - kStep, c2, a, best);
        }
        for (; v < end; v += kThreads) {
            const uint4 u[1] = {row.read(v)};
            take<DT, 1, TOP>(u, v, c2, a, best);
        }
        odd = odd || a.s != a.s;
        a = warp_sums(a);
        if (lane == 0) sh.sums[piece * kWarps + warp] = a;
    }
    if (TOP) {
        uint32_t group = best_word(best);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) group = max(group, __shfl_xor_sync(0xffffffffu, group, d));
        if (lane % 8 == 0) sh.groups[threadIdx.x / 8] = group;
        if (warp == 0) sh.list[lane] = 0ull;
        if (threadIdx.x == 0) sh.threads = sh.count = 0;
    }
    const bool rare_piece = __syncthreads_or(odd);
    uint64_t top = 0;
    if (TOP) top = piece_top<DT>(sh, row, v0, v1, p.K, best, rare_piece);

    if (p.cluster > 1) {
        cluster_wait();  // of the arrival at the start
        if (rank) {
            if (threadIdx.x < (p1 - p0) * kWarps) {
                const int i = p0 * kWarps + threadIdx.x;
                put(in_first(&sh.sums[i].R), sh.sums[i].R);
                put(in_first(&sh.sums[i].s), sh.sums[i].s);
                put(in_first(&sh.sums[i].t), sh.sums[i].t);
            }
        }
        if (TOP && warp == 0) put(in_first(&sh.top[rank][lane]), lane < p.K ? top : (uint64_t)0);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (rank) return;
        if (TOP) {
            // The CTAs' lists are sorted: a key's rank is the number before it in
            // each, found by bisection.
            const int lists = p.cluster, i = threadIdx.x / 32;
            __syncthreads();  // the piece's list has been read
            if (threadIdx.x < 32) sh.list[threadIdx.x] = 0ull;
            __syncthreads();
            const uint64_t key = i < lists ? sh.top[i][lane] : 0ull;
            int rank = 0;
            for (int l = 0; l < lists; ++l) {
                int n = 0;
#pragma unroll
                for (int d = 16; d; d >>= 1) n += sh.top[l][n + d - 1] > key ? d : 0;
                rank += n + (sh.top[l][n] > key ? 1 : 0);
            }
            if (key && rank < p.K) sh.list[rank] = key;
            __syncthreads();
            top = sh.list[lane];
        }
    }
    // Every warp joins all pieces' warps: lane l has entries l, l + 32, ...
    Sums a = {kFloor * c2, 0.0f, 0.0f};
    for (int i = lane; i < p.pieces * kWarps; i += 32) {
        const Sums b = sh.sums[i];
        const float R = fmaxf(a.R, b.R), da = fmaxf(a.R - R, kFar), db = fmaxf(b.R - R, kFar), fa = ex2(da), fb = ex2(db);
        a = {R, a.s * fa + b.s * fb, fa * fmaf(da, a.s, a.t) + fb * fmaf(db, b.s, b.t)};
    }
    a = warp_sums(a);

    Result out;
    out.rare = false;
    out.c = p.scale;
    out.c2 = c2;
    out.R = a.R;
    out.log2s = log2f(a.s);
    out.lse = (a.R + out.log2s) * kLn2;
    out.entropy = (out.log2s - a.t / a.s) * kLn2;
    const bool fine = a.s > 0.0f && a.s < INFINITY && fabsf(a.t) < INFINITY && fabsf(a.R) < kWide;
    if (!fine) rare_row<DT>(sh, row, p.scale, out);
    if ((int)threadIdx.x < p.ntok) p.logprob[r * p.ldp + threadIdx.x] = out.logprob(given);
    if (threadIdx.x == 0) {
        if (p.lse) p.lse[r] = out.lse;
        if (p.entropy) p.entropy[r] = out.entropy;
    }
    if (TOP && warp == 0 && lane < p.K) {
        bool exact;
        float x = key_value(top, exact);
        if ((uint32_t)(top >> 32) == 0xFFFFFFFFu) x = NAN;
        if ((uint32_t)(top >> 32) == 0x80000000u) x = 0.0f;
        p.top_idx[r * p.ldo + lane] = (int32_t)key_index(top);
        if (p.top_logprob) p.top_logprob[r * p.ldo + lane] = out.logprob(x);
    }
}

template <int DT>
mr_status launch(const Params &p, int64_t rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (p.deep)
        return mr_host::cuda_status(p.K ? cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, true, true>, p)
                                        : cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, false, true>, p));
    return mr_host::cuda_status(p.K ? cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, true, false>, p)
                                    : cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, false, false>, p));
}

}  // namespace logprobs
}  // namespace mr

extern "C" mr_status token_logprobs(const void *logits, int64_t ldl, int32_t dtype, int32_t m, int32_t n, float scale,
                                    const int32_t *tokens, int64_t ldt, int32_t ntok, float *logprob, int64_t ldp,
                                    float *lse, float *entropy, int32_t topk, int32_t *top_idx, float *top_logprob,
                                    int64_t ldo, void *stream) {
    if (!logits || m < 1 || n < 1 || ntok < 0 || topk < 0 || topk > n) return MR_ERR_INVALID_ARG;
    if (dtype != MR_F16 && dtype != MR_BF16 && dtype != MR_F32) return MR_ERR_INVALID_ARG;
    if (!(scale >= 1e-6f && scale <= 1e6f)) return MR_ERR_INVALID_ARG;
    if (ldl < n) return MR_ERR_INVALID_ARG;
    if (ntok && (!tokens || !logprob || ldt < ntok || ldp < ntok)) return MR_ERR_INVALID_ARG;
    if (topk && (!top_idx || ldo < topk)) return MR_ERR_INVALID_ARG;
    if (!topk && (top_idx || top_logprob)) return MR_ERR_INVALID_ARG;
    if (!ntok && !topk && !lse && !entropy) return MR_ERR_INVALID_ARG;
    const int size = dtype == MR_F32 ? 4 : 2;
    if (((uintptr_t)logits & (uintptr_t)(size - 1)) || ((uintptr_t)tokens & 3u) || ((uintptr_t)logprob & 3u) ||
        ((uintptr_t)lse & 3u) || ((uintptr_t)entropy & 3u) || ((uintptr_t)top_idx & 3u) || ((uintptr_t)top_logprob & 3u))
        return MR_ERR_MISALIGNED;
    if (topk > mr::logprobs::kMaxK || ntok > mr::logprobs::kMaxTokens || n > (1 << 30)) return MR_ERR_UNSUPPORTED;
    mr::logprobs::Params p = {};
    p.x = static_cast<const uint8_t *>(logits);
    p.ld = ldl * size;
    p.tokens = tokens;
    p.ldt = ldt;
    p.logprob = logprob;
    p.ldp = ldp;
    p.lse = lse;
    p.entropy = entropy;
    p.top_idx = top_idx;
    p.top_logprob = top_logprob;
    p.ldo = ldo;
    p.n = n;
    p.ntok = ntok;
    p.K = topk;
    p.scale = scale;
    p.pieces = 1;
    while (p.pieces < mr::logprobs::kMaxPieces && (int64_t)n * size > p.pieces * mr::logprobs::kPieceBytes)
        p.pieces *= 2;
    // As many CTAs a row (a piece each at the most) as leave 4.5 of them to an
    // SM, 5 without top-k (us at 1, 2, 4, 8 CTAs a row, top 5: 64 rows of 131072 fp32
    // 28.7, 18.6, 14.0, 14.7; 128 rows 31.5, 23.5, 18.6, 24.3; 256 rows of bf16 30.6, 20.9,
    // 25.6, 25.7; 512 rows 34.3, 39.3, 46.3, 46.3).
    const int64_t sms = mr_host::sm_count();
    p.cluster = 1;
    while (p.cluster < p.pieces && (int64_t)m * p.cluster * 4 <= sms * (topk ? 9 : 10)) p.cluster *= 2;
    // Loads ahead, unless there are more CTAs than that form holds at once and a
    // CTA's share of a row is short (us with and without, top 5: one row of 131072 fp32
    // 6.0, 6.5; 1024 rows 100, 112; 2048 rows of bf16 109.5, 110.3; 700 rows of 50021 f16 26.4,
    // 21.7; 306 rows of 50021 fp32 20.4, 18.3; 2048 rows of 4096 fp32 22.1, 20.1).
    p.deep = (int64_t)m * p.cluster <= 4 * sms || (int64_t)n * size >= p.cluster * 4 * mr::logprobs::kPieceBytes;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MR_F32: return mr::logprobs::launch<MR_F32>(p, m, s);
        case MR_BF16: return mr::logprobs::launch<MR_BF16>(p, m, s);
        default: return mr::logprobs::launch<MR_F16>(p, m, s);
    }
}
