// token_logprobs: log probabilities of given tokens, the entropy and the most
// likely alternatives of every row of logits, in one pass over them.
//
//   lse = log sum_j exp(c x_j),  logprob(v) = c x_v - lse,
//   entropy = lse - sum_j p_j c x_j,  top-k by (value desc, index asc)
//
// HBM-bound when there are many rows, latency-bound when there are few.  A row
// is cut into up to 8 pieces (about 64 KB each), one CTA of a cluster each;
// how many depends on the row's bytes alone.  Threads read 16 bytes a load,
// strided by the CTA, and keep a running reference R (the largest c x log2 e so
// far), s = sum 2^d and t = sum d 2^d with d = c x log2 e - R, all in fp32: the
// exponentials are one fma and one ex2 a logit, and everything after the loop is a
// log2 of s.  Threads, warps and pieces are joined in a fixed order.
//
// Top-k without a second pass: a thread also keeps its largest value and the
// 16-byte vector that first had it.  The k best of a piece lie in the k threads
// whose (value, vector) are best: any other element has k better ones.  Only
// those threads' vectors are looked at again (k of 256, from cache), and of
// them only what reaches the k-th thread's best.
#include "topk_core.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mr {
namespace logprobs {

using namespace mr::topk;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 32;
constexpr int kMaxTokens = kThreads;
constexpr int kMaxCluster = 8;
constexpr int64_t kPieceBytes = 64 * 1024;
constexpr int kUnroll = 4;
constexpr int kCandidates = 1024;
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// Logits are taken as no less than this in the sums, so that a masked (-inf)
// one gives d 2^d = 0 and not NaN.  A row whose largest logit is near it or
// below is summed again, without the bound (`rare_row`).
constexpr float kFloor = -0x1p100f;

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
    int n, ntok, K, cluster;
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

// ---- 16 bytes of logits as fp32 -------------------------------------------

template <int DT>
struct Type;
template <>
struct Type<MR_F32> {
    using T = float;
    static constexpr int E = 4;
    static __device__ __forceinline__ float value(T v) { return v; }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
};
template <>
struct Type<MR_BF16> {
    using T = uint16_t;
    static constexpr int E = 8;
    static __device__ __forceinline__ float value(T v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Type<MR_F16> {
    using T = uint16_t;
    static constexpr int E = 8;
    static __device__ __forceinline__ float value(T v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
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
    int lead, n, vectors;
    __device__ Row(const Params &p, int64_t row) {
        x = reinterpret_cast<const T *>(p.x + row * p.ld);
        lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        n = p.n;
        vectors = (int)(((int64_t)lead + n + E - 1) / E);
    }
    __device__ __forceinline__ int64_t first(int v) const { return (int64_t)v * E - lead; }
    __device__ __forceinline__ bool whole(int v) const { return first(v) >= 0 && first(v) + E <= n; }
    __device__ __forceinline__ uint4 load(int v) const {
        return __ldcs(reinterpret_cast<const uint4 *>(x + first(v)));
    }
    // Any vector, absent elements as -inf; only what is in the row is read.
    __device__ __forceinline__ void read(int v, float (&out)[E]) const {
        if (whole(v)) {
            Type<DT>::unpack(*reinterpret_cast<const uint4 *>(x + first(v)), out);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int64_t j = first(v) + i;
                out[i] = j >= 0 && j < n ? Type<DT>::value(x[j]) : -INFINITY;
            }
        }
    }
};

// ---- sums -----------------------------------------------------------------

struct Sums {
    float R, s, t;
};

__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
    const float R = fmaxf(a.R, b.R), da = a.R - R, db = b.R - R, fa = ex2(da), fb = ex2(db);
    return {R, a.s * fa + b.s * fb, fa * fmaf(da, a.s, a.t) + fb * fmaf(db, b.s, b.t)};
}

struct Best {
    float value;
    int vector;
};

// `count` vectors' values into the sums and the best.
template <int E, int U, bool TOP>
__device__ __forceinline__ void take(const float (&v)[U][E], int first, int stride, float c, Sums &a, Best &best) {
    float top[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        top[u] = v[u][0];
#pragma unroll
        for (int i = 1; i < E; ++i) top[u] = fmaxf(top[u], v[u][i]);
        if (TOP && top[u] > best.value) {
            best.value = top[u];
            best.vector = first + u * stride;
        }
    }
    float m = top[0];
#pragma unroll
    for (int u = 1; u < U; ++u) m = fmaxf(m, top[u]);
    const float R = fmaxf(a.R, fmaxf(m, kFloor) * c), d0 = a.R - R, f = ex2(d0);
    a.t = f * fmaf(d0, a.s, a.t);
    a.s *= f;
    a.R = R;
    float s[2] = {}, t[2] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = fmaf(max_nan(v[u][i], kFloor), c, -R), e = ex2(d);
            s[i & 1] += e;
            t[i & 1] = fmaf(e, d, t[i & 1]);
        }
    a.s += s[0] + s[1];
    a.t += t[0] + t[1];
}

// ---- top-k of a piece -----------------------------------------------------

struct Shared {
    uint64_t best[kThreads];
    uint64_t list[32];
    uint64_t cand[kCandidates];
    alignas(16) uint64_t scratch[kWarps][64];
    uint64_t part[kWarps][32];
    Sums sums[kWarps];
    float wide[kWarps];
    int count;
    // written by the cluster's CTAs into the first one's
    uint64_t top[kMaxCluster][32];
    Sums piece[kMaxCluster];
};

// Keys of one vector's elements (0 for absent ones).
template <int DT>
__device__ __forceinline__ void vector_keys(const Row<DT> &row, int v, bool on, uint64_t (&key)[Type<DT>::E]) {
    constexpr int E = Type<DT>::E;
    float x[E];
    if (on) row.read(v, x);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int64_t j = row.first(v) + i;
        key[i] = on && j >= 0 && j < row.n ? make_key(x[i], (uint32_t)j) : 0ull;
    }
}

// The piece's K best keys, one a lane of warp 0.
template <int DT>
__device__ uint64_t piece_top(Shared &sh, const Row<DT> &row, int v0, int v1, int K, const Best &best, bool rare) {
    constexpr int E = Type<DT>::E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (rare) {  // a NaN or an infinity in the piece: every element as a key
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
    sh.best[threadIdx.x] = best.vector >= 0 ? make_key(best.value, (uint32_t)best.vector) : 0ull;
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    if (warp == 0) {
        uint64_t key[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) key[w] = sh.best[32 * w + lane];
        sh.list[lane] = warp_topk_merge<kWarps>(key, 0ull, K, lane, sh.scratch[0]);
    }
    __syncthreads();
    // Elements of the listed threads that reach the K-th one's best: a larger
    // value, or the same in a vector not after it.
    const uint64_t tau = sh.list[K - 1];
    const uint32_t tau_word = (uint32_t)(tau >> 32);
    const int tau_vector = tau ? (int)key_index(tau) : 0x7FFFFFFF;
    const int rounds = (v1 - v0 + kThreads - 1) / kThreads;
    for (int e = threadIdx.x; e < K * rounds; e += kThreads) {
        const uint64_t who = sh.list[e / rounds];
        if (!who) continue;
        const int v = v0 + ((int)key_index(who) - v0) % kThreads + (e % rounds) * kThreads;
        if (v >= v1) continue;
        uint64_t key[E];
        vector_keys<DT>(row, v, true, key);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint32_t w = (uint32_t)(key[i] >> 32);
            if (key[i] && (w > tau_word || (w == tau_word && v <= tau_vector))) {
                const int at = atomicAdd(&sh.count, 1);  // the order does not matter: keys are ranked
                if (at < kCandidates) sh.cand[at] = key[i];
            }
        }
    }
    __syncthreads();
    if (warp) return 0;
    uint64_t run = 0;
    if (sh.count <= kCandidates) {
        for (int at = 0; at < sh.count; at += 128) {
            uint64_t key[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) key[i] = at + 32 * i + lane < sh.count ? sh.cand[at + 32 * i + lane] : 0ull;
            run = warp_topk_merge<4>(key, run, K, lane, sh.scratch[0]);
        }
    } else {  // heavy ties: every element of the listed threads
        for (int at = 0; at < K * rounds; at += 32) {
            const int e = at + lane;
            const uint64_t who = e < K * rounds ? sh.list[e / rounds] : 0ull;
            const int v = who ? v0 + ((int)key_index(who) - v0) % kThreads + (e % rounds) * kThreads : v1;
            uint64_t key[E];
            vector_keys<DT>(row, v, v < v1, key);
            run = warp_topk_merge<E>(key, run, K, lane, sh.scratch[0]);
        }
    }
    return run;
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
        if (!rare) return (fmaf(x, c2, -R) - log2s) * kLn2;
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

// A row with a NaN or an infinity, or with no logit above -2^99: the formulas
// as they stand, two more passes by the cluster's first CTA.
template <int DT>
__device__ void rare_row(Shared &sh, const Row<DT> &row, float c, Result &r) {
    float M = -INFINITY;
    for (int j = threadIdx.x; j < row.n; j += kThreads) M = max_nan(M, Type<DT>::value(row.x[j]));
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
        const float d = (Type<DT>::value(row.x[j]) - M) * c, e = expf(d);
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

template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const Params p) {
    constexpr int E = Type<DT>::E;
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t r = blockIdx.x / p.cluster;
    const Row<DT> row(p, r);
    const int v0 = (int)((int64_t)row.vectors * rank / p.cluster);
    const int v1 = (int)((int64_t)row.vectors * (rank + 1) / p.cluster);
    const float c2 = p.scale * kLog2E;
    if (p.cluster > 1) cluster_arrive();  // every CTA of the cluster runs before any writes to the first
    grid_launch_dependents();
    grid_dependency_wait();

    // The given tokens' logits, ahead of the pass.
    float given = NAN;
    if (rank == 0 && (int)threadIdx.x < p.ntok) {
        const int32_t v = p.tokens[r * p.ldt + threadIdx.x];
        if (v >= 0 && v < p.n) given = Type<DT>::value(row.x[v]);
    }

    Sums a = {kFloor * c2, 0.0f, 0.0f};
    Best best = {-INFINITY, v0 + (int)threadIdx.x < v1 ? v0 + (int)threadIdx.x : -1};
    int v = v0 + threadIdx.x;
    for (; v + (kUnroll - 1) * kThreads < v1; v += kUnroll * kThreads) {
        float x[kUnroll][E];
        if (row.whole(v) && row.whole(v + (kUnroll - 1) * kThreads)) {
            uint4 u[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) u[i] = row.load(v + i * kThreads);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) Type<DT>::unpack(u[i], x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) row.read(v + i * kThreads, x[i]);
        }
        take<E, kUnroll, TOP>(x, v, kThreads, c2, a, best);
    }
    for (; v < v1; v += kThreads) {
        float x[1][E];
        row.read(v, x[0]);
        take<E, 1, TOP>(x, v, kThreads, c2, a, best);
    }

    const bool odd = !(a.s == a.s);  // a NaN or +inf: not seen by the maxima
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const Sums b = {__shfl_xor_sync(0xffffffffu, a.R, d), __shfl_xor_sync(0xffffffffu, a.s, d),
                        __shfl_xor_sync(0xffffffffu, a.t, d)};
        a = (lane & d) ? join(b, a) : join(a, b);
    }
    if (lane == 0) sh.sums[warp] = a;
    const bool rare_piece = __syncthreads_or(odd);
    a = sh.sums[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) a = join(a, sh.sums[w]);
    uint64_t top = 0;
    if (TOP) top = piece_top<DT>(sh, row, v0, v1, p.K, best, rare_piece);

    if (p.cluster > 1) {
        cluster_wait();  // of the arrival at the start
        if (threadIdx.x == 0) {
            put(in_first(&sh.piece[rank].R), a.R);
            put(in_first(&sh.piece[rank].s), a.s);
            put(in_first(&sh.piece[rank].t), a.t);
        }
        if (TOP && warp == 0) put(in_first(&sh.top[rank][lane]), lane < p.K ? top : (uint64_t)0);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (rank) return;
        a = sh.piece[0];
        for (int i = 1; i < p.cluster; ++i) a = join(a, sh.piece[i]);
        if (TOP && warp == 0) {
            uint64_t key[kMaxCluster];
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i) key[i] = i < p.cluster ? sh.top[i][lane] : 0ull;
            top = warp_topk_merge<kMaxCluster>(key, 0ull, p.K, lane, sh.scratch[0]);
        }
    }

    Result out;
    out.rare = false;
    out.c2 = c2;
    out.R = a.R;
    out.log2s = log2f(a.s);
    out.lse = (a.R + out.log2s) * kLn2;
    out.entropy = (out.log2s - a.t / a.s) * kLn2;
    const bool fine = a.s > 0.0f && a.s < INFINITY && a.R > 0.5f * kFloor * c2 && a.R < INFINITY;
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
    return mr_host::cuda_status(p.K ? cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, true>, p)
                                    : cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, false>, p));
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
    p.cluster = 1;
    while (p.cluster < mr::logprobs::kMaxCluster && (int64_t)n * size > p.cluster * mr::logprobs::kPieceBytes)
        p.cluster *= 2;
    if ((int64_t)m * p.cluster > (int64_t)INT32_MAX) return MR_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MR_F32: return mr::logprobs::launch<MR_F32>(p, m, s);
        case MR_BF16: return mr::logprobs::launch<MR_BF16>(p, m, s);
        default: return mr::logprobs::launch<MR_F16>(p, m, s);
    }
}
