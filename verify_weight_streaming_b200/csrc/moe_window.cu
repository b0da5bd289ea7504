// moe_window_bf16 / moe_window_w4: the routed experts of a verify window.
//
//   y[t] = sum_s w[t,s] * Wd[e] . h,   h = silu(Wg[e] . x_t) * (Wu[e] . x_t),   e = ids[t,s] - base
//
// HBM-bound: every expert that some row picked is read once, and a weight
// value meets only the few rows that picked it.  Each CTA finds the distinct
// experts among the m * topk choices itself (no list in memory, no extra
// launch) and the flat list of (expert, tile) is cut into equal runs.
//
//  * up kernel: a tile is 8 gate rows and the 8 up rows of the same columns,
//    one 16-row operand of the matrix instruction; a warp takes a tile and a
//    quarter of k and stores its partial sums.
//  * down kernel: adds the quarters in order, applies the activation, and
//    multiplies by the down projection.  h is fp32; the tensor core takes it
//    as three bf16 pieces whose sum is exact, as three columns of the 8 that
//    an instruction has (most experts serve one or two rows), so no
//    precision is lost between the two products and no instruction added.
//  * combine kernel: the weighted sum over a row's choices, in their order.
//
// The split of k depends on the sizes of the expert alone and sums run in a
// fixed order, so a row's bits depend on its own x, ids and weights only.
#include "w4_core.cuh"

namespace mr {
namespace moe {

using namespace mr::w4;

constexpr int kMaxRows = 16;
constexpr int kMaxTopk = 32;
constexpr int kMaxSlots = kMaxRows * kMaxTopk;
constexpr int kChunk = 8;        // choices of one expert that share a pass over its weight
constexpr int kSplit = 4;        // parts of k in the up projection
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

struct Params {
    const uint8_t *X;
    int64_t ldx;                  // bytes
    const int32_t *ids;
    const float *wts;
    int64_t ldr;
    const uint8_t *Wu, *Wd;
    int64_t ldu, ldd, eu, ed;     // bytes: row strides (bf16) and expert strides
    float *part;                  // [slot][kSplit][2 * inter]
    float *down;                  // [slot][hidden]
    void *Y;
    int64_t ldy;
    int m, topk, experts, base, hidden, inter;
    int cap;                      // choices per chunk: min(kChunk, m)
    int block;                    // bytes of a ring stage
    int stages;
    int out_bf16, softmax;
    uint32_t fmt;
};

// The chunks of a call: up to `cap` choices (slots t * topk + s) of one expert.
struct Chunks {
    int32_t ids[kMaxSlots];
    uint32_t lead[kMaxSlots / 32];
    int32_t expert[kMaxSlots];
    int32_t count[kMaxSlots];
    uint16_t slot[kMaxSlots][kChunk];
    int n;
};
constexpr int kChunkBytes = (sizeof(Chunks) + 127) / 128 * 128;  // at the start of dynamic shared memory

// Built by every thread of the CTA; deterministic (chunks in the order of
// their first slot).
__device__ void build_chunks(Chunks &c, const Params &p) {
    const int S = p.m * p.topk, lane = threadIdx.x & 31;
    for (int s = threadIdx.x; s < S; s += kThreads) {
        // from L2: the producer of ids may have run while this grid was starting
        const int64_t e = (int64_t)__ldcg(p.ids + (s / p.topk) * p.ldr + s % p.topk);
        c.ids[s] = (e >= p.base && e - p.base < p.experts) ? (int32_t)(e - p.base) : -1;
        c.count[s] = 0;
    }
    __syncthreads();
    int rank[kMaxSlots / kThreads], lead[kMaxSlots / kThreads];
#pragma unroll
    for (int i = 0; i < kMaxSlots / kThreads; ++i) {
        const int s = i * kThreads + threadIdx.x;
        const int e = s < S ? c.ids[s] : -1;
        int n = 0, first = s;
        if (e >= 0) {
            for (int q = 0; q < s; ++q)
                if (c.ids[q] == e) {
                    if (n % p.cap == 0) first = q;
                    ++n;
                }
            if (n % p.cap == 0) first = s;
        }
        rank[i] = n;
        lead[i] = first;
        const uint32_t bits = __ballot_sync(0xffffffffu, e >= 0 && first == s);
        if (lane == 0) c.lead[s / 32] = bits;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxSlots / kThreads; ++i) {
        const int s = i * kThreads + threadIdx.x;
        const int e = s < S ? c.ids[s] : -1;
        if (e < 0) continue;
        int chunk = __popc(c.lead[lead[i] / 32] & ((1u << (lead[i] & 31)) - 1u));
        for (int w = 0; w < lead[i] / 32; ++w) chunk += __popc(c.lead[w]);
        c.slot[chunk][rank[i] % p.cap] = (uint16_t)s;
        atomicAdd(&c.count[chunk], 1);
        if (lead[i] == s) c.expert[chunk] = e;
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < kMaxSlots / 32; ++w) n += __popc(c.lead[w]);
        c.n = n;
    }
    __syncthreads();
}

__host__ __device__ inline int row_stride(int k) { return (k + kBlockK - 1) / kBlockK * kBlockK * 2 + 64; }

// ---- up projection --------------------------------------------------------

// G = 0: bf16 rows; else 4-bit groups of G.
template <int G>
__global__ void __launch_bounds__(kThreads) up_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem_base[];
    Chunks &chunks = *reinterpret_cast<Chunks *>(smem_base);
    uint8_t *smem = smem_base + kChunkBytes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int kblocks = (p.hidden + kBlockK - 1) / kBlockK, tiles = p.inter / 8, xs = row_stride(p.hidden);
    const uint32_t x0 = smem_u32(smem), ring = x0 + p.m * xs + warp * p.stages * p.block;
    grid_dependency_wait();
    grid_launch_dependents();  // after the wait: the next grid may read ids at once
    build_chunks(chunks, p);

    const int64_t items = (int64_t)chunks.n * tiles * kSplit;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    auto from = [&](int64_t i) { return kblocks * (int)(i % kSplit) / kSplit; };
    auto to = [&](int64_t i) { return kblocks * ((int)(i % kSplit) + 1) / kSplit; };
    // the next block to request
    int64_t ri = i0 + warp;
    int rkb = 0, rend = 0;
    const uint8_t *src0 = nullptr, *src8 = nullptr;
    auto aim = [&]() {  // first item from ri on that has blocks
        for (; ri < i1; ri += kWarps) {
            rkb = from(ri);
            rend = to(ri);
            if (rkb < rend) break;
        }
        if (ri >= i1) return;
        const int unit = (int)(ri / kSplit), tile = unit % tiles;
        const uint8_t *w = p.Wu + (int64_t)chunks.expert[unit / tiles] * p.eu;
        if (G) {
            src0 = w + (int64_t)tile * kblocks * p.block;
        } else {
            src0 = w + (int64_t)(tile * 8 + g) * p.ldu;
            src8 = src0 + (int64_t)p.inter * p.ldu;
        }
    };
    aim();
    auto request = [&](int stage) {
        if (ri < i1) {
            const uint32_t dst = ring + stage * p.block;
            if (G)
                issue_block(dst, src0 + (int64_t)rkb * p.block, p.block, lane);
            else
                issue_block_bf16(dst, reinterpret_cast<const uint16_t *>(src0) + rkb * kBlockK,
                                 reinterpret_cast<const uint16_t *>(src8) + rkb * kBlockK, true, true,
                                 p.hidden - rkb * kBlockK, lane);
            if (++rkb == rend) {
                ri += kWarps;
                aim();
            }
        }
        cp_async_commit();
    };
    constexpr int kStages = G ? 8 : 2;
#pragma unroll
    for (int s = 0; s < kStages; ++s) request(s);

    const int pieces = kblocks * (kBlockK / 8), live = p.hidden / 8;
    for (int e = threadIdx.x; e < p.m * pieces; e += kThreads) {
        const int r = e / pieces, c = e % pieces;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < live) v = *reinterpret_cast<const uint4 *>(p.X + r * p.ldx + 16 * c);
        *reinterpret_cast<uint4 *>(smem + r * xs + 16 * c) = v;
    }
    __syncthreads();

    int stage = 0;
    for (int64_t i = i0 + warp; i < i1; i += kWarps) {
        const int unit = (int)(i / kSplit), chunk = unit / tiles, tile = unit % tiles, slice = (int)(i % kSplit);
        const int count = chunks.count[chunk];
        const bool on[1] = {g < count};
        const uint32_t xb = x0 + (on[0] ? chunks.slot[chunk][g] / p.topk : 0) * xs + 16 * t;
        float C[1][4] = {};
        for (int kb = from(i); kb < to(i); ++kb) {
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const uint32_t x[1] = {xb + kb * (kBlockK * 2)};
            if constexpr (G)
                consume_block<G, false, 1>(ring + stage * p.block, p.fmt, x, on, C, lane);
            else
                consume_block_bf16<1>(ring + stage * p.block, x, on, C, lane);
            __syncwarp();
            request(stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (2 * t + h < count) {
                float *out = p.part + ((int64_t)chunks.slot[chunk][2 * t + h] * kSplit + slice) * 2 * p.inter +
                             tile * 8 + g;
                out[0] = C[0][h];
                out[p.inter] = C[0][2 + h];
            }
    }
}

// ---- activation and down projection ---------------------------------------

template <int G, int NT>
__device__ __forceinline__ void down_block(uint32_t stage, uint32_t fmt, uint32_t h0, int hs, int kb, int count,
                                           float (&C)[4][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
    bool on[NT];
    uint32_t x[NT];
    float D[NT][4];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int i = 2 * c + (g >> 2), piece = g & 3;  // column g: piece of choice i
        on[c] = piece < 3 && i < count;
        x[c] = h0 + (on[c] ? i * 3 + piece : 0) * hs + kb * (kBlockK * 2) + 16 * t;
#pragma unroll
        for (int e = 0; e < 4; ++e) D[c][e] = C[c][e];
    }
    if constexpr (G)
        consume_block<G, false, NT>(stage, fmt, x, on, D, lane);
    else
        consume_block_bf16<NT>(stage, x, on, D, lane);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) C[c][e] = D[c][e];
}

template <int G>
__global__ void __launch_bounds__(kThreads) down_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem_base[];
    Chunks &chunks = *reinterpret_cast<Chunks *>(smem_base);
    uint8_t *smem = smem_base + kChunkBytes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int kblocks = (p.inter + kBlockK - 1) / kBlockK, tiles = (p.hidden + kTileRows - 1) / kTileRows;
    const int hs = row_stride(p.inter);
    const uint32_t h0 = smem_u32(smem), ring = h0 + 3 * p.cap * hs + warp * p.stages * p.block;
    grid_launch_dependents();
    build_chunks(chunks, p);

    const int64_t units = (int64_t)chunks.n * tiles;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    int64_t ru = u0 + warp;
    int rkb = 0;
    const uint8_t *src0 = nullptr, *src8 = nullptr;
    bool on0 = false, on8 = false;
    auto aim = [&]() {
        if (ru >= u1) return;
        const int tile = (int)(ru % tiles);
        const uint8_t *w = p.Wd + (int64_t)chunks.expert[ru / tiles] * p.ed;
        if (G) {
            src0 = w + (int64_t)tile * kblocks * p.block;
        } else {
            const int row = tile * kTileRows + g;
            on0 = row < p.hidden;
            on8 = row + 8 < p.hidden;
            src0 = on0 ? w + (int64_t)row * p.ldd : w;
            src8 = on8 ? w + (int64_t)(row + 8) * p.ldd : w;
        }
    };
    aim();
    auto request = [&](int stage) {
        if (ru < u1) {
            const uint32_t dst = ring + stage * p.block;
            if (G)
                issue_block(dst, src0 + (int64_t)rkb * p.block, p.block, lane);
            else
                issue_block_bf16(dst, reinterpret_cast<const uint16_t *>(src0) + rkb * kBlockK,
                                 reinterpret_cast<const uint16_t *>(src8) + rkb * kBlockK, on0, on8,
                                 p.inter - rkb * kBlockK, lane);
            if (++rkb == kblocks) {
                rkb = 0;
                ru += kWarps;
                aim();
            }
        }
        cp_async_commit();
    };
    constexpr int kStages = G ? 8 : 2;
#pragma unroll
    for (int s = 0; s < kStages; ++s) request(s);

    grid_dependency_wait();  // the up projection's partial sums
    int stage = 0;
    int64_t u = u0 + warp;
    for (int chunk = (int)(u0 / tiles); u0 < u1 && chunk <= (int)((u1 - 1) / tiles); ++chunk) {
        const int count = chunks.count[chunk], width = kblocks * kBlockK;
        __syncthreads();  // the chunk before is done with h
        for (int e = threadIdx.x; e < count * width; e += kThreads) {
            const int i = e / width, j = e % width;
            float h = 0.0f;
            if (j < p.inter) {
                const float *q = p.part + (int64_t)chunks.slot[chunk][i] * kSplit * 2 * p.inter + j;
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int s = 0; s < kSplit; ++s) {
                    gate += q[(int64_t)s * 2 * p.inter];
                    up += q[(int64_t)s * 2 * p.inter + p.inter];
                }
                h = gate / (1.0f + expf(-gate)) * up;
            }
            // h = hi + mid + lo exactly: each piece takes the next 8 bits
            const uint32_t hi = __float_as_uint(h) & 0xFFFF0000u;
            const bool finite = (hi & 0x7F800000u) != 0x7F800000u;
            const float r = finite ? h - __uint_as_float(hi) : 0.0f;
            const uint32_t mid = __float_as_uint(r) & 0xFFFF0000u;
            const uint32_t lo = __float_as_uint(r - __uint_as_float(mid));
            uint8_t *row = smem + (3 * i) * hs + 2 * j;
            *reinterpret_cast<uint16_t *>(row) = (uint16_t)(hi >> 16);
            *reinterpret_cast<uint16_t *>(row + hs) = (uint16_t)(mid >> 16);
            *reinterpret_cast<uint16_t *>(row + 2 * hs) = (uint16_t)(lo >> 16);
        }
        __syncthreads();
        const int64_t end = min(u1, (int64_t)(chunk + 1) * tiles);
        for (; u < end; u += kWarps) {
            const int tile = (int)(u - (int64_t)chunk * tiles);
            float C[4][4] = {};
            for (int kb = 0; kb < kblocks; ++kb) {
                cp_async_wait<kStages - 1>();
                __syncwarp();
                const uint32_t at = ring + stage * p.block;
                if (count <= 2)
                    down_block<G, 1>(at, p.fmt, h0, hs, kb, count, C, lane);
                else if (count <= 4)
                    down_block<G, 2>(at, p.fmt, h0, hs, kb, count, C, lane);
                else
                    down_block<G, 4>(at, p.fmt, h0, hs, kb, count, C, lane);
                __syncwarp();
                request(stage);
                stage = stage + 1 == kStages ? 0 : stage + 1;
            }
            // The pieces of a choice lie in lanes t = 0, 1 or t = 2, 3.
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (2 * c >= count) break;
                float r0 = C[c][0] + C[c][1], r8 = C[c][2] + C[c][3];
                r0 += __shfl_xor_sync(0xffffffffu, r0, 1);
                r8 += __shfl_xor_sync(0xffffffffu, r8, 1);
                const int i = 2 * c + (t >> 1), row = tile * kTileRows + g + 8 * (t & 1);
                if (i < count && row < p.hidden)
                    p.down[(int64_t)chunks.slot[chunk][i] * p.hidden + row] = (t & 1) ? r8 : r0;
            }
        }
    }
}

// ---- weighted sum over a row's choices -------------------------------------

__global__ void __launch_bounds__(128) combine_kernel(const Params p) {
    __shared__ float w[kMaxTopk];
    const int row = blockIdx.y;
    grid_launch_dependents();
    grid_dependency_wait();
    if (threadIdx.x < 32) {
        const int s = threadIdx.x;
        const int64_t e = s < p.topk ? (int64_t)p.ids[row * p.ldr + s] : -1;
        float v = s < p.topk && e >= 0 ? p.wts[row * p.ldr + s] : -INFINITY;
        if (p.softmax) {
            float top = v;
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            v = e >= 0 ? expf(v - top) : 0.0f;
            float sum = v;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            v /= sum;
        }
        w[s] = v;
    }
    __syncthreads();
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= p.hidden) return;
    float y = 0.0f;
    for (int s = 0; s < p.topk; ++s) {
        const int64_t e = p.ids[row * p.ldr + s];
        if (e < p.base || e - p.base >= p.experts) continue;
        y = fmaf(w[s], p.down[(int64_t)(row * p.topk + s) * p.hidden + j], y);
    }
    if (p.out_bf16)
        static_cast<__nv_bfloat16 *>(p.Y)[row * p.ldy + j] = __float2bfloat16_rn(y);
    else
        static_cast<float *>(p.Y)[row * p.ldy + j] = y;
}

cudaError_t launch_one(void (*kernel)(Params), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const Params &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // Every kernel waits for its predecessor before it reads what that wrote.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

size_t up_smem(const Params &p) {
    return kChunkBytes + (size_t)p.m * row_stride(p.hidden) + (size_t)kWarps * p.stages * p.block;
}
size_t down_smem(const Params &p) {
    return kChunkBytes + (size_t)3 * p.cap * row_stride(p.inter) + (size_t)kWarps * p.stages * p.block;
}

template <int G>
mr_status launch(const Params &p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready_up{0}, ready_down{0};
    if (!allow_smem(up_kernel<G>, ready_up) || !allow_smem(down_kernel<G>, ready_down)) return MR_ERR_CUDA;
    const int sms = mr_host::sm_count();
    const size_t sm_bytes = (size_t)mr_host::max_smem_optin() + 1024, fixed = 1024;
    auto grid = [&](size_t smem) { return dim3((unsigned)(sms * (2 * (smem + fixed) <= sm_bytes ? 2 : 1))); };
    cudaError_t e = launch_one(up_kernel<G>, grid(up_smem(p)), kThreads, up_smem(p), stream, p);
    if (e == cudaSuccess) e = launch_one(down_kernel<G>, grid(down_smem(p)), kThreads, down_smem(p), stream, p);
    if (e == cudaSuccess)
        e = launch_one(combine_kernel, dim3((unsigned)((p.hidden + 127) / 128), (unsigned)p.m), 128, 0, stream, p);
    return mr_host::cuda_status(e);
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }
size_t part_bytes(int m, int topk, int inter) { return align256((size_t)m * topk * kSplit * 2 * inter * sizeof(float)); }
size_t down_bytes(int m, int topk, int hidden) { return align256((size_t)m * topk * hidden * sizeof(float)); }

constexpr int kMaxSize = 1 << 20;  // hidden, inter: far beyond what shared memory holds

bool sizes_ok(int m, int topk, int hidden, int inter) { return m >= 1 && topk >= 1 && hidden >= 1 && inter >= 1; }
bool sizes_supported(int m, int topk, int hidden, int inter) {
    return m <= kMaxRows && topk <= kMaxTopk && hidden <= kMaxSize && inter <= kMaxSize;
}

mr_status run(Params p, int out_dtype, uint32_t flags, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!p.X || !p.ids || !p.wts || !p.Wu || !p.Wd || !p.Y || !workspace) return MR_ERR_INVALID_ARG;
    if (!sizes_ok(p.m, p.topk, p.hidden, p.inter) || p.experts < 1 || p.base < 0) return MR_ERR_INVALID_ARG;
    if ((int64_t)p.base + p.experts > (int64_t)INT32_MAX) return MR_ERR_INVALID_ARG;
    if (out_dtype != MR_F32 && out_dtype != MR_BF16) return MR_ERR_INVALID_ARG;
    if (flags & ~MR_MOE_SOFTMAX) return MR_ERR_INVALID_ARG;
    if (p.ldx < 2 * (int64_t)p.hidden || p.ldr < p.topk || p.ldy < p.hidden) return MR_ERR_INVALID_ARG;
    if (((uintptr_t)p.X & 15u) || p.ldx % 16 || ((uintptr_t)p.Wu & 15u) || ((uintptr_t)p.Wd & 15u) ||
        ((uintptr_t)p.ids & 3u) || ((uintptr_t)p.wts & 3u) || ((uintptr_t)p.Y & (out_dtype == MR_F32 ? 3u : 1u)) ||
        ((uintptr_t)workspace & 255u))
        return MR_ERR_MISALIGNED;
    if (p.hidden % 8 || p.inter % 8) return MR_ERR_MISALIGNED;
    if (!sizes_supported(p.m, p.topk, p.hidden, p.inter)) return MR_ERR_UNSUPPORTED;
    if (workspace_bytes < moe_window_workspace_bytes(p.m, p.topk, p.hidden, p.inter)) return MR_ERR_INVALID_ARG;
    p.part = static_cast<float *>(workspace);
    p.down = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + part_bytes(p.m, p.topk, p.inter));
    p.cap = std::min(kChunk, p.m);
    p.out_bf16 = out_dtype == MR_BF16;
    p.softmax = (flags & MR_MOE_SOFTMAX) != 0;
    const int G = (int)(p.fmt & MR_W4_GROUP_MASK);
    p.block = G ? block_bytes(p.fmt) : kBlockBf16;
    p.stages = G ? 8 : 2;
    const int optin = mr_host::max_smem_optin();
    const size_t most = std::max(up_smem(p), down_smem(p));
    if (most > (size_t)(optin > 0 ? optin : 232448)) return MR_ERR_UNSUPPORTED;
    if (optin <= 0) return MR_ERR_CUDA;
    switch (G) {
        case 0: return launch<0>(p, stream);
        case 32: return launch<32>(p, stream);
        case 64: return launch<64>(p, stream);
        default: return launch<128>(p, stream);
    }
}

}  // namespace moe
}  // namespace mr

extern "C" size_t moe_window_workspace_bytes(int32_t m, int32_t topk, int32_t hidden, int32_t inter) {
    if (!mr::moe::sizes_ok(m, topk, hidden, inter) || !mr::moe::sizes_supported(m, topk, hidden, inter)) return 0;
    return mr::moe::part_bytes(m, topk, inter) + mr::moe::down_bytes(m, topk, hidden);
}

extern "C" mr_status moe_window_bf16(const void *X, int64_t ldx, const int32_t *ids, const float *weights, int64_t ldr,
                                     const void *Wup, int64_t ldu, int64_t stride_up, const void *Wdown, int64_t ldd,
                                     int64_t stride_down, void *Y, int64_t ldy, int32_t m, int32_t topk,
                                     int32_t experts, int32_t hidden, int32_t inter, int32_t expert_base,
                                     int32_t out_dtype, uint32_t flags, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    if (ldu < hidden || ldd < inter || stride_up < 0 || stride_down < 0) return MR_ERR_INVALID_ARG;
    if (ldu % 8 || ldd % 8 || stride_up % 8 || stride_down % 8) return MR_ERR_MISALIGNED;
    mr::moe::Params p = {};
    p.X = static_cast<const uint8_t *>(X);
    p.ldx = 2 * ldx;
    p.ids = ids;
    p.wts = weights;
    p.ldr = ldr;
    p.Wu = static_cast<const uint8_t *>(Wup);
    p.Wd = static_cast<const uint8_t *>(Wdown);
    p.ldu = 2 * ldu;
    p.ldd = 2 * ldd;
    p.eu = 2 * stride_up;
    p.ed = 2 * stride_down;
    p.Y = Y;
    p.ldy = ldy;
    p.m = m;
    p.topk = topk;
    p.experts = experts;
    p.base = expert_base;
    p.hidden = hidden;
    p.inter = inter;
    return mr::moe::run(p, out_dtype, flags, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" mr_status moe_window_w4(const void *X, int64_t ldx, const int32_t *ids, const float *weights, int64_t ldr,
                                   const void *up, size_t up_bytes, const void *down, size_t down_bytes, void *Y,
                                   int64_t ldy, int32_t m, int32_t topk, int32_t experts, int32_t hidden,
                                   int32_t inter, int32_t expert_base, uint32_t fmt, int32_t out_dtype,
                                   uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
    if (inter > (1 << 30)) return MR_ERR_UNSUPPORTED;
    mr_status st = mr::w4::check_format(2 * inter, hidden, fmt);
    if (st == MR_OK) st = mr::w4::check_format(hidden, inter, fmt);
    if (st != MR_OK) return st;
    const size_t eu = w4_packed_bytes(2 * inter, hidden, fmt, 1), ed = w4_packed_bytes(hidden, inter, fmt, 0);
    if (experts < 1 || up_bytes / (size_t)experts < eu || down_bytes / (size_t)experts < ed) return MR_ERR_INVALID_ARG;
    mr::moe::Params p = {};
    p.X = static_cast<const uint8_t *>(X);
    p.ldx = 2 * ldx;
    p.ids = ids;
    p.wts = weights;
    p.ldr = ldr;
    p.Wu = static_cast<const uint8_t *>(up);
    p.Wd = static_cast<const uint8_t *>(down);
    p.eu = (int64_t)eu;
    p.ed = (int64_t)ed;
    p.Y = Y;
    p.ldy = ldy;
    p.m = m;
    p.topk = topk;
    p.experts = experts;
    p.base = expert_base;
    p.hidden = hidden;
    p.inter = inter;
    p.fmt = fmt;
    return mr::moe::run(p, out_dtype, flags, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
