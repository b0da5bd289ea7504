// moe_window_bf16 / moe_window_w4: the routed experts of a verify window.
//
//   y[t] = sum_s w[t,s] * Wd[e] . h,   h = silu(Wg[e] . x_t) * (Wu[e] . x_t),   e = ids[t,s] - base
//
// HBM-bound with bf16 weights (16 rows of 512 experts, top 10, 2560 x 640: 216 us,
// 6.3 TB/s; one row 26.9 us, of which 12 are the kernels' starts and ends), bound by
// unpacking with 4-bit ones (8 rows 57 us): every expert that some row picked is read
// once, and a weight value meets only the few rows that picked it.  Each CTA finds the distinct
// experts among the m * topk choices itself (no list in memory, no extra
// launch) and the flat list of (expert, tile) is cut into equal runs.
//
//  * up kernel: a tile is 8 gate rows and the 8 up rows of the same columns,
//    one 16-row operand of the matrix instruction.  k is summed in quarters,
//    one warp each while tiles are few, all four in one warp when there are
//    enough tiles to keep the warps busy; either way the quarters are added
//    in order.
//  * down kernel: applies the activation and multiplies by the down
//    projection.  h is fp32; the tensor core takes it as three bf16 pieces
//    whose sum is exact, as three columns of the 8 that an instruction has (most
//    experts serve one or two rows), so no precision is lost between the two
//    products and no instruction added.
//  * combine kernel: the weighted sum over a row's choices, in their order.
//    (Added up instead by the warp that stores a tile's last share, it took
//    323 us in place of 234 at 16 rows: a few warps get most of that work.)
//
// The three are launched programmatically: as a kernel's CTAs leave, the next
// one's build their lists and request their first weights (down) or compute the
// softmax (combine) before the rest has finished.
// The split of k depends on the sizes of the expert alone and sums run in a
// fixed order, so a row's bits depend on its own x, ids and weights only.
#include "w4_core.cuh"

#include <type_traits>

namespace mr {
namespace moe {

using namespace mr::w4;

constexpr int kMaxRows = 16;
constexpr int kMaxTopk = 32;
constexpr int kMaxSlots = kMaxRows * kMaxTopk;
constexpr int kChunk = 8;        // choices of one expert that share a pass over its weight
constexpr int kSplit = kKW;      // parts of k in the up projection

struct Params {
    const uint8_t *X;
    int64_t ldx;                  // bytes
    const int32_t *ids;
    const float *wts;
    int64_t ldr;
    const uint8_t *Wu, *Wd;
    int64_t ldu, ldd, eu, ed;     // bytes: row strides (bf16) and expert strides
    float *part;                  // [slot][1 or kSplit][2 * inter]
    float *down;                  // [slot][hidden]
    void *Y;
    int64_t ldy;
    int m, topk, experts, base, hidden, inter;
    int cap;                      // choices per chunk: min(kChunk, m)
    int block;                    // bytes of a block of weight
    int per_up, slots_up, per_down, slots_down;  // ring stages, as in mrgemv_w4
    int up_warps;                 // warps of the up kernel's grid
    int out_bf16, softmax;
    uint32_t fmt;
};

// The chunks of a call: up to `cap` choices (slots t * topk + s) of one expert,
// in the order of their first slots.
constexpr int kTable = 1024;
struct alignas(16) Chunks {
    int32_t ids[kMaxSlots];
    int32_t expert[kMaxSlots];
    int32_t count[kMaxSlots];
    uint32_t lead[kMaxSlots / 32];      // slots that open a chunk
    union {
        uint16_t slot[kMaxSlots][kChunk];
        struct {                        // while it is built, by expert
            int first[kTable], seen[kTable];
        } table;
    };
    int n;
};
constexpr int kChunkBytes = (sizeof(Chunks) + 127) / 128 * 128;  // at the start of dynamic shared memory

// A thread's slots' experts, -1 where there is none held here: loaded ahead of
// build_chunks, from L2 (the producer of ids may have run while this grid was
// starting).
template <int WARPS>
struct Choices {
    static constexpr int N = kMaxSlots / (WARPS * 32);
    int e[N];
    __device__ __forceinline__ explicit Choices(const Params &p) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = i * WARPS * 32 + threadIdx.x;
            e[i] = -1;
            if (s < p.m * p.topk) {
                const int64_t id = (int64_t)__ldcg(p.ids + (s / p.topk) * p.ldr + s % p.topk);
                if (id >= p.base && id - p.base < p.experts) e[i] = (int)(id - p.base);
            }
        }
    }
};

// Built by every thread of the CTA, the same in every CTA.  With a table entry
// an expert, an atomic minimum finds its first slot and an atomic count the
// slots' places (in any order: a place changes no result).  Where there are more
// experts than entries, or one has choices for several chunks (whose members
// must be the same in every CTA), places come from a scan of the slots before.
template <int WARPS>
__device__ void build_chunks(Chunks &c, const Params &p, const Choices<WARPS> &mine) {
    constexpr int N = Choices<WARPS>::N, kThreads = WARPS * 32;
    const int S = p.m * p.topk, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kTable; i += kThreads) {
        c.table.first[i] = kMaxSlots;
        c.table.seen[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) c.count[i * kThreads + threadIdx.x] = 0;
    __syncthreads();
    int place[N], first[N];
    bool scan = p.experts > kTable;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int s = i * kThreads + threadIdx.x, e = mine.e[i];
        c.ids[s] = e;
        if (e >= 0 && p.experts <= kTable) {
            atomicMin(&c.table.first[e], s);
            place[i] = atomicAdd(&c.table.seen[e], 1);
            scan = scan || place[i] >= p.cap;
        }
    }
    scan = __syncthreads_or(scan);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int s = i * kThreads + threadIdx.x, e = mine.e[i];
        if (!scan) {
            first[i] = e >= 0 ? c.table.first[e] : -1;
        } else {
            place[i] = 0;
            first[i] = e >= 0 ? s : -1;
            for (int q = 0; e >= 0 && q < s; ++q)
                if (c.ids[q] == e) {
                    if (place[i] == 0) first[i] = q;
                    place[i] = place[i] + 1 == p.cap ? 0 : place[i] + 1;
                }
            if (place[i] == 0 && e >= 0) first[i] = s;
        }
        const uint32_t leads = __ballot_sync(0xffffffffu, first[i] == s);
        if (lane == 0) c.lead[s / 32] = leads;
    }
    __syncthreads();  // the table has been read
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int s = i * kThreads + threadIdx.x;
        if (first[i] < 0) continue;
        int chunk = __popc(c.lead[first[i] / 32] & ((1u << (first[i] & 31)) - 1u));
        for (int w = 0; w < first[i] / 32; ++w) chunk += __popc(c.lead[w]);
        c.slot[chunk][place[i]] = (uint16_t)s;
        atomicAdd(&c.count[chunk], 1);
        if (first[i] == s) c.expert[chunk] = mine.e[i];
    }
    if (threadIdx.x < 32) {
        const int n = __reduce_add_sync(0xffffffffu, lane < (S + 31) / 32 ? __popc(c.lead[lane]) : 0);
        if (lane == 0) c.n = n;
    }
    __syncthreads();
}

__host__ __device__ inline int row_stride(int k) { return (k + kBlockK - 1) / kBlockK * kBlockK * 2 + 64; }

// The stream of a warp's weight blocks: packed 4-bit blocks come through a Ring
// (bulk copies of up to `per` blocks), bf16 rows through cp.async, where every
// lane copies the bytes it reads itself.

// Whether a warp of the up kernel sums all quarters of a tile itself: when
// that still gives every warp two tiles.  (The down projection has no quarters:
// with its shorter k they cost more in partial sums than they balanced, one bf16
// row 29.8 us without, 31.3 with.)
__device__ __forceinline__ bool whole_up(const Params &p, int chunks) {
    return chunks * (p.inter / 8) >= 2 * p.up_warps;
}

// ---- up projection --------------------------------------------------------

// G = 0: bf16 rows, STAGES blocks in flight; else 4-bit groups of G.
template <int G, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) up_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem_base[];
    Chunks &chunks = *reinterpret_cast<Chunks *>(smem_base);
    uint8_t *smem = smem_base + kChunkBytes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int kblocks = (p.hidden + kBlockK - 1) / kBlockK, tiles = p.inter / 8, xs = row_stride(p.hidden);
    const uint32_t x0 = smem_u32(smem), ring0 = x0 + (p.m + 1) * xs;
    const int ring_bytes = p.slots_up * p.per_up * p.block;
    Ring ring(ring0 + warp * ring_bytes, ring0 + WARPS * ring_bytes + warp * p.slots_up * 8, p.slots_up,
              p.per_up * p.block);
    if (G) ring.init(lane);
    grid_dependency_wait();
    grid_launch_dependents();  // after the wait: the next grid may read ids at once
    const Choices<WARPS> choices(p);
    // The rows, and one of zeros, on their way while the chunks are built.
    const int pieces = kblocks * (kBlockK / 8), live = p.hidden / 8;
    for (int r = warp; r <= p.m; r += WARPS)
        for (int c = lane; c < pieces; c += 32) {
            const bool in = r < p.m && c < live;
            cp_async16_zfill(x0 + r * xs + 16 * c, in ? p.X + r * p.ldx + 16 * c : p.X, in);
        }
    cp_async_commit();
    build_chunks<WARPS>(chunks, p, choices);

    // This CTA's run of items (tiles, or quarters of them), a warp every
    // WARPS-th: a warp of quarters always has the same one.
    const bool whole = whole_up(p, chunks.n);
    const int shift = whole ? 0 : 2, parts = whole ? 1 : kSplit;
    const int64_t items = (int64_t)(chunks.n * tiles) << shift;
    const int i0 = (int)(items * blockIdx.x / gridDim.x) + warp, i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
    const int slice = whole ? 0 : i0 & 3, step = WARPS >> shift;
    int left = i0 < i1 ? (i1 - i0 + WARPS - 1) / WARPS : 0;  // items of this warp
    int chunk = (i0 >> shift) / tiles, tile = (i0 >> shift) % tiles;

    // the next blocks to request
    const int kb0 = quarter_begin(kblocks, slice), kb1 = whole ? kblocks : quarter_begin(kblocks, slice + 1);
    int rleft = kb0 < kb1 ? left : 0, rchunk = chunk, rtile = tile, rkb = kb0;
    const uint8_t *src0 = nullptr, *src8 = nullptr;
    auto aim = [&]() {
        const uint8_t *w = p.Wu + (int64_t)chunks.expert[rchunk] * p.eu;
        if (G) {
            src0 = w + (int64_t)(rtile * kblocks + kb0) * p.block;
        } else {
            src0 = w + (int64_t)(rtile * 8 + g) * p.ldu + kb0 * kBlockK * 2;
            src8 = src0 + (int64_t)p.inter * p.ldu;
        }
    };
    if (rleft) aim();
    int rstage = 0;  // bf16: the stage of the next request
    auto request = [&]() {
        if (rleft) {
            const int count = G ? min(p.per_up, kb1 - rkb) : 1;
            if (G) {
                ring.request(src0, count * p.block, lane);
                src0 += count * p.block;
            } else {
                issue_block_bf16(ring.data + rstage * p.block, reinterpret_cast<const uint16_t *>(src0),
                                 reinterpret_cast<const uint16_t *>(src8), true, true, p.hidden - rkb * kBlockK, lane);
                src0 += kBlockK * 2;
                src8 += kBlockK * 2;
            }
            rkb += count;
            if (rkb == kb1) {
                rkb = kb0;
                rtile += step;
                while (rtile >= tiles) {
                    rtile -= tiles;
                    ++rchunk;
                }
                if (--rleft) aim();
            }
        }
        if (!G) {
            cp_async_commit();
            rstage = rstage + 1 == STAGES ? 0 : rstage + 1;
        }
    };
    const int slots = G ? p.slots_up : STAGES;
    for (int s = 0; s < slots; ++s) request();
    cp_async_wait<G ? 0 : STAGES>();  // the rows
    __syncthreads();

    int stage = 0;
    for (; left; --left) {
        const int count = chunks.count[chunk];
        const uint32_t xb[1] = {x0 + (g < count ? chunks.slot[chunk][g] / p.topk : p.m) * xs + 16 * t};
        float S[1][4];
        if constexpr (G) {
            sum_quarters<G, false, 1>(ring, request, kblocks, kb0, kb1, p.per_up, p.block, p.fmt, xb, S, lane);
        } else {
            for (int q = slice; q < (whole ? kSplit : slice + 1); ++q) {
                float C[1][4] = {};
                for (int kb = quarter_begin(kblocks, q); kb < quarter_begin(kblocks, q + 1); ++kb) {
                    cp_async_wait<STAGES - 1>();
                    const uint32_t x[1] = {xb[0] + kb * (kBlockK * 2)};
                    consume_block_bf16<1>(ring.data + stage * p.block, x, C, lane);
                    request();
                    stage = stage + 1 == STAGES ? 0 : stage + 1;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) S[0][e] = q == slice ? C[0][e] : S[0][e] + C[0][e];
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (2 * t + h < count) {
                float *out = p.part + (int64_t)(chunks.slot[chunk][2 * t + h] * parts + slice) * 2 * p.inter +
                             tile * 8 + g;
                out[0] = S[0][h];
                out[p.inter] = S[0][2 + h];
            }
        tile += step;
        while (tile >= tiles) {
            tile -= tiles;
            ++chunk;
        }
    }
}

// ---- activation and down projection ----------------------------------------

// A chunk's activations in fp32 as three bf16 rows each, hi + mid + lo.
template <int THREADS>
__device__ void stage_activations(uint8_t *smem, const Params &p, const Chunks &c, int chunk, int parts, int hs,
                                  int width) {
    // four columns a thread: all of its loads are in flight together
    const int quads = width / 4;
    for (int e = threadIdx.x; e < c.count[chunk] * quads; e += THREADS) {
        const int i = e / quads, j = 4 * (e % quads);
        float gate[4] = {}, up[4] = {};
        if (j < p.inter) {
            const float *q = p.part + (int64_t)c.slot[chunk][i] * parts * 2 * p.inter + j;
            float4 v[2 * kSplit];
#pragma unroll
            for (int s = 0; s < kSplit; ++s)
                if (s < parts) {
                    v[2 * s] = *reinterpret_cast<const float4 *>(q + 2 * s * p.inter);
                    v[2 * s + 1] = *reinterpret_cast<const float4 *>(q + (2 * s + 1) * p.inter);
                }
#pragma unroll
            for (int s = 0; s < kSplit; ++s)
                if (s < parts) {
                    const float a[4] = {v[2 * s].x, v[2 * s].y, v[2 * s].z, v[2 * s].w};
                    const float b[4] = {v[2 * s + 1].x, v[2 * s + 1].y, v[2 * s + 1].z, v[2 * s + 1].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        gate[x] += a[x];
                        up[x] += b[x];
                    }
                }
        }
        // h = hi + mid + lo exactly: each piece takes the next 8 bits
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float h = gate[x] / (1.0f + expf(-gate[x])) * up[x];
            hi[x] = __float_as_uint(h) & 0xFFFF0000u;
            const bool finite = (hi[x] & 0x7F800000u) != 0x7F800000u;
            const float r = finite ? h - __uint_as_float(hi[x]) : 0.0f;
            mid[x] = __float_as_uint(r) & 0xFFFF0000u;
            lo[x] = __float_as_uint(r - __uint_as_float(mid[x]));
        }
        uint8_t *row = smem + (3 * i) * hs + 2 * j;
        *reinterpret_cast<uint2 *>(row) = make_uint2(hi[0] >> 16 | hi[1], hi[2] >> 16 | hi[3]);
        *reinterpret_cast<uint2 *>(row + hs) = make_uint2(mid[0] >> 16 | mid[1], mid[2] >> 16 | mid[3]);
        *reinterpret_cast<uint2 *>(row + 2 * hs) =
            make_uint2(lo[0] >> 16 | (lo[1] & 0xFFFF0000u), lo[2] >> 16 | (lo[3] & 0xFFFF0000u));
    }
}

template <int G, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) down_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem_base[];
    Chunks &chunks = *reinterpret_cast<Chunks *>(smem_base);
    uint8_t *smem = smem_base + kChunkBytes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int kblocks = (p.inter + kBlockK - 1) / kBlockK, tiles = (p.hidden + kTileRows - 1) / kTileRows;
    const int hs = row_stride(p.inter), zero_row = 3 * p.cap;
    const uint32_t h0 = smem_u32(smem), ring0 = h0 + (zero_row + 1) * hs;
    const int ring_bytes = p.slots_down * p.per_down * p.block;
    Ring ring(ring0 + warp * ring_bytes, ring0 + WARPS * ring_bytes + warp * p.slots_down * 8, p.slots_down,
              p.per_down * p.block);
    grid_launch_dependents();
    const Choices<WARPS> choices(p);
    if (G) ring.init(lane);
    build_chunks<WARPS>(chunks, p, choices);

    const int64_t units = (int64_t)chunks.n * tiles;
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    int ru = u0 + warp, rkb = 0, rchunk = ru / tiles, rtile = ru % tiles;
    const uint8_t *src0 = nullptr, *src8 = nullptr;
    bool on0 = false, on8 = false;
    auto aim = [&]() {
        const uint8_t *w = p.Wd + (int64_t)chunks.expert[rchunk] * p.ed;
        if (G) {
            src0 = w + (int64_t)(rtile * kblocks) * p.block;
        } else {
            const int row = rtile * kTileRows + g;
            on0 = row < p.hidden;
            on8 = row + 8 < p.hidden;
            src0 = on0 ? w + (int64_t)row * p.ldd : w;
            src8 = on8 ? w + (int64_t)(row + 8) * p.ldd : w;
        }
    };
    if (ru < u1) aim();
    auto request = [&](int stage) {
        if (ru < u1) {
            const int count = G ? min(p.per_down, kblocks - rkb) : 1;
            if (G)
                ring.request(src0 + rkb * p.block, count * p.block, lane);
            else
                issue_block_bf16(ring.data + stage * p.block, reinterpret_cast<const uint16_t *>(src0) + rkb * kBlockK,
                                 reinterpret_cast<const uint16_t *>(src8) + rkb * kBlockK, on0, on8,
                                 p.inter - rkb * kBlockK, lane);
            rkb += count;
            if (rkb == kblocks) {
                rkb = 0;
                ru += WARPS;
                rtile += WARPS;
                while (rtile >= tiles) {
                    rtile -= tiles;
                    ++rchunk;
                }
                if (ru < u1) aim();
            }
        }
        if (!G) cp_async_commit();
    };
    const int slots = G ? p.slots_down : STAGES;
    for (int s = 0; s < slots; ++s) request(s);
    for (int e = threadIdx.x; e < hs / 16; e += WARPS * 32)
        *reinterpret_cast<uint4 *>(smem + zero_row * hs + 16 * e) = make_uint4(0, 0, 0, 0);

    grid_dependency_wait();  // the up projection's partial sums
    if (u0 >= u1) return;
    const int parts = whole_up(p, chunks.n) ? 1 : kSplit;
    int stage = 0;
    // The address of a lane's column of column tile c: piece g % 4 of choice
    // 2c + g / 4, zeros for the fourth and for choices that are not there.
    auto column = [&](int c, int count) {
        const int i = 2 * c + (g >> 2), piece = g & 3;
        return h0 + (piece < 3 && i < count ? i * 3 + piece : zero_row) * hs + 16 * t;
    };
    // One tile of the chunk whose activations are staged.  NT column tiles of
    // two choices a pass, and PASSES passes over a stage.
    auto product = [&](auto nt, auto ps, int chunk, int tile, int count) {
        constexpr int NT = decltype(nt)::value, PASSES = decltype(ps)::value;
        uint32_t xb[PASSES][NT];
        float C[PASSES][NT][4] = {};
#pragma unroll
        for (int q = 0; q < PASSES; ++q)
#pragma unroll
            for (int c = 0; c < NT; ++c) xb[q][c] = column(q * NT + c, count);
        auto one = [&](uint32_t at, int kb) {
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                uint32_t x[NT];
#pragma unroll
                for (int c = 0; c < NT; ++c) x[c] = xb[q][c] + kb * (kBlockK * 2);
                if constexpr (G)
                    consume_block<G, false, NT>(at, p.fmt, x, C[q], lane);
                else
                    consume_block_bf16<NT>(at, x, C[q], lane);
            }
        };
        if constexpr (G) {
            for (int kb = 0; kb < kblocks; kb += p.per_down) {
                const uint32_t at = ring.wait();
                const int blocks = min(p.per_down, kblocks - kb);
#pragma unroll 1
                for (int b = 0; b < blocks; ++b) one(at + b * p.block, kb + b);
                ring.done();
                request(0);
            }
        } else {
            for (int kb = 0; kb < kblocks; ++kb) {
                cp_async_wait<STAGES - 1>();
                one(ring.data + stage * p.block, kb);
                request(stage);
                stage = stage + 1 == STAGES ? 0 : stage + 1;
            }
        }
        // The pieces of a choice lie in lanes t = 0, 1 or t = 2, 3.
#pragma unroll
        for (int q = 0; q < PASSES; ++q)
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                float r0 = C[q][c][0] + C[q][c][1], r8 = C[q][c][2] + C[q][c][3];
                r0 += __shfl_xor_sync(0xffffffffu, r0, 1);
                r8 += __shfl_xor_sync(0xffffffffu, r8, 1);
                const int i = 2 * (q * NT + c) + (t >> 1), row = tile * kTileRows + g + 8 * (t & 1);
                if (i < count && row < p.hidden)
                    p.down[(int64_t)chunks.slot[chunk][i] * p.hidden + row] = (t & 1) ? r8 : r0;
            }
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    int u = u0 + warp;
    for (int chunk = u0 / tiles; chunk <= (u1 - 1) / tiles; ++chunk) {
        const int count = chunks.count[chunk];
        __syncthreads();  // the chunk before is done with the activations
        stage_activations<WARPS * 32>(smem, p, chunks, chunk, parts, hs, kblocks * kBlockK);
        __syncthreads();
        const int end = min(u1, (chunk + 1) * tiles);
        for (; u < end; u += WARPS) {
            const int tile = u - chunk * tiles;
            if (count <= 2)
                product(One{}, One{}, chunk, tile, count);
            else if (count <= 4)
                product(Two{}, One{}, chunk, tile, count);
            else
                product(Two{}, Two{}, chunk, tile, count);
        }
    }
}

// ---- weighted sum over a row's choices -------------------------------------

__global__ void __launch_bounds__(128) combine_kernel(const Params p) {
    __shared__ float w[kMaxTopk];
    __shared__ int held[kMaxTopk];
    const int row = blockIdx.y;
    grid_launch_dependents();
    if (threadIdx.x < 32) {
        const int s = threadIdx.x;
        const int64_t e = s < p.topk ? (int64_t)__ldcg(p.ids + row * p.ldr + s) : -1;
        float v = e >= 0 ? __ldcg(p.wts + row * p.ldr + s) : -INFINITY;
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
        held[s] = e >= p.base && e - p.base < p.experts;
    }
    __syncthreads();
    grid_dependency_wait();
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= p.hidden) return;
    float y = 0.0f;
    for (int s0 = 0; s0 < p.topk; s0 += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = s0 + i < p.topk && held[s0 + i] ? p.down[(int64_t)(row * p.topk + s0 + i) * p.hidden + j] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (s0 + i < p.topk && held[s0 + i]) y = fmaf(w[s0 + i], v[i], y);
    }
    if (p.out_bf16)
        static_cast<__nv_bfloat16 *>(p.Y)[row * p.ldy + j] = __float2bfloat16_rn(y);
    else
        static_cast<float *>(p.Y)[row * p.ldy + j] = y;
}

template <class K>
cudaError_t launch_one(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Params &p) {
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

// Warps of a CTA, its CTAs to an SM and its shared memory.
struct Plan {
    int warps = 0, per_sm = 0, stages = 0;
    size_t smem = 0;
};

// A plan of `per_sm` CTAs of `warps` within `limit` bytes each; `length`:
// consecutive blocks a warp can use (packed blocks), `stages`: blocks in flight
// (bf16).
Plan fit(size_t limit, int per_sm, int warps, int stages, size_t fixed, int length, int block, bool packed, int &per,
         int &slots) {
    Plan out;
    fixed += 32 * warps;  // barriers
    const int blocks = limit > fixed ? (int)((limit - fixed) / warps / block) : 0;
    if (blocks < (packed ? 2 : stages)) return out;
    per = packed ? std::min(length, blocks / 2) : 1;
    slots = packed ? std::min(4, blocks / per) : stages;
    out.warps = warps;
    out.per_sm = per_sm;
    out.stages = stages;
    out.smem = fixed + (size_t)warps * slots * per * block;
    return out;
}

// Two CTAs of 8 warps share an SM where the activations leave each a ring (40 KB
// of packed blocks, two bf16 blocks a warp); otherwise one CTA of 16 warps, or for
// bf16 of 8 with a deeper ring.  (One CTA of 8 of each kernel sharing an SM, so
// that the down projection stands ready when the up projection ends, was
// slower: one bf16 row 28.4 us against 26.8, 8 rows of 4-bit experts 71 against 57.)
Plan plan(size_t optin, size_t fixed, int length, int block, bool packed, int &per, int &slots) {
    const size_t half = (optin + 1024) / 2 - 1024;
    Plan out;
    if (packed) {
        if (fixed + 40 * 1024 < half) out = fit(half, 2, 8, 0, fixed, length, block, true, per, slots);
        if (!out.warps) out = fit(optin, 1, 16, 0, fixed, length, block, true, per, slots);
        return out;
    }
    const int tries[4][2] = {{8, 2}, {16, 2}, {8, 3}, {8, 2}};  // warps, stages; the first in half an SM
    for (int i = 0; i < 4 && !out.warps; ++i)
        out = fit(i ? optin : half, i ? 1 : 2, tries[i][0], tries[i][1], fixed, 1, block, false, per, slots);
    return out;
}
Plan up_plan(Params &p, size_t optin) {
    const int kblocks = (p.hidden + kBlockK - 1) / kBlockK;
    return plan(optin, kChunkBytes + (size_t)(p.m + 1) * row_stride(p.hidden), (kblocks + kSplit - 1) / kSplit,
                p.block, p.fmt != 0, p.per_up, p.slots_up);
}
Plan down_plan(Params &p, size_t optin) {
    const int kblocks = (p.inter + kBlockK - 1) / kBlockK;
    return plan(optin, kChunkBytes + (size_t)(3 * p.cap + 1) * row_stride(p.inter), kblocks, p.block, p.fmt != 0,
                p.per_down, p.slots_down);
}

dim3 grid_of(const Plan &pl) { return dim3((unsigned)(mr_host::sm_count() * pl.per_sm)); }

template <int G, int WARPS, int STAGES>
cudaError_t launch_up(const Params &p, const Plan &pl, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(up_kernel<G, WARPS, STAGES>, ready)) return cudaErrorInvalidValue;
    return launch_one(up_kernel<G, WARPS, STAGES>, grid_of(pl),
                      WARPS * 32, pl.smem, stream, p);
}
template <int G, int WARPS, int STAGES>
cudaError_t launch_down(const Params &p, const Plan &pl, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(down_kernel<G, WARPS, STAGES>, ready)) return cudaErrorInvalidValue;
    return launch_one(down_kernel<G, WARPS, STAGES>, grid_of(pl),
                      WARPS * 32, pl.smem, stream, p);
}

template <int G>
mr_status launch(const Params &p, const Plan &up, const Plan &down, cudaStream_t stream) {
    cudaError_t e;
    if constexpr (G) {
        e = up.warps == 8 ? launch_up<G, 8, 0>(p, up, stream) : launch_up<G, 16, 0>(p, up, stream);
        if (e == cudaSuccess)
            e = down.warps == 8 ? launch_down<G, 8, 0>(p, down, stream) : launch_down<G, 16, 0>(p, down, stream);
    } else {
        e = up.warps == 16   ? launch_up<0, 16, 2>(p, up, stream)
            : up.stages == 3 ? launch_up<0, 8, 3>(p, up, stream)
                             : launch_up<0, 8, 2>(p, up, stream);
        if (e == cudaSuccess)
            e = down.warps == 16   ? launch_down<0, 16, 2>(p, down, stream)
                : down.stages == 3 ? launch_down<0, 8, 3>(p, down, stream)
                                   : launch_down<0, 8, 2>(p, down, stream);
    }
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
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part = reinterpret_cast<float *>(ws);
    p.down = reinterpret_cast<float *>(ws + part_bytes(p.m, p.topk, p.inter));
    p.cap = std::min(kChunk, p.m);
    p.out_bf16 = out_dtype == MR_BF16;
    p.softmax = (flags & MR_MOE_SOFTMAX) != 0;
    p.block = p.fmt ? block_bytes(p.fmt) : kBlockBf16;
    const int optin = mr_host::max_smem_optin();
    const size_t most = (size_t)(optin > 0 ? optin : 232448);
    const Plan up = up_plan(p, most), down = down_plan(p, most);
    if (!up.warps || !down.warps) return MR_ERR_UNSUPPORTED;
    if (optin <= 0) return MR_ERR_CUDA;
    p.up_warps = (int)grid_of(up).x * up.warps;
    switch (p.fmt & MR_W4_GROUP_MASK) {
        case 0: return launch<0>(p, up, down, stream);
        case 32: return launch<32>(p, up, down, stream);
        case 64: return launch<64>(p, up, down, stream);
        default: return launch<128>(p, up, down, stream);
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
    if (inter < 1) return MR_ERR_INVALID_ARG;
    if (inter > mr::moe::kMaxSize) return MR_ERR_UNSUPPORTED;  // before it is doubled
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
