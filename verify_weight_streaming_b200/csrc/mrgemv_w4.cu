// w4_pack and mrgemv_w4: multi-row product with a 4-bit weight, fp32 output.
//
//   C[i][j] = sum_groups s[j][grp] * sum_{p in grp} A[i][p] * (q[j][p] - z[j][grp])
//
// The weight is read once for all m <= 16 rows, like mrgemv_bf16's.  At the
// HBM rate an SM receives about 46 values a clock, so neither conversions nor
// FMAs fit on the CUDA cores for more than a row or two: the values are
// unpacked to exact small integers (1.4 instructions a value) and multiplied
// on the tensor core, 256 values x 8 rows an instruction.
//
// Work: a tile is 16 weight rows, one contiguous run of the packed weight.
// KW = 4 warps (one worker) share a tile, each a contiguous quarter of its
// blocks, and add their quarters in order through shared memory.  The split is
// a function of k alone and a column of the matrix instruction never sees its
// neighbours, so row i of the output has the same bits for every m.
#include "w4_core.cuh"

namespace mr {
namespace w4 {

// ---- packing --------------------------------------------------------------

// One warp lays out one block: lane 4g + t gathers, for rows g and g + 8, the
// words of k [32j + 8t, 32j + 8t + 8), j = 0..3.  Rows past the weight's and
// columns past k become zeros of weight (value 8 or zero point, scale 0).
__global__ void __launch_bounds__(256) pack_kernel(const uint8_t *__restrict__ q, const uint16_t *__restrict__ scales,
                                                   const uint8_t *__restrict__ zeros, uint8_t *__restrict__ packed,
                                                   int64_t total_blocks, int n, int k, int tiles,
                                                   int kblocks, uint32_t fmt, int paired) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = (int)(fmt & MR_W4_GROUP_MASK), groups = k / G, per_block = kBlockK / G;
    const int bb = block_bytes(fmt), half = n / 2;
    for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < total_blocks; b += (int64_t)gridDim.x * 8) {
        const int kb = (int)(b % kblocks);
        const int64_t tile_all = b / kblocks;
        const int tile = (int)(tile_all % tiles);
        const int64_t mat = tile_all / tiles;
        auto source_row = [&](int r) -> int64_t {  // row r of the tile in the weight, or -1
            if (paired) {
                const int j = tile * 8 + (r & 7);
                return j < half ? mat * n + (r < 8 ? j : half + j) : -1;
            }
            const int j = tile * kTileRows + r;
            return j < n ? mat * n + j : -1;
        };
        uint8_t *out = packed + b * bb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = source_row(g + 8 * h);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = kb * kBlockK + 32 * j + 8 * t;
                uint32_t v = 0x88888888u;
                if (row >= 0 && p < k) v = *reinterpret_cast<const uint32_t *>(q + row * (k / 2) + p / 2);
                // byte i: value 2i low, value 2i + 1 high -> nibbles i and 4 + i
                const uint32_t lo = v & 0x0F0F0F0Fu, hi = (v >> 4) & 0x0F0F0F0Fu;
                auto squeeze = [](uint32_t x) {
                    return (x & 0xFu) | ((x >> 4) & 0xF0u) | ((x >> 8) & 0xF00u) | ((x >> 12) & 0xF000u);
                };
                w[j] = squeeze(lo) | (squeeze(hi) << 16);
            }
            *reinterpret_cast<uint4 *>(out + 512 * h + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        for (int e = lane; e < per_block * kTileRows; e += 32) {
            const int64_t row = source_row(e % kTileRows);
            const int grp = kb * per_block + e / kTileRows;
            const bool in = row >= 0 && grp < groups;
            reinterpret_cast<uint16_t *>(out + kBlockQ)[e] = in ? scales[row * groups + grp] : (uint16_t)0;
            if (fmt & MR_W4_ZEROS)
                out[kBlockQ + 32 * per_block + e] = in ? (uint8_t)(zeros[row * groups + grp] & 15u) : (uint8_t)8;
        }
    }
}

// ---- product --------------------------------------------------------------

constexpr int kMaxRows = 16;
constexpr int kMaxK = 1 << 20;               // far beyond what shared memory holds
constexpr int kWarps = 8;
constexpr int kKW = 4;                       // warps that share a tile
constexpr int kWorkers = kWarps / kKW;
constexpr int kRedCol = 20;                  // floats between columns of a partial tile (no bank conflicts)
constexpr int kStages = 4;

struct Params {
    const uint8_t *A;
    int64_t lda;       // bytes
    const uint8_t *W;
    float *C;
    int64_t ldc;
    int m, n, k, tiles, kblocks, block;
    uint32_t fmt;
};

__host__ __device__ inline int x_stride(int kblocks) { return kblocks * kBlockK * 2 + 64; }  // odd multiple of 64
__host__ __device__ constexpr int red_floats(int NT) { return kWorkers * 2 * kKW * 8 * NT * kRedCol; }

inline size_t smem_bytes(int m, int kblocks, int block) {
    return (size_t)m * x_stride(kblocks) + (size_t)kWarps * kStages * block +
           sizeof(float) * red_floats(m > 8 ? 2 : 1);
}

template <int G, bool F16, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) gemv_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int worker = warp / kKW, slice = warp % kKW, g = lane >> 2, t = lane & 3;
    const int xs = x_stride(p.kblocks);
    const uint32_t x0 = smem_u32(smem);
    const uint32_t ring = x0 + p.m * xs + warp * kStages * p.block;
    float *red = reinterpret_cast<float *>(smem + p.m * xs + kWarps * kStages * p.block) +
                 worker * 2 * kKW * 8 * NT * kRedCol;
    grid_launch_dependents();

    // This warp's blocks: its quarter [kb0, kb1) of tile first, first + step, ...
    const int kb0 = p.kblocks * slice / kKW, kb1 = p.kblocks * (slice + 1) / kKW;
    const int first = blockIdx.x * kWorkers + worker, step = gridDim.x * kWorkers;
    int itile = first, ikb = kb0;  // the next block to request
    auto request = [&](int stage) {
        if (itile < p.tiles && kb0 < kb1) {
            issue_block(ring + stage * p.block, p.W + ((int64_t)itile * p.kblocks + ikb) * p.block, p.block, lane);
            if (++ikb == kb1) {
                ikb = kb0;
                itile += step;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) request(s);

    // The weight streams while the activations' producer finishes.
    grid_dependency_wait();
    const int chunks = p.kblocks * (kBlockK / 8), live = p.k / 8;
    for (int e = threadIdx.x; e < p.m * chunks; e += kWarps * 32) {
        const int r = e / chunks, c = e % chunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < live) v = *reinterpret_cast<const uint4 *>(p.A + r * p.lda + 16 * c);
        *reinterpret_cast<uint4 *>(smem + r * xs + 16 * c) = v;
    }
    __syncthreads();

    bool on[NT];
    uint32_t xb[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        on[c] = 8 * c + g < p.m;
        xb[c] = x0 + (on[c] ? 8 * c + g : 0) * xs + 16 * t;
    }
    int stage = 0, buf = 0;
    for (int tile = first; tile < p.tiles; tile += step) {
        float C[NT][4] = {};
        for (int kb = kb0; kb < kb1; ++kb) {
            cp_async_wait<kStages - 1>();
            __syncwarp();  // every lane's part of the block has arrived
            uint32_t x[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) x[c] = xb[c] + kb * (kBlockK * 2);
            consume_block<G, F16, NT>(ring + stage * p.block, p.fmt, x, on, C, lane);
            __syncwarp();  // every lane has read it
            request(stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        // Quarters in order.  Two buffers: a warp writes buffer b again only
        // after the barrier of the tile between, which the others reach after
        // reading b.
        float *mine = red + (buf * kKW + slice) * 8 * NT * kRedCol;
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            mine[(8 * c + 2 * t) * kRedCol + g] = C[c][0];
            mine[(8 * c + 2 * t + 1) * kRedCol + g] = C[c][1];
            mine[(8 * c + 2 * t) * kRedCol + g + 8] = C[c][2];
            mine[(8 * c + 2 * t + 1) * kRedCol + g + 8] = C[c][3];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "n"(kKW * 32) : "memory");
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const int col = 8 * c + (threadIdx.x % (kKW * 32)) / kTileRows, r = threadIdx.x % kTileRows;
            const float *from = red + buf * kKW * 8 * NT * kRedCol + col * kRedCol + r;
            float sum = from[0];
#pragma unroll
            for (int s = 1; s < kKW; ++s) sum += from[s * 8 * NT * kRedCol];
            const int row = tile * kTileRows + r;
            if (col < p.m && row < p.n) p.C[col * p.ldc + row] = sum;
        }
        buf ^= 1;
    }
}

template <int G, bool F16, int NT>
mr_status launch(const Params &p, size_t smem, uint32_t flags, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    auto kernel = gemv_kernel<G, F16, NT>;
    if (!allow_smem(kernel, ready)) return MR_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    const int per_sm = 2 * (smem + 1024) <= (size_t)mr_host::max_smem_optin() + 1024 ? 2 : 1;
    cfg.gridDim = dim3((unsigned)std::min((p.tiles + kWorkers - 1) / kWorkers, mr_host::sm_count() * per_sm));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (flags & MR_GEMV_PDL) ? 1 : 0;
    return mr_host::cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <int G>
mr_status launch_group(const Params &p, bool f16, size_t smem, uint32_t flags, cudaStream_t stream) {
    if (f16) return p.m > 8 ? launch<G, true, 2>(p, smem, flags, stream) : launch<G, true, 1>(p, smem, flags, stream);
    return p.m > 8 ? launch<G, false, 2>(p, smem, flags, stream) : launch<G, false, 1>(p, smem, flags, stream);
}

// MR_OK, or why a weight of n x k cannot be packed in this format.
mr_status check_format(int32_t n, int32_t k, uint32_t fmt) {
    const uint32_t G = fmt & MR_W4_GROUP_MASK;
    if (fmt & ~(MR_W4_GROUP_MASK | MR_W4_ZEROS | MR_W4_SCALE_F16)) return MR_ERR_INVALID_ARG;
    if (n < 1 || k < 1 || G == 0) return MR_ERR_INVALID_ARG;
    if (G != 32 && G != 64 && G != 128) return MR_ERR_UNSUPPORTED;
    if (k % (int)G) return MR_ERR_INVALID_ARG;
    return MR_OK;
}

int tiles_of(int32_t n, int32_t paired) { return paired ? (n / 2 + 7) / 8 : (int)(((int64_t)n + 15) / 16); }
int kblocks_of(int32_t k) { return (int)(((int64_t)k + kBlockK - 1) / kBlockK); }

}  // namespace w4
}  // namespace mr

extern "C" size_t w4_packed_bytes(int32_t n, int32_t k, uint32_t fmt, int32_t paired) {
    if (mr::w4::check_format(n, k, fmt) != MR_OK || (paired && n % 2)) return 0;
    return (size_t)mr::w4::tiles_of(n, paired) * mr::w4::kblocks_of(k) * mr::w4::block_bytes(fmt);
}

extern "C" mr_status w4_pack(const void *q, const void *scales, const void *zeros, void *packed, size_t packed_bytes,
                             int32_t count, int32_t n, int32_t k, uint32_t fmt, int32_t paired, void *stream) {
    if (!q || !scales || !packed || count < 1) return MR_ERR_INVALID_ARG;
    const mr_status st = mr::w4::check_format(n, k, fmt);
    if (st != MR_OK) return st;
    if (((fmt & MR_W4_ZEROS) != 0) != (zeros != nullptr)) return MR_ERR_INVALID_ARG;
    if (paired && n % 2) return MR_ERR_INVALID_ARG;
    if (packed_bytes / (size_t)count < w4_packed_bytes(n, k, fmt, paired)) return MR_ERR_INVALID_ARG;
    if (((uintptr_t)q & 3u) || ((uintptr_t)scales & 1u) || ((uintptr_t)packed & 15u)) return MR_ERR_MISALIGNED;
    const int tiles = mr::w4::tiles_of(n, paired), kblocks = mr::w4::kblocks_of(k);
    const int64_t blocks = (int64_t)count * tiles * kblocks;
    const int sms = mr_host::sm_count() > 0 ? mr_host::sm_count() : 148;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((blocks + 7) / 8, (int64_t)sms * 16));
    cfg.blockDim = dim3(256);
    cfg.stream = static_cast<cudaStream_t>(stream);
    return mr_host::cuda_status(cudaLaunchKernelEx(
        &cfg, mr::w4::pack_kernel, static_cast<const uint8_t *>(q), static_cast<const uint16_t *>(scales),
        static_cast<const uint8_t *>(zeros), static_cast<uint8_t *>(packed), blocks, (int)n, (int)k,
        tiles, kblocks, fmt, (int)(paired != 0)));
}

extern "C" mr_status mrgemv_w4(const void *A, int64_t lda, const void *packed, size_t packed_bytes, float *C,
                               int64_t ldc, int32_t m, int32_t n, int32_t k, int32_t in_dtype, uint32_t fmt,
                               uint32_t flags, void *stream) {
    if (!A || !packed || !C || m < 1) return MR_ERR_INVALID_ARG;
    if (in_dtype != MR_F16 && in_dtype != MR_BF16) return MR_ERR_INVALID_ARG;
    const mr_status st = mr::w4::check_format(n, k, fmt);
    if (st != MR_OK) return st;
    if (lda < k || ldc < n || (flags & ~MR_GEMV_PDL)) return MR_ERR_INVALID_ARG;
    if (packed_bytes < w4_packed_bytes(n, k, fmt, 0)) return MR_ERR_INVALID_ARG;
    if (((uintptr_t)A & 15u) || ((uintptr_t)packed & 15u) || ((uintptr_t)C & 3u) || lda % 8) return MR_ERR_MISALIGNED;
    if (m > mr::w4::kMaxRows || k > mr::w4::kMaxK) return MR_ERR_UNSUPPORTED;
    mr::w4::Params p;
    p.A = static_cast<const uint8_t *>(A);
    p.lda = 2 * lda;
    p.W = static_cast<const uint8_t *>(packed);
    p.C = C;
    p.ldc = ldc;
    p.m = m;
    p.n = n;
    p.k = k;
    p.tiles = mr::w4::tiles_of(n, 0);
    p.kblocks = mr::w4::kblocks_of(k);
    p.block = mr::w4::block_bytes(fmt);
    p.fmt = fmt;
    const size_t smem = mr::w4::smem_bytes(m, p.kblocks, p.block);
    const int optin = mr_host::max_smem_optin();
    if (smem > (size_t)(optin > 0 ? optin : 232448)) return MR_ERR_UNSUPPORTED;
    if (optin <= 0) return MR_ERR_CUDA;
    const bool f16 = in_dtype == MR_F16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (fmt & MR_W4_GROUP_MASK) {
        case 32: return mr::w4::launch_group<32>(p, f16, smem, flags, s);
        case 64: return mr::w4::launch_group<64>(p, f16, smem, flags, s);
        default: return mr::w4::launch_group<128>(p, f16, smem, flags, s);
    }
}
