// w4_pack and mrgemv_w4: multi-row product with a 4-bit weight, fp32 output.
//
//   C[i][j] = sum_groups s[j][grp] * sum_{p in grp} A[i][p] * (q[j][p] - z[j][grp])
//
// The weight is read once for all m <= 16 rows, like mrgemv_bf16's.  At the
// HBM rate an SM receives about 46 values a clock, so neither conversions nor
// FMAs fit on the CUDA cores for more than a row or two: the values are
// unpacked to exact small integers and multiplied on the tensor core, 256
// values x 8 rows an instruction.  131072 x 2560 at m = 4: 40.4 us, 4.3 TB/s of
// weight; bound by issue (consume_block).  512 x 2560 at m = 1: 4.0 us, 2.9 in a
// programmatic chain (mrgemv_bf16 there: 3.9 and 2.2): 32 tiles keep 16 CTAs, and
// the rows arrive before any block is taken.
//
// Work: a tile is 16 weight rows, one contiguous run of the packed weight, and
// its k is summed in quarters, added in order.  As many tiles as fill whole
// rounds of all the grid's warps go one to a warp, which then never waits for
// another; the rest, and all of a narrow weight's, go to four warps each, a
// quarter to a warp, joined through shared memory (131072 x 2560, m = 4: 46.0 us
// with every tile in quarters).  The quarters are a function of k alone and a
// column of the matrix instruction never sees its neighbours, so row i of the
// output has the same bits for every m.
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
        for (int e = lane; e < per_block * kTileRows; e += 32) {  // [g][half][group]
            const int64_t row = source_row(e / (2 * per_block) + 8 * (e / per_block % 2));
            const int grp = kb * per_block + e % per_block;
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

struct Params {
    const uint8_t *A;
    int64_t lda;       // bytes
    const uint8_t *W;
    float *C;
    int64_t ldc;
    int m, n, k, tiles, kblocks, block;
    int per, slots;    // blocks of a ring stage, stages of a warp's ring
    uint32_t fmt;
};

// Bytes between activation rows in shared memory: an odd multiple of 64, so
// that the eight 16-byte pieces of a load phase (two rows) miss no bank twice.
__host__ __device__ inline int64_t x_stride(int kblocks) { return (int64_t)kblocks * kBlockK * 2 + 64; }
// The quarters of a tile on their way to the first warp: two buffers of three.
__host__ __device__ constexpr int red_bytes(int warps, int NT) { return warps / kKW * 2 * (kKW - 1) * NT * 512; }

template <int G, bool F16, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) gemv_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int worker = warp / kKW, slice = warp % kKW, g = lane >> 2, t = lane & 3;
    const int xs = (int)x_stride(p.kblocks), x_bytes = (p.m + 1) * xs;
    const uint32_t x0 = smem_u32(smem), red = x0 + x_bytes + worker * 2 * (kKW - 1) * NT * 512;
    const uint32_t ring0 = x0 + x_bytes + red_bytes(WARPS, NT);
    const int ring_bytes = p.slots * p.per * p.block;
    Ring ring(ring0 + warp * ring_bytes, ring0 + WARPS * ring_bytes + warp * p.slots * 8, p.slots, p.per * p.block);
    ring.init(lane);

    // Items: whole tiles [0, whole), then quarters of the others.  A warp takes
    // item `first`, first + step, ...; step and `whole` are multiples of four,
    // so the quarters of a tile are four neighbouring warps'.
    const int first = blockIdx.x * WARPS + warp, step = gridDim.x * WARPS;
    const int whole = p.tiles / step * step;
    // The next request: `rleft` blocks from rsrc on, then item ritem.
    const int64_t tile_bytes = (int64_t)p.kblocks * p.block;
    const int qb = quarter_begin(p.kblocks, slice), qe = quarter_begin(p.kblocks, slice + 1);
    int ritem = first, rleft = 0;
    const uint8_t *rsrc = nullptr;
    auto request = [&]() {
        while (rleft == 0) {
            if (ritem < whole) {
                rsrc = p.W + ritem * tile_bytes;
                rleft = p.kblocks;
            } else {
                const int tile = whole + (ritem - whole) / kKW;
                if (tile >= p.tiles) return;
                rsrc = p.W + tile * tile_bytes + qb * p.block;
                rleft = qe - qb;
            }
            ritem += step;
        }
        const int count = min(p.per, rleft);
        ring.request(rsrc, count * p.block, lane);
        rsrc += count * p.block;
        rleft -= count;
    };
    for (int s = 0; s < p.slots; ++s) request();

    // The weight streams while the activations' producer finishes.
    grid_dependency_wait();
    // After the wait: the next kernel may read ahead a weight that the one before this wrote (and chains of
    // narrow products are faster than with the trigger at entry: 512 x 2560, m = 1 2.9 us against 3.1).
    grid_launch_dependents();
    const int chunks = p.kblocks * (kBlockK / 8), live = p.k / 8;
    for (int r = warp; r <= p.m; r += WARPS)
        for (int c = lane; c < chunks; c += 32) {
            const bool in = r < p.m && c < live;
            cp_async16_zfill(x0 + r * xs + 16 * c, in ? p.A + r * p.lda + 16 * c : p.A, in);
        }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();

    uint32_t xb[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) xb[c] = x0 + min(8 * c + g, p.m) * xs + 16 * t;
    auto store = [&](int tile, const float (&S)[NT][4]) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = 8 * c + 2 * t + (e & 1), row = tile * kTileRows + g + 8 * (e >> 1);
                if (col < p.m && row < p.n) p.C[col * p.ldc + row] = S[c][e];
            }
    };
    int item = first;
    for (; item < whole; item += step) {
        float S[NT][4];
        sum_quarters<G, F16, NT>(ring, request, p.kblocks, 0, p.kblocks, p.per, p.block, p.fmt, xb, S, lane);
        store(item, S);
    }
    int buf = 0;
    for (int tile; (tile = whole + (item - whole) / kKW) < p.tiles; item += step) {
        float S[NT][4];
        sum_quarters<G, F16, NT>(ring, request, p.kblocks, qb, qe, p.per, p.block, p.fmt, xb, S, lane);
        // The first warp adds the quarters in order.  Two buffers: a warp
        // writes one again only after the barrier of the tile between, which
        // the first warp reaches after reading it.
        const uint32_t part = red + buf * (kKW - 1) * NT * 512 + 16 * lane;
        if (slice) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(part + ((slice - 1) * NT + c) * 512),
                             "f"(S[c][0]), "f"(S[c][1]), "f"(S[c][2]), "f"(S[c][3])
                             : "memory");
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "n"(kKW * 32) : "memory");
        if (slice == 0) {
#pragma unroll
            for (int s = 0; s < kKW - 1; ++s)
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const uint4 v = lds128(part + (s * NT + c) * 512);
                    S[c][0] += __uint_as_float(v.x);
                    S[c][1] += __uint_as_float(v.y);
                    S[c][2] += __uint_as_float(v.z);
                    S[c][3] += __uint_as_float(v.w);
                }
            store(tile, S);
        }
        buf ^= 1;
    }
}

// Shared memory and the launch's shape.  Two CTAs of 8 warps share an SM when
// the activations leave each of them 40 KB of ring (the next launch's CTA then
// also finds room under programmatic launch); otherwise, or where every warp gets
// two tiles or more, one of 16 warps, whose rings are longer as the activations
// are there once (131072 x 2560, m = 4: 42.2 and 40.3 us).  A stage holds a warp's
// whole quarter of a tile where two of them fit (five blocks a stage there; with
// three 42.8 us, with two 45.1).
struct Plan {
    int warps = 0;
    size_t smem = 0;
};

Plan plan(Params &p, size_t optin) {
    Plan out;
    const int NT = p.m > 8 ? 2 : 1, quarter = (p.kblocks + kKW - 1) / kKW;
    const bool deep = p.tiles >= 2 * 16 * mr_host::sm_count();
    for (int warps : {8, 16}) {
        if (warps == 8 && deep) continue;
        const size_t limit = warps == 8 ? (optin + 1024) / 2 - 1024 : optin;
        const size_t fixed = (size_t)(p.m + 1) * x_stride(p.kblocks) + red_bytes(warps, NT) + 8 * 4 * warps;
        if (fixed + (warps == 8 ? 40 * 1024 : 2 * warps * p.block) > limit) continue;
        const int blocks = (int)((limit - fixed) / warps / p.block);  // a warp's ring, at least 2
        p.per = std::min(quarter, blocks / 2);
        p.slots = std::min(4, blocks / p.per);
        out.warps = warps;
        out.smem = fixed + (size_t)warps * p.slots * p.per * p.block;
        return out;
    }
    return out;
}

template <int G, bool F16, int NT, int WARPS>
mr_status launch(const Params &p, const Plan &pl, uint32_t flags, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    auto kernel = gemv_kernel<G, F16, NT, WARPS>;
    if (!allow_smem(kernel, ready)) return MR_ERR_CUDA;
    constexpr int kWorkers = WARPS / kKW;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min((p.tiles + kWorkers - 1) / kWorkers, mr_host::sm_count() * (16 / WARPS)));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (flags & MR_GEMV_PDL) ? 1 : 0;
    return mr_host::cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <int G, bool F16>
mr_status launch_rows(const Params &p, const Plan &pl, uint32_t flags, cudaStream_t stream) {
    if (p.m > 8)
        return pl.warps == 8 ? launch<G, F16, 2, 8>(p, pl, flags, stream) : launch<G, F16, 2, 16>(p, pl, flags, stream);
    return pl.warps == 8 ? launch<G, F16, 1, 8>(p, pl, flags, stream) : launch<G, F16, 1, 16>(p, pl, flags, stream);
}

template <int G>
mr_status launch_group(const Params &p, const Plan &pl, bool f16, uint32_t flags, cudaStream_t stream) {
    return f16 ? launch_rows<G, true>(p, pl, flags, stream) : launch_rows<G, false>(p, pl, flags, stream);
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
    const int optin = mr_host::max_smem_optin();
    const mr::w4::Plan pl = mr::w4::plan(p, (size_t)(optin > 0 ? optin : 232448));
    if (!pl.warps) return MR_ERR_UNSUPPORTED;
    if (optin <= 0) return MR_ERR_CUDA;
    const bool f16 = in_dtype == MR_F16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (fmt & MR_W4_GROUP_MASK) {
        case 32: return mr::w4::launch_group<32>(p, pl, f16, flags, s);
        case 64: return mr::w4::launch_group<64>(p, pl, f16, flags, s);
        default: return mr::w4::launch_group<128>(p, pl, f16, flags, s);
    }
}
