// Shared pieces of the kernels that stream a weight past a few activation
// columns on mma.sync m16n8k16 (mrgemv_w4, moe_window_*).
//
// Orientation.  A tile is 16 weight rows (the M of the instruction); the
// activations of up to 8 tokens are its N columns.  The instruction's k index
// may be any permutation of the real one as long as both operands use the
// same: lane l = 4g + t takes, of every 32 consecutive k, the 8 values
// [8t, 8t + 8) of rows g and g + 8, and the same 8 values of column g.  Those
// are one 16-byte load per row and column, and they feed two instructions.
// Nothing is rearranged between memory and the tensor core.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"

namespace mr {
namespace w4 {

constexpr int kTileRows = 16;
constexpr int kBlockK = 128;        // k values of one packed block
constexpr int kBlockQ = 1024;       // bytes of a block's 4-bit values

// Bytes of one packed block (16 rows x 128 k) of format `fmt`: the values,
// 16 scales a group, and 16 zero points a group when the format has them.
__host__ __device__ inline int block_bytes(uint32_t fmt) {
    const int groups = kBlockK / (int)(fmt & MR_W4_GROUP_MASK);
    return kBlockQ + groups * 32 + ((fmt & MR_W4_ZEROS) ? groups * 16 : 0);
}

// ---- asynchronous copies into the issuing lane's own bytes ----------------

// 16 bytes, or zeros when !valid (nothing is read then).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// ---- the matrix instruction -----------------------------------------------

// d += a (16 x 16, row) . b (16 x 8, col), fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a . b
template <bool F16>
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---- 4-bit values ---------------------------------------------------------

// One word holds 8 values: nibble i is value 2i, nibble 4 + i is value 2i + 1.
// Pair i is (q - z) of both, exact: the nibble is put into the mantissa of 128
// (bf16) or 1024 (f16) and the zero point taken off again.  bf16: the low bits,
// whose spacing is 1, and -(128 + z) is added (`minus`, both halves).  f16 has room
// for a second nibble above (UPPER): the odd pairs become 1024 + 16 q, and a sixteenth
// of that minus 64 + z (`minus16`), which saves two of three shifts a word
// (131072 x 2560 at m = 4, G = 128: 40.3 -> 37.6 us) but needs a second constant a group
// (6144 x 2560 at m = 16, G = 32 with zero points: 7.4 -> 7.7), so groups of 32 go without.
// `one` is 128 or 1024 in both halves, kept in a register by `magic`: with mask
// and constant both known, the compiler emits two logic operations for the one.
template <bool F16>
__device__ __forceinline__ uint32_t magic(uint32_t fmt) {
    return (F16 ? 0x64006400u : 0x43004300u) + (fmt >> 31);  // no format has bit 31
}

struct Zero {
    uint32_t minus, minus16;
    template <bool F16>
    static __device__ __forceinline__ Zero of(uint32_t z) {
        return {z * 0x00010001u + (F16 ? 0xE400E400u : 0xC300C300u), z * 0x00100010u + 0xD400D400u};
    }
};

template <bool F16, bool UPPER>
__device__ __forceinline__ uint32_t pair(uint32_t word, int i, uint32_t one, const Zero &zero) {
    uint32_t v, r;
    if constexpr (F16) {
        const uint32_t w = UPPER ? word >> (8 * (i / 2)) : word >> (4 * i);
        if (UPPER && (i & 1)) {
            asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(v) : "r"(w), "r"(one));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x2C002C00u), "r"(zero.minus16));
        } else {
            asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(v) : "r"(w), "r"(one));
            asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero.minus));
        }
    } else {
        asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "r"(one));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x3F803F80u), "r"(zero.minus));
    }
    return r;
}

// A stored 16-bit scale in fp32 (exact).
__device__ __forceinline__ float scale_value(uint16_t bits, bool f16) {
    return f16 ? __half2float(__ushort_as_half(bits)) : __uint_as_float((uint32_t)bits << 16);
}

template <int BYTES>
struct Word;
template <>
struct Word<2> {
    static __device__ __forceinline__ void read(uint32_t addr, uint32_t (&w)[1]) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
        w[0] = v;
    }
};
template <>
struct Word<4> {
    static __device__ __forceinline__ void read(uint32_t addr, uint32_t (&w)[1]) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    }
};
template <>
struct Word<8> {
    static __device__ __forceinline__ void read(uint32_t addr, uint32_t (&w)[2]) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    }
};
template <>
struct Word<16> {
    static __device__ __forceinline__ void read(uint32_t addr, uint32_t (&w)[4]) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr)
                     : "memory");
    }
};

// C += (one packed block) . (the activation columns).  x[c] is the shared
// address of this lane's 16 bytes of column g of column tile c at the block's
// first k (a row of zeros where that column does not exist).  The values of a
// group are summed by the tensor core as small exact integers times the
// activations and take their scale once, in fp32: the sum of at most 128
// products is the longest chain of the matrix instruction's own additions,
// which round towards zero, so its error does not grow with k.
//
// What bounds it is issue: 134 instructions a block at NT = 1 and G = 128, 60 of
// them on the ALU pipe (7 shifts and masks for 8 values), 32 exact subtractions,
// and 8 matrix instructions that take about 7 slots each: 46 cycles a block with
// 16 warps on the SM, 60 at NT = 2 (57 and 74 for groups of 32 with zero points), where
// the HBM rate leaves a block 38 to 44.  A group of 128 runs as two chains of four
// instructions instead of one of eight.
template <int G, bool F16, int NT>
__device__ __forceinline__ void consume_block(uint32_t stage, uint32_t fmt, const uint32_t (&x)[NT],
                                              float (&C)[NT][4], int lane) {
    constexpr int kGroups = kBlockK / G, kChains = G >= 128 ? 2 : 1;
    const int g = lane >> 2;
    const uint32_t one = magic<F16>(fmt);
    const uint4 v0 = lds128(stage + 16 * lane), v8 = lds128(stage + 512 + 16 * lane);
    const uint32_t q0[4] = {v0.x, v0.y, v0.z, v0.w}, q8[4] = {v8.x, v8.y, v8.z, v8.w};
    // scales and zero points of rows g and g + 8, one read each
    uint32_t sw[kGroups], zw[(kGroups + 1) / 2];
    Word<4 * kGroups>::read(stage + kBlockQ + 4 * kGroups * g, sw);
    const bool sf16 = (fmt & MR_W4_SCALE_F16) != 0, zeros = (fmt & MR_W4_ZEROS) != 0;
    if (zeros) Word<2 * kGroups>::read(stage + kBlockQ + 32 * kGroups + 2 * kGroups * g, zw);
    auto scale_of = [&](int i) {  // i: half * kGroups + group
        return scale_value((uint16_t)(sw[i / 2] >> (16 * (i & 1))), sf16);
    };
    auto zero_of = [&](int i) { return Zero::of<F16>((zw[i / 4] >> (8 * (i & 3))) & 0xFFu); };
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
        Zero z0 = Zero::of<F16>(8u), z8 = z0;
        if (zeros) {
            z0 = zero_of(gi);
            z8 = zero_of(kGroups + gi);
        }
        float acc[kChains][NT][4];
#pragma unroll
        for (int j = gi * (G / 32); j < (gi + 1) * (G / 32); ++j) {
            uint32_t a0[4], a8[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a0[i] = pair<F16, (G > 32)>(q0[j], i, one, z0);
                a8[i] = pair<F16, (G > 32)>(q8[j], i, one, z8);
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const uint4 b = lds128(x[c] + 64 * j);
                if (j == gi * (G / 32))
                    mma_first<F16>(acc[0][c], a0[0], a8[0], a0[1], a8[1], b.x, b.y);
                else
                    mma<F16>(acc[0][c], a0[0], a8[0], a0[1], a8[1], b.x, b.y);
                if (kChains > 1 && j == gi * (G / 32))
                    mma_first<F16>(acc[kChains - 1][c], a0[2], a8[2], a0[3], a8[3], b.z, b.w);
                else
                    mma<F16>(acc[kChains - 1][c], a0[2], a8[2], a0[3], a8[3], b.z, b.w);
            }
        }
        const float s0 = scale_of(gi), s8 = scale_of(kGroups + gi);
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float sum = kChains > 1 ? acc[0][c][e] + acc[kChains - 1][c][e] : acc[0][c][e];
                C[c][e] = fmaf(e < 2 ? s0 : s8, sum, C[c][e]);
            }
    }
}

// ---- the same for a bf16 weight in row-major order ------------------------

constexpr int kBlockBf16 = kTileRows * kBlockK * 2;

// Request 16 rows x 128 k: `row0` and `row8` are this lane's rows g and g + 8
// at the block's first k (on0 / on8: whether they exist), `live` the k values
// left in the row.  Every lane copies exactly the bytes that it reads back.
__device__ __forceinline__ void issue_block_bf16(uint32_t stage, const uint16_t *row0, const uint16_t *row8, bool on0,
                                                 bool on8, int live, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = 32 * j + 8 * t;
        const bool in = p < live;
        cp_async16_zfill(stage + (2 * j) * 512 + 16 * lane, in && on0 ? row0 + p : row0, in && on0);
        cp_async16_zfill(stage + (2 * j + 1) * 512 + 16 * lane, in && on8 ? row8 + p : row0, in && on8);
    }
}

// C += (the block) . (the activation columns); the tensor core's own sums end
// with the block, as in consume_block.
template <int NT>
__device__ __forceinline__ void consume_block_bf16(uint32_t stage, const uint32_t (&x)[NT], float (&C)[NT][4],
                                                   int lane) {
    float acc[2][NT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v0 = lds128(stage + (2 * j) * 512 + 16 * lane);
        const uint4 v8 = lds128(stage + (2 * j + 1) * 512 + 16 * lane);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const uint4 b = lds128(x[c] + 64 * j);
            if (j == 0) {
                mma_first<false>(acc[0][c], v0.x, v8.x, v0.y, v8.y, b.x, b.y);
                mma_first<false>(acc[1][c], v0.z, v8.z, v0.w, v8.w, b.z, b.w);
            } else {
                mma<false>(acc[0][c], v0.x, v8.x, v0.y, v8.y, b.x, b.y);
                mma<false>(acc[1][c], v0.z, v8.z, v0.w, v8.w, b.z, b.w);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) C[c][i] += acc[0][c][i] + acc[1][c][i];
}

// ---- a warp's ring of packed blocks ---------------------------------------

// `slots` stages of up to `per` consecutive blocks, each filled by one bulk copy
// that lane 0 requests and an mbarrier counts.  Requests and takes go through
// the stages in the same order; a stage is requested again only after every
// lane has read it (__syncwarp), so a wait is never more than one phase ahead.
struct Ring {
    uint32_t data, bars;
    int slots, stage_bytes;
    int put_at = 0, take_at = 0;
    uint32_t parity = 0;
    bool dead = false;  // a wait ran out: no more are tried, and nothing more is requested
    __device__ __forceinline__ Ring(uint32_t d, uint32_t b, int n, int bytes)
        : data(d), bars(b), slots(n), stage_bytes(bytes) {}
    __device__ __forceinline__ void init(int lane) const {
        if (lane == 0) {
            for (int i = 0; i < slots; ++i) mbar_init(bars + 8 * i, 1);
            fence_mbar_init();
        }
        __syncwarp();
    }
    __device__ __forceinline__ void request(const uint8_t *src, int bytes, int lane) {
        if (lane == 0 && !dead) {
            mbar_arrive_expect_tx(bars + 8 * put_at, (uint32_t)bytes);
            bulk_g2s(data + put_at * stage_bytes, src, (uint32_t)bytes, bars + 8 * put_at);
        }
        put_at = put_at + 1 == slots ? 0 : put_at + 1;
    }
    __device__ __forceinline__ uint32_t wait() {  // the next stage, once its bytes have arrived
        if (!dead && !mbar_wait_bounded(bars + 8 * take_at, parity, MR_DEVERR_GEMV_TIMEOUT)) {
            dead = true;
            drain();
        }
        return data + take_at * stage_bytes;
    }
    // After a wait that ran out: a bounded one for each copy on its way, this one's too, so that
    // none lands in shared memory that the CTA has left.
    __device__ __forceinline__ void drain() const {
        int at = take_at, count = put_at > take_at ? put_at - take_at : put_at - take_at + slots;
        uint32_t phase = parity;
#pragma unroll 1
        for (; count > 0; --count) {
            mbar_wait_bounded(bars + 8 * at, phase, MR_DEVERR_GEMV_TIMEOUT);
            if (++at == slots) {
                at = 0;
                phase ^= 1u;
            }
        }
    }
    __device__ __forceinline__ void done() {  // this lane has read the stage
        __syncwarp();
        if (++take_at == slots) {
            take_at = 0;
            parity ^= 1u;
        }
    }
};

// ---- quarters of k ---------------------------------------------------------

// k is summed in kKW = 4 quarters of its blocks, added in order: the split that
// lets four warps share a tile, kept by a warp that has a tile to itself, so
// that an output's bits do not depend on which of the two it was.
constexpr int kKW = 4;
__device__ __forceinline__ int quarter_begin(int kblocks, int q) { return kblocks * q / kKW; }

// S = the quarters of blocks [begin, end) of a tile, in order; `request` asks
// for the blocks that follow, a stage at a time.
template <int G, bool F16, int NT, class Request>
__device__ __forceinline__ void sum_quarters(Ring &ring, Request &request, int kblocks, int begin, int end, int per,
                                             int block, uint32_t fmt, const uint32_t (&xb)[NT], float (&S)[NT][4],
                                             int lane) {
    float C[NT][4] = {};
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[c][e] = 0.0f;
    int q = 0, close = 0;  // the quarter's end
    auto next = [&](int kb) {
        while (close <= kb && q < kKW) close = quarter_begin(kblocks, ++q);
    };
    next(begin);
    for (int kb = begin; kb < end; kb += per) {
        uint32_t at = ring.wait();
        const int stop = min(kb + per, end);
#pragma unroll 1
        for (int b = kb; b < stop; ++b, at += block) {
            uint32_t x[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) x[c] = xb[c] + b * (kBlockK * 2);
            consume_block<G, F16, NT>(at, fmt, x, C, lane);
            if (b + 1 == close) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[c][e] += C[c][e];
                        C[c][e] = 0.0f;
                    }
                next(b + 1);
            }
        }
        ring.done();
        request();
    }
}

// Allow `kernel` all the shared memory the device offers, once per device.
template <class K>
bool allow_smem(K kernel, std::atomic<uint64_t> &done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, mr_host::max_smem_optin()) !=
        cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

}  // namespace w4
}  // namespace mr
