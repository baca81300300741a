// qk_attn_chunk.cuh -- what the two many-row forms of attention over the 4-bit
// cache share: accesses to shared memory, the work of a thread block, a row's
// state, outputs, and the join of the parts of a head's splits.
#pragma once

#include <atomic>

#include "qk_attn.cuh"
#include "qk_internal.h"
#include "qk_tc.cuh"

namespace qk {
namespace chunk {
using namespace attn;

constexpr int kTile = 64;                  // keys a tile
constexpr int kTileBlocks = kTile / kBlockTokens;
constexpr float kMost = 16384.0f;          // the largest P, and sum of 16
constexpr float kFresh = 4.0f;             // and of a row's largest when its reference moves

// One operand row's 16-byte chunk (8 elements from element 8 * c) in 128-byte swizzle.
__device__ __forceinline__ uint32_t operand_chunk(int row, int c, int rows)
{
    return static_cast<uint32_t>((c >> 3) * rows * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t a)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr)
{
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void lds128(uint32_t (&w)[4], uint32_t addr)
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
}

// a * b + c on fp16 pairs, rounded once, subnormals kept.
__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

__device__ __forceinline__ void lds64(uint32_t &a, uint32_t &b, uint32_t addr)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}

// N neighbouring words by the widest load that N allows.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr)
{
    if constexpr (N == 4) {
        lds128(w, addr);
    } else if constexpr (N == 2) {
        lds64(w[0], w[1], addr);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = lds32(addr + 4 * i);
    }
}

// One thread of the warp, the same each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A wait whose outcome the whole warp shares (a limit may run out for one lane and not another).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit_ns));
}

// A 16-bit element's value.
__device__ __forceinline__ float float_of(uint32_t bits, bool bf16)
{
    return bf16 ? __uint_as_float(bits << 16) : half_bits_to_float(bits);
}

// Two values as a pair of 16-bit elements.
__device__ __forceinline__ uint32_t pack_as(float lo, float hi, bool bf16)
{
    if (!bf16) return pack_half(lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Splits of a head that have blocks, at least one: each takes the same number.
__device__ __forceinline__ int active_splits(const AttnArgs &a, int blocks)
{
    const int per = max((blocks + a.splits - 1) / a.splits, a.min_blocks);
    return blocks > per ? (blocks + per - 1) / per : 1;
}

// What a thread block works on.
struct Work {
    int64_t b;
    int hk, tile, split;
    Sequence seq;
    Span span;
    int n, first, rows;          // rows of the sequence and head; this block's
    int active;                  // splits with blocks (at least one)
    int nblk, ntiles;            // 16-token blocks and key tiles of this split
    int64_t blk0;                // its first block in the sequence
    int two;                     // both row tiles hold rows
};

// One row's state.
struct Row {
    float m, l, to_log2;
    int lo, hi;
};

// This thread block's work: split, head, row tile, sequence.  False where it has none.
__device__ __forceinline__ bool find_work(const AttnArgs &a, int tile_rows, int D, Work &w)
{
    int64_t u = blockIdx.x;
    w.split = static_cast<int>(u % a.splits);
    u /= a.splits;
    w.hk = static_cast<int>(u % a.n_kv);
    u /= a.n_kv;
    w.tile = static_cast<int>(u % a.tiles);
    w.b = u / a.tiles;
    w.seq = sequence_of(a, w.b);
    if (w.seq.bad) {
        if (w.split == 0) poison_rows(a, w.seq, w.hk, w.tile, a.rep * D);
        return false;
    }
    w.n = static_cast<int>(w.seq.r1 - w.seq.r0) * a.rep;
    w.first = w.tile * tile_rows;
    if (w.first >= w.n) return false;
    w.rows = min(tile_rows, w.n - w.first);
    w.two = w.rows > 128;
    w.span = span_of(a, w.seq, w.first, w.rows);
    const int per = max((w.span.blocks + a.splits - 1) / a.splits, a.min_blocks);
    w.active = active_splits(a, w.span.blocks);
    if (w.split >= w.active) return false;
    const int b0 = w.split * per;
    w.nblk = min(w.span.blocks - b0, per);
    w.ntiles = (w.nblk + kTileBlocks - 1) / kTileBlocks;
    w.blk0 = w.span.blk_lo + b0;
    return true;
}

// 16 channels of a row out; wide: 16 bytes an access.
__device__ __forceinline__ void store16(const AttnArgs &a, int64_t to, const float (&x)[16], bool wide)
{
    if (!wide) {
#pragma unroll
        for (int i = 0; i < 16; ++i) store_float_as(a.out, to + i, a.out_type, x[i]);
    } else if (a.out_type == QK_F32) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
        const bool bf16 = a.out_type == QK_BF16;
#pragma unroll
        for (int i = 0; i < 16; i += 8)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + to + i) =
                make_uint4(pack_as(x[i], x[i + 1], bf16), pack_as(x[i + 2], x[i + 3], bf16), pack_as(x[i + 4], x[i + 5], bf16),
                           pack_as(x[i + 6], x[i + 7], bf16));
    }
}

// Launches the tiles' kernel and, where heads are split, the join of their parts.
cudaError_t launch_tiles(void (*kern)(const AttnArgs), std::atomic<uint64_t> &done, int smem, int threads, const AttnArgs &a, int D,
                         int rows, int64_t groups, cudaStream_t st);

}  // namespace chunk
}  // namespace qk
