// qk_attn.cuh -- what the two forms of attention over the 4-bit cache share.
#pragma once

#include "qk_device.cuh"
#include "qk_kv4.cuh"

namespace qk {
namespace attn {

constexpr float kNoMax = -3.0e38f;      // a row's reference before it has seen a key

struct AttnArgs {
    const uint8_t *pages;
    int64_t n_pages;
    int n_kv, page_blocks, rep;      // page_blocks: 16-token blocks a page
    const void *q;
    int64_t ldq;
    int q_type;
    const int32_t *page_table;
    int64_t ld_pages, max_pages;
    const int32_t *lens, *q_start;
    int64_t T, max_q, window;
    float scale_log2;                // scale * log2(e)
    void *out;
    int64_t ldo;
    int out_type;
    int tiles, items;                // row tiles a sequence, and of all sequences
    int cut;                         // thread blocks that cut heads share (0: one a head and item)
    int sms;
    int *counters;
    float *parts;
    void *plan;                      // many rows: how the blocks are shared out
    int *err;
    uint64_t wait_ns;
    int skip_block;                  // test hook: this block of thread block 0 (its first warp's) is never copied
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// n - 8 as an fp16 pair, of nibble AT (0 or 1) of both halves of a word: the nibble in the mantissa of 1024 (where
// the lowest bit counts 1) or of 64 (where bit 4 does), less the constant.
template <int AT>
__device__ __forceinline__ uint32_t signed_nibbles(uint32_t w)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(AT ? 0x00F000F0 : 0x000F000F), "n"(AT ? 0x54005400 : 0x64006400));
    const uint32_t bias = AT ? 0x54805480u : 0x64086408u;   // 72, 1032
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&r), *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// A call's rows and keys as a thread block sees them.
struct Sequence {
    int64_t r0, r1;       // its query rows
    int64_t len;
    bool bad;             // an index out of range
};
__device__ __forceinline__ Sequence sequence_of(const AttnArgs &a, int64_t b)
{
    Sequence s;
    s.r0 = b * a.max_q, s.r1 = s.r0 + a.max_q;
    if (a.q_start) s.r0 = a.q_start[b], s.r1 = a.q_start[b + 1];
    s.len = a.lens[b];
    s.bad = s.r0 < 0 || s.r1 > a.T || s.r1 < s.r0 || s.r1 - s.r0 > a.max_q || s.len < 0 ||
            s.len > a.max_pages * a.page_blocks * kBlockTokens;
    return s;
}

// Every row that q_start names becomes NaN, shared out over the row tiles.
__device__ __forceinline__ void poison_rows(const AttnArgs &a, const Sequence &s, int hk, int tile, int width)
{
    if (threadIdx.x == 0 && tile == 0) record_error(a.err, kErrBadIndex);
    for (int64_t row = (s.r0 < 0 ? 0 : s.r0) + tile; row < (s.r1 > a.T ? a.T : s.r1); row += a.tiles)
        for (int i = threadIdx.x; i < width; i += blockDim.x)
            store_float_as(a.out, row * a.ldo + static_cast<int64_t>(hk) * width + i, a.out_type,
                           __int_as_float(0x7FC00000));
}

// The 16-token blocks that the rows [first, first + rows) of a sequence see.
struct Span {
    int64_t pos0, pos1;          // positions of the first and the last row
    int64_t key_lo, key_hi;      // keys that some row sees
    int64_t blk_lo;
    int blocks;                  // at most 2^27: lengths are below 2^31
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, const Sequence &s, int first, int rows)
{
    Span p;
    p.pos0 = s.len - (s.r1 - s.r0) + first / a.rep, p.pos1 = s.len - (s.r1 - s.r0) + (first + rows - 1) / a.rep;
    p.key_lo = a.window > 0 && p.pos0 - a.window + 1 > 0 ? p.pos0 - a.window + 1 : 0;
    p.key_hi = p.pos1 + 1 > 0 ? p.pos1 + 1 : 0;
    p.blk_lo = p.key_lo / kBlockTokens;
    p.blocks = p.key_hi > p.key_lo ? static_cast<int>((p.key_hi + kBlockTokens - 1) / kBlockTokens - p.blk_lo) : 0;
    return p;
}

__device__ __forceinline__ int clamp_key(int64_t k) { return static_cast<int>(k < -1 ? -1 : (k > INT32_MAX ? INT32_MAX : k)); }

// Thread blocks an SM holds of the few-row form: two (128 registers a thread), one where accumulators and queries
// need more.
constexpr int kWarps = 8;
__host__ __device__ constexpr int rows_blocks_per_sm(int G, int NT) { return G <= 4 && NT <= 2 ? 2 : 1; }
constexpr int kRowItems = 512;           // row tiles of all sequences whose heads may be split

// The few-row form (qk_attn_rows.cuh), by head size: rows of `pieces` fp16 pieces in `sets` sets of 8 columns.
cudaError_t rows_launch_64(const AttnArgs &a, int pieces, int sets, int64_t grid, cudaStream_t st);
cudaError_t rows_launch_96(const AttnArgs &a, int pieces, int sets, int64_t grid, cudaStream_t st);
cudaError_t rows_launch_128(const AttnArgs &a, int pieces, int sets, int64_t grid, cudaStream_t st);
cudaError_t rows_launch_256(const AttnArgs &a, int pieces, int sets, int64_t grid, cudaStream_t st);

// The many-row forms, on the 5th-generation tensor cores: tiles of kChunkRows rows in bf16 (qk_attn_chunk.cu), of
// kChunkRows32 in fp32 and fp16 (qk_attn_chunk32.cu).
constexpr int kChunkRows = 256, kChunkRows32 = 128;
cudaError_t chunk_launch(const AttnArgs &a, int D, int64_t groups, cudaStream_t st);
cudaError_t chunk32_launch(const AttnArgs &a, int D, int64_t groups, cudaStream_t st);
__host__ __device__ inline int64_t chunk_part_bytes(int D, int rows)
{
    return (static_cast<int64_t>(rows) * D + 2 * rows) * 4;
}

}  // namespace attn
}  // namespace qk
