// qk_moe.cuh -- what the kernels of the experts' feed-forward products share:
// the call's sizes, the plan that groups the assignments by expert, and the
// operands' layout.
//
// An assignment is a place (t, j) of ids [T][top_k].  The plan sorts the live
// ones by expert (stable, so nothing depends on the order of atomics); `place`
// is an assignment's place in that order.  Eight neighbouring places of one
// expert are an octet, the 8 columns of an m16n8k16 product, and up to kSetOctets
// octets a set, the columns that share one pass over the expert's weights.
//
// Operands: a row x is held as fp16 pieces hi + lo of x * 2^e, 2^e the power of
// two that puts the row's largest magnitude into [2^14, 2^15): a value is then
// exact to 2^-23 of itself, or to 2^-39 of the row's largest.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_kv4.cuh"

namespace qk {
namespace moe {

constexpr int kMaxExperts = 1024;
constexpr int kSetOctets = 2;
constexpr int kTileBoxRows = 32;                  // rows of a TMA box of a tile set's operands
constexpr int kRowWarps = 16;                     // warps of a thread block of the few-token products
// Assignments up to which no plan is made (qk_moe_few.cuh), which reads an expert again for each of its tokens.  8 of
// 128 experts of 768 x 2048, Q4_K and Q6_K, calls one after another in a graph: one token 19.3 us, with the plan 38.2; three
// 50.2 and 59.6; four 63.6 and 66.9, five 82.2 and 68.4; where 8 experts have all tokens three take 48.6 and 40.1.
constexpr int kMaxFew = 24;
constexpr int kMaxFewCols = 8192;                 // a row of x has to fit into shared memory
constexpr int kUnit = 256;                        // columns of a unit of the products' loops
constexpr int kPieceBytes = 8 * 32 * 16;          // an octet's unit, one piece: 8 steps of 16 bytes a lane
constexpr int kSumBytes = 32 * 8;                 // the sums of its sub-blocks (Q4_K)

struct ExpertSet {
    int expert, first, count, octet;              // first place, places, first octet
};

struct Plan {
    int *head;                // [0] sets, [1] tile sets, [2] live places
    int *place;               // [A] place of an assignment; -1 none, -2 an id out of range
    int *column;              // [A] octet * 8 + column of a place; -1: of a tile set
    ExpertSet *sets;
    ExpertSet *tile_sets;     // (octet is not used)
};

// Expert e's row r is row `first_row + e * expert_rows + r` of w.
struct Weights {
    const uint8_t *w;
    int64_t expert_rows, row_bytes;
};

// Rows [A or T][ld] to operands.
struct PackArgs {
    Plan plan;
    const void *x;
    int64_t ld;
    int type, top_k;          // row of a place: x[assignment / top_k], or x[place] where top_k == 0
    int64_t tokens;
    bool vec;                 // rows start on four values
    int cols, units, pieces, fmt;
    uint8_t *out;
    __half *tile_out;         // rows of the tile sets, hi pieces [place][tile_cols]; lo ones tile_lo further
    int64_t tile_lo;
    int tile_cols;
    float *scale;             // [place] 2^-e
};

struct RowsArgs {
    Plan plan;
    Weights a, b;             // gate and up; or down twice
    int cols, units, pieces;
    int rows, tiles;          // output columns and 16-row tiles (8 + 8 where gate and up are paired)
    int sms;
    const uint8_t *x;         // operands, octet after octet
    const float *scale;
    float *out;               // [place][rows]
    uint64_t wait_ns;
    int *err;
};

struct TileArgs {
    Plan plan;
    Weights a, b;             // as above
    int cols, chunks, pieces, w_pieces;      // chunks: stages of a row
    int rows, tiles;          // output columns and 128-row tiles (64 + 64 where paired)
    const float *scale;
    float *out;
    int skip_chunk;           // test hook: the first cluster never loads this chunk of its (-1: none)
    uint64_t wait_ns;
    int *err;
};

// The two launches of few assignments.
struct FewArgs {
    const int32_t *ids;
    int experts, top_k;
    Weights a, b;             // gate and up; or down
    int cols, rows;
    const void *x;
    int64_t ldx;
    int x_type;
    bool vec;                 // rows of x start on four values
    float *h;                 // [assignment], groups of 16
    const float *weights;
    void *y;
    int64_t ldy;
    int y_type;
    int *err;
};

// The tokens' operands: rows [rows][cols] of fp16 pieces.
struct TileOperands {
    const void *hi, *lo;
    int64_t rows, cols;
};

__host__ __device__ constexpr int64_t octet_unit_bytes(int fmt, int pieces)
{
    return pieces * kPieceBytes + (fmt == kFmtQ4K ? kSumBytes : 0);
}
__host__ __device__ constexpr int unit_bytes(int fmt) { return fmt == kFmtQ4K ? 144 : fmt == kFmtQ80 ? 272 : 210; }
__host__ __device__ inline int64_t row_bytes_of(int fmt, int64_t K)
{
    return fmt == kFmtQ80 ? (K + 31) / 32 * 34 : (K + 255) / 256 * unit_bytes(fmt);
}

cudaError_t few_gate_q4k(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st);
cudaError_t few_down_q4k(const FewArgs &a, int64_t T, cudaStream_t st);
cudaError_t few_gate_q80(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st);
cudaError_t few_down_q80(const FewArgs &a, int64_t T, cudaStream_t st);
cudaError_t few_gate_q6k(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st);
cudaError_t few_down_q6k(const FewArgs &a, int64_t T, cudaStream_t st);
cudaError_t rows_launch_q4k(const RowsArgs &a, bool paired, int sms, cudaStream_t st);
cudaError_t rows_launch_q80(const RowsArgs &a, bool paired, int sms, cudaStream_t st);
cudaError_t rows_launch_q6k(const RowsArgs &a, bool paired, int sms, cudaStream_t st);
cudaError_t tile_launch_q4k(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st);
cudaError_t tile_launch_q80(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st);
cudaError_t tile_launch_q6k(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st);

// Four neighbouring values of a row, 0 past its end.
__device__ __forceinline__ float4 four(const void *x, int64_t row, int k, int cols, int type, bool vec)
{
    if (vec && k + 4 <= cols) {
        if (type == QK_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + row + k);
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(x) + row + k);
        if (type == QK_F16) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
            return make_float4(a.x, a.y, b.x, b.y);
        }
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
    }
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = k + i < cols ? load_as_float(x, row + k + i, type) : 0.0f;
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch that may start while the kernel before it drains (its threads call wait_for_previous() before they read
// what that one writes).
template <class Kern, class Args>
cudaError_t launch_chained(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t st, bool chained, const Args &a)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at, cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace moe
}  // namespace qk
