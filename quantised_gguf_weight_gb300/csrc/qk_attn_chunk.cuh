// qk_attn_chunk.cuh -- what the two many-row forms of attention over the 4-bit
// cache share: accesses to shared memory, the work of a thread block, a row's
// state, outputs, and the join of a cut head's parts.
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

// Products of fp16 pairs, rounded once, subnormals kept.
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// a * b + c on fp16 pairs, rounded once, subnormals kept.
__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// The power of two taken off the scales of a 16-token block whose largest has the fp16 bits `top`.  Times 2^6 an fp16
// scale is below 2^12, and its products with n - 8 in fp16's range, up to 2^6; above it more is taken off.  It is the
// same for nearly every block: a row's probabilities carry the values' power, and where one block took off much more
// than the others, theirs would sink below fp16's range.
__device__ __forceinline__ int power_of(uint32_t top) { return max(static_cast<int>(top >> 10) - 26, -6); }

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

// Two values as a pair of 16-bit elements.
__device__ __forceinline__ uint32_t pack_as(float lo, float hi, bool bf16)
{
    if (!bf16) return pack_half(lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// How a call's blocks are shared out where heads are few: found on the device from the lengths by a kernel of one
// thread block (every thread block finding it for itself cost as much, and registers).  A head of an item (a row tile of a sequence) is cut into parts of `per` 16-token blocks, each a thread
// block's; `per` is the longest item's blocks over one of kCuts, the one whose estimated time is least: of the
// longest part, or of all parts over the GPU, with kPartFixed blocks' time for a part's start and end (about 15 us,
// a block 0.26 us in 16 bits, 0.35 in fp32), and for cut heads the join of the parts.
// Whole and cut so: 8 x 64 fp32 queries over up to 5000 keys, uneven, 108 us and 78; 64 fp32 queries over 16384 keys
// 361 and 62, bf16 266 and 40; 8 x 64 over 4096 keys each, bf16 78 and 66, but fp32, where nothing can be cut, 105
// and 115.
constexpr int kItems = 512;              // items of a call whose heads may be cut
constexpr int kCutChoices = 16;
constexpr float kPartFixed = 50.0f, kJoinFixed = 25.0f, kJoinBytes = 400.0e3f;      // in blocks; bytes a block's time
__host__ __device__ constexpr int cut_of(int c)
{
    return c < 10 ? c + 1 : c == 10 ? 12 : c == 11 ? 14 : c == 12 ? 16 : c == 13 ? 19 : c == 14 ? 25 : 38;
}
__host__ __device__ inline int part_of(int longest, int c)
{
    const int per = ((longest + cut_of(c) - 1) / cut_of(c) + kTileBlocks - 1) / kTileBlocks * kTileBlocks;      // whole tiles
    return per > 16 ? per : 16;
}
__host__ __device__ inline float part_cost(float all_blocks, int parts, int per, int sms, int64_t part_bytes, bool cut)
{
    const float spread = (all_blocks + kPartFixed * parts) / sms + 0.5f * per;           // uneven parts, packed
    const float rounds = (parts + sms - 1) / sms * (all_blocks / parts + kPartFixed);      // even ones
    const float run = parts <= sms ? per + kPartFixed : spread > rounds ? spread : rounds;
    return run + (cut ? kJoinFixed + parts * static_cast<float>(part_bytes) / kJoinBytes : 0.0f);
}

// The sharing out lies in the workspace's plan: for each thread block item, head, part and blocks a part (item -1:
// none), for each item its first thread block and parts a head, and at the end whether any head is cut.
constexpr int kPlanBytes = 16384, kPlanBlocks = (kPlanBytes - kItems * 8) / 16 - 1;
__device__ __forceinline__ int4 *plan_of_blocks(const AttnArgs &a) { return static_cast<int4 *>(a.plan); }
__device__ __forceinline__ int2 *plan_of_items(const AttnArgs &a) { return reinterpret_cast<int2 *>(plan_of_blocks(a) + kPlanBlocks); }
__device__ __forceinline__ int *plan_any(const AttnArgs &a) { return reinterpret_cast<int *>(plan_of_items(a) + kItems); }

// What a thread block works on, in few registers.  Keys and positions count from the part's first key.
struct Work {
    int b, hk, first, rows;      // sequence, head; this block's rows of them
    int active;                  // parts of the head (at least one)
    int nblk, ntiles;            // 16-token blocks and key tiles of this part
    int blk0;                    // its first block in the sequence
    int r0;                      // the sequence's first row among the queries
    int pos;                     // and its position
    int lo, hi;                  // keys that some row sees
};

// One row's state.
struct Row {
    float m, l, to_log2;
    int lo, hi;
};

// This thread block's work; false where it has none.
__device__ __forceinline__ bool find_work(const AttnArgs &a, int tile_rows, int D, Work &w)
{
    int item = static_cast<int>(blockIdx.x / a.n_kv), per = INT32_MAX;
    w.hk = static_cast<int>(blockIdx.x) - item * a.n_kv;
    int split = 0;
    w.active = 1;
    if (a.cut) {
        const int4 mine = plan_of_blocks(a)[blockIdx.x];
        item = mine.x;
        if (item < 0) return false;
        w.hk = mine.y, split = mine.z, per = mine.w;
        w.active = plan_of_items(a)[item].y;
    }
    w.b = item / a.tiles;
    const int tile = item - w.b * a.tiles;
    const Sequence seq = sequence_of(a, w.b);
    if (seq.bad) {
        if (split == 0) poison_rows(a, seq, w.hk, tile, a.rep * D);
        return false;
    }
    const int n = static_cast<int>(seq.r1 - seq.r0) * a.rep;
    w.first = tile * tile_rows;
    if (w.first >= n) return false;
    w.rows = min(tile_rows, n - w.first);
    const Span span = span_of(a, seq, w.first, w.rows);
    const int b0 = split ? split * per : 0;
    w.nblk = min(span.blocks - b0, per);
    w.ntiles = (w.nblk + kTileBlocks - 1) / kTileBlocks;
    w.blk0 = static_cast<int>(span.blk_lo) + b0;
    const int64_t base = static_cast<int64_t>(w.blk0) * kBlockTokens;
    w.r0 = static_cast<int>(seq.r0);
    w.pos = static_cast<int>(seq.len - (seq.r1 - seq.r0) - base);
    w.lo = clamp_key(span.key_lo - base), w.hi = clamp_key(span.key_hi - base);
    return true;
}

// Where a row of this block begins among rows of stride ld (rows beyond them: where the first does).
__device__ __forceinline__ int64_t row_at(const AttnArgs &a, const Work &w, int row, bool in, int64_t ld, int D)
{
    const int r = w.first + (in ? row : 0), i = r / a.rep;
    return (static_cast<int64_t>(w.r0) + i) * ld + (static_cast<int64_t>(w.hk) * a.rep + (r - i * a.rep)) * D;
}

// The keys that a row sees.
__device__ __forceinline__ void row_keys(const AttnArgs &a, const Work &w, int row, int &lo, int &hi)
{
    const int64_t pos = static_cast<int64_t>(w.pos) + (w.first + row) / a.rep;
    lo = clamp_key(a.window > 0 ? pos - a.window + 1 : -1);
    hi = clamp_key(pos + 1);
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

// Launches the tiles' kernel and, where heads may be cut, the plan before and the join of the parts after.
cudaError_t launch_tiles(void (*kern)(const AttnArgs), std::atomic<uint64_t> &done, int smem, int threads, const AttnArgs &a, int D,
                         int rows, int64_t groups, cudaStream_t st);

}  // namespace chunk
}  // namespace qk
