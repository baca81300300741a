// qk_moe_tile.cuh -- the experts' products for many tokens an expert: tiles of
// 128 weight rows x up to 128 tokens on the tcgen05 tensor cores.
//
// Pairs of thread blocks keep going over their items; a product (cta_group::2)
// is 256 rows, half of them each block's, x the set's tokens, half of which each
// block holds.  A block's warps have roles: groups of four take the weights
// apart, a thread a row, and leave them as the A operand in tensor memory; one
// issues the pair's products (in the even block); one fetches the tokens'
// operands by TMA; two copy the weights' bytes (rows of 34 to 272 bytes of a
// unit: by TMA, about six cycles for each, gate and up of 4096 tokens took 1.5
// times as long); eight turn finished accumulators into outputs while the next
// item's products run, and look over a later item's rows for their largest scale.
//
// Weights are fp16 after a power of two a row that puts the largest value that
// the row's scales allow into [2^14, 2^15): for bf16 activations and outputs,
// which are coarser than that, once rounded (Q8_0), or twice (Q6_K: scale and
// product; Q4_K: minimum and sum), 2^-11 at most each.  Else they are two such
// pieces, and fp32 activations too (qk_moe.cuh); the product of the two low
// pieces is left out, 2^-22 of the product.
//
// Measured, 8 of 128 experts of 768 x 2048, Q4_K: 4096 bf16 tokens, gate and up
// 218 us (0.95 PFLOP/s, the tensor cores 43% busy), down 150 (0.69; 268 MB of
// outputs); 512 fp16 tokens 166 and 107 (Q6_K).  Taking the weights apart bounds
// it: a scheduler issues 0.52 to 0.64 instructions a cycle, and an expert of few
// tokens costs its weights' 4.7 million values whatever their number.
//
// Why A is in tensor memory and the tokens are shared: a product of 128 x 128 x
// 16 takes 64 cycles, in which shared memory moves 8 KB.  One block's tokens
// alone would be 4 KB written and 4 KB read, and A as much again (from shared
// memory, measured, a product of 192 tokens takes 145 cycles where one from
// tensor memory takes 100); half of the tokens leaves room.
#pragma once

#include "qk_moe.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace moe {

constexpr int kDeqWarp = 4;                                  // first warp that takes weights apart
// Stages whose products one accumulator takes with fp32 accuracy: each product cuts the sum towards zero, so that the error
// goes with their number (of a result 0.9e-6, 1.5e-6 and 2.8e-6 with 1, 2 and 4 stages; 400 tokens 80, 72 and 70 us).
constexpr int kFlush = 1;
constexpr int kEpiWarps = 8;                                 // two threads share a row's tokens
// Groups of four warps that take weights apart: three, or the two that fp32 sums leave registers for.
__host__ __device__ constexpr int tile_groups(int PB) { return PB == 1 ? 3 : 2; }
__host__ __device__ constexpr int tile_epi_warp(int PB) { return kDeqWarp + 4 * tile_groups(PB); }
__host__ __device__ constexpr int tile_threads(int PB) { return 32 * (tile_epi_warp(PB) + kEpiWarps); }
constexpr int kStages = 4;                                   // of the weights' operand
constexpr int kMaxN = 128;                                   // tokens of a set
// Columns of a stage: eight products for each (a wait costs the issuing warp as much as three of them).
__host__ __device__ constexpr int tile_cols_of_stage(int PA) { return PA == 1 ? 128 : 64; }
__host__ __device__ constexpr int tile_b_bytes(int PA, int PB) { return kMaxN / 2 * 2 * tile_cols_of_stage(PA) * PB; }
// The weights' bytes, a unit of 256 columns of each of 128 rows at a time: 16-byte chunks that hold it wherever it starts,
// in a pitch of 4 (mod 8) words, so that eight rows' chunks lie in different banks.
constexpr int kRawStages = 3;
__host__ __device__ constexpr int tile_chunks(int FMT) { return FMT == kFmtQ4K ? 9 : FMT == kFmtQ80 ? 18 : 14; }
__host__ __device__ constexpr int tile_pitch(int FMT) { return FMT == kFmtQ4K ? 144 : FMT == kFmtQ80 ? 304 : 240; }
// Stages of the tokens' operand: as many as shared memory holds (a refill takes 3000 cycles, a stage's products 500).
__host__ __device__ constexpr int tile_b_stages(int FMT, int PA, int PB)
{
    const int room = (222 * 1024 - kRawStages * 128 * tile_pitch(FMT)) / tile_b_bytes(PA, PB);
    return room < 8 ? room : 8;
}
__host__ __device__ constexpr int tile_smem(int FMT, int PA, int PB)
{
    return tile_b_stages(FMT, PA, PB) * tile_b_bytes(PA, PB) + kRawStages * 128 * tile_pitch(FMT) + 1024;
}

struct TileShared {
    uint64_t full[kStages], empty[kStages], b_full[8], b_empty[8], raw_full[kRawStages], raw_empty[kRawStages], acc_full[2], acc_empty[2], rs_full[4];
    float row_scale[4][128];                                 // 2^s of the rows of an item and of the next two
    float token_scale[kEpiWarps][64];                        // 2^-e of a warp's tokens
    uint32_t tmem;
    int abort;
};

// A bounded wait; one that runs out ends every other of the block.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const TileArgs &a, volatile int *abort)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t deadline = globaltimer_ns() + a.wait_ns;
    for (uint32_t i = 1; !*abort; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 31u) == 0 && globaltimer_ns() > deadline) {
            *abort = 1;
            record_error(a.err, kErrTimeout);
        }
    }
    return false;
}
__device__ __forceinline__ bool tile_wait_warp(uint32_t bar, uint32_t parity, const TileArgs &a, volatile int *abort)
{
    return __all_sync(~0u, tile_wait(bar, parity, a, abort));
}

// A test that may sleep a while before it says no, for arrivals from the other block, too.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// One lane of the (converged) warp is elected.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// D[tmem of both blocks] (+)= A[tmem of both] * B^T, M = 256.
__device__ __forceinline__ void tc_mma_f16_tmem_a_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t tile_h2(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 tile_b2(uint32_t b) { return *reinterpret_cast<__half2 *>(&b); }
template <uint32_t MASK>
__device__ __forceinline__ __half2 tile_field(uint32_t w)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "n"(0x64006400));
    return tile_b2(r);
}

// The row of the item's tile that thread `row` of it has: its first byte.
template <bool PAIRED>
__device__ __forceinline__ const uint8_t *tile_row(const TileArgs &a, int expert, int tile, int row)
{
    if constexpr (PAIRED) {
        // lanes 0..15 of a quarter have gate rows, 16..31 the up rows of the same outputs
        const Weights &w = row & 16 ? a.b : a.a;
        const int p = min(tile * 64 + (row >> 5) * 16 + (row & 15), a.rows - 1);
        return w.w + (expert * w.expert_rows + p) * w.row_bytes;
    } else {
        return a.a.w + (expert * a.a.expert_rows + min(tile * 128 + row, a.rows - 1)) * a.a.row_bytes;
    }
}

__device__ __forceinline__ float half_at(const uint8_t *p)
{
    return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short *>(p))));
}

// 2^s that puts the largest magnitude that a row's scales allow into [2^14, 2^15).
template <int FMT>
__device__ __forceinline__ float row_scale_of(const uint8_t *row, int cols)
{
    float most = 0.0f;
    const auto take = [&](float v) {
        v = fabsf(v);
        if (v < INFINITY) most = fmaxf(most, v);             // one that is not finite shows in the result anyway
    };
    if constexpr (FMT == kFmtQ4K) {
#pragma unroll 8
        for (int u = 0; u < (cols + 255) / 256; ++u) {
            const uint32_t h = __ldg(reinterpret_cast<const uint32_t *>(row + 144 * u));
            const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            take(fabsf(d.x) * 945.0f + fabsf(d.y) * 63.0f);
        }
    } else if constexpr (FMT == kFmtQ80) {
#pragma unroll 16
        for (int u = 0; u < (cols + 31) / 32; ++u) take(half_at(row + 34 * u) * 128.0f);
    } else {
#pragma unroll 8
        for (int u = 0; u < (cols + 255) / 256; ++u) take(half_at(row + 210 * u + 208) * 4096.0f);
    }
    const int ex = most == 0.0f ? 141 : max(static_cast<int>(__float_as_uint(most) >> 23), 15);
    return __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);
}

// A stage's bytes of a row, in registers.  Q8_0, Q6_K: words from a 4-byte boundary on; `sh` is 16 where the bytes start
// two later.
template <int FMT, int KC>
struct Raw {
    static constexpr int kWords = FMT == kFmtQ4K ? KC / 8 + 4 : FMT == kFmtQ80 ? KC / 64 * 17 + 1 : 27 + 3 + 1;
    uint32_t w[kWords], sh;
};

__device__ __forceinline__ uint4 tile_lds128(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}
__device__ __forceinline__ uint32_t tile_lds32(uint32_t p)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
    return v;
}
// N words that hold 4 (N - 1) + 2 bytes from p on.
template <int N>
__device__ __forceinline__ void tile_words(uint32_t *w, uint32_t p)
{
    const uint32_t q = p & ~3u;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = tile_lds32(q + 4 * i);
}

// Stage c of the row whose unit lies at `p`.
template <int FMT, int KC>
__device__ __forceinline__ void load_raw(Raw<FMT, KC> &r, uint32_t p, int c)
{
    const int part = c & (256 / KC - 1);
    if constexpr (FMT == kFmtQ4K) {
#pragma unroll
        for (int i = 0; i < KC / 32; ++i) {
            const uint4 v = tile_lds128(p + 16 + part * (KC / 2) + 16 * i);
            r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
        }
        const uint4 h = tile_lds128(p);
        r.w[KC / 8] = h.x, r.w[KC / 8 + 1] = h.y, r.w[KC / 8 + 2] = h.z, r.w[KC / 8 + 3] = h.w;
    } else if constexpr (FMT == kFmtQ80) {
        tile_words<Raw<FMT, KC>::kWords>(r.w, p + 34 * (KC / 32) * part);
        r.sh = ((p + 34 * (KC / 32) * part) & 2) * 8;
    } else {
        const int half = KC == 128 ? part : part >> 1;
        tile_words<9>(r.w, p + 64 * half);                       // low nibbles, 0..31
        tile_words<9>(r.w + 9, p + 64 * half + 32);              // 32..63
        tile_words<9>(r.w + 18, p + 128 + 32 * half);            // high bits
        tile_words<3>(r.w + 27, p + 192 + 8 * half);             // scales
        r.sh = (p & 2) * 8;
        r.w[30] = tile_lds32((p + 208) & ~3u) >> r.sh;           // d
    }
}

// a b + c and a + c in fp32, a and b the halves AT of fp16 pairs
template <int AT>
__device__ __forceinline__ uint16_t half_of(__half2 v)
{
    return static_cast<uint16_t>(AT ? tile_h2(v) >> 16 : tile_h2(v) & 0xffffu);
}
__device__ __forceinline__ float fma_half(uint16_t a, uint16_t b, float c)
{
    float r;
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(r) : "h"(a), "h"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float add_half(uint16_t a, float c)
{
    float r;
    asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(r) : "h"(a), "f"(c));
    return r;
}

// fp16 pairs of 32 values: hi pieces, and lo where PA == 2, the rest to 2^-22 of the value.
template <int PA>
struct Pieces {
    uint32_t hi[16], lo[PA == 2 ? 16 : 1];
    // whole numbers t times d (exact in fp16) less m, of which mh is the fp16
    __device__ __forceinline__ void set(int i, __half2 t, __half2 d, float m, __half2 mh)
    {
        const __half2 h = __hfma2(t, d, __hneg2(mh));
        hi[i] = tile_h2(h);
        if constexpr (PA == 2) {
            // t d - (m + h): the sum's rounding is 2^-24 of m
            const float a = fma_half(half_of<0>(t), half_of<0>(d), -add_half(half_of<0>(h), m));
            const float b = fma_half(half_of<1>(t), half_of<0>(d), -add_half(half_of<1>(h), m));
            lo[i] = tile_h2(__floats2half2_rn(a, b));
        }
    }
    // whole numbers q times dh + dl: a product's rest is a fused multiply-add away
    __device__ __forceinline__ void set(int i, __half2 q, __half2 dh, __half2 dl, bool rest)
    {
        const __half2 h = __hmul2(q, dh);
        hi[i] = tile_h2(h);
        if constexpr (PA == 2) {
            const __half2 e = __hfma2(q, dh, __hneg2(h));
            lo[i] = tile_h2(rest ? __hfma2(q, dl, e) : e);
        }
    }
};

// Values 32 k .. 32 k + 31 of a stage, times 2^s, as fp16 pairs in the order (0, 2), (1, 3) of every four columns.
template <int FMT, int PA, int KC>
__device__ __forceinline__ void take_apart(Pieces<PA> &o, const Raw<FMT, KC> &r, int c, int cols, float up, int k)
{
    if constexpr (FMT == kFmtQ4K) {
        const __half2 k1024 = __float2half2_rn(1024.0f);
        const float2 d2 = __half22float2(tile_b2(r.w[KC / 8]));
        const int pair = (c * (KC / 64) + (k >> 1)) & 3, high = k & 1, sh = (pair & 1) * 16 + 8 * high;     // sub-block 2 pair + high
        const uint32_t A = r.w[KC / 8 + 1] >> sh, B = r.w[KC / 8 + 2] >> sh, C = r.w[KC / 8 + 3] >> sh;
        const uint32_t sc = pair < 2 ? A & 0x3fu : (C & 0x0fu) | ((A >> 2) & 0x30u);
        const uint32_t mm = pair < 2 ? B & 0x3fu : ((C >> 4) & 0x0fu) | ((B >> 2) & 0x30u);
        const __half2 s0 = __hsub2(tile_b2(0x64006400u | sc | sc << 16), k1024);
        const float m = d2.y * up * static_cast<float>(mm);
        const __half2 dh = __float2half2_rn(d2.x * up), mh = __float2half2_rn(m);
        const __half2 mul = high ? __hmul2(s0, __float2half2_rn(0.0625f)) : s0;
        const __half2 add = __hmul2(s0, __float2half2_rn(high ? -64.0f : -1024.0f));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = r.w[8 * (k >> 1) + i];
            // scale times quant, exact
            const __half2 a = __hfma2(high ? tile_field<0x00f000f0>(v) : tile_field<0x000f000f>(v), mul, add);
            const __half2 b = __hfma2(high ? tile_field<0x00f000f0>(v >> 8) : tile_field<0x000f000f>(v >> 8), mul, add);
            o.set(2 * i, a, dh, m, mh), o.set(2 * i + 1, b, dh, m, mh);
        }
    } else if constexpr (FMT == kFmtQ80) {
        // block k: d at byte 34 k, then the quants; none past the row's end
        const int first = c * (KC / 32), base = 17 * (k >> 1);
        const auto at = [&](int i) { return __funnelshift_r(r.w[i], r.w[i + 1], r.sh); };
        const __half2 bias = __float2half2_rn(1152.0f);
        const float d = first + k < (cols + 31) / 32 ? half_bits_to_float(k & 1 ? at(base + 8) >> 16 : at(base)) * up : 0.0f;
        const __half2 dh = __float2half2_rn(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t q = (k & 1 ? at(base + 9 + i) : __funnelshift_r(at(base + i), at(base + i + 1), 16)) ^ 0x80808080u;
            o.set(2 * i, __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4240)), bias), dh, dh, false);
            o.set(2 * i + 1, __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4341)), bias), dh, dh, false);
        }
    } else {
        // 32 columns t of the half
        const int t = KC == 128 ? k : 2 * (c & 1) + k;
        const float d0 = half_bits_to_float(r.w[30]) * up;
        const __half2 bias = __float2half2_rn(1056.0f);
        const uint32_t scales = __funnelshift_r(r.w[27 + (t >> 1)], r.w[28 + (t >> 1)], r.sh) >> (16 * (t & 1));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float d = d0 * static_cast<float>(static_cast<int8_t>(scales >> (8 * u)));
            const __half2 dh = __float2half2_rn(d), dl = __float2half2_rn(d - __low2float(dh));
#pragma unroll
            for (int i = 4 * u; i < 4 * u + 4; ++i) {
                const uint32_t low = __funnelshift_r(r.w[9 * (k & 1) + i], r.w[9 * (k & 1) + i + 1], r.sh) >> (t & 2 ? 4 : 0);
                const uint32_t high = __funnelshift_r(r.w[18 + i], r.w[19 + i], r.sh) >> (2 * t);
                const uint32_t q = (low & 0x0f0f0f0fu) | ((high & 0x03030303u) << 4);
                o.set(2 * i, __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4240)), bias), dh, dl, true);
                o.set(2 * i + 1, __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4341)), bias), dh, dl, true);
            }
        }
    }
}

struct TileMaps {
    CUtensorMap hi, lo;              // the tokens' operands
};

template <int FMT, int PA, int PB, bool PAIRED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(tile_threads(PB), 1)
tile_kernel(const __grid_constant__ TileMaps maps, const TileArgs a)
{
    constexpr int KC = tile_cols_of_stage(PA), kStage = tile_b_bytes(PA, PB), kBStages = tile_b_stages(FMT, PA, PB), kPitch = tile_pitch(FMT), kRaw = 128 * kPitch;
    constexpr int kGroups = tile_groups(PB), kEpiWarp = tile_epi_warp(PB), kParts = 256 / KC;      // stages of a unit
    constexpr uint32_t kACols = KC / 2 * PA, kA0 = 2 * kMaxN;         // tensor-memory columns of a stage of A, and of the first
    static_assert(kA0 + kStages * kACols == 512, "all of tensor memory");
    extern __shared__ uint8_t raw_smem[];
    __shared__ TileShared sh;
    const uint32_t b_base = (smem_u32(raw_smem) + 1023u) & ~1023u, raw_base = b_base + kBStages * kStage;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 8);             // (even block) a group's four warps of each block
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < kBStages; ++i) mbar_init(smem_u32(&sh.b_full[i]), 1), mbar_init(smem_u32(&sh.b_empty[i]), 1);
        for (int i = 0; i < kRawStages; ++i) mbar_init(smem_u32(&sh.raw_full[i]), 64), mbar_init(smem_u32(&sh.raw_empty[i]), 4 * kParts);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.acc_full[i]), 1), mbar_init(smem_u32(&sh.acc_empty[i]), 2 * kEpiWarps);
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh.rs_full[i]), 4);
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.hi);
        if (PB == 2) tma_prefetch_desc(&maps.lo);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&sh.tmem), 512);
        tmem_relinquish_pair();
    }
    let_next_start();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t taddr = *static_cast<volatile uint32_t *>(&sh.tmem);
    wait_for_previous();

    const int pairs = (a.tiles + 1) / 2;
    const int items = a.plan.head[1] * pairs, first = blockIdx.x >> 1, step = gridDim.x >> 1;      // (the caller sees to 31 bits)
    const int nk = a.chunks;
    const int per = PB == 2 ? kFlush : nk;                     // stages an accumulator takes
    const auto set_of = [&](int item) { return a.plan.tile_sets[item / pairs]; };
    const auto tile_of = [&](int item) { return item % pairs * 2 + rank; };
    const auto columns_of = [](int count) { return (count + 31) / 32 * 32; };       // of a product: a pair's are multiples of 32
    // an arrival on a barrier of the even block
    const auto arrive_even = [&](uint64_t *bar) {
        if (rank == 0) mbar_arrive(smem_u32(bar));
        else mbar_arrive_remote(mapa_shared(smem_u32(bar), 0));
    };

    // What the warps that issue copies and products go by: they stay together and elect a lane for each, and all that
    // steers them comes from votes, reductions and counters, so that operands are in the warp's uniform registers.  (A
    // thread of a branch of its own, or in a loop whose end it has read from memory, takes 100 to 118 cycles a product and
    // 250 a copy, measured; this form N / 2 and 30.)
    const auto ready = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(~0u, mbar_try_wait_cluster(bar, parity))) return true;
        const uint64_t deadline = globaltimer_ns() + a.wait_ns;
        for (unsigned i = 1;; ++i) {
            if (__all_sync(~0u, mbar_try_wait_cluster(bar, parity))) return true;
            if ((i & 7u) == 0) {
                const bool late = globaltimer_ns() > deadline;
                if (late) *abort = 1, record_error(a.err, kErrTimeout);
                if (__any_sync(~0u, late || *abort)) return false;
            }
        }
    };
    const unsigned end = __reduce_max_sync(~0u, static_cast<unsigned>(items));

    if (warp == 0) {
        const uint64_t keep = l2_evict_last_policy();
        unsigned n = 0;
        bool ok = true;
        for (unsigned item = first; item < end && ok; item += step) {
            const ExpertSet s = set_of(item);
            const unsigned cols = __reduce_max_sync(~0u, static_cast<unsigned>(columns_of(s.count)));
            const unsigned boxes = (cols / 2 + kTileBoxRows - 1) / kTileBoxRows;
            const int y = __reduce_max_sync(~0u, s.first) + rank * static_cast<int>(cols / 2);
            for (int c = 0; c < nk; ++c, ++n) {
                const unsigned st = n % kBStages;
                if (n >= kBStages && !ready(smem_u32(&sh.b_empty[st]), (n / kBStages - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t full = smem_u32(&sh.b_full[st]), to = b_base + st * kStage;
                const uint32_t full0 = rank == 0 ? full : mapa_shared(full, 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full, 2 * boxes * kTileBoxRows * 2 * KC * PB);
                    if (!(a.skip_chunk >= 0 && static_cast<int>(n) == a.skip_chunk && blockIdx.x < 2))       // test hook
                        for (unsigned b = 0; b < boxes; ++b)
#pragma unroll
                            for (int k = 0; k < KC / 64; ++k) {
                                const uint32_t at = to + k * (kMaxN / 2 * 128) + b * (kTileBoxRows * 128);
                                tma_load_2d_peer(at, &maps.hi, c * KC + k * 64, y + b * kTileBoxRows, full0, keep);
                                if (PB == 2)
                                    tma_load_2d_peer(at + kStage / 2, &maps.lo, c * KC + k * 64, y + b * kTileBoxRows, full0, keep);
                            }
                }
            }
        }
        // every copy lands before the blocks leave (both blocks' are counted on the even one's barriers)
        if (rank == 0)
            for (unsigned t = n > kBStages ? n - kBStages : 0; t < n; ++t)
                mbar_wait(smem_u32(&sh.b_full[t % kBStages]), (t / kBStages) & 1, a.wait_ns);
        __syncwarp();
    } else if (warp == 1) {
        unsigned n = 0, q = 0;                                 // stages and accumulators so far
        bool ok = rank == 0;
        const uint32_t tmem = __reduce_max_sync(~0u, taddr);
        const uint64_t desc0 = smem_desc_sw128_kmajor(b_base);
        for (unsigned item = first; item < end && ok; item += step) {
            const uint32_t idesc = idesc_f16_f32(256, columns_of(__reduce_max_sync(~0u, set_of(item).count)));
            for (int c = 0, of = 0; c < nk; ++c, ++n) {
                const unsigned st = n % kStages, sb = n % kBStages, buf = q & 1;
                const bool fresh = of == 0, last = c + 1 == nk || of + 1 == per;
                if (fresh && q >= 2 && !ready(smem_u32(&sh.acc_empty[buf]), (q / 2 - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (!ready(smem_u32(&sh.b_full[sb]), (n / kBStages) & 1) || !ready(smem_u32(&sh.full[st]), (n / kStages) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + buf * kMaxN, at = tmem + kA0 + st * kACols;
                const uint64_t b = desc0 + static_cast<uint64_t>(sb * (kStage >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < KC / 16; ++k) {
                        const uint64_t bk = b + (k >> 2) * (kMaxN / 2 * 128 >> 4) + 2 * (k & 3);
                        tc_mma_f16_tmem_a_pair(d, at + 8 * k, bk, idesc, !fresh || k > 0);
                        if constexpr (PA == 2) tc_mma_f16_tmem_a_pair(d, at + KC / 2 + 8 * k, bk, idesc, 1);
                        if constexpr (PB == 2) tc_mma_f16_tmem_a_pair(d, at + 8 * k, bk + (kStage >> 5), idesc, 1);
                    }
                    tc_commit_pair(smem_u32(&sh.empty[st]), 3);
                    tc_commit_pair(smem_u32(&sh.b_empty[sb]), 3);
                    if (last) tc_commit_pair(smem_u32(&sh.acc_full[buf]), 3);
                }
                of = last ? 0 : of + 1;
                q += last;
            }
        }
        // products in flight end before tensor memory is freed; the other block sees their last arrivals as well
        for (unsigned t = n > kBStages ? n - kBStages : 0; t < n; ++t) mbar_wait(smem_u32(&sh.b_empty[t % kBStages]), (t / kBStages) & 1, a.wait_ns);
        if (n > 0) mbar_wait(smem_u32(&sh.empty[(n - 1) % kStages]), ((n - 1) / kStages) & 1, a.wait_ns);
        __syncwarp();
    } else if (warp < kDeqWarp) {
        // the weights' bytes, 16 at a time: four lanes a row, eight rows an instruction, 64 rows a warp
        constexpr int UB = unit_bytes(FMT), CH = tile_chunks(FMT);
        const int units = (nk + kParts - 1) / kParts, row0 = (warp - 2) * 64 + (lane >> 2), ch0 = lane & 3;
        int n = 0;                                             // units so far
        bool ok = true;
        for (int item = first; item < items && ok; item += step) {
            const int expert = set_of(item).expert, tile = tile_of(item);
            const uint8_t *at[8];
#pragma unroll
            for (int o = 0; o < 8; ++o) at[o] = tile_row<PAIRED>(a, expert, tile, row0 + 8 * o);
            for (int u = 0; u < units; ++u, ++n) {
                const int st = n % kRawStages;
                if (n >= kRawStages && !tile_wait_warp(smem_u32(&sh.raw_empty[st]), (n / kRawStages - 1) & 1, a, abort)) {
                    ok = false;
                    break;
                }
                const uint32_t to = raw_base + st * kRaw + row0 * kPitch + 16 * ch0;
                const int64_t off = static_cast<int64_t>(u) * UB;
                const int left = static_cast<int>(min(static_cast<int64_t>(UB), a.a.row_bytes - off));      // bytes of the unit
#pragma unroll
                for (int o = 0; o < 8; ++o) {
                    const uint8_t *from = at[o] + off;
                    int bytes = left - 16 * ch0;               // from this lane's first chunk on
                    if constexpr (FMT != kFmtQ4K) {
                        const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
                        from -= skew, bytes += skew;
                    }
                    from += 16 * ch0;
#pragma unroll
                    for (int i = 0; i < (CH + 3) / 4; ++i)
                        if (16 * 4 * i < bytes)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 8 * o * kPitch + 64 * i), "l"(from + 64 * i)
                                         : "memory");
                }
                // arrives when this thread's copies have landed
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.raw_full[st])) : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < kEpiWarp) {
        // takes stages' weights apart: group h has every kGroups-th stage of the block's
        const int group = (warp - kDeqWarp) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        int n = group, it = 0, c = group;
        int item = first;
        while (c >= nk && item < items) c -= nk, ++it, item += step;
        uint32_t start = 0;                                    // low bits of the address of the thread's row
        float up = 0.0f;
        int have = -1;
        while (item < items) {
            const int st = n % kStages, u = it * ((nk + kParts - 1) / kParts) + c / kParts, rs = u % kRawStages;
            if (have != it) {
                start = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(tile_row<PAIRED>(a, set_of(item).expert, tile_of(item), row)));
                if (!tile_wait_warp(smem_u32(&sh.rs_full[it & 3]), (it / 4) & 1, a, abort)) break;
                up = sh.row_scale[it & 3][row];
                have = it;
            }
            if (!tile_wait_warp(smem_u32(&sh.raw_full[rs]), (u / kRawStages) & 1, a, abort)) break;
            Raw<FMT, KC> raw;
            load_raw<FMT, KC>(raw, raw_base + rs * kRaw + row * kPitch + ((start + c / kParts * unit_bytes(FMT)) & 15), c);
            __syncwarp();
            // (a row's last stage arrives for those that its last unit lacks, too)
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&sh.raw_empty[rs])),
                             "r"(c + 1 == nk ? kParts - c % kParts : 1)
                             : "memory");
            if (n >= kStages && !tile_wait_warp(smem_u32(&sh.empty[st]), (n / kStages - 1) & 1, a, abort)) break;
            tc_fence_after();
            const uint32_t to = taddr + (static_cast<uint32_t>(quarter * 32) << 16) + kA0 + st * kACols;
#pragma unroll
            for (int k = 0; k < KC / 32; ++k) {
                Pieces<PA> o;
                take_apart<FMT, PA, KC>(o, raw, c, a.cols, up, k);
                tmem_st_32x32b_x16(to + 16 * k, o.hi);
                if constexpr (PA == 2) tmem_st_32x32b_x16(to + KC / 2 + 16 * k, o.lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even(&sh.full[st]);
            n += kGroups, c += kGroups;
            while (c >= nk && item < items) c -= nk, ++it, item += step;
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, part = (warp - kEpiWarp) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        int it = 0, q = 0;
        bool ok = true;
        // the scales of item number i's rows, by the first four warps
        const auto look_over = [&](int i) {
            const int item = first + i * step;
            if (part != 0 || item >= items) return;
            sh.row_scale[i & 3][row] = row_scale_of<FMT>(tile_row<PAIRED>(a, set_of(item).expert, tile_of(item), row), a.cols);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.rs_full[i & 3]));
        };
        look_over(0), look_over(1);
        for (int item = first; item < items && ok; item += step, ++it) {
            const ExpertSet s = set_of(item);
            const int tile = tile_of(item);
            float back = 0.0f;
            // a warp's 64 tokens from c_first on
            const int c_first = part * 64;
            float *ts = sh.token_scale[warp - kEpiWarp];
            __syncwarp();                                      // every lane has read the last item's
#pragma unroll
            for (int j = lane; j < 64; j += 32) ts[j] = c_first + j < s.count ? a.scale[s.first + c_first + j] : 0.0f;
            __syncwarp();
            // 32 tokens' sums of this thread's row, from the warp's token c0 on
            const auto emit = [&](const uint32_t (&v)[32], int c0) {
                const int left = s.count - c_first - c0;
                const float *t = ts + c0;
                if constexpr (PAIRED) {
                    const int p = tile * 64 + quarter * 16 + (lane & 15);
                    const bool low = lane < 16;
                    float *out = a.out + static_cast<int64_t>(s.first + c_first + c0 + !low) * a.rows + p;
                    const int64_t next = 2 * static_cast<int64_t>(a.rows);
                    const int mine = p < a.rows ? left - !low : 0;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        // this half of the warp keeps one token of two and gets its other row's sum
                        const float keep = __uint_as_float(low ? v[j] : v[j + 1]) * back, give = __uint_as_float(low ? v[j + 1] : v[j]) * back;
                        const float got = __shfl_xor_sync(~0u, give, 16), tj = t[j + !low];
                        const float h = silu((low ? keep : got) * tj) * ((low ? got : keep) * tj);
                        if (j < mine) *out = h;
                        out += next;
                    }
                } else {
                    const int p = tile * 128 + row;
                    float *out = a.out + static_cast<int64_t>(s.first + c_first + c0) * a.rows + p;
                    const int mine = p < a.rows ? left : 0;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j < mine) *out = __uint_as_float(v[j]) * back * t[j];
                        out += a.rows;
                    }
                }
            };
            const auto ready = [&]() {
                if (!tile_wait_warp(smem_u32(&sh.acc_full[q & 1]), (q / 2) & 1, a, abort)) return ok = false;
                tc_fence_after();
                if (back == 0.0f) back = 1.0f / sh.row_scale[it & 3][row];      // a power of two
                return true;
            };
            const auto drained = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_even(&sh.acc_empty[q & 1]);
                ++q;
            };
            if constexpr (PB == 2) {
                float sum[2][32];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[h][j] = 0.0f;
                for (int c = 0; c < nk && ok; c += per) {
                    if (!ready()) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (c_first + h * 32 >= s.count) continue;
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(taddr + lanes + (q & 1) * kMaxN + c_first + h * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[h][j] += __uint_as_float(v[j]);
                    }
                    drained();
                }
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (c_first + h * 32 >= s.count) continue;
                    uint32_t v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sum[h][j]);
                    emit(v, h * 32);
                }
            } else {
                if (!ready()) break;
#pragma unroll 1
                for (int c0 = 0; c0 < 64 && c_first + c0 < s.count; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + lanes + (q & 1) * kMaxN + c_first + c0, v);
                    tmem_ld_wait();
                    emit(v, c0);
                }
                drained();
            }
            // the slot's last item was done when this one's sums were: every thread had read its scale before
            look_over(it + 2);
        }
    }
    tc_fence_before();
    cluster_sync();              // neither block leaves while the other may still write to it
    if (warp == 1) tmem_dealloc_pair(taddr, 512);
}

template <int FMT, int PA, int PB, bool PAIRED>
cudaError_t tile_launch_as(const TileOperands &t, const TileArgs &a, int sms, cudaStream_t st)
{
    const auto kern = tile_kernel<FMT, PA, PB, PAIRED>;
    constexpr int smem = tile_smem(FMT, PA, PB);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    TileMaps maps;
    const gemm::EncodeTiledFn enc = gemm::encode_fn();
    if (!enc) return cudaErrorNotSupported;
    // boxes of 64 columns and kTileBoxRows rows
    const auto encode = [&](CUtensorMap *m, const void *p) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.cols), static_cast<cuuint64_t>(t.rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * t.cols)};
        const cuuint32_t box[2] = {64, kTileBoxRows}, one[2] = {1, 1};
        return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    bool ok = encode(&maps.hi, t.hi);
    maps.lo = maps.hi;
    if (PB == 2) ok = ok && encode(&maps.lo, t.lo);
    if (!ok) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2)), cfg.blockDim = dim3(tile_threads(PB));
    cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

template <int FMT, bool PAIRED>
cudaError_t tile_launch_pieces(const TileOperands &t, const TileArgs &a, int sms, cudaStream_t st)
{
    if (a.w_pieces == 1) return tile_launch_as<FMT, 1, 1, PAIRED>(t, a, sms, st);
    return a.pieces == 1 ? tile_launch_as<FMT, 2, 1, PAIRED>(t, a, sms, st) : tile_launch_as<FMT, 2, 2, PAIRED>(t, a, sms, st);
}

template <int FMT>
cudaError_t tile_launch(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st)
{
    return paired ? tile_launch_pieces<FMT, true>(t, a, sms, st) : tile_launch_pieces<FMT, false>(t, a, sms, st);
}

}  // namespace moe
}  // namespace qk
