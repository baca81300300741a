// qk_moe_tile.cuh -- the experts' products for many tokens an expert: tiles of
// 128 weight rows x up to 128 tokens on the tcgen05 tensor cores.
//
// Pairs of thread blocks keep going over their items; a product (cta_group::2)
// is 256 rows, half of them each block's, x the set's tokens, half of which each
// block holds.  A block's warps have roles: groups of four take the weights
// apart, a thread a row, and leave them as the A operand in tensor memory; one
// issues the pair's products (in the even block); one fetches the tokens'
// operands, and Q4_K's bytes, by TMA; eight turn finished accumulators into
// outputs while the next item's products run; two look over the next item's
// rows for their largest scale.
//
// Weights are fp16 after a power of two a row that puts the largest value that
// the row's scales allow into [2^14, 2^15): one rounding (Q4_K: the minimum's
// and the sum's) of 2^-12 for bf16 activations and outputs.  Else they are two
// such pieces, and fp32 activations too (qk_moe.cuh); the product of the two
// low pieces is left out.
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
constexpr int kFlush = 4;                                    // stages whose products one accumulator takes, with fp32 accuracy
constexpr int kEpiWarps = 8;                                 // two threads share a row's tokens
// Groups of four warps that take weights apart.  More than two need the registers that fp32 sums, or bytes fetched a
// stage ahead by the threads themselves (all formats but Q4_K), take.
__host__ __device__ constexpr int tile_groups(int FMT, int PB) { return FMT == kFmtQ4K && PB == 1 ? 3 : 2; }
__host__ __device__ constexpr int tile_epi_warp(int FMT, int PB) { return kDeqWarp + 4 * tile_groups(FMT, PB); }
__host__ __device__ constexpr int tile_threads(int FMT, int PB) { return 32 * (tile_epi_warp(FMT, PB) + kEpiWarps); }
constexpr int kStages = 4;                                   // of both operands
constexpr int kMaxN = 128;                                   // tokens of a set
// Columns of a stage: eight products for each (a wait costs the issuing warp as much as three of them).
__host__ __device__ constexpr int tile_cols_of_stage(int PA) { return PA == 1 ? 128 : 64; }
__host__ __device__ constexpr int tile_b_bytes(int PA, int PB) { return kMaxN / 2 * 2 * tile_cols_of_stage(PA) * PB; }
// Q4_K's bytes of a stage: [128 rows] of half its columns' number, and of 16 for the scales.
__host__ __device__ constexpr int tile_raw_bytes(int FMT, int PA) { return FMT == kFmtQ4K ? 128 * (tile_cols_of_stage(PA) / 2 + 16) : 0; }
__host__ __device__ constexpr int tile_smem(int FMT, int PA, int PB)
{
    return kStages * (tile_b_bytes(PA, PB) + tile_raw_bytes(FMT, PA)) + 1024;
}

struct TileShared {
    uint64_t full[kStages], empty[kStages], raw_full[kStages], raw_empty[kStages], acc_full[2], acc_empty[2], rs_full[2], rs_empty[2];
    float row_scale[2][128];                                 // 2^s of the rows
    float token_scale[kEpiWarps][64];                        // 2^-e of a warp's tokens
    uint32_t tmem;
    int abort;
};

// A bounded wait; one that runs out ends every other of the block.  POLL: without sleeping, and for arrivals from the
// other block.
template <bool POLL = false>
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const TileArgs &a, volatile int *abort)
{
    const auto test = [&]() { return POLL ? mbar_test(bar, parity) : mbar_try_wait(bar, parity); };
    if (test()) return true;
    const uint64_t deadline = globaltimer_ns() + a.wait_ns;
    for (uint32_t i = 1; !*abort; ++i) {
        if (test()) return true;
        if ((i & 31u) == 0 && globaltimer_ns() > deadline) {
            *abort = 1;
            record_error(a.err, kErrTimeout);
        }
    }
    return false;
}
template <bool POLL = false>
__device__ __forceinline__ bool tile_wait_warp(uint32_t bar, uint32_t parity, const TileArgs &a, volatile int *abort)
{
    return __all_sync(~0u, tile_wait<POLL>(bar, parity, a, abort));
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

// A stage's bytes of a row, in registers.
template <int FMT, int KC>
struct Raw {
    static constexpr int kWords = FMT == kFmtQ4K ? KC / 8 + 4 : FMT == kFmtQ80 ? KC / 64 * 17 + 1 : 27;
    uint32_t w[kWords];
};

// The 32-bit words that hold N words from a 2-byte aligned place on (one more where it is off).
template <int N>
__device__ __forceinline__ void load_words2(uint32_t *w, const uint8_t *p)
{
    const uint32_t *q = reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(q + i);
    w[N] = reinterpret_cast<uintptr_t>(p) & 2 ? __ldg(q + N) : 0u;
}

template <int FMT, int KC>
__device__ __forceinline__ void load_raw(Raw<FMT, KC> &r, const uint8_t *row, int c, int cols)
{
    if constexpr (FMT == kFmtQ4K) {
        const int pair = c * (KC / 64);
        const uint8_t *blk = row + 144 * (pair >> 2);
        const uint4 *q = reinterpret_cast<const uint4 *>(blk + 16 + 32 * (pair & 3));
#pragma unroll
        for (int i = 0; i < KC / 32; ++i) {
            const uint4 v = __ldg(q + i);
            r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
        }
        const uint4 h = __ldg(reinterpret_cast<const uint4 *>(blk));
        r.w[KC / 8] = h.x, r.w[KC / 8 + 1] = h.y, r.w[KC / 8 + 2] = h.z, r.w[KC / 8 + 3] = h.w;
    } else if constexpr (FMT == kFmtQ80) {
        // the words that the row's own blocks have bytes in
        const int first = c * (KC / 32), blocks = min(KC / 32, (cols + 31) / 32 - first);
        const uint8_t *p = row + 34 * static_cast<int64_t>(first);
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 2);
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p - off);
#pragma unroll
        for (int i = 0; i < Raw<FMT, KC>::kWords; ++i) r.w[i] = 4 * i < 34 * blocks + off ? __ldg(q + i) : 0u;
    } else {
        const int half = c * KC / 128;
        const uint8_t *blk = row + 210 * (half >> 1);
        load_words2<8>(r.w, blk + 64 * (half & 1));                  // low nibbles, 0..31
        load_words2<8>(r.w + 9, blk + 64 * (half & 1) + 32);         // 32..63
        load_words2<8>(r.w + 18, blk + 128 + 32 * (half & 1));       // high bits
    }
}

// fp16 pairs of 32 values: hi pieces, and lo where PA == 2.
template <int PA>
struct Pieces {
    uint32_t hi[16], lo[PA == 2 ? 16 : 1];
    __device__ __forceinline__ void set(int i, float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        hi[i] = tile_h2(h);
        if constexpr (PA == 2) {
            const float2 f = __half22float2(h);
            lo[i] = tile_h2(__floats2half2_rn(a - f.x, b - f.y));
        }
    }
    // two pairs of integers times d, plus m
    __device__ __forceinline__ void set4(int i, __half2 a, __half2 b, float d, float m, __half2 dh, __half2 mh)
    {
        if constexpr (PA == 1) {
            hi[i] = tile_h2(__hfma2(a, dh, mh)), hi[i + 1] = tile_h2(__hfma2(b, dh, mh));
        } else {
            const float2 x = __half22float2(a), y = __half22float2(b);
            set(i, fmaf(x.x, d, m), fmaf(x.y, d, m)), set(i + 1, fmaf(y.x, d, m), fmaf(y.y, d, m));
        }
    }
};

// Values 32 k .. 32 k + 31 of a stage, times 2^s, as fp16 pairs in the order (0, 2), (1, 3) of every four columns.
template <int FMT, int PA, int KC>
__device__ __forceinline__ void take_apart(Pieces<PA> &o, const Raw<FMT, KC> &r, const uint8_t *row, int c, int cols, float up, int k)
{
    if constexpr (FMT == kFmtQ4K) {
        const __half2 k1024 = __float2half2_rn(1024.0f);
        const float2 d2 = __half22float2(tile_b2(r.w[KC / 8]));
        const int pair = (c * (KC / 64) + (k >> 1)) & 3, high = k & 1, sh = (pair & 1) * 16 + 8 * high;     // sub-block 2 pair + high
        const uint32_t A = r.w[KC / 8 + 1] >> sh, B = r.w[KC / 8 + 2] >> sh, C = r.w[KC / 8 + 3] >> sh;
        const uint32_t sc = pair < 2 ? A & 0x3fu : (C & 0x0fu) | ((A >> 2) & 0x30u);
        const uint32_t mm = pair < 2 ? B & 0x3fu : ((C >> 4) & 0x0fu) | ((B >> 2) & 0x30u);
        const __half2 s0 = __hsub2(tile_b2(0x64006400u | sc | sc << 16), k1024);
        const float d = d2.x * up, m = -d2.y * up * static_cast<float>(mm);
        const __half2 dh = __float2half2_rn(d), mh = __float2half2_rn(m);
        const __half2 mul = high ? __hmul2(s0, __float2half2_rn(0.0625f)) : s0;
        const __half2 add = __hmul2(s0, __float2half2_rn(high ? -64.0f : -1024.0f));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = r.w[8 * (k >> 1) + i];
            // scale times quant, exact
            const __half2 a = __hfma2(high ? tile_field<0x00f000f0>(v) : tile_field<0x000f000f>(v), mul, add);
            const __half2 b = __hfma2(high ? tile_field<0x00f000f0>(v >> 8) : tile_field<0x000f000f>(v >> 8), mul, add);
            o.set4(2 * i, a, b, d, m, dh, mh);
        }
    } else if constexpr (FMT == kFmtQ80) {
        // block k: d at byte 34 k, then the quants; none past the row's end
        const int first = c * (KC / 32), base = 17 * (k >> 1);
        const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + 34 * static_cast<int64_t>(first)) & 2) * 8;
        const auto at = [&](int i) { return __funnelshift_r(r.w[i], r.w[i + 1], sh); };
        const __half2 bias = __float2half2_rn(1152.0f), zero = __float2half2_rn(0.0f);
        const float d = first + k < (cols + 31) / 32 ? half_bits_to_float(k & 1 ? at(base + 8) >> 16 : at(base)) * up : 0.0f;
        const __half2 dh = __float2half2_rn(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t q = (k & 1 ? at(base + 9 + i) : __funnelshift_r(at(base + i), at(base + i + 1), 16)) ^ 0x80808080u;
            o.set4(2 * i, __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4240)), bias), __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4341)), bias),
                   d, 0.0f, dh, zero);
        }
    } else {
        // 32 columns t of the half
        const int half = c * KC / 128, t = KC == 128 ? k : 2 * (c & 1) + k;
        const uint8_t *blk = row + 210 * (half >> 1);
        const float d0 = half_at(blk + 208) * up;
        const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(blk) & 2) * 8;
        const __half2 bias = __float2half2_rn(1056.0f), zero = __float2half2_rn(0.0f);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float d = d0 * static_cast<float>(static_cast<int8_t>(__ldg(blk + 192 + 8 * (half & 1) + 2 * t + u)));
            const __half2 dh = __float2half2_rn(d);
#pragma unroll
            for (int i = 4 * u; i < 4 * u + 4; ++i) {
                const uint32_t low = __funnelshift_r(r.w[9 * (k & 1) + i], r.w[9 * (k & 1) + i + 1], sh) >> (t & 2 ? 4 : 0);
                const uint32_t high = __funnelshift_r(r.w[18 + i], r.w[19 + i], sh) >> (2 * t);
                const uint32_t q = (low & 0x0f0f0f0fu) | ((high & 0x03030303u) << 4);
                o.set4(2 * i, __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4240)), bias), __hsub2(tile_b2(__byte_perm(q, 0x64u, 0x4341)), bias),
                       d, 0.0f, dh, zero);
            }
        }
    }
}

struct TileMaps {
    CUtensorMap hi, lo;              // the tokens' operands
    CUtensorMap wa, wb, ha, hb;      // Q4_K: nibbles and scales of a's and b's rows
};

template <int FMT, int PA, int PB, bool PAIRED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(tile_threads(FMT, PB), 1)
tile_kernel(const __grid_constant__ TileMaps maps, const TileArgs a)
{
    constexpr int KC = tile_cols_of_stage(PA), kStage = tile_b_bytes(PA, PB), kRaw = tile_raw_bytes(FMT, PA);
    constexpr int kGroups = tile_groups(FMT, PB), kEpiWarp = tile_epi_warp(FMT, PB);
    constexpr bool kCopied = FMT == kFmtQ4K;                 // the weights' bytes come by TMA
    constexpr uint32_t kACols = KC / 2 * PA, kA0 = 2 * kMaxN;         // tensor-memory columns of a stage of A, and of the first
    static_assert(kA0 + kStages * kACols == 512, "all of tensor memory");
    extern __shared__ uint8_t raw_smem[];
    __shared__ TileShared sh;
    const uint32_t b_base = (smem_u32(raw_smem) + 1023u) & ~1023u, raw_base = b_base + kStages * kStage;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 9);             // (even block) a group's four warps of each block, and the copies
            mbar_init(smem_u32(&sh.empty[i]), 1), mbar_init(smem_u32(&sh.raw_full[i]), 1), mbar_init(smem_u32(&sh.raw_empty[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1), mbar_init(smem_u32(&sh.acc_empty[i]), 2 * kEpiWarps);
            mbar_init(smem_u32(&sh.rs_full[i]), 2), mbar_init(smem_u32(&sh.rs_empty[i]), kEpiWarps);
        }
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.hi);
        if (PB == 2) tma_prefetch_desc(&maps.lo);
        if (kCopied) tma_prefetch_desc(&maps.wa), tma_prefetch_desc(&maps.wb), tma_prefetch_desc(&maps.ha), tma_prefetch_desc(&maps.hb);
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
    const int64_t items = static_cast<int64_t>(a.plan.head[3]) * pairs, first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int nk = a.chunks;
    const int per = PB == 2 ? kFlush : nk;                     // stages an accumulator takes
    const auto set_of = [&](int64_t item) { return a.plan.tile_sets[item / pairs]; };
    const auto tile_of = [&](int64_t item) { return static_cast<int>(item % pairs) * 2 + rank; };
    const auto columns_of = [](int count) { return (count + 31) / 32 * 32; };       // of a product: a pair's are multiples of 32
    // an arrival on a barrier of the even block
    const auto arrive_even = [&](uint64_t *bar) {
        if (rank == 0) mbar_arrive(smem_u32(bar));
        else mbar_arrive_remote(mapa_shared(smem_u32(bar), 0));
    };

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_evict_last_policy(), once = l2_evict_first_policy();
            int n = 0, nr = 0;
            bool ok = true;
            // the weights' bytes run ahead of the tokens by as much as their own barriers allow
            int64_t raw_item = first;
            int raw_c = 0;
            const auto weights = [&]() {
                if (!kCopied || raw_item >= items) return;
                const int st = nr % kStages;
                if (nr >= kStages && !mbar_test(smem_u32(&sh.raw_empty[st]), (nr / kStages - 1) & 1)) return;
                const uint32_t bar = smem_u32(&sh.raw_full[st]), to = raw_base + st * kRaw;
                mbar_arrive_expect_tx(bar, kRaw);
                const int e = set_of(raw_item).expert, tile = tile_of(raw_item), pair = raw_c * (KC / 64);
                const int r0 = static_cast<int>(e * a.a.expert_rows) + tile * (PAIRED ? 64 : 128);
                const int r1 = PAIRED ? static_cast<int>(e * a.b.expert_rows) + tile * 64 : r0 + 64;
                const int at = 144 * (pair >> 2);
                tma_load_2d(to, &maps.wa, at + 16 + 32 * (pair & 3), r0, bar, once);
                tma_load_2d(to + 64 * (KC / 2), &maps.wb, at + 16 + 32 * (pair & 3), r1, bar, once);
                tma_load_2d(to + 128 * (KC / 2), &maps.ha, at, r0, bar, once);
                tma_load_2d(to + 128 * (KC / 2) + 64 * 16, &maps.hb, at, r1, bar, once);
                ++nr;
                if (++raw_c == nk) raw_c = 0, raw_item += step;
            };
            for (int64_t item = first; item < items && ok; item += step) {
                const ExpertSet s = set_of(item);
                const int cols = columns_of(s.count), boxes = (cols / 2 + kTileBoxRows - 1) / kTileBoxRows;
                const int y = s.first + rank * (cols / 2);
                for (int c = 0; c < nk; ++c, ++n) {
                    const int st = n % kStages;
                    weights();
                    if (n >= kStages) {
                        // a bounded wait in which weights go on
                        uint64_t since = 0;
                        while (!mbar_test(smem_u32(&sh.empty[st]), (n / kStages - 1) & 1)) {
                            weights();
                            const uint64_t now = globaltimer_ns();
                            if (since == 0) since = now;
                            if (*abort || now - since > a.wait_ns) {
                                if (!*abort) record_error(a.err, kErrTimeout);
                                *abort = 1;
                                ok = false;
                                break;
                            }
                        }
                        if (!ok) break;
                    }
                    const uint32_t full = smem_u32(&sh.full[st]), to = b_base + st * kStage;
                    if (rank == 0) mbar_arrive_expect_tx(full, 2 * boxes * kTileBoxRows * 2 * KC * PB);
                    if (a.skip_chunk >= 0 && n == a.skip_chunk && blockIdx.x < 2) continue;     // test hook
                    const uint32_t full0 = rank == 0 ? full : mapa_shared(full, 0);
                    for (int b = 0; b < boxes; ++b)
#pragma unroll
                        for (int k = 0; k < KC / 64; ++k) {
                            const uint32_t at = to + k * (kMaxN / 2 * 128) + b * (kTileBoxRows * 128);
                            tma_load_2d_peer(at, &maps.hi, c * KC + k * 64, y + b * kTileBoxRows, full0, keep);
                            if (PB == 2) tma_load_2d_peer(at + kStage / 2, &maps.lo, c * KC + k * 64, y + b * kTileBoxRows, full0, keep);
                        }
                }
            }
            for (const uint64_t since = globaltimer_ns(); ok && kCopied && nr < n && !*abort;) {
                weights();
                if (globaltimer_ns() - since > a.wait_ns) record_error(a.err, kErrTimeout), *abort = 1;
            }
            // every copy lands before the blocks leave: the tokens of both on the even block's barriers, and this one's weights
            if (rank == 0)
                for (int t = max(0, n - kStages); t < n; ++t) mbar_wait(smem_u32(&sh.full[t % kStages]), (t / kStages) & 1, a.wait_ns);
            for (int t = max(0, nr - kStages); t < nr; ++t) mbar_wait(smem_u32(&sh.raw_full[t % kStages]), (t / kStages) & 1, a.wait_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        // The warp stays together and elects a lane for each product: a thread of a branch of its own takes 118 cycles a
        // product whatever its size (measured), an elected one N / 2.
        int n = 0, q = 0;                                      // stages and accumulators so far
        bool ok = rank == 0;
        const uint64_t desc0 = smem_desc_sw128_kmajor(b_base);
        for (int64_t item = first; item < items && ok; item += step) {
            const uint32_t idesc = idesc_f16_f32(256, columns_of(set_of(item).count));
            for (int c = 0; c < nk; ++c, ++n) {
                const int st = n % kStages, buf = q & 1;
                const bool fresh = c % per == 0, last = c + 1 == nk || (c + 1) % per == 0;
                if ((fresh && q >= 2 && !tile_wait_warp<true>(smem_u32(&sh.acc_empty[buf]), (q / 2 - 1) & 1, a, abort)) ||
                    !tile_wait_warp<true>(smem_u32(&sh.full[st]), (n / kStages) & 1, a, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = taddr + buf * kMaxN, at = taddr + kA0 + st * kACols;
                const uint64_t b = desc0 + static_cast<uint64_t>(st * (kStage >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < KC / 16; ++k) {
                        const uint64_t bk = b + (k >> 2) * (kMaxN / 2 * 128 >> 4) + 2 * (k & 3);
                        tc_mma_f16_tmem_a_pair(d, at + 8 * k, bk, idesc, !fresh || k > 0);
                        if constexpr (PA == 2) tc_mma_f16_tmem_a_pair(d, at + KC / 2 + 8 * k, bk, idesc, 1);
                        if constexpr (PB == 2) tc_mma_f16_tmem_a_pair(d, at + 8 * k, bk + (kStage >> 5), idesc, 1);
                    }
                    tc_commit_pair(smem_u32(&sh.empty[st]), 3);
                    if (last) tc_commit_pair(smem_u32(&sh.acc_full[buf]), 3);
                }
                if (last) ++q;
            }
        }
        // products in flight end before tensor memory is freed; the other block sees their last arrivals as well
        for (int t = max(0, n - kStages); t < n; ++t) mbar_wait(smem_u32(&sh.empty[t % kStages]), (t / kStages) & 1, a.wait_ns);
        __syncwarp();
    } else if (warp < kDeqWarp) {
        // rows' scales, an item ahead
        int it = 0;
        for (int64_t item = first; item < items; item += step, ++it) {
            const int buf = it & 1;
            const ExpertSet s = set_of(item);
            float v[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                v[r] = row_scale_of<FMT>(tile_row<PAIRED>(a, s.expert, tile_of(item), (warp - 2) * 64 + r * 32 + lane), a.cols);
            if (it >= 2 && !tile_wait_warp(smem_u32(&sh.rs_empty[buf]), (it / 2 - 1) & 1, a, abort)) break;
#pragma unroll
            for (int r = 0; r < 2; ++r) sh.row_scale[buf][(warp - 2) * 64 + r * 32 + lane] = v[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.rs_full[buf]));
        }
    } else if (warp < kEpiWarp) {
        // takes stages' weights apart: group h has every kGroups-th stage of the block's
        const int group = (warp - kDeqWarp) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        int n = group, it = 0, c = group;
        int64_t item = first;
        while (c >= nk && item < items) c -= nk, ++it, item += step;
        Raw<FMT, KC> next;
        const uint8_t *at = nullptr;
        if (!kCopied && item < items) {
            // the next stage's bytes are on their way while one is taken apart
            at = tile_row<PAIRED>(a, set_of(item).expert, tile_of(item), row);
            load_raw<FMT, KC>(next, at, c, a.cols);
        }
        // this thread's row among the copied ones: gate's 64, then up's
        const int raw_row = PAIRED ? (row >> 5) * 16 + (row & 15) + (row & 16 ? 64 : 0) : row;
        float up = 0.0f;
        int have = -1;
        while (item < items) {
            const int st = n % kStages;
            Raw<FMT, KC> now;
            const uint8_t *now_at = at;
            const int now_c = c, now_it = it;
            if constexpr (kCopied) {
                if (!tile_wait_warp(smem_u32(&sh.raw_full[st]), (n / kStages) & 1, a, abort)) break;
                const uint32_t from = raw_base + st * kRaw;
                // chunks of 16 bytes are swapped within 64 (32) bytes by the row, as the copy's swizzle does
                const uint32_t x = KC == 128 ? (raw_row >> 1) & 3 : (raw_row >> 2) & 1;
#pragma unroll
                for (int i = 0; i < KC / 32; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(raw_smem + (from - smem_u32(raw_smem)) + raw_row * (KC / 2) + ((i ^ x) * 16));
                    now.w[4 * i] = v.x, now.w[4 * i + 1] = v.y, now.w[4 * i + 2] = v.z, now.w[4 * i + 3] = v.w;
                }
                const uint4 h = *reinterpret_cast<const uint4 *>(raw_smem + (from - smem_u32(raw_smem)) + 128 * (KC / 2) + raw_row * 16);
                now.w[KC / 8] = h.x, now.w[KC / 8 + 1] = h.y, now.w[KC / 8 + 2] = h.z, now.w[KC / 8 + 3] = h.w;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.raw_empty[st]));
            } else {
                now = next;
            }
            c += kGroups;
            bool moved = false;
            while (c >= nk && item < items) c -= nk, ++it, item += step, moved = true;
            if (!kCopied && item < items) {
                if (moved) at = tile_row<PAIRED>(a, set_of(item).expert, tile_of(item), row);
                load_raw<FMT, KC>(next, at, c, a.cols);
            }
            if (have != now_it) {
                if (!tile_wait_warp(smem_u32(&sh.rs_full[now_it & 1]), (now_it / 2) & 1, a, abort)) break;
                up = sh.row_scale[now_it & 1][row];
                have = now_it;
            }
            if (n >= kStages && !tile_wait_warp(smem_u32(&sh.empty[st]), (n / kStages - 1) & 1, a, abort)) break;
            tc_fence_after();
            const uint32_t to = taddr + (static_cast<uint32_t>(quarter * 32) << 16) + kA0 + st * kACols;
#pragma unroll
            for (int k = 0; k < KC / 32; ++k) {
                Pieces<PA> o;
                take_apart<FMT, PA, KC>(o, now, now_at, now_c, a.cols, up, k);
                tmem_st_32x32b_x16(to + 16 * k, o.hi);
                if constexpr (PA == 2) tmem_st_32x32b_x16(to + KC / 2 + 16 * k, o.lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even(&sh.full[st]);
            n += kGroups;
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane, part = (warp - kEpiWarp) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        int it = 0, q = 0;
        bool ok = true;
        for (int64_t item = first; item < items && ok; item += step, ++it) {
            const ExpertSet s = set_of(item);
            const int tile = tile_of(item);
            float back = 0.0f;
            // a warp's 64 tokens from c_first on
            const int c_first = part * 64;
            float *ts = sh.token_scale[warp - kEpiWarp];
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
                if (back == 0.0f) back = 1.0f / sh.row_scale[it & 1][row];      // a power of two
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
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.rs_empty[it & 1]));
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
    constexpr int smem = tile_smem(FMT, PA, PB), KC = tile_cols_of_stage(PA);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    TileMaps maps;
    const gemm::EncodeTiledFn enc = gemm::encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const auto encode = [&](CUtensorMap *m, bool bytes, const void *p, int64_t cols, int64_t rows, int box_cols, int box_rows,
                            CUtensorMapSwizzle swizzle) {
        const int64_t size = bytes ? 1 : 2;
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * size)};
        const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
        return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(p), dims, strides,
                   box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    bool ok = encode(&maps.hi, false, t.hi, t.cols, t.rows, 64, kTileBoxRows, CU_TENSOR_MAP_SWIZZLE_128B);
    maps.lo = maps.hi;
    if (PB == 2) ok = ok && encode(&maps.lo, false, t.lo, t.cols, t.rows, 64, kTileBoxRows, CU_TENSOR_MAP_SWIZZLE_128B);
    maps.wa = maps.wb = maps.ha = maps.hb = maps.hi;
    if (FMT == kFmtQ4K) {
        const CUtensorMapSwizzle swizzle = KC == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
        const auto rows = [&](const Weights &w) { return (a.experts - 1) * w.expert_rows + a.rows; };
        ok = ok && encode(&maps.wa, true, a.a.w, a.a.row_bytes, rows(a.a), KC / 2, 64, swizzle) &&
             encode(&maps.wb, true, a.b.w, a.b.row_bytes, rows(a.b), KC / 2, 64, swizzle) &&
             encode(&maps.ha, true, a.a.w, a.a.row_bytes, rows(a.a), 16, 64, CU_TENSOR_MAP_SWIZZLE_NONE) &&
             encode(&maps.hb, true, a.b.w, a.b.row_bytes, rows(a.b), 16, 64, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2)), cfg.blockDim = dim3(tile_threads(FMT, PB));
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
