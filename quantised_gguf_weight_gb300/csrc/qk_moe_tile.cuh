// qk_moe_tile.cuh -- the experts' products for many tokens an expert: tiles of
// 128 weight rows x up to 128 tokens on the tcgen05 tensor cores.
//
// A thread block keeps going over its items.  Its warps have roles: two groups
// of four take the weights apart, a thread a row, and leave them as the A
// operand in tensor memory; a thread issues the products; a thread fetches the
// tokens' operands by TMA, half of them each of two neighbouring blocks for
// both (they have the same tokens and neighbouring rows); four warps turn
// finished accumulators into outputs while the next item's products run; two
// look over the next item's rows for their largest scale.
//
// Weights are fp16 after a power of two a row that puts the largest value that
// the row's scales allow into [2^14, 2^15): one rounding (Q4_K: the minimum's
// and the sum's) of 2^-12 for bf16 activations and outputs.  Else they are two
// such pieces, and fp32 activations too (qk_moe.cuh); the product of the two
// low pieces is left out.
//
// Why A is in tensor memory: a product of 128 x 128 x 16 takes 64 cycles, in which
// shared memory moves 8 KB; the tokens' operand alone is 4 KB written and 4 KB
// read.  From shared memory (measured) a product of 192 tokens takes 145 cycles
// where one from tensor memory takes 100.
#pragma once

#include "qk_moe.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace moe {

constexpr int kDeqWarp = 4, kDeqGroups = 2, kEpiWarp = 12;   // first warps of the roles
constexpr int kFlush = 4;                                    // stages whose products one accumulator takes, with fp32 accuracy
constexpr int kEpiWarps = 8;                                 // two threads share a row's tokens
constexpr int kTileThreads = 32 * (kEpiWarp + kEpiWarps);
constexpr int kStages = 4;                                   // of both operands
constexpr int kMaxN = 128;                                   // tokens of a set
// Columns of a stage: eight products for each (a wait costs the issuing warp as much as three of them).
__host__ __device__ constexpr int tile_cols_of_stage(int PA) { return PA == 1 ? 128 : 64; }
__host__ __device__ constexpr int tile_b_bytes(int PA, int PB) { return kMaxN * 2 * tile_cols_of_stage(PA) * PB; }
__host__ __device__ constexpr int tile_smem(int PA, int PB) { return kStages * tile_b_bytes(PA, PB) + 1024; }

struct TileShared {
    uint64_t full[kStages], empty_b[kStages], empty_a[kStages], acc_full[2], acc_empty[2], rs_full[2], rs_empty[2];
    float row_scale[2][128];                                 // 2^s of the rows
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

// One lane of the (converged) warp is elected.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void tma_load_2d_both(uint32_t dst, const CUtensorMap *m, int32_t x, int32_t y, uint32_t bar,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5, %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar), "h"(static_cast<uint16_t>(3)), "l"(policy)
        : "memory");
}
// Arrive once on the mbarrier at `bar` of both blocks when every product issued so far by this thread has completed.
__device__ __forceinline__ void tc_commit_both(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
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

template <int FMT, int PA, int PB, bool PAIRED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
tile_kernel(const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo, const TileArgs a)
{
    constexpr int KC = tile_cols_of_stage(PA), kStage = tile_b_bytes(PA, PB);
    constexpr uint32_t kACols = KC / 2 * PA, kA0 = 2 * kMaxN;         // tensor-memory columns of a stage of A, and of the first
    static_assert(kA0 + kStages * kACols == 512, "all of tensor memory");
    extern __shared__ uint8_t raw_smem[];
    __shared__ TileShared sh;
    const uint32_t b_base = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 5);                     // a group's four warps, and the copies
            mbar_init(smem_u32(&sh.empty_b[i]), 2), mbar_init(smem_u32(&sh.empty_a[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1), mbar_init(smem_u32(&sh.acc_empty[i]), kEpiWarps);
            mbar_init(smem_u32(&sh.rs_full[i]), 2), mbar_init(smem_u32(&sh.rs_empty[i]), kEpiWarps);
        }
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_hi);
        if (PB == 2) tma_prefetch_desc(&map_lo);
    }
    if (warp == 1) {
        tmem_alloc_1(smem_u32(&sh.tmem), 512);
        tmem_relinquish_1();
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

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_evict_last_policy();
            int n = 0;
            bool ok = true;
            for (int64_t item = first; item < items && ok; item += step) {
                const ExpertSet s = set_of(item);
                const int boxes = (s.count + kTileBoxRows - 1) / kTileBoxRows;
                for (int c = 0; c < nk; ++c, ++n) {
                    const int st = n % kStages;
                    if (n >= kStages && !tile_wait(smem_u32(&sh.empty_b[st]), (n / kStages - 1) & 1, a, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = smem_u32(&sh.full[st]), to = b_base + st * kStage;
                    mbar_arrive_expect_tx(full, boxes * kTileBoxRows * 2 * KC * PB);
                    if (a.skip_chunk >= 0 && n == a.skip_chunk && blockIdx.x < 2) continue;     // test hook
                    for (int b = rank; b < boxes; b += 2)
#pragma unroll
                        for (int k = 0; k < KC / 64; ++k) {
                            const uint32_t at = to + k * (kMaxN * 128) + b * (kTileBoxRows * 128);
                            tma_load_2d_both(at, &map_hi, c * KC + k * 64, s.first + b * kTileBoxRows, full, keep);
                            if (PB == 2)
                                tma_load_2d_both(at + kStage / 2, &map_lo, c * KC + k * 64, s.first + b * kTileBoxRows, full, keep);
                        }
                }
            }
            // every copy that this block has asked for lands before it leaves (the other's, too: the closing barrier)
            for (int t = max(0, n - kStages); t < n; ++t) mbar_wait(smem_u32(&sh.full[t % kStages]), (t / kStages) & 1, a.wait_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        // The warp stays together and elects a lane for each product: a thread of a branch of its own takes 118 cycles a
        // product whatever its size (measured), an elected one N / 2.
        int n = 0, q = 0;                                      // stages and accumulators so far
        bool ok = true;
        const uint64_t desc0 = smem_desc_sw128_kmajor(b_base);
        for (int64_t item = first; item < items && ok; item += step) {
            const int count = set_of(item).count;
            const uint32_t idesc = idesc_f16_f32(128, (count + 15) / 16 * 16);
            for (int c = 0; c < nk; ++c, ++n) {
                const int st = n % kStages, buf = q & 1;
                const bool fresh = c % per == 0, last = c + 1 == nk || (c + 1) % per == 0;
                if ((fresh && q >= 2 && !tile_wait_warp(smem_u32(&sh.acc_empty[buf]), (q / 2 - 1) & 1, a, abort)) ||
                    !tile_wait_warp(smem_u32(&sh.full[st]), (n / kStages) & 1, a, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = taddr + buf * kMaxN, at = taddr + kA0 + st * kACols;
                const uint64_t b = desc0 + static_cast<uint64_t>(st * (kStage >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < KC / 16; ++k) {
                        const uint64_t bk = b + (k >> 2) * (kMaxN * 128 >> 4) + 2 * (k & 3);
                        tc_mma_f16_tmem_a(d, at + 8 * k, bk, idesc, !fresh || k > 0);
                        if constexpr (PA == 2) tc_mma_f16_tmem_a(d, at + KC / 2 + 8 * k, bk, idesc, 1);
                        if constexpr (PB == 2) tc_mma_f16_tmem_a(d, at + 8 * k, bk + (kStage >> 5), idesc, 1);
                    }
                    tc_commit_1(smem_u32(&sh.empty_a[st]));
                    tc_commit_both(smem_u32(&sh.empty_b[st]));
                    if (last) tc_commit_1(smem_u32(&sh.acc_full[buf]));
                }
                if (last) ++q;
            }
        }
        // products in flight end before tensor memory is freed
        if (n > 0) mbar_wait(smem_u32(&sh.empty_a[(n - 1) % kStages]), ((n - 1) / kStages) & 1, a.wait_ns);
        // and the other block's arrivals have come before this one leaves
        for (int t = max(0, n - kStages); t < n; ++t) mbar_wait(smem_u32(&sh.empty_b[t % kStages]), (t / kStages) & 1, a.wait_ns);
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
        // takes stages' weights apart: group h has every other stage of the block's
        const int group = (warp - kDeqWarp) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        int n = group, it = 0, c = group;
        int64_t item = first;
        while (c >= nk) c -= nk, ++it, item += step;
        // the next stage's bytes are on their way while one is taken apart
        Raw<FMT, KC> next;
        const uint8_t *at = nullptr;
        if (item < items) {
            at = tile_row<PAIRED>(a, set_of(item).expert, tile_of(item), row);
            load_raw<FMT, KC>(next, at, c, a.cols);
        }
        float up = 0.0f;
        int have = -1;
        while (item < items) {
            const Raw<FMT, KC> now = next;
            const uint8_t *now_at = at;
            const int now_c = c, now_it = it;
            c += kDeqGroups;
            bool moved = false;
            while (c >= nk) c -= nk, ++it, item += step, moved = true;
            if (item < items) {
                if (moved) at = tile_row<PAIRED>(a, set_of(item).expert, tile_of(item), row);
                load_raw<FMT, KC>(next, at, c, a.cols);
            }
            if (have != now_it) {
                if (!tile_wait_warp(smem_u32(&sh.rs_full[now_it & 1]), (now_it / 2) & 1, a, abort)) break;
                up = sh.row_scale[now_it & 1][row];
                have = now_it;
            }
            const int st = n % kStages;
            if (n >= kStages && !tile_wait_warp(smem_u32(&sh.empty_a[st]), (n / kStages - 1) & 1, a, abort)) break;
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
            if (lane == 0) mbar_arrive(smem_u32(&sh.full[st]));
            n += kDeqGroups;
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
                if (lane == 0) mbar_arrive(smem_u32(&sh.acc_empty[q & 1]));
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
    if (warp == 1) tmem_dealloc_1(taddr, 512);
}

template <int FMT, int PA, int PB, bool PAIRED>
cudaError_t tile_launch_as(const CUtensorMap &hi, const CUtensorMap &lo, const TileArgs &a, int sms, cudaStream_t st)
{
    const auto kern = tile_kernel<FMT, PA, PB, PAIRED>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem(PA, PB));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2)), cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tile_smem(PA, PB), cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, hi, lo, a);
}

template <int FMT, bool PAIRED>
cudaError_t tile_launch_pieces(const CUtensorMap &hi, const CUtensorMap &lo, const TileArgs &a, int sms, cudaStream_t st)
{
    if (a.w_pieces == 1) return tile_launch_as<FMT, 1, 1, PAIRED>(hi, lo, a, sms, st);
    return a.pieces == 1 ? tile_launch_as<FMT, 2, 1, PAIRED>(hi, lo, a, sms, st) : tile_launch_as<FMT, 2, 2, PAIRED>(hi, lo, a, sms, st);
}

template <int FMT>
cudaError_t tile_launch(const CUtensorMap &hi, const CUtensorMap &lo, const TileArgs &a, bool paired, int sms, cudaStream_t st)
{
    return paired ? tile_launch_pieces<FMT, true>(hi, lo, a, sms, st) : tile_launch_pieces<FMT, false>(hi, lo, a, sms, st);
}

}  // namespace moe
}  // namespace qk
