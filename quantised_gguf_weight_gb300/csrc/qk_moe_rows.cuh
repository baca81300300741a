// qk_moe_rows.cuh -- the experts' products for few tokens an expert: a pass
// over the expert's weights for every 16 tokens, in the m16n8k16 products of
// the tensor cores.
//
// The weights are the 16-row operand.  Quants are exact in fp16 (Q4_K: quant
// times sub-block scale, at most 945, too), so a product's only roundings are
// those of the activations' pieces (qk_moe.cuh) and of the fp32 sums:
//   Q4_K  sum over a super-block of (sc q) x by one product chain, of m by one
//         more product with the sub-blocks' sums of x; then d and dmin in fp32
//   Q8_0  a product chain a block of 32, then d in fp32
//   Q6_K  a product a sub-block of 16, then d sc in fp32
// A lane of a product holds four values of each of its rows; which columns they
// are is free as long as both operands agree, so that a lane's values lie
// together in the block (operands are laid out to match, qk_moe.cu).
//
// A warp takes a tile of 16 rows (8 gate rows and their 8 up rows, so that a
// lane has both sums of an output), or a part of its columns where tiles are few.
// Its weights come through a ring of its own in shared memory, 16 bytes an
// asynchronous copy, which runs on from one item to the next; the tokens'
// operands come through a ring that the thread block's warps share, one bulk copy
// an octet and unit.  (With operands read through L1 instead, 8 KB for every 2.3
// KB of weights, 64 tokens of 8 of 128 experts took 132 us for gate and up.)
//
// Measured, 64 fp32 tokens of 8 of 128 experts of 768 x 2048 in Q4_K: gate and up
// 87 us, 2.4 TB/s of weights, down 52; 16 bf16 tokens of 6 of 64 experts of 1408 x
// 2048 in Q8_0: 104 us, 2.7 TB/s, and 61.  What bounds it is the way from shared
// memory into the products: a scheduler issues 0.44 to 0.54 instructions a cycle
// and its warps wait most for the queue of shared-memory loads (Q8_0: eight for a
// row pair's 32 columns, in blocks of 34 bytes).
#pragma once

#include <type_traits>

#include "qk_moe.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace moe {

constexpr int kRowTiles = 1;                      // 16-row tiles of a warp
// Shared-memory pitch of a row's unit: 16-byte chunks that hold it wherever it starts.  Q4_K's starts on one.
__host__ __device__ constexpr int row_pitch(int fmt) { return fmt == kFmtQ4K ? 144 : fmt == kFmtQ80 ? 288 : 224; }
__host__ __device__ constexpr int row_chunks(int fmt) { return fmt == kFmtQ4K ? 9 : fmt == kFmtQ80 ? 18 : 14; }
__host__ __device__ constexpr int ring_stages(int fmt) { return fmt == kFmtQ4K ? 3 : 2; }
constexpr int kOpStages = 4;                      // units of the tokens' operands
__host__ __device__ constexpr int ring_bytes(int fmt) { return ring_stages(fmt) * kRowTiles * 16 * row_pitch(fmt); }
__host__ __device__ constexpr int op_bytes(int fmt, int P) { return kSetOctets * static_cast<int>(octet_unit_bytes(fmt, P)); }
__host__ __device__ constexpr int rows_smem(int fmt, int P) { return kRowWarps * ring_bytes(fmt) + kOpStages * op_bytes(fmt, P); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t b) { return *reinterpret_cast<__half2 *>(&b); }
// (w & mask) | 0x64006400: the field in the mantissa of 1024
template <uint32_t MASK>
__device__ __forceinline__ __half2 field1024(uint32_t w)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "n"(0x64006400));
    return bits_h2(r);
}

__device__ __forceinline__ uint32_t lds32(uint32_t p)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t p)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
    return v;
}
__device__ __forceinline__ int lds_s8(uint32_t p)
{
    int v;
    asm volatile("ld.shared.s8 %0, [%1];" : "=r"(v) : "r"(p));
    return v;
}
// the 32-bit word at a 2-byte aligned place
__device__ __forceinline__ uint32_t lds32_2(uint32_t p)
{
    const uint32_t q = p & ~3u;
    return __funnelshift_r(lds32(q), lds32(q + 4), (p & 2u) * 8);
}

// The products of one unit (256 columns): total[m][n] += rows (g, g + 8) of tile m x octet n's columns.
// st: the tiles' unit in shared memory; al[m][2]: byte offsets of rows g and g + 8 inside their chunks; x: the octets'
// operands, step i of piece p at 512 i + 4096 p.
template <int FMT, int P, int NT>
__device__ __forceinline__ void unit_products(float (&total)[kRowTiles][NT][4], uint32_t st, const uint32_t (&al)[kRowTiles][2],
                                              int blocks, uint32_t x, int lane)
{
    constexpr int M = kRowTiles, OB = static_cast<int>(octet_unit_bytes(FMT, P));
    const int g = lane >> 2, c = lane & 3;
    x += lane * 16;
    const auto row = [&](int m, int r) { return st + (16 * m + 8 * r + g) * row_pitch(FMT) + al[m][r]; };
    if constexpr (FMT == kFmtQ4K) {
        // lane c has sub-blocks 2c and 2c + 1: 32 bytes of nibbles.  The low and the high nibbles' products are summed apart:
        // the tensor cores cut a sum at 2^-24 of it, so short sums are the more exact.
        float dd[M][2], dm[M][2];
        __half2 sl[M][2], sb[M][2], shi[M][2], shb[M][2];     // scale of the low nibbles' sub-block, -1024 of it; high: / 16, -64
        float acc[M][NT][2][4], low[M][NT][4];
#pragma unroll
        for (int t = 0; t < M; ++t) {
            uint32_t m[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 h = lds128(row(t, r));
                const float2 d2 = __half22float2(bits_h2(h.x));
                dd[t][r] = d2.x, dm[t][r] = d2.y;
                const int sh = (c & 1) * 16;
                const uint32_t A = h.y >> sh, B = h.z >> sh, C = h.w >> sh;
                const uint32_t sc = c < 2 ? A & 0x3f3fu : (C & 0x0f0fu) | ((A >> 2) & 0x3030u);
                const uint32_t mm = c < 2 ? B & 0x3f3fu : ((C >> 4) & 0x0f0fu) | ((B >> 2) & 0x3030u);
                const __half2 k1024 = __float2half2_rn(1024.0f);
                const __half2 s0 = __hsub2(bits_h2(__byte_perm(sc, 0x64u, 0x4040)), k1024);
                const __half2 s1 = __hsub2(bits_h2(__byte_perm(sc, 0x64u, 0x4141)), k1024);
                sl[t][r] = s0, sb[t][r] = __hmul2(s0, __float2half2_rn(-1024.0f));
                shi[t][r] = __hmul2(s1, __float2half2_rn(0.0625f)), shb[t][r] = __hmul2(s1, __float2half2_rn(-64.0f));
                m[r] = h2_bits(__hmul2(__hsub2(bits_h2(__byte_perm(mm, 0x64u, 0x4140)), k1024), __float2half2_rn(32.0f)));
            }
            const uint32_t a[4] = {m[0], m[1], m[0], m[1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t][n][0][j] = acc[t][n][1][j] = low[t][n][j] = 0.0f;
                const uint32_t at = x - lane * 8 + n * OB + P * kPieceBytes;
                mma16(low[t][n], a, lds32(at), lds32(at + 4));
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint4 w[M][2];
#pragma unroll
            for (int t = 0; t < M; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) w[t][r] = lds128(row(t, r) + 16 + 32 * c + 16 * q);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4 o[NT][P];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int p = 0; p < P; ++p) o[n][p] = lds128(x + n * OB + p * kPieceBytes + (4 * q + k) * 512);
#pragma unroll
                for (int t = 0; t < M; ++t) {
                    const uint32_t v0 = k == 0 ? w[t][0].x : k == 1 ? w[t][0].y : k == 2 ? w[t][0].z : w[t][0].w;
                    const uint32_t v1 = k == 0 ? w[t][1].x : k == 1 ? w[t][1].y : k == 2 ? w[t][1].z : w[t][1].w;
                    const uint32_t a[4] = {h2_bits(__hfma2(field1024<0x000f000f>(v0), sl[t][0], sb[t][0])),
                                           h2_bits(__hfma2(field1024<0x000f000f>(v1), sl[t][1], sb[t][1])),
                                           h2_bits(__hfma2(field1024<0x000f000f>(v0 >> 8), sl[t][0], sb[t][0])),
                                           h2_bits(__hfma2(field1024<0x000f000f>(v1 >> 8), sl[t][1], sb[t][1]))};
                    const uint32_t b[4] = {h2_bits(__hfma2(field1024<0x00f000f0>(v0), shi[t][0], shb[t][0])),
                                           h2_bits(__hfma2(field1024<0x00f000f0>(v1), shi[t][1], shb[t][1])),
                                           h2_bits(__hfma2(field1024<0x00f000f0>(v0 >> 8), shi[t][0], shb[t][0])),
                                           h2_bits(__hfma2(field1024<0x00f000f0>(v1 >> 8), shi[t][1], shb[t][1]))};
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16(acc[t][n][0], a, o[n][p].x, o[n][p].y);
                            mma16(acc[t][n][1], b, o[n][p].z, o[n][p].w);
                        }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    total[t][n][j] += dd[t][j >> 1] * (acc[t][n][0][j] + acc[t][n][1][j]) - dm[t][j >> 1] * low[t][n][j];
    } else if constexpr (FMT == kFmtQ80) {
        const __half2 bias = __float2half2_rn(1152.0f);
        const auto pair = [&](uint32_t v, int sel) { return h2_bits(__hsub2(bits_h2(__byte_perm(v, 0x64u, sel)), bias)); };
#pragma unroll 2
        for (int i = 0; i < blocks; ++i) {
            uint4 o[NT][P];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < P; ++p) o[n][p] = lds128(x + n * OB + p * kPieceBytes + i * 512);
#pragma unroll
            for (int t = 0; t < M; ++t) {
                uint32_t v[2][2];
                float dd[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t blk = row(t, r) + 34 * i;
                    dd[r] = half_bits_to_float(lds16(blk));
                    const uint32_t p = blk + 2 + 8 * c, q = p & ~3u, sh = (p & 2u) * 8;
                    const uint32_t w0 = lds32(q), w1 = lds32(q + 4), w2 = sh ? lds32(q + 8) : 0u;
                    v[r][0] = __funnelshift_r(w0, w1, sh) ^ 0x80808080u, v[r][1] = __funnelshift_r(w1, w2, sh) ^ 0x80808080u;
                }
                const uint32_t a[4] = {pair(v[0][0], 0x4240), pair(v[1][0], 0x4240), pair(v[0][0], 0x4341), pair(v[1][0], 0x4341)};
                const uint32_t b[4] = {pair(v[0][1], 0x4240), pair(v[1][1], 0x4240), pair(v[0][1], 0x4341), pair(v[1][1], 0x4341)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        mma16(acc, a, o[n][p].x, o[n][p].y);
                        mma16(acc, b, o[n][p].z, o[n][p].w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) total[t][n][j] += dd[j >> 1] * acc[j];
                }
            }
        }
    } else {
        const __half2 bias = __float2half2_rn(1056.0f);
        const auto pair = [&](uint32_t v, int sel) { return h2_bits(__hsub2(bits_h2(__byte_perm(v, 0x64u, sel)), bias)); };
        float dd[M][2];
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) dd[t][r] = half_bits_to_float(lds16(row(t, r) + 208));
#pragma unroll 1
        for (int hu = 0; hu < 4; ++hu) {             // half n = hu / 2, 16 positions u = hu % 2
            uint4 o[NT][P][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k) o[n][p][k] = lds128(x + n * OB + p * kPieceBytes + (2 * hu + k) * 512);
#pragma unroll
            for (int s = 0; s < M; ++s) {
                uint32_t A[2], B[2], H[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t blk = row(s, r) + 16 * (hu & 1) + 4 * c;
                    A[r] = lds32_2(blk + 64 * (hu >> 1)), B[r] = lds32_2(blk + 64 * (hu >> 1) + 32);
                    H[r] = lds32_2(blk + 128 + 32 * (hu >> 1));
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    uint32_t v[2];
                    float ds[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t lowb = ((t & 1 ? B[r] : A[r]) >> (t & 2 ? 4 : 0)) & 0x0f0f0f0fu;
                        const uint32_t high = (t < 2 ? H[r] << (4 - 2 * t) : H[r] >> (2 * t - 4)) & 0x30303030u;
                        v[r] = lowb | high;
                        ds[r] = dd[s][r] * lds_s8(row(s, r) + 192 + 8 * (hu >> 1) + 2 * t + (hu & 1));
                    }
                    const uint32_t a[4] = {pair(v[0], 0x4240), pair(v[1], 0x4240), pair(v[0], 0x4341), pair(v[1], 0x4341)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const uint4 q = o[n][p][t >> 1];
                            mma16(acc, a, t & 1 ? q.z : q.x, t & 1 ? q.w : q.y);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) total[s][n][j] += ds[j >> 1] * acc[j];
                    }
                }
            }
        }
    }
}

struct RowsShared {
    uint64_t full[kOpStages], empty[kOpStages];
    float join[kRowWarps * kRowTiles * kSetOctets * 4 * 32];
    int abort;
    int failed;                // a computing warp has left its units; written before the parts' barrier only
};

// A bounded wait of a whole warp; one that runs out ends every other of the block.
__device__ __forceinline__ bool rows_wait(uint32_t bar, uint32_t parity, const RowsArgs &a, volatile int *abort)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t deadline = globaltimer_ns() + a.wait_ns;
        for (uint32_t i = 1; !*abort && !(ok = mbar_try_wait(bar, parity)); ++i)
            if ((i & 31u) == 0 && globaltimer_ns() > deadline) {
                *abort = 1;
                record_error(a.err, kErrTimeout);
            }
    }
    return __all_sync(~0u, ok);
}

// A warp's way through its items' units: item, the pair of tiles in it, the units [u, u1) left of it.
struct Cursor {
    int item, u, u1;
};

template <int FMT, int P, bool PAIRED>
__global__ void __launch_bounds__((kRowWarps + 1) * 32, 1) rows_kernel(const RowsArgs a)
{
    constexpr int S = ring_stages(FMT), UB = unit_bytes(FMT), PITCH = row_pitch(FMT), CH = row_chunks(FMT), M = kRowTiles;
    constexpr int OB = static_cast<int>(octet_unit_bytes(FMT, P)), OPS = op_bytes(FMT, P), SLOT = M * 16 * PITCH;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ RowsShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &sh.abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kOpStages; ++i) mbar_init(smem_u32(&sh.full[i]), 1), mbar_init(smem_u32(&sh.empty[i]), kRowWarps);
        sh.abort = sh.failed = 0;
        fence_barrier_init();
    }
    __syncthreads();
    let_next_start();
    wait_for_previous();
    // warps that share a pair's units: enough for every SM's warps to have work where pairs are few
    const int sets = a.plan.head[0], pairs = (a.tiles + M - 1) / M;
    int kw = 1;
    while (kw < kRowWarps && 2 * kw <= a.units && static_cast<int64_t>(sets) * pairs * kw < kRowWarps * a.sms) kw *= 2;
    const int per = kRowWarps / kw, blocks = (pairs + per - 1) / per, items = sets * blocks;      // (the caller sees to 31 bits)
    const uint32_t ops = smem_u32(smem) + kRowWarps * ring_bytes(FMT);

    if (warp == kRowWarps) {
        // the tokens' operands, every unit of every item
        const uint64_t keep = l2_evict_last_policy();
        int n = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const ExpertSet s = a.plan.sets[item / blocks];
            const int octets = (s.count + 7) / 8;
            bool ok = true;
            for (int u = 0; u < a.units && ok; ++u, ++n) {
                const int st = n % kOpStages;
                if (n >= kOpStages && !(ok = rows_wait(smem_u32(&sh.empty[st]), (n / kOpStages - 1) & 1, a, abort))) break;
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&sh.full[st]);
                    mbar_arrive_expect_tx(bar, octets * OB);
                    for (int o = 0; o < octets; ++o)
                        bulk_g2s(ops + st * OPS + o * OB, a.x + (static_cast<int64_t>(s.octet + o) * a.units + u) * OB, OB, bar, keep);
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        for (int t = max(0, n - kOpStages); t < n; ++t) mbar_wait(smem_u32(&sh.full[t % kOpStages]), (t / kOpStages) & 1, a.wait_ns);
        return;
    }

    const int g = lane >> 2, c = lane & 3, part = warp % kw;
    const uint32_t ring = smem_u32(smem) + warp * ring_bytes(FMT);
    const int u0 = a.units * part / kw, u1 = a.units * (part + 1) / kw;
    const auto pair_of = [&](int item) { return item % blocks * per + warp / kw; };
    // rows past the last are read as the last and not written; row i of a pair's 32
    const auto row_of = [&](int expert, int pair, int i) -> const uint8_t * {
        const int tile = pair * M + (i >> 4), row = PAIRED ? min(tile * 8 + (i & 7), a.rows - 1) : min(tile * 16 + (i & 15), a.rows - 1);
        const Weights &w = i & 8 ? a.b : a.a;
        return w.w + (expert * w.expert_rows + row) * w.row_bytes;
    };

    // what is fetched runs S - 1 units ahead of what is computed, over the ends of items
    Cursor f = {static_cast<int>(blockIdx.x), u0, u1};
    const uint8_t *from[2 * M];
    int slot_in = 0;
    const auto aim = [&]() {
        if (f.item >= items) return;
        const int expert = a.plan.sets[f.item / blocks].expert, pair = pair_of(f.item);
#pragma unroll
        for (int o = 0; o < 2 * M; ++o) from[o] = row_of(expert, pair, 8 * o + (lane >> 2));
    };
    aim();
    const auto fetch = [&]() {
        if (f.item < items && pair_of(f.item) < pairs) {
            const int64_t off = static_cast<int64_t>(f.u) * UB;
            const int left = static_cast<int>(min(static_cast<int64_t>(UB), a.a.row_bytes - off)) - 16 * c;
            const uint32_t to = ring + slot_in * SLOT + (lane >> 2) * PITCH + 16 * c;
#pragma unroll
            for (int o = 0; o < 2 * M; ++o) {
                const uint8_t *p = from[o] + off;
                int bytes = left;
                if constexpr (FMT != kFmtQ4K) {
                    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
                    p -= skew, bytes += skew;
                }
                p += 16 * c;
#pragma unroll
                for (int i = 0; i < (CH + 3) / 4; ++i)
                    if (64 * i < bytes) cp_async16(to + 8 * o * PITCH + 64 * i, p + 64 * i);
            }
        }
        cp_async_commit();
        slot_in = slot_in + 1 == S ? 0 : slot_in + 1;
        if (++f.u >= f.u1 && f.item < items) f.item += gridDim.x, f.u = u0, aim();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch();

    int slot = 0, n = 0;
    const auto run = [&](auto nt, const ExpertSet &s, int pair) -> bool {
        constexpr int NT = decltype(nt)::value;
        float total[M][NT][4];
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) total[t][k][j] = 0.0f;
        uint32_t start[M][2];
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) start[t][r] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row_of(s.expert, pair, 16 * t + 8 * r + g)) & 15);
        bool ok = true;
        for (int u = 0; u < a.units; ++u, ++n) {
            const int st = n % kOpStages;
            const bool mine = u >= u0 && u < u1;
            if (mine) cp_async_wait<S - 2>();
            if (!(ok = rows_wait(smem_u32(&sh.full[st]), (n / kOpStages) & 1, a, abort))) break;
            if (mine) {
                __syncwarp();                // everyone's copies of this unit have landed, and the slot before it is free
                fetch();
                if (pair < pairs) {
                    uint32_t al[M][2];
#pragma unroll
                    for (int t = 0; t < M; ++t)
#pragma unroll
                        for (int r = 0; r < 2; ++r) al[t][r] = (start[t][r] + (UB % 16 ? u * UB : 0)) & 15;
                    const int in_row = FMT == kFmtQ80 ? min(8, (a.cols + 31) / 32 - 8 * u) : 8;
                    unit_products<FMT, P, NT>(total, ring + slot * SLOT, al, in_row, ops + st * OPS, lane);
                }
                slot = slot + 1 == S ? 0 : slot + 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st]));
        }
        if (kw == 1 && !ok) return false;
        if (kw > 1) {
            // parts of a pair, added in their order; a warp that gave up comes to the barriers, too, and takes all along
            if (!ok) *static_cast<volatile int *>(&sh.failed) = 1;
            float *join = sh.join + warp * (M * kSetOctets * 4 * 32) + lane;
#pragma unroll
            for (int t = 0; t < M; ++t)
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) join[((t * NT + k) * 4 + j) * 32] = total[t][k][j];
            named_bar_sync(1, kRowWarps * 32);
            ok = *static_cast<volatile int *>(&sh.failed) == 0;
            if (part == 0)
                for (int w = 1; w < kw; ++w)
#pragma unroll
                    for (int t = 0; t < M; ++t)
#pragma unroll
                        for (int k = 0; k < NT; ++k)
#pragma unroll
                            for (int j = 0; j < 4; ++j) total[t][k][j] += join[w * (M * kSetOctets * 4 * 32) + ((t * NT + k) * 4 + j) * 32];
            named_bar_sync(1, kRowWarps * 32);
            if (part != 0 || !ok) return ok;
        }
        if (pair >= pairs) return true;
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = k * 8 + 2 * c + j;
                    if (col >= s.count) continue;
                    const int64_t place = s.first + col;
                    const float back = a.scale[place];
                    float *out = a.out + place * a.rows;
                    if constexpr (PAIRED) {
                        const int row = (pair * M + t) * 8 + g;
                        if (row < a.rows) out[row] = silu(total[t][k][j] * back) * (total[t][k][2 + j] * back);
                    } else {
                        const int row = (pair * M + t) * 16 + g;
                        if (row < a.rows) out[row] = total[t][k][j] * back;
                        if (row + 8 < a.rows) out[row + 8] = total[t][k][2 + j] * back;
                    }
                }
        return true;
    };
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const ExpertSet s = a.plan.sets[item / blocks];
        const int pair = pair_of(item);
        if (!(s.count <= 8 ? run(std::integral_constant<int, 1>{}, s, pair) : run(std::integral_constant<int, kSetOctets>{}, s, pair))) break;
    }
    cp_async_wait<0>();
}

template <int FMT, int P, bool PAIRED>
cudaError_t rows_launch_as(const RowsArgs &a, int sms, cudaStream_t st)
{
    constexpr size_t smem = rows_smem(FMT, P);
    const auto kern = rows_kernel<FMT, P, PAIRED>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_chained(kern, dim3(sms), (kRowWarps + 1) * 32, smem, st, true, a);
}

template <int FMT>
cudaError_t rows_launch(const RowsArgs &a, bool paired, int sms, cudaStream_t st)
{
    if (a.pieces == 2) return paired ? rows_launch_as<FMT, 2, true>(a, sms, st) : rows_launch_as<FMT, 2, false>(a, sms, st);
    return paired ? rows_launch_as<FMT, 1, true>(a, sms, st) : rows_launch_as<FMT, 1, false>(a, sms, st);
}

}  // namespace moe
}  // namespace qk
