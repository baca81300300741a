// qk_moe_rows.cuh -- the experts' products for few tokens an expert: a pass
// over the expert's weights for every 32 tokens, in the m16n8k16 products of
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
// lane has both sums of an output), or a part of its columns where tiles are
// few; its weights come through a ring of its own in shared memory, 16 bytes an
// asynchronous copy, so nothing waits for other warps.
#pragma once

#include "qk_moe.cuh"

namespace qk {
namespace moe {

// Shared-memory pitch of a row's unit: 16-byte chunks that hold it wherever it starts.  Q4_K's starts on one.
__host__ __device__ constexpr int row_pitch(int fmt) { return fmt == kFmtQ4K ? 144 : fmt == kFmtQ80 ? 288 : 224; }
__host__ __device__ constexpr int ring_stages(int fmt) { return fmt == kFmtQ4K ? 4 : fmt == kFmtQ80 ? 2 : 3; }

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

// Operand words of an octet's unit: step i of piece p.
__device__ __forceinline__ uint4 operand(const uint8_t *unit, int p, int i, int lane)
{
    return __ldg(reinterpret_cast<const uint4 *>(unit + p * kPieceBytes + i * 512 + lane * 16));
}

// The products of one unit (256 columns): total[n] += rows (g, g + 8) x octet n's columns.
// st: the tile's unit in shared memory; al[2]: byte offsets of rows g and g + 8 inside their chunks.
template <int FMT, int P, int NT>
__device__ __forceinline__ void unit_products(float (&total)[NT][4], uint32_t st, const uint32_t (&al)[2], int blocks,
                                              const uint8_t *x, int64_t octet_bytes, int lane)
{
    const int g = lane >> 2, c = lane & 3;
    const uint32_t row0 = st + g * row_pitch(FMT) + al[0], row1 = st + (g + 8) * row_pitch(FMT) + al[1];
    if constexpr (FMT == kFmtQ4K) {
        // lane c has sub-blocks 2c and 2c + 1: 32 bytes of nibbles
        float dd[2], dm[2];
        __half2 sl[2], sb[2], shi[2], shb[2];     // scale of the low nibbles' sub-block, -1024 of it; high: / 16, -64
        uint32_t m[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint4 h = lds128(r ? row1 : row0);
            const float2 d2 = __half22float2(bits_h2(h.x));
            dd[r] = d2.x, dm[r] = d2.y;
            const int sh = (c & 1) * 16;
            const uint32_t A = h.y >> sh, B = h.z >> sh, C = h.w >> sh;
            const uint32_t sc = c < 2 ? A & 0x3f3fu : (C & 0x0f0fu) | ((A >> 2) & 0x3030u);
            const uint32_t mm = c < 2 ? B & 0x3f3fu : ((C >> 4) & 0x0f0fu) | ((B >> 2) & 0x3030u);
            const __half2 k1024 = __float2half2_rn(1024.0f);
            const __half2 s0 = __hsub2(bits_h2(__byte_perm(sc, 0x64u, 0x4040)), k1024);
            const __half2 s1 = __hsub2(bits_h2(__byte_perm(sc, 0x64u, 0x4141)), k1024);
            sl[r] = s0, sb[r] = __hmul2(s0, __float2half2_rn(-1024.0f));
            shi[r] = __hmul2(s1, __float2half2_rn(0.0625f)), shb[r] = __hmul2(s1, __float2half2_rn(-64.0f));
            m[r] = h2_bits(__hmul2(__hsub2(bits_h2(__byte_perm(mm, 0x64u, 0x4140)), k1024), __float2half2_rn(32.0f)));
        }
        float acc[NT][4], low[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = low[n][j] = 0.0f;
            const uint2 s = __ldg(reinterpret_cast<const uint2 *>(x + n * octet_bytes + P * kPieceBytes + lane * 8));
            const uint32_t a[4] = {m[0], m[1], m[0], m[1]};
            mma16(low[n], a, s.x, s.y);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint4 w0 = lds128(row0 + 16 + 32 * c + 16 * q), w1 = lds128(row1 + 16 + 32 * c + 16 * q);
            const uint32_t v0[4] = {w0.x, w0.y, w0.z, w0.w}, v1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a[4] = {h2_bits(__hfma2(field1024<0x000f000f>(v0[k]), sl[0], sb[0])),
                                       h2_bits(__hfma2(field1024<0x000f000f>(v1[k]), sl[1], sb[1])),
                                       h2_bits(__hfma2(field1024<0x000f000f>(v0[k] >> 8), sl[0], sb[0])),
                                       h2_bits(__hfma2(field1024<0x000f000f>(v1[k] >> 8), sl[1], sb[1]))};
                const uint32_t b[4] = {h2_bits(__hfma2(field1024<0x00f000f0>(v0[k]), shi[0], shb[0])),
                                       h2_bits(__hfma2(field1024<0x00f000f0>(v1[k]), shi[1], shb[1])),
                                       h2_bits(__hfma2(field1024<0x00f000f0>(v0[k] >> 8), shi[0], shb[0])),
                                       h2_bits(__hfma2(field1024<0x00f000f0>(v1[k] >> 8), shi[1], shb[1]))};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint4 o = operand(x + n * octet_bytes, p, 4 * q + k, lane);
                        mma16(acc[n], a, o.x, o.y);
                        mma16(acc[n], b, o.z, o.w);
                    }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                total[n][j] += dd[j >> 1] * acc[n][j] - dm[j >> 1] * low[n][j];
    } else if constexpr (FMT == kFmtQ80) {
        const __half2 bias = __float2half2_rn(1152.0f);
        const auto pair = [&](uint32_t v, int sel) { return h2_bits(__hsub2(bits_h2(__byte_perm(v, 0x64u, sel)), bias)); };
#pragma unroll 2
        for (int i = 0; i < blocks; ++i) {
            uint32_t v[2][2];
            float dd[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t blk = (r ? row1 : row0) + 34 * i;
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
                    const uint4 o = operand(x + n * octet_bytes, p, i, lane);
                    mma16(acc, a, o.x, o.y);
                    mma16(acc, b, o.z, o.w);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) total[n][j] += dd[j >> 1] * acc[j];
            }
        }
    } else {
        const __half2 bias = __float2half2_rn(1056.0f);
        const auto pair = [&](uint32_t v, int sel) { return h2_bits(__hsub2(bits_h2(__byte_perm(v, 0x64u, sel)), bias)); };
        const float dd[2] = {half_bits_to_float(lds16(row0 + 208)), half_bits_to_float(lds16(row1 + 208))};
#pragma unroll 1
        for (int hu = 0; hu < 4; ++hu) {             // half n = hu / 2, 16 positions u = hu % 2
            uint32_t A[2], B[2], H[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t blk = (r ? row1 : row0) + 16 * (hu & 1) + 4 * c;
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
                    ds[r] = dd[r] * lds_s8((r ? row1 : row0) + 192 + 8 * (hu >> 1) + 2 * t + (hu & 1));
                }
                const uint32_t a[4] = {pair(v[0], 0x4240), pair(v[1], 0x4240), pair(v[0], 0x4341), pair(v[1], 0x4341)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint4 o = operand(x + n * octet_bytes, p, 2 * hu + (t >> 1), lane);
                        mma16(acc, a, t & 1 ? o.z : o.x, t & 1 ? o.w : o.y);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) total[n][j] += ds[j >> 1] * acc[j];
                }
            }
        }
    }
}

// One tile's units [u0, u1) for a set of NT octets.
template <int FMT, int P, int NT>
__device__ __forceinline__ void tile_products(float (&total)[NT][4], const RowsArgs &a, const uint8_t *mine,
                                              const uint32_t (&al)[2], uint32_t ring, int u0, int u1, int octet, int lane)
{
    constexpr int S = ring_stages(FMT), UB = unit_bytes(FMT), PITCH = row_pitch(FMT), CH = PITCH / 16;
    const int64_t ub = octet_unit_bytes(FMT, P), octet_bytes = ub * a.units;
    const uint8_t *x = a.x + octet * octet_bytes;
    const int r = lane >> 1, half = lane & 1;
    const uint8_t *row_end = mine + a.a.row_bytes;
    const uint32_t dst = ring + r * PITCH;
    const auto fetch = [&](int u, int slot) {
        const uint8_t *from = mine + static_cast<int64_t>(u) * UB;
        const uint8_t *end = from + UB < row_end ? from + UB : row_end;
        from -= reinterpret_cast<uintptr_t>(from) & 15;
#pragma unroll
        for (int i = 0; i < (CH + 1) / 2; ++i) {
            const int ch = 2 * i + half;
            if (ch < CH && from + 16 * ch < end) cp_async16(dst + slot * 16 * PITCH + 16 * ch, from + 16 * ch);
        }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (u0 + i < u1) fetch(u0 + i, i);
        cp_async_commit();
    }
    int slot = 0;
    uint32_t at[2] = {al[0], al[1]};
    for (int u = u0; u < u1; ++u) {
        cp_async_wait<S - 2>();
        __syncwarp();                // everyone's copies of this unit have landed, and the slot before it is free
        const int next = u + S - 1, into = slot == 0 ? S - 1 : slot - 1;
        if (next < u1) fetch(next, into);
        cp_async_commit();
        // a unit of Q6_K is no whole number of chunks
        if constexpr (UB % 16 != 0) at[0] = (al[0] + u * UB) & 15, at[1] = (al[1] + u * UB) & 15;
        const int blocks = FMT == kFmtQ80 ? min(8, (a.cols + 31) / 32 - 8 * u) : 8;
        unit_products<FMT, P, NT>(total, ring + slot * 16 * PITCH, at, blocks, x + u * ub, octet_bytes, lane);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
}

template <int FMT, int P, bool PAIRED, int NT>
__device__ __forceinline__ void set_tile(const RowsArgs &a, const ExpertSet &s, int tile, int part, int kw, uint32_t ring,
                                         float *join, int lane, int warp)
{
    const int g = lane >> 2, c = lane & 3, r = lane >> 1;
    float total[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[n][j] = 0.0f;
    if (tile < a.tiles) {
        // rows past the last are read as the last and not written
        const auto row_of = [&](int i) -> const uint8_t * {
            const int row = PAIRED ? min(tile * 8 + (i & 7), a.rows - 1) : min(tile * 16 + i, a.rows - 1);
            const Weights &w = i < 8 ? a.a : a.b;
            return w.w + (s.expert * w.expert_rows + row) * w.row_bytes;
        };
        const uint32_t al[2] = {static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row_of(g)) & 15),
                                static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row_of(g + 8)) & 15)};
        const int u0 = a.units * part / kw, u1 = a.units * (part + 1) / kw;
        tile_products<FMT, P, NT>(total, a, row_of(r), al, ring, u0, u1, s.octet, lane);
    }
    if (kw > 1) {
        // parts of a tile, added in their order
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) join[((warp * NT + n) * 4 + j) * 32 + lane] = total[n][j];
        __syncthreads();
        if (part == 0)
            for (int k = 1; k < kw; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) total[n][j] += join[(((warp + k) * NT + n) * 4 + j) * 32 + lane];
        __syncthreads();
        if (part != 0) return;
    }
    if (tile >= a.tiles) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = n * 8 + 2 * c + j;
            if (col >= s.count) continue;
            const int64_t place = s.first + col;
            const float back = a.scale[place];
            float *out = a.out + place * a.rows;
            if constexpr (PAIRED) {
                const int row = tile * 8 + g;
                if (row < a.rows) out[row] = silu(total[n][j] * back) * (total[n][2 + j] * back);
            } else {
                const int row = tile * 16 + g;
                if (row < a.rows) out[row] = total[n][j] * back;
                if (row + 8 < a.rows) out[row + 8] = total[n][2 + j] * back;
            }
        }
}

template <int FMT, int P, bool PAIRED>
__global__ void __launch_bounds__(kRowWarps * 32, 2) rows_kernel(const RowsArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float join[kRowWarps * kSetOctets * 4 * 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem) + warp * ring_stages(FMT) * 16 * row_pitch(FMT);
    let_next_start();
    wait_for_previous();
    // warps that share a tile's units: enough for every SM's 16 warps to have work where tiles are few
    const int64_t sets = a.plan.head[0];
    int kw = 1;
    while (kw < kRowWarps && 2 * kw <= a.units && sets * a.tiles * kw < 16 * a.sms) kw *= 2;
    const int per = kRowWarps / kw, blocks = (a.tiles + per - 1) / per;
    const int64_t items = sets * blocks;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const ExpertSet s = a.plan.sets[i / blocks];
        const int tile = static_cast<int>(i % blocks) * per + warp / kw, part = warp % kw;
        if (s.count <= 8) set_tile<FMT, P, PAIRED, 1>(a, s, tile, part, kw, ring, join, lane, warp);
        else if (s.count <= 16) set_tile<FMT, P, PAIRED, 2>(a, s, tile, part, kw, ring, join, lane, warp);
        else set_tile<FMT, P, PAIRED, 4>(a, s, tile, part, kw, ring, join, lane, warp);
    }
}

template <int FMT, int P, bool PAIRED>
cudaError_t rows_launch_as(const RowsArgs &a, int sms, cudaStream_t st)
{
    constexpr size_t smem = kRowWarps * ring_stages(FMT) * 16 * row_pitch(FMT);
    const auto kern = rows_kernel<FMT, P, PAIRED>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_chained(kern, dim3(2 * sms), kRowWarps * 32, smem, st, true, a);
}

template <int FMT>
cudaError_t rows_launch(const RowsArgs &a, bool paired, int sms, cudaStream_t st)
{
    if (a.pieces == 2) return paired ? rows_launch_as<FMT, 2, true>(a, sms, st) : rows_launch_as<FMT, 2, false>(a, sms, st);
    return paired ? rows_launch_as<FMT, 1, true>(a, sms, st) : rows_launch_as<FMT, 1, false>(a, sms, st);
}

}  // namespace moe
}  // namespace qk
