// qk_attn_rows.cuh -- attention over the 4-bit paged cache for few query rows a
// key/value head (single tokens, short chunks), and heads of 256 channels.
//
// Mathematics.  With K_j = d_jg (n_jc - 8) in each 32-channel group g,
//   s_j = scale * sum_g d_jg (sum_c q_c n_jc - 8 sum_c q_c)
//   o_c = sum_j (p_j e_jg) (n_jc - 8)     (e: the values' scales)
// so both products run on the tensor cores (m16n8k16, fp16 in, fp32 out) with
// the nibbles themselves as the 16-row operand: S^T = K Q^T takes 16 keys by 8
// query columns, O^T = V^T P^T 16 channels by 8 columns.  Grouped heads are
// few, and as columns they fill the products' narrow side; the other way round
// (queries as the 16 rows) four heads left 12 rows of every product empty, and
// a block took 32 products and 432 instructions instead of 16 and 352.
// The scores' accumulator, rounded to fp16 and transposed by movmatrix, is the
// second product's operand as it stands: the cache's token order is made for
// it.
//
// For the scores a nibble under a mask is the fp16 subnormal n * 2^-24 (or
// 16 n * 2^-24), so a word of 8 nibbles becomes four fp16 pairs in four masks
// and a shift.  For the values n - 8 is formed in normal fp16 (one more
// subtraction a pair): sums over keys are not exact, and the tensor cores cut
// them relative to the operands' exponents, which a subnormal hides (2e-6 of
// the sum instead of 1e-7).  Scales stay in fp32, on the scores and on the
// probabilities.
//
// fp32 queries keep fp32 accuracy: a row's query (and probability) is two
// fp16 pieces of 22 bits together, in neighbouring columns.  A probability's
// second piece is held 2^11 times as large: what fp16's least value cuts off is
// below 2^-36, next to leading terms of 2^7 and more.  (At 2^-25, a group of
// values 2^-16 of the largest was 5e-5 off; it took 202 us for 64 x 16 rows over
// 4096 keys, this 206.)
//
// The softmax is one pass: P_j = 2^(z_j - M) against a reference M that moves
// only when a P could leave fp16's range next to its value scale, so most
// blocks need no shuffle and no rescaling.
//
// Blocks of 16 tokens arrive by bulk copies in a ring of stages of each warp
// (no barrier across warps in the loop).  Where heads are fewer than the
// thread blocks that the GPU holds, each head's blocks are split evenly over
// several thread blocks, by the lengths found on the device, and the last of
// them to finish joins their parts in their order; else a thread block has a
// head to itself.  (One line of all heads' blocks cut into equal pieces that
// cross heads, a thread block going through several heads, balanced better
// but cost 12% more instructions a block: 64 x 8192 tokens 149 us against
// 146.)
//
// What bounds it: latency, at 16 warps an SM.  64 sequences of 8192 tokens, 8
// heads of 128 with 4 queries each in bf16, are 604 MB in 147 us (4.1 TB/s, 61%
// of the copy rate): 352 warp instructions a block of 16 tokens, a third of them
// taking nibbles apart, with the issue slots 60% and the integer pipe 52% busy
// and no pipe full; 128 registers a thread leave no room for more warps.  Two
// column sets of 16-bit rows spill at that (462 bytes of stores, 500 of loads at
// 128 channels, 202 and 160 at 96), and are taken where they measured faster all
// the same.  Short calls are their fixed part, dependent reads (lengths, page
// table, first blocks) and the join: 1 x 32768 18 us, 4 of them before the
// first block, 6.5 over the keys, 5 for parts and join.
#pragma once

#include <atomic>

#include "qk_attn.cuh"
#include "qk_internal.h"

namespace qk {
namespace attn {

constexpr float kTwo24 = 16777216.0f;
constexpr float kRest = 2048.0f;      // what a probability's second piece is multiplied by

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 fp16 matrix of a warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// N 32-bit words from shared memory at a multiple of the widest load that N allows.
template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], uint32_t addr)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(addr + 4 * i));
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i]), "=r"(w[i + 1]) : "r"(addr + 4 * i));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(addr + 4 * i));
    }
}

// G fp16 scales of one token as floats.
template <int G>
__device__ __forceinline__ void load_scales(float (&d)[G], uint32_t addr)
{
    if constexpr (G % 2 == 0) {
        uint32_t w[G / 2];
        lds(w, addr);
#pragma unroll
        for (int g = 0; g < G; g += 2) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[g / 2]));
            d[g] = f.x, d[g + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr + 2 * g));
            d[g] = __half2float(__ushort_as_half(h));
        }
    }
}

// A warp's tile: NT sets of 8 columns; PIECES 1: a column is a row, 2: a row
// has its two pieces in columns 2k, 2k + 1.
constexpr int kMaxItems = kRowItems;

template <int G, int PIECES, int NT>
struct Shape {
    static constexpr int D = 32 * G, RT = NT * 8 / PIECES;
    static constexpr int NR = 2 / PIECES;                             // rows of a lane in each column set
    static constexpr int block_bytes = 18 * D;
    static constexpr int blocks_per_sm = rows_blocks_per_sm(G, NT);
    static constexpr int NST = G <= 2 ? 6 : 4;
    static constexpr bool q_in_regs = G * NT <= 4;
    static constexpr int frag_bytes = NT * G * 2 * 32 * 8;
    static constexpr int part_stride = D + 4;                         // floats a row, padded
    static constexpr int part_bytes = RT * part_stride * 4 + RT * 8;  // and (M, l) of each row
    static constexpr int ring_bytes = NST * block_bytes;
    static constexpr int warp_bytes = ((ring_bytes > part_bytes ? ring_bytes : part_bytes) + 127) / 128 * 128;
    static constexpr int bars_at = frag_bytes + kWarps * warp_bytes;
    static constexpr int misc_at = bars_at + kWarps * NST * 8;        // the scan's sums, where this thread block stands
    static constexpr int init_at = misc_at + kWarps * 4 + 32;         // [group][column], then [row]
    static constexpr int smem = init_at + NT * 8 * G * 4 + RT * 4;
    static constexpr int part_floats = RT * D + 2 * RT;               // in the workspace
    static_assert(smem <= 227 * 1024, "shared memory of a block");
};

// One warp's running state.  A lane (r = lane/4, c = lane%4) has, in each column set, rows 2c, 2c + 1 (or c).
template <int G, int PIECES, int NT>
struct State {
    static constexpr int NR = Shape<G, PIECES, NT>::NR;
    float o[NT][G][2][4];        // [..][m][x]: channel 32g + 4r + m (+ 2 for x >= 2), column 2c + x%2
    float m[NT][NR], l[NT][NR];
    float limit;                 // exponents above it leave fp16's range
    uint32_t scale_lim;          // largest value scale seen (fp16 bits, twice)
};

// What a lane needs of its query rows.
template <int G, int PIECES, int NT>
struct Query {
    static constexpr int NR = Shape<G, PIECES, NT>::NR;
    uint32_t b[Shape<G, PIECES, NT>::q_in_regs ? NT * G * 4 : 1];    // operand fragments [set][group][step][2]
    float init[NT][G][2];        // -8 * 2^-24 * (the group's sum of q') of columns 2c, 2c + 1
    float to_log2[NT][NR];       // score -> exponent
    int lo[NT][NR], hi[NT][NR];  // keys [lo, hi) of each row, from the split's first block
};

template <int G, int PIECES, int NT, bool MASK>
__device__ __forceinline__ void block16(State<G, PIECES, NT> &S, const Query<G, PIECES, NT> &Q, uint32_t blk,
                                        uint32_t qfrag, int key0, int all_lo, int all_hi, int lane)
{
    using Sh = Shape<G, PIECES, NT>;
    constexpr int Gp = kv4_gp(G), NR = Sh::NR, D = Sh::D;
    const int tok = 4 * (lane >> 3) + ((lane >> 2) & 1);      // the lane's tokens: tok and tok + 2

    // scores: s[set][token h][row]
    float s[NT][2][NR];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < NR; ++r) s[n][0][r] = s[n][1][r] = 0.0f;
    {
        float dk[2][G];
        load_scales<G>(dk[0], blk + 16 * D + tok * 2 * G);
        load_scales<G>(dk[1], blk + 16 * D + (tok + 2) * 2 * G);
#pragma unroll
        for (int pl = 0; pl < G / Gp; ++pl) {
            uint32_t kw[2][Gp];
            lds(kw[0], blk + pl * 256 * Gp + lane * 4 * Gp);
            lds(kw[1], blk + pl * 256 * Gp + 128 * Gp + lane * 4 * Gp);
#pragma unroll
            for (int gp = 0; gp < Gp; ++gp) {
                const int g = pl * Gp + gp;
                const uint32_t w0 = kw[0][gp], w1 = kw[1][gp], x0 = w0 >> 8, x1 = w1 >> 8;
                const uint32_t a0[4] = {w0 & 0x000F000Fu, w1 & 0x000F000Fu, x0 & 0x000F000Fu, x1 & 0x000F000Fu};
                const uint32_t a1[4] = {w0 & 0x00F000F0u, w1 & 0x00F000F0u, x0 & 0x00F000F0u, x1 & 0x00F000F0u};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t q[4];
                    if constexpr (Sh::q_in_regs) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) q[k] = Q.b[(n * G + g) * 4 + k];
                    } else {
                        lds(q, qfrag + ((n * G + g) * 32 + lane) * 16);
                    }
                    float c[4] = {Q.init[n][g][0], Q.init[n][g][1], Q.init[n][g][0], Q.init[n][g][1]};
                    mma_f16(c, a0, q[0], q[1]);
                    mma_f16(c, a1, q[2], q[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (PIECES == 2) {
                            s[n][h][0] = fmaf(dk[h][g], c[2 * h] + c[2 * h + 1], s[n][h][0]);
                        } else {
                            s[n][h][0] = fmaf(dk[h][g], c[2 * h], s[n][h][0]);
                            s[n][h][NR - 1] = fmaf(dk[h][g], c[2 * h + 1], s[n][h][NR - 1]);
                        }
                    }
                }
            }
        }
    }

    // the value scales' largest magnitude: each lane looks at G/4 of the block's 8G words
    {
        bool grown = false;
        uint32_t w[(8 * G + 31) / 32];
#pragma unroll
        for (int i = 0; i < (8 * G + 31) / 32; ++i) {
            const int at = i * 32 + lane;
            w[i] = 0;
            if (8 * G % 32 == 0 || at < 8 * G) {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(blk + 17 * D + 4 * at));
                w[i] &= 0x7FFF7FFFu;
                if (MASK) {   // slots without a token may hold anything
                    const int t0 = key0 + 2 * at / G, t1 = key0 + (2 * at + 1) / G;
                    if (t0 < all_lo || t0 >= all_hi) w[i] &= 0xFFFF0000u;
                    if (t1 < all_lo || t1 >= all_hi) w[i] &= 0x0000FFFFu;
                }
            }
            grown |= __vmaxu2(w[i], S.scale_lim) != S.scale_lim;
        }
        if (__any_sync(0xFFFFFFFFu, grown)) {
            // one that is not finite makes its channels NaN as it is, and shall not move rows that do not see it
            uint32_t m = S.scale_lim & 0xFFFFu;
#pragma unroll
            for (int i = 0; i < (8 * G + 31) / 32; ++i) {
                const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
                m = max(m, max(lo < 0x7C00u ? lo : 0u, hi < 0x7C00u ? hi : 0u));
            }
            m = redux_max_u32(0xFFFFFFFFu, m);
            S.scale_lim = m | m << 16;
            // |scale| < 2^(e + 1): probabilities up to 2^limit keep P * scale below 2^14
            const int e = m >= 0x0400u ? static_cast<int>(m >> 10) - 15 : -15;
            S.limit = static_cast<float>(13 - e);
        }
    }

    // exponents against the reference
    float p[NT][2][NR];
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                if (MASK) {
                    const int t = key0 + tok + 2 * h;
                    if (t < Q.lo[n][r] || t >= Q.hi[n][r]) s[n][h][r] = -INFINITY;
                }
                p[n][h][r] = fmaf(s[n][h][r], Q.to_log2[n][r], -S.m[n][r]);
                over |= p[n][h][r] > S.limit;
            }
    if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float z = fmaxf(s[n][0][r], s[n][1][r]) * Q.to_log2[n][r];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) z = fmaxf(z, __shfl_xor_sync(0xFFFFFFFFu, z, x));
                if (z - S.m[n][r] > S.limit) {      // the row's new largest sits 2^6 below the limit
                    const float m = z - (S.limit - 6.0f), f = ex2(S.m[n][r] - m);
                    S.m[n][r] = m;
                    S.l[n][r] *= f;
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (PIECES == 2 || (x & 1) == r) S.o[n][g][k][x] *= f;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) p[n][h][r] = fmaf(s[n][h][r], Q.to_log2[n][r], -S.m[n][r]);
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            p[n][0][r] = ex2(p[n][0][r]), p[n][1][r] = ex2(p[n][1][r]);
            S.l[n][r] += p[n][0][r] + p[n][1][r];
        }

    // values
    float dv[2][G];
    load_scales<G>(dv[0], blk + 17 * D + tok * 2 * G);
    load_scales<G>(dv[1], blk + 17 * D + (tok + 2) * 2 * G);
#pragma unroll
    for (int pl = 0; pl < G / Gp; ++pl) {
        uint32_t vw[2][Gp];
        lds(vw[0], blk + 8 * D + pl * 256 * Gp + lane * 4 * Gp);
        lds(vw[1], blk + 8 * D + pl * 256 * Gp + 128 * Gp + lane * 4 * Gp);
#pragma unroll
        for (int gp = 0; gp < Gp; ++gp) {
            const int g = pl * Gp + gp;
            const uint32_t w0 = vw[0][gp], w1 = vw[1][gp], x0 = w0 >> 8, x1 = w1 >> 8;
            const uint32_t a0[4] = {signed_nibbles<0>(w0), signed_nibbles<0>(x0), signed_nibbles<0>(w1), signed_nibbles<0>(x1)};
            const uint32_t a1[4] = {signed_nibbles<1>(w0), signed_nibbles<1>(x0), signed_nibbles<1>(w1), signed_nibbles<1>(x1)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t b[2];
                float x[2][NR];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        x[h][r] = p[n][h][r] * dv[h][g];
                        if (MASK) {   // 0 * (a scale that is not of a key the row sees) may be NaN
                            const int t = key0 + tok + 2 * h;
                            if (t < Q.lo[n][r] || t >= Q.hi[n][r]) x[h][r] = 0.0f;
                        }
                    }
                if constexpr (PIECES == 2) {
                    // rounded to 11 bits, and what that left (exact), times kRest.  x is rounded again beside its rest: two
                    // byte permutes to pair them from the first rounding took 6% more (64 x 16 rows 219 us, this 206)
                    const uint32_t lead = pack_half(x[0][0], x[1][0]);
                    const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&lead));
                    b[0] = transpose8(pack_half(x[0][0], fmaf(x[0][0], kRest, l.x * -kRest)));
                    b[1] = transpose8(pack_half(x[1][0], fmaf(x[1][0], kRest, l.y * -kRest)));
                } else {
                    b[0] = transpose8(pack_half(x[0][0], x[0][NR - 1])), b[1] = transpose8(pack_half(x[1][0], x[1][NR - 1]));
                }
                mma_f16(S.o[n][g][0], a0, b[0], b[1]);
                mma_f16(S.o[n][g][1], a1, b[0], b[1]);
            }
        }
    }
}

// Rows without a key are 0.
__device__ __forceinline__ void zero_rows(const AttnArgs &a, const Sequence &s, int hk, int first, int row_tile, int D)
{
    const int n = static_cast<int>(s.r1 - s.r0) * a.rep;
    for (int row = first; row < n && row < first + row_tile; ++row) {
        const int64_t at = (s.r0 + row / a.rep) * a.ldo + (static_cast<int64_t>(hk) * a.rep + row % a.rep) * D;
        for (int i = threadIdx.x; i < D; i += blockDim.x) store_float_as(a.out, at + i, a.out_type, 0.0f);
    }
}

// Four channels of a row out, divided by the row's sum.
__device__ __forceinline__ void store_row4(const AttnArgs &a, int64_t at, const float4 &v, float l)
{
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) store_float_as(a.out, at + e, a.out_type, l == 0.0f ? 0.0f : x[e] / l);
}

// The parts of the thread blocks that share a head: `count` from c_first on.  Rows' references and sums come first,
// into shared memory, a batch of parts at a time; then a thread takes four channels of every `ways`-th part, and the
// ways are added in order.
template <int RT, int D, class OutAt>
__device__ __forceinline__ void join_parts(const AttnArgs &a, int c_first, int count, int rows, float *buf, int buf_floats,
                                           OutAt out_at)
{
    constexpr int part_floats = RT * D + 2 * RT, kThreads = kWarps * 32, kAhead = 20;
    auto part = [&](int p) { return a.parts + static_cast<int64_t>(c_first + p) * part_floats; };
    const int cols = rows * (D / 4);
    const int ways = cols >= kThreads ? 1 : kThreads / cols;
    float *sum = buf, *ml = buf + (ways > 1 ? ways * cols * 4 : 0);
    const int batch = (buf_floats - static_cast<int>(ml - buf)) / (2 * rows);      // parts whose (M, l) fit beside the sums
    for (int i0 = 0; i0 < cols; i0 += kThreads) {        // more than one round only where ways is 1
        const int i = i0 + static_cast<int>(threadIdx.x), way = i / cols;
        const int col = ways > 1 ? i % cols : i, row = col / (D / 4), ch = col % (D / 4) * 4;
        const bool on = ways > 1 ? way < ways : i < cols;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float m = kNoMax, l = 0.0f;
        for (int p0 = 0; p0 < count; p0 += batch) {
            const int n = min(batch, count - p0);
            __syncthreads();
            for (int j = threadIdx.x; j < 2 * rows * n; j += kThreads)
                ml[j] = __ldcg(part(p0 + j / (2 * rows)) + RT * D + j % (2 * rows));
            __syncthreads();
            if (on) {
                float m2 = m;
                for (int p = 0; p < n; ++p) m2 = fmaxf(m2, ml[2 * rows * p + 2 * row]);
                const float f0 = ex2(m - m2);
                m = m2, l *= f0, v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
                for (int p = 0; p < n; ++p) l = fmaf(ex2(ml[2 * rows * p + 2 * row] - m), ml[2 * rows * p + 2 * row + 1], l);
                const int start = ways > 1 ? way : 0;
                for (int p = start; p < n; p += kAhead * ways) {      // that many parts on their way at once
                    float4 x[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        x[k] = p + k * ways < n ? __ldcg(reinterpret_cast<const float4 *>(part(p0 + p + k * ways) + row * D + ch))
                                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        const float f = p + k * ways < n ? ex2(ml[2 * rows * (p + k * ways) + 2 * row] - m) : 0.0f;
                        v.x = fmaf(f, x[k].x, v.x), v.y = fmaf(f, x[k].y, v.y);
                        v.z = fmaf(f, x[k].z, v.z), v.w = fmaf(f, x[k].w, v.w);
                    }
                }
            }
        }
        if (ways == 1) {
            if (on) store_row4(a, out_at(row) + ch, v, l);
        } else {
            __syncthreads();
            if (on) *reinterpret_cast<float4 *>(sum + (way * cols + col) * 4) = v;
            __syncthreads();
            if (on && way == 0) {
                for (int y = 1; y < ways; ++y) {
                    const float4 x = *reinterpret_cast<const float4 *>(sum + (y * cols + col) * 4);
                    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                }
                store_row4(a, out_at(row) + ch, v, l);
            }
        }
    }
}

template <int G, int PIECES, int NT>
__global__ void __launch_bounds__(kWarps * 32, Shape<G, PIECES, NT>::blocks_per_sm) rows_kernel(const AttnArgs a)
{
    using Sh = Shape<G, PIECES, NT>;
    constexpr int D = Sh::D, RT = Sh::RT, NST = Sh::NST, NR = Sh::NR, kThreads = kWarps * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + Sh::frag_bytes + warp * Sh::warp_bytes;
    const uint32_t bars = smem_u32(smem + Sh::bars_at) + warp * NST * 8;
    int *sums = reinterpret_cast<int *>(smem + Sh::misc_at), *stand = sums + kWarps;
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // This thread block's item (row tile of a sequence), head and split.
    auto blocks_of = [&](int item, int *why) -> int {
        const Sequence s = sequence_of(a, item / a.tiles);
        const int at = item % a.tiles * RT, n = s.bad ? 0 : static_cast<int>(s.r1 - s.r0) * a.rep;
        const int blocks = at < n ? span_of(a, s, at, min(RT, n - at)).blocks : 0;
        *why = s.bad ? 1 : (at < n && blocks == 0 ? 2 : 0);
        return blocks;
    };
    auto rows_without_blocks = [&](int item, int hk, int why) {
        const Sequence s = sequence_of(a, item / a.tiles);
        if (why == 1) poison_rows(a, s, hk, item % a.tiles, a.rep * D);
        else zero_rows(a, s, hk, item % a.tiles * RT, RT, D);
    };
    int item = static_cast<int>(blockIdx.x / a.n_kv), hk = static_cast<int>(blockIdx.x) - item * a.n_kv;
    int b0 = 0, c_first = 0, active = 1, per = INT32_MAX;
    if (a.cut && a.items == 1) {
        // one item: as below, without a scan
        int why;
        const int n = blocks_of(0, &why);
        if (n == 0) {
            if (why && blockIdx.x == 0)
                for (int h = 0; h < a.n_kv; ++h) rows_without_blocks(0, h, why);
            return;
        }
        const int room = a.cut - a.n_kv;
        per = max((n * a.n_kv + room - 1) / room, 2 * kWarps);
        active = (n + per - 1) / per;
        if (static_cast<int>(blockIdx.x) >= active * a.n_kv) return;
        item = 0, hk = static_cast<int>(blockIdx.x) / active;
        const int split = static_cast<int>(blockIdx.x) - hk * active;
        b0 = split * per, c_first = static_cast<int>(blockIdx.x) - split;
    } else if (a.cut) {
        // Every item's blocks (below 2^31 in all: the host sees to it), two items a thread; from their sum the blocks
        // a split takes, so that all splits fit the thread blocks; then which split this one is.
        static_assert(kMaxItems <= 2 * kThreads, "two items a thread");
        int n[2] = {0, 0}, why[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 * static_cast<int>(threadIdx.x) + k < a.items) n[k] = blocks_of(2 * threadIdx.x + k, &why[k]);
        int total = n[0] + n[1];
        total = __reduce_add_sync(0xFFFFFFFFu, total);
        if (lane == 0) sums[warp] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += sums[w];
        total *= a.n_kv;
        const int room = a.cut - a.items * a.n_kv;       // above 0: the host splits where heads are few
        per = max((total + room - 1) / room, 2 * kWarps);
        const int u[2] = {(n[0] + per - 1) / per * a.n_kv, (n[1] + per - 1) / per * a.n_kv};
        int run = u[0] + u[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int below = __shfl_up_sync(0xFFFFFFFFu, run, o);
            if (lane >= o) run += below;
        }
        __syncthreads();
        if (threadIdx.x == 0) stand[0] = -1;
        if (lane == 31) sums[warp] = run;
        __syncthreads();
        for (int w = 0; w < warp; ++w) run += sums[w];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int end = k ? run : run - u[1], begin = end - u[k];
            if (static_cast<int>(blockIdx.x) >= begin && static_cast<int>(blockIdx.x) < end) {
                const int at = static_cast<int>(blockIdx.x) - begin, each = u[k] / a.n_kv;
                stand[0] = 2 * threadIdx.x + k, stand[1] = at / each, stand[2] = at % each, stand[3] = each;
            }
        }
        // rows without blocks: the thread block of the item's number, and so on round
        if (__syncthreads_or(why[0] | why[1]))
            for (int it = blockIdx.x; it < a.items; it += gridDim.x) {
                int w;
                blocks_of(it, &w);
                if (w)
                    for (int h = 0; h < a.n_kv; ++h) rows_without_blocks(it, h, w);
            }
        item = stand[0], hk = stand[1], active = stand[3];
        if (item < 0) return;
        b0 = stand[2] * per, c_first = static_cast<int>(blockIdx.x) - stand[2];
    } else {
        int why;
        if (blocks_of(item, &why) == 0) {
            if (why) rows_without_blocks(item, hk, why);
            return;
        }
    }
    const int64_t b = item / a.tiles;
    const Sequence seq = sequence_of(a, b);
    const int64_t r0 = seq.r0;
    const int first = item % a.tiles * RT, rows = min(RT, static_cast<int>(seq.r1 - r0) * a.rep - first);
    const Span span = span_of(a, seq, first, rows);
    const int b1 = span.blocks - b0 < per ? span.blocks : b0 + per;
    const int nk = b1 - b0 > warp ? (b1 - b0 - warp + kWarps - 1) / kWarps : 0;

    // addresses of this warp's next 32 blocks, one a lane
    const uint64_t policy = l2_evict_first_policy();
    bool poison = false;
    const uint8_t *addr = nullptr;
    auto look_up = [&](int k) {
        addr = a.pages;
        if (k + lane < nk) {
            const uint32_t blk = static_cast<uint32_t>(span.blk_lo) + b0 + warp + kWarps * (k + lane);      // below 2^27
            const uint32_t pg = blk / static_cast<uint32_t>(a.page_blocks);
            const int32_t page = a.page_table[b * a.ld_pages + pg];
            if (page < 0 || page >= a.n_pages) {
                poison = true;
                record_error(a.err, kErrBadIndex);
            } else {
                addr += ((static_cast<int64_t>(page) * a.n_kv + hk) * a.page_blocks + (blk - pg * a.page_blocks)) *
                        static_cast<int64_t>(Sh::block_bytes);
            }
        }
    };
    auto issue = [&](int k) {        // by the lane that holds the address
        if (lane == (k & 31) && !(k == a.skip_block && blockIdx.x == 0 && warp == 0)) {
            const uint32_t bar = bars + 8 * (k % NST);
            mbar_arrive_expect_tx(bar, Sh::block_bytes);
            bulk_g2s(smem_u32(ring) + (k % NST) * Sh::block_bytes, addr, Sh::block_bytes, bar, policy);
        }
    };
    // this warp's first query row is on its way meanwhile
    auto load_row = [&](int row, float (&x)[G]) {
        const bool in = row < rows;
        const int i = in ? (first + row) / a.rep : 0;
        const int64_t at = (r0 + i) * a.ldq + (static_cast<int64_t>(hk) * a.rep + (first + row - i * a.rep)) * D;
#pragma unroll
        for (int g = 0; g < G; ++g) x[g] = in ? load_as_float(a.q, at + 32 * g + lane, a.q_type) : 0.0f;
    };
    float x[G];
    load_row(warp, x);
    if (nk > 0) look_up(0);
    for (int k = 0; k < NST && k < nk; ++k) issue(k);

    // query rows: scaled by a power of two to [2^10, 2^11), fp16 pieces in fragment order.  Two pieces are whole
    // numbers and multiples of 2^-12, so that every product and sum of a group is exact in the tensor cores (which
    // cut what they add at 2^-24 of the largest term: with floating pieces a score lost four bits to that, 1.2e-5
    // of an output over 32768 keys instead of 1e-6).  One warp takes a row, a lane one channel of each group.
    const uint32_t qfrag = smem_u32(smem);
    float *col_init = reinterpret_cast<float *>(smem + Sh::init_at);     // [group][column]
    float *row_log2 = col_init + NT * 8 * G;                             // [row]
    for (int row = warp; row < RT; row += kWarps) {
        if (row != warp) load_row(row, x);
        float big = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) big = fmaxf(big, fabsf(x[g]));
        big = __uint_as_float(redux_max_u32(0xFFFFFFFFu, __float_as_uint(big)));
        int e = 127;
        if (big > 0.0f && big < INFINITY) e = 127 + 10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127);
        e = min(e, 250);
        // the scale's sign goes to the query, so that -inf masks a score whatever the scale
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e) << 23), a.scale_log2);
        // exponent of 2 per unit of (q' n 2^-24), never 0: scale * log2(e) * 2^24 / up
        if (lane == 0) row_log2[row] = fmaxf(a.scale_log2 * kTwo24 / up, 1.2e-38f);
        const int col = row * PIECES, j = lane & 7, st = j & 1;
        // the pair's register of the fragment (x[st], x[st + 4]) or (x[st + 2], x[st + 6]), and the half in it
        const int at_half = st * 8 + ((j >> 1) & 1) * 4 + (j >> 2) * 2;
        uint8_t *to = smem + ((col >> 3) * G * 32 + (col & 7) * 4 + (lane >> 3)) * 16 + at_half;
        const float sixteenth = st ? 0.0625f : 1.0f;     // odd channels' nibbles come 16 times as large
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float v = x[g] * up, rest = 0.0f;
            if (PIECES == 2) {
                const float lead = rintf(v);
                rest = rintf((v - lead) * 4096.0f) * (1.0f / 4096.0f);
                v = lead;
                *reinterpret_cast<__half *>(to + g * 512 + 64) = __float2half_rn(rest * sixteenth);   // the next column
            } else {
                v = __half2float(__float2half_rn(v));
            }
            *reinterpret_cast<__half *>(to + g * 512) = __float2half_rn(v * sixteenth);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
                if (PIECES == 2) rest += __shfl_xor_sync(0xFFFFFFFFu, rest, o);
            }
            if (lane == 0) {
                col_init[NT * 8 * g + col] = v * (-8.0f / kTwo24);
                if (PIECES == 2) col_init[NT * 8 * g + col + 1] = rest * (-8.0f / kTwo24);
            }
        }
    }

    State<G, PIECES, NT> S;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 8; ++k) S.o[n][g][k >> 2][k & 3] = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r) S.m[n][r] = kNoMax, S.l[n][r] = 0.0f;
    }
    S.limit = 28.0f;
    S.scale_lim = 0;
    __syncthreads();

    const int64_t base = (span.blk_lo + b0) * kBlockTokens;      // the first key of this split
    Query<G, PIECES, NT> Q;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = n * (8 / PIECES) + c * NR + r;
            Q.to_log2[n][r] = row_log2[row];
            const int64_t pos = seq.len - (seq.r1 - r0) + (row < rows ? (first + row) / a.rep : 0);
            Q.lo[n][r] = clamp_key(a.window > 0 ? pos - a.window + 1 - base : -1);
            Q.hi[n][r] = row < rows ? clamp_key(pos + 1 - base) : -1;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int x = 0; x < 2; ++x) Q.init[n][g][x] = col_init[NT * 8 * g + n * 8 + 2 * c + x];
            if constexpr (Sh::q_in_regs) {
                uint32_t q[4];
                lds(q, qfrag + ((n * G + g) * 32 + lane) * 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) Q.b[(n * G + g) * 4 + k] = q[k];
            }
        }
    }

    // keys every row sees, counted from the split's first block
    const int64_t last_lo = a.window > 0 ? span.pos1 - a.window + 1 - base : 0;
    const int64_t first_hi = span.pos0 + 1 - base;
    const int all_lo = clamp_key(span.key_lo - base), all_hi = clamp_key(span.key_hi - base);
    bool dead = false;
    for (int k = 0; k < nk; ++k) {
        // the warp shares the outcome: a limit may run out for one lane and not another
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bars + 8 * (k % NST), (k / NST) & 1, a.wait_ns))) {
            // give up: the copies still in flight are waited for before their memory is used for anything else
            dead = true;
            for (int i = k; i < nk && i < k + NST; ++i) mbar_wait(bars + 8 * (i % NST), (i / NST) & 1, a.wait_ns);
            break;
        }
        const uint32_t blk = smem_u32(ring) + (k % NST) * Sh::block_bytes;
        const int key0 = (warp + kWarps * k) * kBlockTokens;
        if (key0 >= last_lo && key0 + kBlockTokens <= first_hi)
            block16<G, PIECES, NT, false>(S, Q, blk, qfrag, key0, all_lo, all_hi, lane);
        else
            block16<G, PIECES, NT, true>(S, Q, blk, qfrag, key0, all_lo, all_hi, lane);
        __syncwarp();
        const int next = k + NST;
        if (next < nk) {
            if ((next & 31) == 0) look_up(next);
            issue(next);
        }
    }
    if (__any_sync(0xFFFFFFFFu, dead) && lane == 0) record_error(a.err, kErrTimeout);
    poison = __any_sync(0xFFFFFFFFu, poison || dead);

    // the warp's part: rows of D values and (M, l), in its own ring
    float *part = reinterpret_cast<float *>(ring);
    float *ml = part + RT * Sh::part_stride;
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float l = S.l[n][r];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
            if (poison) l = __int_as_float(0x7FC00000);
            const int row = n * (8 / PIECES) + c * NR + r;
            if (r8 == 0) ml[2 * row] = S.m[n][r], ml[2 * row + 1] = l;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float v[4];      // channels 32g + 4 r8 + 0..3
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        v[m + 2 * x] = PIECES == 2 ? fmaf(S.o[n][g][m][2 * x + 1], 1.0f / kRest, S.o[n][g][m][2 * x])
                                                   : S.o[n][g][m][2 * x + r];
                *reinterpret_cast<float4 *>(part + row * Sh::part_stride + 32 * g + 4 * r8) =
                    make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    __syncthreads();

    // join the warps' parts; a thread takes four channels of a row
    const uint8_t *rings = smem + Sh::frag_bytes;
    auto warp_part = [&](int w) { return reinterpret_cast<const float *>(rings + w * Sh::warp_bytes); };
    auto out_at = [&](int row) {
        const int i = (first + row) / a.rep;
        return (r0 + i) * a.ldo + (static_cast<int64_t>(hk) * a.rep + first + row - i * a.rep) * D;
    };
    float *mine = active > 1 ? a.parts + static_cast<int64_t>(blockIdx.x) * Sh::part_floats : nullptr;
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), ch = i % (D / 4) * 4;
        float m = kNoMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_part(w)[RT * Sh::part_stride + 2 * row]);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(warp_part(w)[RT * Sh::part_stride + 2 * row] - m);
            const float4 x = *reinterpret_cast<const float4 *>(warp_part(w) + row * Sh::part_stride + ch);
            v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
            l = fmaf(f, warp_part(w)[RT * Sh::part_stride + 2 * row + 1], l);
        }
        if (mine) {
            *reinterpret_cast<float4 *>(mine + row * D + ch) = v;
            if (ch == 0) mine[RT * D + 2 * row] = m, mine[RT * D + 2 * row + 1] = l;
        } else {
            store_row4(a, out_at(row) + ch, v, l);
        }
    }
    if (!mine) return;

    // the last of the head's thread blocks to get here joins their parts, in their order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        int *counter = a.counters + static_cast<int64_t>(item) * a.n_kv + hk;
        const int seen = atomicAdd(counter, 1);
        if (seen == active - 1) *counter = 0;
        stand[0] = seen == active - 1;
    }
    __syncthreads();
    if (!stand[0]) return;
    __threadfence();
    join_parts<RT, D>(a, c_first, active, rows, reinterpret_cast<float *>(smem + Sh::frag_bytes),
                      kWarps * Sh::warp_bytes / 4, out_at);
}

template <int G, int PIECES, int NT>
cudaError_t launch_rows(const AttnArgs &a, int64_t grid, cudaStream_t st)
{
    const auto kern = rows_kernel<G, PIECES, NT>;
    constexpr int smem = Shape<G, PIECES, NT>::smem;
    // once a device; two threads that find it undone both do it
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = library_programmatic() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// Column sets: 1 or 2, and 4 for fp32 rows where the accumulators leave room for them.
template <int G>
cudaError_t launch_rows_of(const AttnArgs &a, int pieces, int sets, int64_t grid, cudaStream_t st)
{
    if (sets == 1) return pieces == 2 ? launch_rows<G, 2, 1>(a, grid, st) : launch_rows<G, 1, 1>(a, grid, st);
    if (sets == 2) return pieces == 2 ? launch_rows<G, 2, 2>(a, grid, st) : launch_rows<G, 1, 2>(a, grid, st);
    if constexpr (G <= 4)
        if (pieces == 2) return launch_rows<G, 2, 4>(a, grid, st);
    return cudaErrorInvalidValue;
}

}  // namespace attn
}  // namespace qk
