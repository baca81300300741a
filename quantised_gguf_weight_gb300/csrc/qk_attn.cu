// qk_attn.cu -- attention over the 4-bit paged cache (qk_attn_q4): the form
// for few query rows a key/value head (single tokens, short chunks), and the
// entry point.
//
// Mathematics.  With K_j = d_jg (n_jc - 8) in each 32-channel group g,
//   s_j = scale * sum_g d_jg (sum_c q_c n_jc - 8 sum_c q_c)
//   o_c = sum_j (p_j e_jg) (n_jc - 8)     (e: the values' scales)
// so both products run on the tensor cores (m16n8k16, fp16 in, fp32 out) with
// the nibbles themselves as one operand.  For the scores a nibble under a mask
// is the fp16 subnormal n * 2^-24 (or 16 n * 2^-24), so a word of 8 nibbles
// becomes four fp16 pairs in four masks and a shift.  For the values n - 8 is
// formed in normal fp16 (one more subtraction a pair): sums over keys are not
// exact, and the tensor cores cut them relative to the operands' exponents,
// which a subnormal hides (2e-6 of the sum instead of 1e-7).  Scales stay in
// fp32, on the scores and on the probabilities.
//
// fp32 queries keep fp32 accuracy: a row's query (and probability) is two
// fp16 pieces of 22 bits together, the second in the tile's rows 8..15, which
// a group of at most 8 query heads leaves empty, so it costs no products.
// 16-bit queries are one piece, and rows 8..15 hold more rows.
//
// The softmax is one pass: P_j = 2^(z_j - M) against a reference M that moves
// only when a P could leave fp16's range next to its value scale, so most
// blocks need no shuffle and no rescaling.
//
// Blocks of 16 tokens arrive by bulk copies in a ring of stages of each warp
// (no barrier across warps in the loop); a sequence's blocks are split over
// thread blocks, and the last to finish joins the parts in a fixed order.
#include <atomic>
#include <cmath>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_attn.cuh"

namespace qk {
using namespace attn;
namespace {

constexpr int kWarps = 8;
constexpr float kTwo24 = 16777216.0f;

// Thread blocks an SM holds: two (128 registers a thread), one where a head of 256 channels needs more.
template <int G>
constexpr int kBlocksPerSm = G <= 4 ? 2 : 1;

// Forms of a row tile.
constexpr int kTwoPiece = 0;    // 8 rows, fp32 queries
constexpr int kOnePiece8 = 1;   // 8 rows, 16-bit queries
constexpr int kOnePiece16 = 2;  // 16 rows, 16-bit queries

__device__ __forceinline__ void mma_f16(float &c0, float &c1, float &c2, float &c3, uint32_t a0, uint32_t a1,
                                        uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Half i of packed fp16 words.
template <int N>
__device__ __forceinline__ float half_at(const uint32_t (&w)[N], int i)
{
    const __half2 h = *reinterpret_cast<const __half2 *>(&w[i >> 1]);
    return i & 1 ? __high2float(h) : __low2float(h);
}

// One warp's running state.
template <int G, int MODE>
struct State {
    static constexpr int NR = MODE == kOnePiece16 ? 2 : 1;       // rows of a lane: lane/4 (and + 8)
    float o[G][4][4];                                            // [group][n-tile j]: channels 32g + 4n + j
    float m[NR], l[NR];
    float limit;                                                 // exponents above it leave fp16's range
    uint32_t scale_lim;                                          // largest value scale seen (fp16 bits, twice)
};

// What a lane needs of its query rows; the fragments themselves are in shared memory.
template <int G, int MODE>
struct Query {
    static constexpr int NR = State<G, MODE>::NR;
    float init[G][2];                                            // -8 * 2^-24 * (the group's sum of q'), rows r, r + 8
    float to_log2[NR];                                           // score -> exponent
    int lo[NR], hi[NR];                                          // keys [lo, hi) of each row, from the tile's first block
};

template <int G, int MODE, bool MASK>
__device__ __forceinline__ void block16(State<G, MODE> &S, const Query<G, MODE> &Q, uint32_t blk, uint32_t qfrag,
                                        int key0, int all_lo, int all_hi, int lane)
{
    constexpr int Gp = kv4_gp(G), NR = State<G, MODE>::NR, D = 32 * G;
    const int c = lane & 3;

    // scores: s[row][tile h][token e] for tokens 4c + 2h + e
    float s[NR][2][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r][0][0] = s[r][0][1] = s[r][1][0] = s[r][1][1] = 0.0f;
    uint32_t ks[2 * G];
    lds(ks, blk + 16 * D + c * 8 * G);
#pragma unroll
    for (int pl = 0; pl < G / Gp; ++pl) {
        uint32_t kw[2][Gp];
        lds(kw[0], blk + pl * 256 * Gp + lane * 4 * Gp);
        lds(kw[1], blk + pl * 256 * Gp + 128 * Gp + lane * 4 * Gp);
#pragma unroll
        for (int gp = 0; gp < Gp; ++gp) {
            const int g = pl * Gp + gp;
            uint32_t a[2][4];
#pragma unroll
            for (int st = 0; st < 2; ++st) lds(a[st], qfrag + ((g * 2 + st) * 32 + lane) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w = kw[h][gp], w8 = w >> 8;
                float c0 = Q.init[g][0], c1 = c0, c2 = MODE == kOnePiece8 ? 0.0f : Q.init[g][1], c3 = c2;
                mma_f16(c0, c1, c2, c3, a[0][0], a[0][1], a[0][2], a[0][3], w & 0x000F000Fu, w8 & 0x000F000Fu);
                mma_f16(c0, c1, c2, c3, a[1][0], a[1][1], a[1][2], a[1][3], w & 0x00F000F0u, w8 & 0x00F000F0u);
                const float d0 = half_at(ks, (2 * h) * G + g), d1 = half_at(ks, (2 * h + 1) * G + g);
                if constexpr (MODE == kTwoPiece) c0 += c2, c1 += c3;
                s[0][h][0] = fmaf(d0, c0, s[0][h][0]);
                s[0][h][1] = fmaf(d1, c1, s[0][h][1]);
                if constexpr (MODE == kOnePiece16) {
                    s[NR - 1][h][0] = fmaf(d0, c2, s[NR - 1][h][0]);
                    s[NR - 1][h][1] = fmaf(d1, c3, s[NR - 1][h][1]);
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
            uint32_t m = S.scale_lim & 0xFFFFu;
#pragma unroll
            for (int i = 0; i < (8 * G + 31) / 32; ++i) m = max(m, max(w[i] & 0xFFFFu, w[i] >> 16));
            m = min(redux_max_u32(0xFFFFFFFFu, m), 0x7BFFu);
            S.scale_lim = m | m << 16;
            // |scale| < 2^(e + 1): probabilities up to 2^limit keep P * scale below 2^14
            const int e = m >= 0x0400u ? static_cast<int>(m >> 10) - 15 : -15;
            S.limit = static_cast<float>(13 - e);
        }
    }

    // exponents against the reference
    float p[NR][2][2];
    bool over = false;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (MASK) {
                    const int t = key0 + 4 * c + 2 * h + e;
                    if (t < Q.lo[r] || t >= Q.hi[r]) s[r][h][e] = -INFINITY;
                }
                p[r][h][e] = fmaf(s[r][h][e], Q.to_log2[r], -S.m[r]);
                over |= p[r][h][e] > S.limit;
            }
    if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float z = fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][1][0], s[r][1][1])) * Q.to_log2[r];
            z = fmaxf(z, __shfl_xor_sync(0xFFFFFFFFu, z, 1));
            z = fmaxf(z, __shfl_xor_sync(0xFFFFFFFFu, z, 2));
            if (z - S.m[r] > S.limit) {      // the row's new largest sits 2^6 below the limit
                const float m = z - (S.limit - 6.0f), f = ex2(S.m[r] - m);
                S.m[r] = m;
                S.l[r] *= f;
#pragma unroll
                for (int g = 0; g < G; ++g) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        S.o[g][j][2 * r] *= f;
                        S.o[g][j][2 * r + 1] *= f;
                        if constexpr (MODE == kTwoPiece) S.o[g][j][2] *= f, S.o[g][j][3] *= f;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) p[r][h][e] = fmaf(s[r][h][e], Q.to_log2[r], -S.m[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) p[r][h][e] = ex2(p[r][h][e]);
        S.l[r] += (p[r][0][0] + p[r][0][1]) + (p[r][1][0] + p[r][1][1]);
    }

    // values
    uint32_t vs[2 * G];
    lds(vs, blk + 17 * D + c * 8 * G);
#pragma unroll
    for (int pl = 0; pl < G / Gp; ++pl) {
        uint32_t vw[2][Gp];
        lds(vw[0], blk + 8 * D + pl * 256 * Gp + lane * 4 * Gp);
        lds(vw[1], blk + 8 * D + pl * 256 * Gp + 128 * Gp + lane * 4 * Gp);
#pragma unroll
        for (int gp = 0; gp < Gp; ++gp) {
            const int g = pl * Gp + gp;
            float x[NR][2][2];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[r][h][e] = p[r][h][e] * half_at(vs, (2 * h + e) * G + g);
                        if (MASK) {   // 0 * (a scale that is not of a key the row sees) may be NaN
                            const int t = key0 + 4 * c + 2 * h + e;
                            if (t < Q.lo[r] || t >= Q.hi[r]) x[r][h][e] = 0.0f;
                        }
                    }
            uint32_t a0, a1 = 0, a2, a3 = 0;
            if constexpr (MODE == kTwoPiece) {
                float f[2][2];   // the leading 11 bits
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        f[h][e] = __uint_as_float(__float_as_uint(x[0][h][e]) & 0xFFFFE000u);
                a0 = pack_half(f[0][0], f[0][1]);
                a2 = pack_half(f[1][0], f[1][1]);
                a1 = pack_half(x[0][0][0] - f[0][0], x[0][0][1] - f[0][1]);
                a3 = pack_half(x[0][1][0] - f[1][0], x[0][1][1] - f[1][1]);
            } else {
                a0 = pack_half(x[0][0][0], x[0][0][1]);
                a2 = pack_half(x[0][1][0], x[0][1][1]);
                if constexpr (NR == 2) {
                    a1 = pack_half(x[NR - 1][0][0], x[NR - 1][0][1]);
                    a3 = pack_half(x[NR - 1][1][0], x[NR - 1][1][1]);
                }
            }
            const uint32_t u0 = vw[0][gp], u1 = vw[1][gp], v0 = u0 >> 8, v1 = u1 >> 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b0 = j & 1 ? signed_nibbles<1>(j & 2 ? v0 : u0) : signed_nibbles<0>(j & 2 ? v0 : u0);
                const uint32_t b1 = j & 1 ? signed_nibbles<1>(j & 2 ? v1 : u1) : signed_nibbles<0>(j & 2 ? v1 : u1);
                mma_f16(S.o[g][j][0], S.o[g][j][1], S.o[g][j][2], S.o[g][j][3], a0, a1, a2, a3, b0, b1);
            }
        }
    }
}

// Shared memory: query fragments, the warps' rings (later their parts), barriers.
template <int G, int MODE>
struct Shape {
    static constexpr int D = 32 * G, RT = MODE == kOnePiece16 ? 16 : 8;
    static constexpr int block_bytes = 18 * D;
    static constexpr int NST = G <= 2 ? 6 : 4;
    static constexpr int frag_bytes = G * 2 * 32 * 16;
    static constexpr int part_bytes = RT * (D + 4) * 4 + RT * 8;      // rows padded by 4 floats; (M, l) of each row
    static constexpr int ring_bytes = NST * block_bytes;
    static constexpr int warp_bytes = ((ring_bytes > part_bytes ? ring_bytes : part_bytes) + 127) / 128 * 128;
    static constexpr int bars_at = frag_bytes + kWarps * warp_bytes;
    static constexpr int init_at = bars_at + kWarps * NST * 8 + 16;   // after the barriers and the join's flag
    static constexpr int smem = init_at + 16 * G * 4 + 16 * 4;
    static constexpr int part_floats = RT * D + 2 * RT;               // in the workspace
};

template <int G, int MODE>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm<G>) attn_kernel(const AttnArgs a)
{
    using Sh = Shape<G, MODE>;
    constexpr int D = Sh::D, RT = Sh::RT, NST = Sh::NST, NR = State<G, MODE>::NR;
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + Sh::frag_bytes + warp * Sh::warp_bytes;
    const uint32_t bars = smem_u32(smem + Sh::bars_at) + warp * NST * 8;
    int *shared_flag = reinterpret_cast<int *>(smem + Sh::bars_at + kWarps * NST * 8);
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
    }
    __syncwarp();

    // unit: row tile, split, head, sequence
    int64_t u = blockIdx.x;
    const int tile = static_cast<int>(u % a.tiles);
    u /= a.tiles;
    const int split = static_cast<int>(u % a.splits);
    u /= a.splits;
    const int hk = static_cast<int>(u % a.n_kv);
    const int64_t b = u / a.n_kv;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Sequence seq = sequence_of(a, b);
    if (seq.bad) {
        if (split == 0) poison_rows(a, seq, hk, tile, a.rep * D);
        return;
    }
    const int64_t r0 = seq.r0, r1 = seq.r1, L = seq.len;
    const int n = static_cast<int>(r1 - r0) * a.rep;      // rows of this sequence and head
    const int first = tile * RT;
    if (first >= n) return;
    const int rows = min(RT, n - first);
    const Span span = span_of(a, seq, first, rows);
    const int active = span.active;
    if (split >= active) return;
    const int64_t blk_lo = span.blk_lo, nblk = span.blocks, per = span.per, pos0 = span.pos0, pos1 = span.pos1;
    const int64_t b0 = split * per, b1 = nblk < b0 + per ? nblk : b0 + per;    // blocks from blk_lo
    const int nk = b1 - b0 > warp ? static_cast<int>((b1 - b0 - warp + kWarps - 1) / kWarps) : 0;

    // addresses of this warp's next 32 blocks, one a lane
    const uint64_t policy = l2_evict_first_policy();
    bool poison = false;
    const uint8_t *addr = nullptr;
    auto look_up = [&](int k) {
        addr = a.pages;
        if (k + lane < nk) {
            const int64_t blk = blk_lo + b0 + warp + static_cast<int64_t>(kWarps) * (k + lane);
            const int64_t pg = blk / a.page_blocks;
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
    auto issue = [&](int k) {
        const uint64_t from = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(addr), k & 31);
        if (lane == 0 && !(k == a.skip_block && blockIdx.x == 0 && warp == 0)) {
            const uint32_t bar = bars + 8 * (k % NST);
            mbar_arrive_expect_tx(bar, Sh::block_bytes);
            bulk_g2s(smem_u32(ring) + (k % NST) * Sh::block_bytes, reinterpret_cast<const void *>(from),
                     Sh::block_bytes, bar, policy);
        }
    };
    if (nk > 0) look_up(0);
    for (int k = 0; k < NST && k < nk; ++k) issue(k);

    // query rows: scaled by a power of two to [2^10, 2^11), fp16 pieces in fragment order.  Two pieces are whole
    // numbers and multiples of 2^-12, so that every product and sum of a group is exact in the tensor cores (which
    // cut what they add at 2^-24 of the largest term: with floating pieces a score lost four bits to that, 1.2e-5
    // of an output over 32768 keys instead of 1e-6).  One warp takes a row, a lane one channel of each group.
    const uint32_t qfrag = smem_u32(smem);
    float *row_init = reinterpret_cast<float *>(smem + Sh::init_at);     // [group][16]
    float *row_log2 = row_init + 16 * G;                                 // [row]
    for (int row = warp; row < RT; row += kWarps) {
        const bool in = row < rows;
        const int i = in ? (first + row) / a.rep : 0;
        const int64_t at = (r0 + i) * a.ldq + (static_cast<int64_t>(hk) * a.rep + (first + row - i * a.rep)) * D;
        float x[G], big = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            x[g] = in ? load_as_float(a.q, at + 32 * g + lane, a.q_type) : 0.0f;
            big = fmaxf(big, fabsf(x[g]));
        }
        big = __uint_as_float(redux_max_u32(0xFFFFFFFFu, __float_as_uint(big)));
        int e = 127;
        if (big > 0.0f && big < INFINITY) e = 127 + 10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127);
        e = min(e, 250);
        // the scale's sign goes to the query, so that -inf masks a score whatever the scale
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e) << 23), a.scale_log2);
        // exponent of 2 per unit of (q' n 2^-24), never 0: scale * log2(e) * 2^24 / up
        if (lane == 0) row_log2[row] = fmaxf(a.scale_log2 * kTwo24 / up, 1.2e-38f);
        const int j = lane & 7, st = j & 1;
        // the pair's register of the fragment (x[st], x[st + 4]) or (x[st + 2], x[st + 6]), and the half in it
        const int flane = (row & 7) * 4 + (lane >> 3), second = (j >> 1) & 1, upper = j >> 2;
        const float sixteenth = st ? 0.0625f : 1.0f;     // odd channels' nibbles come 16 times as large
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float v = x[g] * up, rest = 0.0f;
            if (MODE == kTwoPiece) {
                const float lead = rintf(v);
                rest = rintf((v - lead) * 4096.0f) * (1.0f / 4096.0f);
                v = lead;
            } else {
                v = __half2float(__float2half_rn(v));
            }
            uint8_t *to = smem + ((g * 2 + st) * 32 + flane) * 16 + 8 * second + 2 * upper;
            const __half lead = __float2half_rn(v * sixteenth);
            if constexpr (MODE == kOnePiece16) {
                *reinterpret_cast<__half *>(to + 4 * (row >> 3)) = lead;
            } else {
                *reinterpret_cast<__half *>(to) = lead;
                *reinterpret_cast<__half *>(to + 4) = __float2half_rn(rest * sixteenth);   // 0 with one piece
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
                if (MODE == kTwoPiece) rest += __shfl_xor_sync(0xFFFFFFFFu, rest, o);
            }
            if (lane == 0) {
                row_init[16 * g + row] = v * (-8.0f / kTwo24);
                if (MODE != kOnePiece16) row_init[16 * g + 8 + row] = rest * (-8.0f / kTwo24);
            }
        }
    }

    State<G, MODE> S;
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) S.o[g][j][k] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) S.m[k] = kNoMax, S.l[k] = 0.0f;
    S.limit = 28.0f;
    S.scale_lim = 0;
    __syncthreads();

    const int64_t base = (blk_lo + b0) * kBlockTokens;
    Query<G, MODE> Q;
#pragma unroll
    for (int half = 0; half < NR; ++half) {
        const int row = r8 + 8 * half;
        Q.to_log2[half] = row_log2[row];
        const int64_t pos = L - (r1 - r0) + (row < rows ? (first + row) / a.rep : 0);
        Q.lo[half] = clamp_key(a.window > 0 ? pos - a.window + 1 - base : -1);
        Q.hi[half] = row < rows ? clamp_key(pos + 1 - base) : -1;
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < 2; ++k) Q.init[g][k] = row_init[16 * g + r8 + 8 * k];

    // keys every row sees, counted from the split's first block
    const int64_t last_lo = a.window > 0 ? pos1 - a.window + 1 - base : 0;
    const int64_t first_hi = pos0 + 1 - base;
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
            block16<G, MODE, false>(S, Q, blk, qfrag, key0, all_lo, all_hi, lane);
        else
            block16<G, MODE, true>(S, Q, blk, qfrag, key0, all_lo, all_hi, lane);
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
    float *ml = part + RT * (D + 4);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NR; ++k) {
        S.l[k] += __shfl_xor_sync(0xFFFFFFFFu, S.l[k], 1);
        S.l[k] += __shfl_xor_sync(0xFFFFFFFFu, S.l[k], 2);
        if (poison) S.l[k] = __int_as_float(0x7FC00000);
        const int row = r8 + 8 * k;
        if (c == 0) ml[2 * row] = S.m[k], ml[2 * row + 1] = S.l[k];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = S.o[g][j][2 * k + x];
                    if constexpr (MODE == kTwoPiece) v += S.o[g][j][2 + x];
                    part[row * (D + 4) + 32 * g + 4 * (2 * c + x) + j] = v;
                }
    }
    __syncthreads();

    // join the warps' parts; a thread takes whole columns of rows
    const uint8_t *rings = smem + Sh::frag_bytes;
    auto warp_part = [&](int w) { return reinterpret_cast<const float *>(rings + w * Sh::warp_bytes); };
    float *mine = nullptr;
    int *counter = nullptr;
    if (active > 1) {
        const int64_t group = (b * a.n_kv + hk) * a.tiles + tile;
        counter = a.counters + group;
        mine = a.parts + (group * a.splits) * Sh::part_floats;
    }
    for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
        const int row = i / D, ch = i % D;
        float m = kNoMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_part(w)[RT * (D + 4) + 2 * row]);
        float v = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(warp_part(w)[RT * (D + 4) + 2 * row] - m);
            v = fmaf(f, warp_part(w)[row * (D + 4) + ch], v);
            l = fmaf(f, warp_part(w)[RT * (D + 4) + 2 * row + 1], l);
        }
        if (active == 1) {
            const int64_t to = (r0 + (first + row) / a.rep) * a.ldo +
                               (static_cast<int64_t>(hk) * a.rep + (first + row) % a.rep) * D + ch;
            store_float_as(a.out, to, a.out_type, l == 0.0f ? 0.0f : v / l);
        } else {
            float *to = mine + static_cast<int64_t>(split) * Sh::part_floats;
            to[i] = v;
            if (ch == 0) to[RT * D + 2 * row] = m, to[RT * D + 2 * row + 1] = l;
        }
    }
    if (active == 1) return;

    // the last split to get here joins all parts, in their order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int seen = atomicAdd(counter, 1);
        if (seen == active - 1) *counter = 0;
        *shared_flag = seen == active - 1;
    }
    __syncthreads();
    if (!*shared_flag) return;
    __threadfence();
    for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
        const int row = i / D, ch = i % D;
        float m = kNoMax;
        for (int w = 0; w < active; ++w) m = fmaxf(m, __ldcg(mine + static_cast<int64_t>(w) * Sh::part_floats + RT * D + 2 * row));
        float v = 0.0f, l = 0.0f;
#pragma unroll 4
        for (int w = 0; w < active; ++w) {
            const float *from = mine + static_cast<int64_t>(w) * Sh::part_floats;
            const float f = ex2(__ldcg(from + RT * D + 2 * row) - m);
            v = fmaf(f, __ldcg(from + i), v);
            l = fmaf(f, __ldcg(from + RT * D + 2 * row + 1), l);
        }
        const int64_t to = (r0 + (first + row) / a.rep) * a.ldo +
                           (static_cast<int64_t>(hk) * a.rep + (first + row) % a.rep) * D + ch;
        store_float_as(a.out, to, a.out_type, l == 0.0f ? 0.0f : v / l);
    }
}

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }

// How a call's rows and keys are cut.
struct Cut {
    int mode, row_tile, tiles, splits;
    int64_t min_blocks, groups;      // groups: sequences * heads * tiles
};

std::atomic<int> g_skip_block{-1};

constexpr int kChunk = 3;                    // Cut::mode of the many-row form (qk_attn_chunk.cu)
constexpr int64_t kChunkFrom = 64;           // rows a sequence and head from which it is taken
constexpr int64_t kCounters = 16384;         // at the start of every workspace, whatever the call
Cut cut_for(int64_t B, int n_kv, int rep, int D, int64_t max_q, int64_t max_len, bool fp32)
{
    Cut c{};
    const int64_t rows = max_q * rep;
    c.mode = fp32 ? kTwoPiece : (rows <= 8 ? kOnePiece8 : kOnePiece16);
    if (!fp32 && rows >= kChunkFrom && D <= 128) c.mode = kChunk;
    c.row_tile = c.mode == kChunk ? kChunkRows : c.mode == kOnePiece16 ? 16 : 8;
    c.tiles = static_cast<int>((rows + c.row_tile - 1) / c.row_tile);
    c.groups = B * n_kv * c.tiles;
    const int64_t blocks = (max_len + kBlockTokens - 1) / kBlockTokens;
    // The split with the least of (rounds of thread blocks) * (steps of a warp + a thread block's start and join,
    // about 10 steps), of splits that leave every warp two blocks.
    int sms = 152, smem = 0;
    device_limits(&sms, &smem);
    if (c.mode == kChunk) {
        // rounds of one thread block an SM, of key tiles of 8 blocks (about 1.2 us each) and 3 tiles' worth of start
        // and end; parts of several splits are written and read again (5 TB/s) by a second kernel (2 us)
        const int64_t tiles = (blocks + 7) / 8;
        double best = 1e30;
        c.splits = 1;
        for (int64_t rounds = 1, last = 0; rounds <= 8; ++rounds) {
            int64_t s = sms * rounds / c.groups;
            if (s * 2 > tiles) s = tiles / 2;
            if (s < 1) s = 1;
            if (s == last) continue;
            last = s;
            const double us = 1.2 * static_cast<double>((c.groups * s + sms - 1) / sms * ((tiles + s - 1) / s + 3)) +
                              (s > 1 ? 2.0 + 2e-7 * static_cast<double>(2 * s * c.groups * chunk_part_bytes(D)) : 0.0);
            if (us < best) best = us, c.splits = static_cast<int>(s);
        }
        c.min_blocks = (tiles + c.splits - 1) / c.splits * 8;
        if (c.min_blocks < 16) c.min_blocks = 16;
        return c;
    }
    const int64_t slots = static_cast<int64_t>(sms) * (D > 128 ? 1 : 2);
    int64_t best = 1, best_cost = INT64_MAX;
    for (int64_t rounds = 1, last = 0; rounds <= 12 && c.groups <= kCounters; ++rounds) {
        // as many splits as `rounds` rounds hold, or one
        int64_t s = slots * rounds / c.groups;
        if (s * 2 * kWarps > blocks) s = blocks / (2 * kWarps);
        if (s < 1) s = 1;
        if (s == last) continue;
        last = s;
        const int64_t per = (blocks + s - 1) / s;
        const int64_t cost = (c.groups * s + slots - 1) / slots * ((per + kWarps - 1) / kWarps + 10);
        if (cost < best_cost) best = s, best_cost = cost;
    }
    c.splits = static_cast<int>(best);
    c.min_blocks = (blocks + best - 1) / best;
    if (c.min_blocks < 2 * kWarps) c.min_blocks = 2 * kWarps;
    return c;
}

int64_t part_bytes_of(const Cut &c, int D)
{
    if (c.mode == kChunk) return chunk_part_bytes(D);
    return (static_cast<int64_t>(c.row_tile) * D + 2 * c.row_tile) * 4;
}

template <int G, int MODE>
cudaError_t launch(const AttnArgs &a, int64_t grid, cudaStream_t st)
{
    const auto kern = attn_kernel<G, MODE>;
    constexpr int smem = Shape<G, MODE>::smem;
    static_assert(smem <= 227 * 1024, "shared memory of a block");
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

template <int G>
cudaError_t launch_mode(const AttnArgs &a, int mode, int64_t grid, cudaStream_t st)
{
    if (mode == kTwoPiece) return launch<G, kTwoPiece>(a, grid, st);
    if (mode == kOnePiece8) return launch<G, kOnePiece8>(a, grid, st);
    return launch<G, kOnePiece16>(a, grid, st);
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

// Test hook, not part of the public header: thread block 0 of every later
// attention launch never copies its 16-token block number `block` (the
// few-row form: of its first warp; -1 restores normal operation), so that a
// bounded wait runs out and the launch records QK_ERR_TIMEOUT.
int qk_debug_attn_skip_block(int block) { return g_skip_block.exchange(block); }

size_t qk_attn_q4_workspace_bytes(int64_t B, int n_q_heads, int n_kv_heads, int head_dim, int64_t max_q,
                                  int64_t max_len)
{
    if (B <= 0 || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || head_dim <= 0 || max_q <= 0 ||
        max_len <= 0 || B > INT32_MAX / max_q)
        return 0;
    size_t most = 0;
    for (const bool fp32 : {true, false}) {
        const Cut c = cut_for(B, n_kv_heads, n_q_heads / n_kv_heads, head_dim, max_q, max_len, fp32);
        const size_t n = c.splits > 1 ? 4 * kCounters + c.groups * c.splits * part_bytes_of(c, head_dim) : 0;
        if (n > most) most = n;
    }
    return most;
}

int qk_attn_q4(const qk_kv_cache_q4 *cache, const void *q, int64_t ldq, int q_type, int n_q_heads,
               const int32_t *page_table, int64_t ld_pages, int64_t max_pages, const int32_t *lens,
               const int32_t *q_start, int64_t B, int64_t T, int64_t max_q, int64_t max_len, float scale,
               int64_t window, void *out, int64_t ldo, int out_type, void *workspace, size_t workspace_bytes,
               qk_stream_t stream)
{
    const int st = kv4_check_cache(cache);
    if (st != QK_OK) return st;
    if (!type_ok(q_type) || !type_ok(out_type)) return QK_ERR_TYPE;
    const int D = cache->head_dim, n_kv = cache->n_kv_heads;
    if (n_q_heads < 1 || n_q_heads % n_kv || B < 0 || T < 0 || max_q < 0 || max_len < 0 || window < 0 ||
        ld_pages < 0 || max_pages < 0 || !std::isfinite(scale))
        return QK_ERR_BAD_DIM;
    const int64_t w = static_cast<int64_t>(n_q_heads) * D;
    if (ldq == 0) ldq = w;
    if (ldo == 0) ldo = w;
    if (max_pages == 0) max_pages = ld_pages;
    if (ldq < w || ldo < w || max_pages > ld_pages) return QK_ERR_BAD_DIM;
    if (!q_start && (B == 0 || max_q == 0 ? T != 0 : T / B != max_q || T % B)) return QK_ERR_BAD_DIM;
    if (T == 0 || B == 0 || max_q == 0) return QK_OK;
    if (!q || !page_table || !lens || !out) return QK_ERR_NULL;
    if (!multiple(q, q_type == QK_F32 ? 4 : 2) || !multiple(out, out_type == QK_F32 ? 4 : 2) ||
        !multiple(page_table, 4) || !multiple(lens, 4) || !multiple(q_start, 4))
        return QK_ERR_ALIGN;
    if (workspace && !multiple(workspace, 256)) return QK_ERR_WORKSPACE;
    const int rep = n_q_heads / n_kv;
    if (n_q_heads > 65535 || B > INT32_MAX / max_q || T > INT32_MAX || max_q > INT32_MAX / rep - 16 ||
        max_pages > INT32_MAX / cache->page_tokens)
        return QK_ERR_TOO_LARGE;
    const int64_t keys = max_pages * cache->page_tokens;
    Cut cut = cut_for(B, n_kv, rep, D, max_q, max_len > 0 && max_len < keys ? max_len : keys, q_type == QK_F32);
    // as many splits as the workspace holds
    const int64_t room = workspace ? static_cast<int64_t>(workspace_bytes) - 4 * kCounters : 0;
    const int64_t fit = room > 0 ? room / (cut.groups * part_bytes_of(cut, D)) : 0;
    if (cut.splits > fit) cut.splits = fit > 1 ? static_cast<int>(fit) : 1;
    const int64_t grid = cut.groups * cut.splits;
    if (grid > INT32_MAX) return QK_ERR_TOO_LARGE;
    AttnArgs a{};
    a.pages = static_cast<const uint8_t *>(cache->pages), a.n_pages = cache->n_pages;
    a.n_kv = n_kv, a.page_blocks = cache->page_tokens / kBlockTokens, a.rep = rep;
    a.q = q, a.ldq = ldq, a.q_type = q_type;
    a.page_table = page_table, a.ld_pages = ld_pages, a.max_pages = max_pages;
    a.lens = lens, a.q_start = q_start, a.T = T, a.max_q = max_q, a.window = window;
    a.scale_log2 = static_cast<float>(scale * 1.4426950408889634074);
    a.out = out, a.ldo = ldo, a.out_type = out_type;
    a.tiles = cut.tiles, a.splits = cut.splits, a.min_blocks = cut.min_blocks;
    a.counters = static_cast<int *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + 4 * kCounters);
    a.err = library_error_word();
    a.wait_ns = library_wait_limit_ns();
    if (!a.err) return QK_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    a.skip_block = g_skip_block.load();
    if (cut.mode == kChunk) return chunk_launch(a, D, cut.groups, s) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
    switch (D) {
    case 64: e = launch_mode<2>(a, cut.mode, grid, s); break;
    case 96: e = launch_mode<3>(a, cut.mode, grid, s); break;
    case 128: e = launch_mode<4>(a, cut.mode, grid, s); break;
    case 256: e = launch_mode<8>(a, cut.mode, grid, s); break;
    }
    return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

}  // extern "C"
