// qk_attn_chunk32.cu -- attention over the 4-bit cache for many query rows a
// key/value head with fp32 or fp16 queries, on the 5th-generation tensor
// cores.
//
// A thread block takes 128 rows (queries x grouped heads) of one key/value
// head and walks the keys in tiles of 64.  fp32 accuracy comes from operands
// of two fp16 pieces and three of their four products:
//   S = Q1 K1^T + Q2 K1^T + Q1 K2^T      O += P1 V1 + P2 V1 + P1 V2
// (1e-6 off over 16384 keys; the few-row form 2e-6)
// Queries, a power of two away from themselves, are whole numbers below 2^11
// and multiples of 2^-12; K = (n - 8) d has 15 bits, K1 its leading 11 and K2
// exactly the rest; P1 and P2 are a probability's first and next 11 bits.  The
// product left out is below 2^-22 of the sum's terms.  fp16 queries are one
// piece, and S two products.  (In the bf16 form, whose K, P and V are rounded to
// 11 bits, fp16 outputs were 4e-4 off, twice their own rounding; bf16's own is
// 1.7e-3.)
//
// The tensor cores cut what they add at about 2^-24 of the largest term, the
// accumulator too, always the same way; over thousands of keys that would be
// 2^-24 a product.  So O takes the products of kFlush tiles and is then added
// to a second accumulator in fp32, which rounds.
//
// Everything but the shared-memory operands K1, K2, V1, V2 (64 KB a tile at
// 128 channels) is in tensor memory: S 64 columns, P1, P2 32 each, Q1, Q2 and
// both accumulators D/2 and D each, 512 at 128 channels.
//
// Scales, references and masks are as in the 16-bit form: K' = K 2^-kk and V'
// = V 2^-kt, whose two pieces hold all their bits.  kk and kt are the same for
// nearly all 16-token blocks.  (With those of each block's largest scale, a
// block with one value 2^16 above the others, of no weight itself, left the other
// blocks' probabilities 2^-16 smaller, and fp32 outputs 1e-4 off.)
//
// Warps: 0-7 softmax (a thread is a row and half of a tile's keys, and for the
// accumulators half of the channels), 8-14 dequantisation (each takes every
// seventh 16-token block and copies its own raw blocks, two ahead; a block's
// values come after the next block's keys, as the scores need those first: 512
// queries of 32 heads over 16384 keys 324 us, both at once 361), 15 issues the
// MMAs.
//
// What bounds it: the softmax warps, 2000 of a tile's 2400 cycles (read S, two
// exponentials' pieces, write P), the tensor cores being busy for 1540.  512
// queries of 32 heads of 128 over 16384 keys take 324 us in fp32 (133 GFLOP, 0.41
// PFLOP/s counted once, 1.2 of products; the few-row form 1287), 312 in fp16 (743).  (With four softmax warps, a thread a whole row, the softmax took
// 3700 cycles a tile, and the tensor cores less than half of that.)
#include "qk_attn_chunk.cuh"
#include "qk_internal.h"

namespace qk {
using namespace attn;
using namespace chunk;
namespace {

constexpr int kSoftmaxWarps = 8, kDequantWarps = 7, kMmaWarp = 15;
constexpr int kThreads = 16 * 32;
constexpr int kStages = 2;                 // tiles of K' and of V'
constexpr int kMetas = 8;                  // tiles whose exponents are kept: more than stages and tiles at work
constexpr int kSlots = 3 * kDequantWarps;  // raw blocks in flight and at work: three a dequantising warp, its own
constexpr int kFlush = 4;                  // tiles whose products one accumulator takes

template <int G>
struct Shape {
    static constexpr int D = 32 * G;
    static constexpr int kblocks = (D + 63) / 64;                    // 64-column blocks of a K-major operand row
    static constexpr int block_bytes = 18 * D;
    static constexpr int k_piece = kblocks * kTile * 128;            // one piece of a tile of K'
    static constexpr int v_piece = D * 128;                          // and of V' transposed: D rows of 64 keys
    static constexpr int k_at = 0;
    static constexpr int v_at = k_at + kStages * 2 * k_piece;
    static constexpr int raw_at = v_at + kStages * 2 * v_piece;
    static constexpr int scale_at = raw_at + kSlots * block_bytes;   // the dequantising warps' scaled scales
    static constexpr int scale_bytes = (4 + 2 * 2) * 16 * G;         // a fp16 pair a key scale, a row of values' a group, twice
    static constexpr int meta_at = scale_at + kDequantWarps * scale_bytes;       // [tile % kMetas][block] (2^kk, kt, 2^-kt, 0)
    static constexpr int bars_at = meta_at + kMetas * kTileBlocks * 16;
    static constexpr int flags_at = bars_at + (kSlots + 4 * kStages + 4) * 8;
    static constexpr int rows_at = flags_at + 16;                    // a float of each row's two threads
    static constexpr int bytes = rows_at + 2 * kChunkRows32 * 4;
    // a warp meets every second tile or more often: no phase of a barrier that it waits for can be taken for an older
    static_assert(kDequantWarps <= kStages * kTileBlocks && kStages >= 2, "phases");
    static constexpr int smem = bytes + 1008;                        // the base is brought to 1024 bytes
    static_assert(smem <= 227 * 1024, "shared memory of a block");
    // tensor memory
    static constexpr int p_col = 64, q_col = 128, o_col = 256, sum_col = 384;      // P: two pieces of 32; Q: two of D/2
    static_assert(D <= 128, "tensor memory");
};

// Barrier addresses.
struct Bars {
    uint32_t at;
    __device__ __forceinline__ uint32_t rfull(int i) const { return at + 8 * i; }
    __device__ __forceinline__ uint32_t kfull(int i) const { return at + 8 * (kSlots + i); }
    __device__ __forceinline__ uint32_t kempty(int i) const { return at + 8 * (kSlots + kStages + i); }
    __device__ __forceinline__ uint32_t vfull(int i) const { return at + 8 * (kSlots + 2 * kStages + i); }
    __device__ __forceinline__ uint32_t vempty(int i) const { return at + 8 * (kSlots + 3 * kStages + i); }
    __device__ __forceinline__ uint32_t sfull() const { return at + 8 * (kSlots + 4 * kStages); }
    __device__ __forceinline__ uint32_t sread() const { return at + 8 * (kSlots + 4 * kStages + 1); }
    __device__ __forceinline__ uint32_t pfull() const { return at + 8 * (kSlots + 4 * kStages + 2); }
    __device__ __forceinline__ uint32_t odone() const { return at + 8 * (kSlots + 4 * kStages + 3); }
};

// m s of fp16 pairs in two pieces: the rounded product, and what it left (exact).
__device__ __forceinline__ void two_pieces(uint32_t m, uint32_t s, uint32_t &lead, uint32_t &rest)
{
    lead = mul_half2(m, s);
    rest = fma_half2(m, s, lead ^ 0x80008000u);
}

// Whether `over` is true in any softmax thread; all of them call it.
__device__ __forceinline__ bool any_softmax(bool over)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(over)), "n"(kSoftmaxWarps * 32)
                 : "memory");
    return r != 0;
}

// P of 32 scores v of a row in two fp16 pieces, and the sums of each block's 16.
template <bool MASK>
__device__ __forceinline__ void exponents32(const Row &R, const uint32_t (&v)[32], const float (&f)[2], const float (&kt)[2],
                                            int key0, uint32_t (&p1)[16], uint32_t (&p2)[16], float (&sum)[2])
{
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const float at = kt[b] - R.m;
        const uint64_t f2 = pack2f(f[b], f[b]), at2 = pack2f(at, at);
        uint64_t total = 0;      // two zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 16 * b + 2 * i;
            float2 z = unpack2f(fma_f32x2(pack2(v[c], v[c + 1]), f2, at2));
            if (MASK) {
                if (key0 + c < R.lo || key0 + c >= R.hi) z.x = -INFINITY;
                if (key0 + c + 1 < R.lo || key0 + c + 1 >= R.hi) z.y = -INFINITY;
            }
            z.x = ex2(z.x), z.y = ex2(z.y);
            total = add_f32x2(total, pack2f(z.x, z.y));
            // the leading 11 bits, and what rounding to them left, itself to 11 (nothing below 2^-25 counts)
            const uint32_t lead = pack_half(z.x, z.y);
            const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&lead));
            p1[8 * b + i] = lead;
            p2[8 * b + i] = pack_half(z.x - l.x, z.y - l.y);
        }
        const float2 t = unpack2f(total);
        sum[b] = t.x + t.y;
    }
}

// The accumulators of 16 channels scaled by a factor.
__device__ __forceinline__ void scale16(uint32_t addr, float factor)
{
    uint32_t w[16];
    tmem_ld_32x32b_x16(addr, w);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * factor);
    tmem_st_32x32b_x16(addr, w);
}

// 32 of a row's 64 scores of one key tile to probabilities.  All softmax threads call it together; ok: this warp's
// waits so far have not run out.  Returns false if any thread's have.
template <int G, bool MASK>
__device__ __forceinline__ bool softmax_tile(Row &R, uint32_t tmem, int half, uint32_t meta, float *rows, int key0,
                                             const Bars &bars, int tile, uint64_t wait_ns, int lane, bool ok)
{
    using Sh = Shape<G>;
    uint32_t v[32];
    tmem_ld_32x32b_x32(tmem + 32 * half, v);
    float f[2], kt[2], inv[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        uint32_t w[4];
        lds128(w, meta + 16 * (2 * half + b));
        f[b] = R.to_log2 * __uint_as_float(w[0]);
        kt[b] = __uint_as_float(w[1]);
        inv[b] = __uint_as_float(w[2]);
    }
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.sread());          // the next scores may come
    uint32_t p1[16], p2[16];
    float sum[2];
    key0 += 32 * half;
    exponents32<MASK>(R, v, f, kt, key0, p1, p2, sum);
    // the last tile's products, which read P and form O
    if (tile > 0) ok = warp_wait(bars.odone(), (tile - 1) & 1, wait_ns) && ok;
    tc_fence_after();
    const float most = fmaxf(sum[0], sum[1]);
    const bool over = any_softmax(most > kMost || !ok);
    if (over && any_softmax(!ok)) return false;
    const uint32_t o_addr = tmem + Sh::o_col + 16 * G * half, sum_addr = tmem + Sh::sum_col + 16 * G * half;
    if (over) {
        // rows past the limit take a new reference; what they have so far is scaled to it
        float top = kNoMax;
        if (most > kMost) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float y = fmaf(__uint_as_float(v[i]), f[i >> 4], kt[i >> 4]);
                if (!MASK || (key0 + i >= R.lo && key0 + i < R.hi)) top = fmaxf(top, y);
            }
        }
        const int row = threadIdx.x & 127;
        rows[kChunkRows32 * half + row] = top;
        any_softmax(false);
        top = fmaxf(top, rows[kChunkRows32 * (1 - half) + row]);
        any_softmax(false);          // both have read it
        float factor = 1.0f;
        if (top > kNoMax) {
            const float m = ceilf(top) - kFresh;
            factor = ex2(R.m - m);
            R.m = m;
            R.l *= factor;
        }
        exponents32<MASK>(R, v, f, kt, key0, p1, p2, sum);
        for (int c = 0; c < G; ++c) {
            if (tile > 0) scale16(o_addr + 16 * c, factor);
            if (tile > kFlush) scale16(sum_addr + 16 * c, factor);
        }
        tmem_st_wait();          // the flush below loads what these stores wrote, and nothing else orders the two
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) R.l = fmaf(sum[b], inv[b], R.l);
    tmem_st_32x32b_x16(tmem + Sh::p_col + 16 * half, p1);
    tmem_st_32x32b_x16(tmem + Sh::p_col + 32 + 16 * half, p2);
    // the accumulator to the sum, before these products begin it anew
    if (tile > 0 && tile % kFlush == 0) {
#pragma unroll 2
        for (int c = 0; c < G; ++c) {
            uint32_t w[16], s[16];
            tmem_ld_32x32b_x16(o_addr + 16 * c, w);
            if (tile > kFlush) tmem_ld_32x32b_x16(sum_addr + 16 * c, s);
            tmem_ld_wait();
            if (tile > kFlush) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(s[i]));
            }
            tmem_st_32x32b_x16(sum_addr + 16 * c, w);
        }
    }
    tmem_st_wait();
    tc_fence_before();
    return true;
}

// 32 channels of a row; wide: 16 bytes a load.
__device__ __forceinline__ void load32(float (&x)[32], const __half *from, bool in, bool wide)
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = in ? __ldg(reinterpret_cast<const uint4 *>(from) + i) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[8 * i + 2 * k] = half_bits_to_float(w[k]), x[8 * i + 2 * k + 1] = half_bits_to_float(w[k] >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = in ? __half2float(from[i]) : 0.0f;
    }
}
__device__ __forceinline__ void load32(float (&x)[32], const float *from, bool in, bool wide)
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 v = in ? __ldg(reinterpret_cast<const float4 *>(from) + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = in ? __ldg(from + i) : 0.0f;
    }
}

template <int G, class Q>
__global__ void __launch_bounds__(kThreads, 1) chunk32_kernel(const AttnArgs a)
{
    using Sh = Shape<G>;
    constexpr int D = Sh::D;
    constexpr bool two_q = sizeof(Q) == 4;       // fp32 queries are two pieces
    extern __shared__ uint8_t smem_raw[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Bars bars{sb + Sh::bars_at};
    uint32_t *flags = reinterpret_cast<uint32_t *>(sm + Sh::flags_at);     // tensor memory address, poison, dead

    asm volatile("griddepcontrol.wait;" ::: "memory");
    Work w;
    if (!find_work(a, kChunkRows32, D, w)) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(bars.rfull(i), 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars.kfull(i), kTileBlocks), mbar_init(bars.kempty(i), 1);
            mbar_init(bars.vfull(i), kTileBlocks), mbar_init(bars.vempty(i), 1);
        }
        mbar_init(bars.sfull(), 1), mbar_init(bars.sread(), kSoftmaxWarps);
        mbar_init(bars.pfull(), kSoftmaxWarps), mbar_init(bars.odone(), 1);
        flags[1] = flags[2] = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_1(sb + Sh::flags_at, 512);
        tmem_relinquish_1();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __reduce_or_sync(0xFFFFFFFFu, flags[0]);      // in a uniform register

    // softmax threads: their row of Q, scaled by a power of two to [2^10, 2^11), in two pieces, channels 0 4 1 5 2 6 3 7
    // of each eight (the order in which masks take a word's nibbles apart), to tensor memory
    Row R{kNoMax, 0.0f, 1.2e-38f, 0, INT32_MAX};
    const bool softmax_warp = warp < kSoftmaxWarps;
    const uint32_t mine_tmem = tmem + (static_cast<uint32_t>(warp & 3) << 21);       // 32 lanes a warp, lane in bits 16..
    const int my_row = threadIdx.x & 127, half = warp >> 2;       // half: of a tile's keys, and of the channels
    const bool row_in = softmax_warp && my_row < w.rows;
    if (softmax_warp) {
        const Q *from = static_cast<const Q *>(a.q) + row_at(a, w, my_row, row_in, a.ldq, D);
        const bool wide = ((reinterpret_cast<uintptr_t>(a.q) | sizeof(Q) * a.ldq) & 15) == 0;
        float big = 0.0f;
#pragma unroll
        for (int c = 0; c < G; ++c) {
            float x[32];
            load32(x, from + 32 * c, row_in, wide);
#pragma unroll
            for (int k = 0; k < 32; ++k) big = fmaxf(big, fabsf(x[k]));
        }
        int e = 127;
        if (big > 0.0f && big < INFINITY) e = 127 + 10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127);
        e = min(e, 250);
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e) << 23), a.scale_log2);
        R.to_log2 = fmaxf(a.scale_log2 / up, 1.2e-38f);
        if (row_in) row_keys(a, w, my_row, R.lo, R.hi);
        for (int c = half; c < G; c += 2) {
            float x[32];
            load32(x, from + 32 * c, row_in, wide);
            uint32_t q1[16], q2[16];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lead[2], rest[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float v = x[8 * k + j + 4 * h] * up;
                        lead[h] = two_q ? rintf(v) : v;
                        rest[h] = two_q ? rintf((v - lead[h]) * 4096.0f) * (1.0f / 4096.0f) : 0.0f;
                    }
                    q1[4 * k + j] = pack_half(lead[0], lead[1]);
                    q2[4 * k + j] = pack_half(rest[0], rest[1]);
                }
            tmem_st_32x32b_x16(mine_tmem + Sh::q_col + 16 * c, q1);
            if (two_q) tmem_st_32x32b_x16(mine_tmem + Sh::q_col + D / 2 + 16 * c, q2);
        }
        tmem_st_wait();
    }
    if (softmax_warp || warp == kMmaWarp) {       // the dequantising warps need no query
        tc_fence_before();
        named_bar_sync(2, (kSoftmaxWarps + 1) * 32);
        tc_fence_after();
    }
    bool dead = false, poison = false;

    if (warp == kMmaWarp) {
        // ------------------------------------------------ the MMAs, by one elected thread; the warp waits together
        if (w.ntiles > 0) {
            constexpr uint32_t idesc_s = idesc_f16_f32(128, kTile), idesc_o = idesc_f16_f32(128, D);
            const uint32_t p_col = tmem + Sh::p_col, q_col = tmem + Sh::q_col, o_col = tmem + Sh::o_col;
            // the small products first
            auto scores = [&](int stage) {
                const uint64_t k0 = smem_desc_sw128_kmajor(sb + Sh::k_at + stage * 2 * Sh::k_piece);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 3; ++x) {
                        if (x == 1 && !two_q) continue;
                        const uint32_t q = q_col + (x == 1 ? D / 2 : 0);
                        const uint64_t kx = k0 + (x == 0 ? Sh::k_piece / 16 : 0);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_f16_tmem_a(tmem, q + 8 * k, kx + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2, idesc_s, x > 0 || k > 0);
                    }
                    tc_commit_1(bars.sfull());
                    tc_commit_1(bars.kempty(stage));
                }
                __syncwarp();
            };
            dead = !warp_wait(bars.kfull(0), 0, a.wait_ns);
            tc_fence_after();
            if (!dead) scores(0);
            for (int i = 0; i < w.ntiles && !dead; ++i) {
                const int stage = i % kStages, next = (i + 1) % kStages;
                if (i + 1 < w.ntiles) {         // the next scores, once these have been read
                    if (!warp_wait(bars.kfull(next), ((i + 1) / kStages) & 1, a.wait_ns) ||
                        !warp_wait(bars.sread(), i & 1, a.wait_ns)) { dead = true; break; }
                    tc_fence_after();
                    scores(next);
                }
                if (!warp_wait(bars.vfull(stage), (i / kStages) & 1, a.wait_ns) || !warp_wait(bars.pfull(), i & 1, a.wait_ns)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                const uint64_t v0 = smem_desc_sw128_kmajor(sb + Sh::v_at + stage * 2 * Sh::v_piece);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 3; ++x) {
                        const uint32_t p = p_col + (x == 1 ? 32 : 0);
                        const uint64_t vx = v0 + (x == 0 ? Sh::v_piece / 16 : 0);
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            tc_mma_f16_tmem_a(o_col, p + 8 * k, vx + 2 * k, idesc_o, i % kFlush != 0 || x > 0 || k > 0);
                    }
                    tc_commit_1(bars.odone());
                    tc_commit_1(bars.vempty(stage));
                }
                __syncwarp();
            }
        }
    } else if (!softmax_warp) {
        // ------------------------------------------------ dequantisation: block j of the part, 16 tokens
        const int r8 = lane >> 2, c = lane & 3, swap = G % 2 == 0 ? r8 & 1 : 0;
        // scales: group sg of tokens st, st + 1
        const int sg = lane % G, st = 2 * (lane / G);
        const bool scale_lane = lane < 8 * G;
        // keys: tokens key_token + 2h; where their 16-byte chunk of group 0 (1, with swap) lies among the block's rows
        const int key_token = 4 * (r8 >> 1) + (r8 & 1);
        uint32_t key_at[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            key_at[h] = key_token * 128 + (((4 * swap + c) ^ ((key_token + 2 * h) & 7)) << 4);
        // values: an item is (g, r, half of the block's tokens): 4 words, channels 32g + 4r + j, 8 tokens a chunk; the items
        // of a quarter of the warp start at other j, so that they too write all eight columns
        constexpr int kItems = (16 * G + 31) / 32;
        const int vr = G == 3 ? (lane >> 1) & 7 : lane >> 2, kp = G == 3 ? lane & 1 : (lane >> 1) & 1;
        const int turn = G == 3 ? (vr >> 1) & 1 : lane & 1, shift = 8 * turn;
        const uint32_t value_at = (4 * vr + 2 * turn) * 128 + (((4 * vr + 2 * turn) & 7) << 4);
        auto group_of = [&](int k) { return G == 3 ? 2 * k + (lane >> 4) : kItems * (lane & 1) + k; };
        const int me = warp - kSoftmaxWarps;
        const uint32_t scales = sb + Sh::scale_at + me * Sh::scale_bytes;      // keys [token][G], values [G][token]
        // this warp's blocks are number me, me + 7, ..; its n-th goes to slot me + 7 (n % 3).  A lane holds the address
        // of one of the next 32
        const int mine = w.nblk > me ? (w.nblk - me + kDequantWarps - 1) / kDequantWarps : 0;
        const uint64_t policy = l2_evict_first_policy();
        const uint8_t *addr = a.pages;
        int issued = 0, arrived = 0;
        auto copy = [&](int n) {
            if (n >= mine) return;
            issued = n + 1;
            if ((n & 31) == 0) {
                addr = a.pages;
                if (n + lane < mine) {
                    const int64_t blk = static_cast<int64_t>(w.blk0) + me + kDequantWarps * (n + lane), pg = blk / a.page_blocks;
                    const int32_t page = a.page_table[static_cast<int64_t>(w.b) * a.ld_pages + pg];
                    if (page < 0 || page >= a.n_pages) {
                        poison = true;
                        record_error(a.err, kErrBadIndex);
                    } else {
                        addr += ((static_cast<int64_t>(page) * a.n_kv + w.hk) * a.page_blocks + (blk - pg * a.page_blocks)) *
                                static_cast<int64_t>(Sh::block_bytes);
                    }
                }
            }
            if (lane == (n & 31) && !(me + kDequantWarps * n == a.skip_block && blockIdx.x == 0)) {
                const int slot = me + kDequantWarps * (n % 3);
                mbar_arrive_expect_tx(bars.rfull(slot), Sh::block_bytes);
                bulk_g2s(sb + Sh::raw_at + slot * Sh::block_bytes, addr, Sh::block_bytes, bars.rfull(slot), policy);
            }
        };
        // Keys of block j, its n-th of this warp.  False if a wait ran out.
        auto keys = [&](int j, int n) {
            const int i = j / kTileBlocks, bi = j % kTileBlocks;      // key tile, block of it
            const bool have = j < w.nblk;
            const int slot = me + kDequantWarps * (n % 3);
            const uint32_t raw = sb + Sh::raw_at + slot * Sh::block_bytes;
            if (have) {
                if (!warp_wait(bars.rfull(slot), (n / 3) & 1, a.wait_ns)) return false;
                arrived = n + 1;
            }
            // scales: a lane has those of one group g of two neighbouring tokens
            uint32_t dk[2] = {0, 0}, dv[2] = {0, 0}, top_k = 0, top_v = 0, odd = 0;
            const bool inner = have && j * kBlockTokens >= w.lo && (j + 1) * kBlockTokens <= w.hi;
            if (scale_lane) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = j * kBlockTokens + st + e;
                    if (inner || (have && key >= w.lo && key < w.hi)) {
                        dk[e] = lds16(raw + 16 * D + 2 * ((st + e) * G + sg));
                        dv[e] = lds16(raw + 17 * D + 2 * ((st + e) * G + sg));
                    }
                    if ((dk[e] & 0x7C00u) != 0x7C00u) top_k = max(top_k, dk[e] & 0x7FFFu);
                    if ((dv[e] & 0x7C00u) != 0x7C00u) top_v = max(top_v, dv[e] & 0x7FFFu);
                    else odd |= 1 << e;
                }
            }
            top_k = redux_max_u32(0xFFFFFFFFu, top_k);
            top_v = redux_max_u32(0xFFFFFFFFu, top_v);
            const int kk = power_of(top_k), kt = power_of(top_v);
            const float down_k = __uint_as_float(static_cast<uint32_t>(127 - kk) << 23);
            const float down_v = __uint_as_float(static_cast<uint32_t>(127 - kt) << 23);
            if (scale_lane) {
                float sv[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sk = half_bits_to_float(dk[e]) * down_k;
                    // a value scale that is not finite counts as 0, and makes the key's scores NaN (below), and with
                    // them the rows that see it
                    sv[e] = odd >> e & 1 ? 0.0f : half_bits_to_float(dv[e]) * down_v;
                    sts32(scales + 4 * ((st + e) * G + sg), pack_half(sk, sk));
                }
                sts32(scales + 64 * G + 32 * G * (n & 1) + 2 * (16 * sg + st), pack_half(sv[0], sv[1]));
            }
            if (lane == 0)
                sts128(sb + Sh::meta_at + (i % kMetas * kTileBlocks + bi) * 16, static_cast<uint32_t>(127 + kk) << 23,
                       __float_as_uint(static_cast<float>(kt)), __float_as_uint(down_v), 0u);
            __syncwarp();
            if (__any_sync(0xFFFFFFFFu, odd)) {
                for (int e = 0; e < 2; ++e)
                    if (odd >> e & 1) sts32(scales + 4 * ((st + e) * G), 0x7FFF7FFFu);
                __syncwarp();
            }
            // keys: lane (r, c) has token 4(r/2) + 2h + r%2, channels 32g + 8c..8c+7 a word
            if (i >= kStages && !warp_wait(bars.kempty(i % kStages), (i / kStages - 1) & 1, a.wait_ns)) return false;
            const uint32_t kb = sb + Sh::k_at + i % kStages * 2 * Sh::k_piece + bi * kBlockTokens * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t words[G];
                lds_words<G>(words, raw + h * 128 * G + lane * 4 * G);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    // odd r take the groups in pairs the other way round: a quarter of the warp then writes all eight
                    // 16-byte columns
                    const uint32_t word = G % 2 == 0 && swap ? words[g ^ (G % 2 == 0)] : words[g], high = word >> 8;
                    const uint32_t s = lds32(scales + 4 * ((key_token + 2 * h) * G + (g ^ swap)));
                    const uint32_t m[4] = {signed_nibbles<0>(word), signed_nibbles<1>(word), signed_nibbles<0>(high), signed_nibbles<1>(high)};
                    uint32_t lead[4], rest[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) two_pieces(m[k], s, lead[k], rest[k]);
                    // chunk 4 (g ^ swap) + c of row t, 16 bytes each: its column of 8 is xored with t % 8
                    const uint32_t at = kb + (g >> 1) * (kTile * 128) + h * 256 + (key_at[h] ^ ((g & 1) << 6));
                    sts128(at, lead[0], lead[1], lead[2], lead[3]);
                    sts128(at + Sh::k_piece, rest[0], rest[1], rest[2], rest[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.kfull(i % kStages));
            return true;
        };
        // And its values.
        auto values = [&](int j, int n) {
            const int i = j / kTileBlocks, bi = j % kTileBlocks;
            const uint32_t raw = sb + Sh::raw_at + (me + kDequantWarps * (n % 3)) * Sh::block_bytes;
            if (i >= kStages && !warp_wait(bars.vempty(i % kStages), (i / kStages - 1) & 1, a.wait_ns)) return false;
            const uint32_t vb = sb + Sh::v_at + i % kStages * 2 * Sh::v_piece, column = (2 * bi + kp) << 4;
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int g = group_of(k);
                if (G != 3 || g < G) {
                    uint32_t words[4], s[4];      // tokens 8kp + 0,1 | 2,3 | 4,5 | 6,7
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        words[e] = lds32(raw + 8 * D + (e & 1) * 128 * G + (vr * 4 + 2 * kp + (e >> 1)) * 4 * G + 4 * g);
                    lds128(s, scales + 64 * G + 32 * G * (n & 1) + 2 * (16 * g + 8 * kp));
#pragma unroll
                    for (int half_j = 0; half_j < 2; ++half_j) {
                        uint32_t src[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) src[e] = words[e] >> (half_j ? 8 - shift : shift);
                        // row 32g + 4r + j with j = 2 (half_j ^ turn) + jj, its columns xored with row % 8
                        const uint32_t row = g * 4096 + (value_at ^ (half_j ? 256 + 32 : 0));
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj) {
                            uint32_t lead[4], rest[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                two_pieces(jj ? signed_nibbles<1>(src[e]) : signed_nibbles<0>(src[e]), s[e], lead[e], rest[e]);
                            const uint32_t at = vb + ((row ^ (jj ? 128 + 16 : 0)) ^ column);
                            sts128(at, lead[0], lead[1], lead[2], lead[3]);
                            sts128(at + Sh::v_piece, rest[0], rest[1], rest[2], rest[3]);
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.vfull(i % kStages));
            return true;
        };
        copy(0);
        copy(1);
        copy(2);
        const int blocks = w.ntiles * kTileBlocks;
        for (int j = me, n = 0; j < blocks + kDequantWarps && !dead; j += kDequantWarps, ++n) {
            if (j < blocks && !keys(j, n)) dead = true;
            if (n > 0 && !dead) {
                if (!values(j - kDequantWarps, n - 1)) dead = true;
                else copy(n + 2);       // into the slot just read
            }
        }
        // copies still in flight when a wait ran out are waited for before the block ends
        if (dead)
            for (int k = arrived; k < issued; ++k) mbar_wait(bars.rfull(me + kDequantWarps * (k % 3)), (k / 3) & 1, a.wait_ns);
        if (__any_sync(0xFFFFFFFFu, poison) && lane == 0) flags[1] = 1;
    } else {
        // ------------------------------------------------ softmax: a thread is a row
        // keys that every row sees
        int see_lo, see_hi, none;
        row_keys(a, w, w.rows - 1, see_lo, none);
        row_keys(a, w, 0, none, see_hi);
        float *rows = reinterpret_cast<float *>(sm + Sh::rows_at);
        for (int i = 0; i < w.ntiles; ++i) {
            const bool ok = warp_wait(bars.sfull(), i & 1, a.wait_ns);
            tc_fence_after();
            const int key0 = i * kTile;
            const uint32_t meta = sb + Sh::meta_at + i % kMetas * kTileBlocks * 16;
            const bool whole = key0 >= see_lo && key0 + kTile <= see_hi;
            if (whole ? !softmax_tile<G, false>(R, mine_tmem, half, meta, rows, key0, bars, i, a.wait_ns, lane, ok)
                      : !softmax_tile<G, true>(R, mine_tmem, half, meta, rows, key0, bars, i, a.wait_ns, lane, ok)) {
                dead = true;
                break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.pfull());
        }
        if (w.ntiles > 0 && !dead && !warp_wait(bars.odone(), (w.ntiles - 1) & 1, a.wait_ns)) dead = true;
        tc_fence_after();
        rows[kChunkRows32 * half + my_row] = R.l;
    }
    if (__any_sync(0xFFFFFFFFu, dead) && lane == 0) {
        record_error(a.err, kErrTimeout);
        flags[2] = 1;
    }
    __syncthreads();
    poison = flags[1] || flags[2];

    // rows out, or to the workspace
    if (softmax_warp) {
        const float *rows = reinterpret_cast<const float *>(sm + Sh::rows_at);
        R.l = poison ? __int_as_float(0x7FC00000) : rows[my_row] + rows[kChunkRows32 + my_row];
        float *part = nullptr;
        if (w.active > 1) {
            part = a.parts + static_cast<int64_t>(blockIdx.x) * (chunk_part_bytes(D, kChunkRows32) / 4);
            if (row_in && half == 0) {
                part[kChunkRows32 * D + 2 * my_row] = R.m;
                part[kChunkRows32 * D + 2 * my_row + 1] = R.l;
            }
            part += my_row * 4;       // a warp's 32 rows of four channels lie side by side
        }
        const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | a.ldo * (a.out_type == QK_F32 ? 4 : 2)) & 15) == 0;
        const int64_t to = row_at(a, w, my_row, row_in, a.ldo, D);
        for (int c = G * half; c < G * half + G; ++c) {
            uint32_t v[16], s[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = s[i] = 0;
            if (w.ntiles > 0 && !flags[2]) {
                tmem_ld_32x32b_x16(mine_tmem + Sh::o_col + 16 * c, v);
                if (w.ntiles > kFlush) tmem_ld_32x32b_x16(mine_tmem + Sh::sum_col + 16 * c, s);
                tmem_ld_wait();
            }
            if (!row_in) continue;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]) + __uint_as_float(s[i]);
            if (part) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4 *>(part + (4 * c + i / 4) * (kChunkRows32 * 4)) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = R.l == 0.0f ? 0.0f : x[i] / R.l;
            store16(a, to + 16 * c, x, wide);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_1(tmem, 512);
    }
}

template <int G, class Q>
cudaError_t launch(const AttnArgs &a, int64_t groups, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    return launch_tiles(chunk32_kernel<G, Q>, done, Shape<G>::smem, kThreads, a, 32 * G, kChunkRows32, groups, st);
}

}  // namespace

namespace attn {

cudaError_t chunk32_launch(const AttnArgs &a, int D, int64_t groups, cudaStream_t st)
{
    const bool half = a.q_type == QK_F16;
    if (D == 64) return half ? launch<2, __half>(a, groups, st) : launch<2, float>(a, groups, st);
    if (D == 96) return half ? launch<3, __half>(a, groups, st) : launch<3, float>(a, groups, st);
    if (D == 128) return half ? launch<4, __half>(a, groups, st) : launch<4, float>(a, groups, st);
    return cudaErrorInvalidValue;
}

}  // namespace attn
}  // namespace qk
