// qk_attn_chunk.cu -- attention over the 4-bit cache for many query rows a
// key/value head (prompt chunks) with bf16 queries, on the 5th-generation
// tensor cores.
//
// A thread block takes 256 rows (queries x grouped heads) of one key/value
// head as two tiles of 128 and walks the keys in tiles of 64:
//   S = Q K'^T        M 128, N 64, K = D
//   O += P V'         M 128, N = D, K = 64
// with K' and V' in shared memory and S, P and O in tensor memory, and Q too
// but for the second tile's at 128 channels, where tensor memory is full.
// (With Q in shared memory and 128 keys a tile the products' operands alone
// filled the shared memory's 128 bytes a clock.)  P has columns of its own, so
// the next scores are formed while these are turned into P.
// K' and V' are the cache's values in fp16, formed once for both row tiles
// straight in the operands' 128-byte-swizzled layouts.
//
// Scales: K' = K 2^-kk and V' = V 2^-kt, products (n - 8) (d 2^-kk) rounded
// once to fp16, which holds them with all its 11 bits from 2^-20 up; kk and kt
// are -6 but for 16-token blocks with scales of 2^6 and more (power_of).  (With
// kk and kt from every block's largest scale, and n - 8 and its product in one
// multiply-add below fp16's normal range, a group or token of scales 2^-12 of
// the block's largest was 0.7% off, one of 2^-18 half.)  2^kk goes to the scores
// and 2^kt to the exponents of P.  Each row
// keeps a reference M (a whole number, so moving it scales by a power of
// two): P = 2^(z + kt - M) stays below 2^14, and M moves only when that would
// be passed, so most tiles need neither a row maximum nor a rescaling of O.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles (a thread is a row), 8-13
// the dequantisation (each takes every sixth 16-token block and copies its own
// raw blocks, two ahead), 14 and 15 issue the MMAs, one for each row tile, so
// that the waits of one are covered by the products of the other.
//
// What bounds it: three things at once.  1024 queries of 32 heads of 128 over
// 16384 keys, 8 key/value heads, 266 GFLOP, take 268 us (1.0 PFLOP/s, 52% of
// the cuBLAS rate); a tile of 64 keys for 256 rows is 2015 cycles, of which the
// softmax warps work 1700 to 1830, the dequantising ones 1450 to 1570 and the
// tensor cores 1210 (busy 60% of the time where a thread block is: 128 of 152
// SMs).
#include "qk_attn_chunk.cuh"
#include "qk_internal.h"

namespace qk {
using namespace attn;
using namespace chunk;
namespace {

// Sixteen warps, so that a thread may have 128 registers.
constexpr int kSoftmaxWarps = 8, kDequantWarps = 6, kMmaWarp = 14;
constexpr int kThreads = 16 * 32;
constexpr int kStages = 3;                 // tiles of K' and of V'
constexpr int kMetas = 8;                  // tiles whose exponents are kept: more than stages and tiles at work
constexpr int kSlots = 2 * kDequantWarps;  // raw blocks in flight: two a dequantising warp, its own

template <int G>
struct ChunkShape {
    static constexpr int D = 32 * G;
    static constexpr int kblocks = (D + 63) / 64;                    // 64-column blocks of a K-major operand row
    static constexpr int block_bytes = 18 * D;
    static constexpr int k_bytes = kblocks * kTile * 128;            // one tile of K'
    static constexpr int v_bytes = D * 128;                          // and of V' transposed: D rows of 64 keys
    static constexpr int k_at = 0;
    static constexpr int v_at = k_at + kStages * k_bytes;
    static constexpr bool q2_in_smem = D > 96;                       // Q of the second row tile
    static constexpr int q2_at = v_at + kStages * v_bytes;
    static constexpr int raw_at = q2_at + (q2_in_smem ? kblocks * 128 * 128 : 0);
    static constexpr int scale_at = raw_at + kSlots * block_bytes;   // the dequantising warps' scaled scales
    static constexpr int scale_bytes = (4 + 2) * 16 * G;             // a fp16 pair a key scale, a row of values' a group
    static constexpr int meta_at = scale_at + kDequantWarps * scale_bytes;       // [tile % kMetas][block] (2^kk, kt, 2^-kt, 0)
    static constexpr int bars_at = meta_at + kMetas * kTileBlocks * 16;
    static constexpr int flags_at = bars_at + (kSlots + 4 * kStages + 8) * 8;
    static constexpr int bytes = flags_at + 16;
    // a warp meets every second tile or more often: no phase of a barrier that it waits for can be taken for an older
    static_assert(kDequantWarps <= 2 * kTileBlocks && kStages >= 2, "phases");
    static constexpr int smem = bytes + 1008;                        // the base is brought to 1024 bytes
    // tensor memory: S 0..127, P 128..191, Q of the first tile 192..255, O after, Q of the second from 448
    static constexpr int p_col = 128, q_col = 192, o_col = 256, q2_col = 448;
    static_assert(q2_in_smem || (o_col + 2 * D <= q2_col && q2_col + D / 2 <= 512), "tensor memory");
};

// Barrier addresses.
struct Bars {
    uint32_t at;
    __device__ __forceinline__ uint32_t rfull(int i) const { return at + 8 * i; }
    __device__ __forceinline__ uint32_t kfull(int i) const { return at + 8 * (kSlots + i); }
    __device__ __forceinline__ uint32_t kempty(int i) const { return at + 8 * (kSlots + kStages + i); }
    __device__ __forceinline__ uint32_t vfull(int i) const { return at + 8 * (kSlots + 2 * kStages + i); }
    __device__ __forceinline__ uint32_t vempty(int i) const { return at + 8 * (kSlots + 3 * kStages + i); }
    __device__ __forceinline__ uint32_t sfull(int x) const { return at + 8 * (kSlots + 4 * kStages + x); }
    __device__ __forceinline__ uint32_t sread(int x) const { return at + 8 * (kSlots + 4 * kStages + 2 + x); }
    __device__ __forceinline__ uint32_t pfull(int x) const { return at + 8 * (kSlots + 4 * kStages + 4 + x); }
    __device__ __forceinline__ uint32_t odone(int x) const { return at + 8 * (kSlots + 4 * kStages + 6 + x); }
};

// P of a row's 64 scores v, as fp16 pairs, and the sums of each block's 16.
template <bool MASK>
__device__ __forceinline__ void exponents64(const Row &R, const uint32_t (&v)[2][32], const float (&f)[4], const float (&kt)[4],
                                            int key0, uint32_t (&p)[32], float (&sum)[4])
{
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float at = kt[b] - R.m;
        const uint64_t f2 = pack2f(f[b], f[b]), at2 = pack2f(at, at);
        uint64_t total = 0;      // two zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 16 * b + 2 * i;
            float2 z = unpack2f(fma_f32x2(pack2(v[c >> 5][c & 31], v[c >> 5][(c & 31) + 1]), f2, at2));
            if (MASK) {
                if (key0 + c < R.lo || key0 + c >= R.hi) z.x = -INFINITY;
                if (key0 + c + 1 < R.lo || key0 + c + 1 >= R.hi) z.y = -INFINITY;
            }
            z.x = ex2(z.x), z.y = ex2(z.y);
            total = add_f32x2(total, pack2f(z.x, z.y));
            p[8 * b + i] = pack_half(z.x, z.y);
        }
        const float2 t = unpack2f(total);
        sum[b] = t.x + t.y;
    }
}

// A row's 64 scores of one key tile to probabilities.  Returns false if the
// wait for the last tile's products (which read P and form O) ran out.
template <int G, bool MASK>
__device__ __forceinline__ bool softmax_tile(Row &R, uint32_t s_addr, uint32_t p_addr, uint32_t o_addr, uint32_t meta,
                                             int key0, uint32_t sread, uint32_t odone, int tile, uint64_t wait_ns, int lane)
{
    constexpr int D = 32 * G;
    uint32_t v[2][32];
    tmem_ld_32x32b_x32(s_addr, v[0]);
    tmem_ld_32x32b_x32(s_addr + 32, v[1]);
    float f[4], kt[4], inv[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t w[4];
        lds128(w, meta + 16 * b);
        f[b] = R.to_log2 * __uint_as_float(w[0]);
        kt[b] = __uint_as_float(w[1]);
        inv[b] = __uint_as_float(w[2]);
    }
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(sread);          // the next scores may come
    uint32_t p[32];
    float sum[4];
    exponents64<MASK>(R, v, f, kt, key0, p, sum);
    if (tile > 0 && !warp_wait(odone, (tile - 1) & 1, wait_ns)) return false;
    tc_fence_after();
    float most = fmaxf(fmaxf(sum[0], sum[1]), fmaxf(sum[2], sum[3]));
    if (__any_sync(0xFFFFFFFFu, most > kMost)) {
        // rows past the limit take a new reference; what they have so far is scaled to it
        float factor = 1.0f;
        if (most > kMost) {
            float top = kNoMax;
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                const float y = fmaf(__uint_as_float(v[i >> 5][i & 31]), f[i >> 4], kt[i >> 4]);
                if (!MASK || (key0 + i >= R.lo && key0 + i < R.hi)) top = fmaxf(top, y);
            }
            const float m = ceilf(top) - kFresh;
            factor = ex2(R.m - m);
            R.m = m;
            R.l *= factor;
        }
        exponents64<MASK>(R, v, f, kt, key0, p, sum);
        if (tile > 0) {
            for (int c = 0; c < D / 16; ++c) {
                uint32_t w[16];
                tmem_ld_32x32b_x16(o_addr + 16 * c, w);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * factor);
                tmem_st_32x32b_x16(o_addr + 16 * c, w);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) R.l = fmaf(sum[b], inv[b], R.l);
    tmem_st_32x32b_x32(p_addr, p);
    tmem_st_wait();
    tc_fence_before();
    return true;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const AttnArgs a)
{
    using Sh = ChunkShape<G>;
    constexpr int D = Sh::D;
    extern __shared__ uint8_t smem_raw[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Bars bars{sb + Sh::bars_at};
    uint32_t *flags = reinterpret_cast<uint32_t *>(sm + Sh::flags_at);     // tensor memory address, poison, dead

    asm volatile("griddepcontrol.wait;" ::: "memory");
    Work w;
    if (!find_work(a, kChunkRows, D, w)) return;
    const int two = w.rows > 128;                // both row tiles hold rows

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(bars.rfull(i), 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars.kfull(i), kTileBlocks), mbar_init(bars.kempty(i), 1 + two);
            mbar_init(bars.vfull(i), kTileBlocks), mbar_init(bars.vempty(i), 1 + two);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bars.sfull(x), 1), mbar_init(bars.sread(x), 4);
            mbar_init(bars.pfull(x), 4), mbar_init(bars.odone(x), 1);
        }
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

    // softmax threads: their row of Q, scaled by a power of two to [2^10, 2^11), channels 0 4 1 5 2 6 3 7 of each
    // eight (the order in which masks take a word's nibbles apart), to tensor memory
    Row R{kNoMax, 0.0f, 1.2e-38f, 0, INT32_MAX};
    const int half = warp >> 2, my_row = threadIdx.x & 127;
    const bool softmax_warp = warp < kSoftmaxWarps;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // 32 lanes a warp, lane in bits 16..
    const bool row_in = softmax_warp && half * 128 + my_row < w.rows;
    if (softmax_warp && (half == 0 || two)) {
        const int64_t at = row_at(a, w, half * 128 + my_row, row_in, a.ldq, D);
        // the row as it is, 16 bytes a load where base and stride allow it (one element a load: 45 us more a call)
        const uint16_t *from = static_cast<const uint16_t *>(a.q) + at;
        uint32_t raw[D / 2], top = 0;
        if (((reinterpret_cast<uintptr_t>(a.q) | 2 * a.ldq) & 15) == 0) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 x = row_in ? __ldg(reinterpret_cast<const uint4 *>(from) + c) : make_uint4(0, 0, 0, 0);
                raw[4 * c] = x.x, raw[4 * c + 1] = x.y, raw[4 * c + 2] = x.z, raw[4 * c + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int c = 0; c < D / 2; ++c) raw[c] = row_in ? __ldg(from + 2 * c) | __ldg(from + 2 * c + 1) << 16 : 0;
        }
#pragma unroll
        for (int c = 0; c < D / 2; ++c) top = __vmaxu2(top, raw[c] & 0x7FFF7FFFu);
        const float big = __uint_as_float(max(top >> 16, top & 0xFFFFu) << 16);
        int e = 127;
        if (big > 0.0f && big < INFINITY) e = 127 + 10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127);
        e = min(e, 250);
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e) << 23), a.scale_log2);
        R.to_log2 = fmaxf(a.scale_log2 / up, 1.2e-38f);
        if (row_in) row_keys(a, w, half * 128 + my_row, R.lo, R.hi);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            uint32_t q[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const uint32_t pair = raw[16 * c + 4 * k + j / 2];
                    x[j] = __uint_as_float(pair << 16) * up, x[j + 1] = __uint_as_float(pair & 0xFFFF0000u) * up;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) q[4 * k + j] = pack_half(x[j], x[j + 4]);
            }
            if (half == 0) {
                tmem_st_32x32b_x16(tmem + lanes + Sh::q_col + 16 * c, q);
            } else if constexpr (!Sh::q2_in_smem) {
                tmem_st_32x32b_x16(tmem + lanes + Sh::q2_col + 16 * c, q);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sts128(sb + Sh::q2_at + operand_chunk(my_row, 4 * c + k, 128), q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
            }
        }
        tmem_st_wait();
        fence_proxy_async_smem();
    }
    if (softmax_warp || warp >= kMmaWarp) {       // the dequantising warps need no query
        tc_fence_before();
        named_bar_sync(2, (kSoftmaxWarps + 2) * 32);
        tc_fence_after();
    }
    bool dead = false, poison = false;

    if (warp >= kMmaWarp) {
        // ------------------------------------------------ the MMAs of row tile x, by one elected thread; the warp waits
        // together and what the instructions take is the warp's, so that it stays in uniform registers
        const int x = warp - kMmaWarp;
        if (w.ntiles > 0 && x <= two) {
            constexpr uint32_t idesc_s = idesc_f16_f32(128, kTile), idesc_o = idesc_f16_f32(128, D);
            const uint32_t s_col = tmem + 64 * x, p_col = tmem + Sh::p_col + 32 * x, o_col = tmem + Sh::o_col + D * x;
            auto scores = [&](int stage) {
                const uint64_t k0 = smem_desc_sw128_kmajor(sb + Sh::k_at + stage * Sh::k_bytes);
                if (elect_one()) {
                    if (Sh::q2_in_smem && x == 1) {
                        const uint64_t q0 = smem_desc_sw128_kmajor(sb + Sh::q2_at);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_f16(s_col, q0 + (k >> 2) * (128 * 128 / 16) + (k & 3) * 2,
                                       k0 + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2, idesc_s, k > 0);
                    } else {
                        const uint32_t q = tmem + (x ? Sh::q2_col : Sh::q_col);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_f16_tmem_a(s_col, q + 8 * k, k0 + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2, idesc_s, k > 0);
                    }
                    tc_commit_1(bars.sfull(x));
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
                        !warp_wait(bars.sread(x), i & 1, a.wait_ns)) { dead = true; break; }
                    tc_fence_after();
                    scores(next);
                }
                if (!warp_wait(bars.vfull(stage), (i / kStages) & 1, a.wait_ns) || !warp_wait(bars.pfull(x), i & 1, a.wait_ns)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                const uint64_t v0 = smem_desc_sw128_kmajor(sb + Sh::v_at + stage * Sh::v_bytes);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_f16_tmem_a(o_col, p_col + 8 * k, v0 + 2 * k, idesc_o, i > 0 || k > 0);
                    tc_commit_1(bars.odone(x));
                    tc_commit_1(bars.vempty(stage));
                }
                __syncwarp();
            }
        }
    } else if (warp >= kSoftmaxWarps) {
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
        const uint32_t scales = sb + Sh::scale_at + (warp - kSoftmaxWarps) * Sh::scale_bytes;      // keys [token][G], values [G][token]
        // this warp's blocks are number me, me + 6, ..; its n-th goes to slot me + 6 (n % 2).  A lane holds the address
        // of one of the next 32
        const int me = warp - kSoftmaxWarps, mine = w.nblk > me ? (w.nblk - me + kDequantWarps - 1) / kDequantWarps : 0;
        const uint64_t policy = l2_evict_first_policy();
        const uint8_t *addr = a.pages;
        auto copy = [&](int n) {
            if (n >= mine) return;
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
                const int slot = me + kDequantWarps * (n & 1);
                mbar_arrive_expect_tx(bars.rfull(slot), Sh::block_bytes);
                bulk_g2s(sb + Sh::raw_at + slot * Sh::block_bytes, addr, Sh::block_bytes, bars.rfull(slot), policy);
            }
        };
        copy(0);
        copy(1);
        int n = 0;
        for (int j = me; j < w.ntiles * kTileBlocks; j += kDequantWarps, ++n) {
            const int i = j / kTileBlocks, bi = j % kTileBlocks;      // key tile, block of it
            const bool have = j < w.nblk;
            const int slot = me + kDequantWarps * (n & 1);
            const uint32_t raw = sb + Sh::raw_at + slot * Sh::block_bytes;
            if (have && !warp_wait(bars.rfull(slot), (n >> 1) & 1, a.wait_ns)) { dead = true; break; }
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
                sts32(scales + 64 * G + 2 * (16 * sg + st), pack_half(sv[0], sv[1]));
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
            if (i >= kStages && !warp_wait(bars.kempty(i % kStages), (i / kStages - 1) & 1, a.wait_ns)) { dead = true; break; }
            const uint32_t kb = sb + Sh::k_at + i % kStages * Sh::k_bytes + bi * kBlockTokens * 128;
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
                    // chunk 4 (g ^ swap) + c of row t, 16 bytes each: its column of 8 is xored with t % 8
                    const uint32_t at = kb + (g >> 1) * (kTile * 128) + h * 256 + (key_at[h] ^ ((g & 1) << 6));
                    sts128(at, mul_half2(signed_nibbles<0>(word), s), mul_half2(signed_nibbles<1>(word), s),
                           mul_half2(signed_nibbles<0>(high), s), mul_half2(signed_nibbles<1>(high), s));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.kfull(i % kStages));
            if (i >= kStages && !warp_wait(bars.vempty(i % kStages), (i / kStages - 1) & 1, a.wait_ns)) { dead = true; break; }
            const uint32_t vb = sb + Sh::v_at + i % kStages * Sh::v_bytes, column = (2 * bi + kp) << 4;
            uint32_t words[kItems][4];      // tokens 8kp + 0,1 | 2,3 | 4,5 | 6,7
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t from = raw + 8 * D + (e & 1) * 128 * G + (vr * 4 + 2 * kp + (e >> 1)) * 4 * G;
                if constexpr (G == 4) {
                    lds64(words[0][e], words[kItems - 1][e], from + 4 * group_of(0));
                } else {
#pragma unroll
                    for (int k = 0; k < kItems; ++k) words[k][e] = group_of(k) < G ? lds32(from + 4 * group_of(k)) : 0;
                }
            }
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int g = group_of(k);
                if (G != 3 || g < G) {
                    uint32_t s[4];
                    lds128(s, scales + 64 * G + 2 * (16 * g + 8 * kp));
#pragma unroll
                    for (int half_j = 0; half_j < 2; ++half_j) {
                        uint32_t src[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) src[e] = words[k][e] >> (half_j ? 8 - shift : shift);
                        // row 32g + 4r + j with j = 2 (half_j ^ turn) + jj, its columns xored with row % 8
                        const uint32_t row = g * 4096 + (value_at ^ (half_j ? 256 + 32 : 0));
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[e] = mul_half2(jj ? signed_nibbles<1>(src[e]) : signed_nibbles<0>(src[e]), s[e]);
                            sts128(vb + ((row ^ (jj ? 128 + 16 : 0)) ^ column), x[0], x[1], x[2], x[3]);
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.vfull(i % kStages));
            copy(n + 2);       // into the slot just read
        }
        // copies still in flight when a wait ran out are waited for before the block ends
        if (dead)
            for (int k = n; k < n + 2 && k < mine; ++k)
                mbar_wait(bars.rfull(me + kDequantWarps * (k & 1)), (k >> 1) & 1, a.wait_ns);
        if (__any_sync(0xFFFFFFFFu, poison) && lane == 0) flags[1] = 1;
    } else if (half == 0 || two) {
        // ------------------------------------------------ softmax: a thread is a row
        const uint32_t s_addr = tmem + lanes + 64 * half, p_addr = tmem + lanes + Sh::p_col + 32 * half,
                       o_addr = tmem + lanes + Sh::o_col + D * half;
        // keys that every row of this tile sees
        const int last = min(w.rows, half * 128 + 128) - 1;
        int see_lo, see_hi, none;
        row_keys(a, w, last, see_lo, none);
        row_keys(a, w, half * 128, none, see_hi);
        for (int i = 0; i < w.ntiles; ++i) {
            if (!warp_wait(bars.sfull(half), i & 1, a.wait_ns)) { dead = true; break; }
            tc_fence_after();
            const int key0 = i * kTile;
            const uint32_t meta = sb + Sh::meta_at + i % kMetas * kTileBlocks * 16;
            const bool whole = key0 >= see_lo && key0 + kTile <= see_hi;
            if (whole ? !softmax_tile<G, false>(R, s_addr, p_addr, o_addr, meta, key0, bars.sread(half), bars.odone(half), i, a.wait_ns, lane)
                      : !softmax_tile<G, true>(R, s_addr, p_addr, o_addr, meta, key0, bars.sread(half), bars.odone(half), i, a.wait_ns, lane)) {
                dead = true;
                break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.pfull(half));
        }
        if (w.ntiles > 0 && !dead && !warp_wait(bars.odone(half), (w.ntiles - 1) & 1, a.wait_ns)) dead = true;
        tc_fence_after();
    }
    if (__any_sync(0xFFFFFFFFu, dead) && lane == 0) {
        record_error(a.err, kErrTimeout);
        flags[2] = 1;
    }
    __syncthreads();
    poison = flags[1] || flags[2];

    // rows out, or to the workspace
    if (softmax_warp && (half == 0 || two)) {
        const uint32_t o_addr = tmem + lanes + Sh::o_col + D * half;
        if (poison) R.l = __int_as_float(0x7FC00000);
        const float inv = R.l == 0.0f ? 0.0f : 1.0f / R.l;
        float *part = nullptr;
        if (w.active > 1) {
            part = a.parts + static_cast<int64_t>(blockIdx.x) * (chunk_part_bytes(D, kChunkRows) / 4);
            if (row_in) {
                part[kChunkRows * D + 2 * (half * 128 + my_row)] = R.m;
                part[kChunkRows * D + 2 * (half * 128 + my_row) + 1] = R.l;
            }
            part += (half * 128 + my_row) * 4;       // a warp's 32 rows of four channels lie side by side
        }
        const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | a.ldo * (a.out_type == QK_F32 ? 4 : 2)) & 15) == 0;
        const int64_t to = row_at(a, w, half * 128 + my_row, row_in, a.ldo, D);
        for (int c = 0; c < D / 16; ++c) {
            uint32_t v[16];
            if (w.ntiles > 0 && !flags[2]) {
                tmem_ld_32x32b_x16(o_addr + 16 * c, v);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0;
            }
            if (!row_in) continue;
            if (part) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<uint4 *>(part + (4 * c + i / 4) * (kChunkRows * 4)) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                continue;
            }
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = R.l == 0.0f ? 0.0f : __uint_as_float(v[i]) * inv;
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

// The plan: a thread an item.
__global__ void __launch_bounds__(kItems) plan_kernel(const AttnArgs a, int D, int tile_rows)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kW = kItems / 32;
    __shared__ int tops[kW], sums[kCutChoices + 1][kW], ends[kW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = static_cast<int>(threadIdx.x);
    int n = 0;
    bool has = false;
    if (item < a.items) {
        const Sequence s = sequence_of(a, item / a.tiles);
        const int at = item % a.tiles * tile_rows, rows = s.bad ? 0 : static_cast<int>(s.r1 - s.r0) * a.rep;
        has = s.bad || at < rows;
        if (at < rows) n = span_of(a, s, at, min(tile_rows, rows - at)).blocks;
    }
    int top = n, all = n;
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    if (lane == 0) tops[warp] = top, sums[kCutChoices][warp] = all;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) top = max(top, tops[w]);
    for (int c = 0; c < kCutChoices; ++c) {
        const int per = part_of(top, c);
        const int parts = __reduce_add_sync(0xFFFFFFFFu, has ? max(1, (n + per - 1) / per) : 0);
        if (lane == 0) sums[c][warp] = parts;
    }
    __syncthreads();
    uint32_t key = 0xFFFFFFFFu;
    if (lane < kCutChoices) {
        int parts = 0;
        float blocks = 0.0f;
#pragma unroll
        for (int w = 0; w < kW; ++w) parts += sums[lane][w], blocks += static_cast<float>(sums[kCutChoices][w]);
        parts *= a.n_kv;
        const float cost = part_cost(blocks * a.n_kv, parts, part_of(top, lane), a.sms, chunk_part_bytes(D, tile_rows), lane > 0);
        if (parts <= a.cut) key = (__float_as_uint(cost) & ~15u) | lane;
    }
    key = __reduce_min_sync(0xFFFFFFFFu, key);
    const int per = part_of(top, static_cast<int>(key & 15u));
    const int count = has ? max(1, (n + per - 1) / per) : 0;
    int run = count * a.n_kv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o) run += below;
    }
    if (lane == 31) ends[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += ends[w];
    if (item < a.items) plan_of_items(a)[item] = make_int2(run - count * a.n_kv, count);
    if (threadIdx.x == 0) *plan_any(a) = top > per;
    // thread blocks: of this warp's items one after another, a lane a thread block
    for (int from = 0; from < 32; ++from) {
        const int parts = __shfl_sync(0xFFFFFFFFu, count, from), end = __shfl_sync(0xFFFFFFFFu, run, from);
        for (int u = lane; u < parts * a.n_kv; u += 32)
            plan_of_blocks(a)[end - parts * a.n_kv + u] = make_int4(32 * warp + from, u / parts, u % parts, per);
    }
    for (int w = warp; w < kW; ++w) run += w > warp ? ends[w] : 0;
    const int used = __shfl_sync(0xFFFFFFFFu, run, 31);
    for (int u = used + static_cast<int>(threadIdx.x); u < a.cut; u += kItems) plan_of_blocks(a)[u] = make_int4(-1, 0, 0, 0);
}

// Joins the parts of cut heads in their order: a warp 8 rows of 16 channels, a lane a row of 4; eight parts are on
// their way at once.
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a, int D, int rows, int64_t groups)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!*plan_any(a)) return;
    const int lane = threadIdx.x & 31, per_group = rows / 8 * (D / 16);
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5), group = item / per_group;
    if (group >= groups) return;
    const int at = static_cast<int>(item - group * per_group);
    const int row = at % (rows / 8) * 8 + (lane & 7), vec = at / (rows / 8) * 4 + (lane >> 3);
    const int of = static_cast<int>(group / a.n_kv), hk = static_cast<int>(group) - of * a.n_kv, tile = of % a.tiles;
    const int2 plan = plan_of_items(a)[of];
    const int active = plan.y;
    if (active <= 1) return;       // not cut, without rows, or with an index out of range
    const Sequence seq = sequence_of(a, of / a.tiles);
    const int n = static_cast<int>(seq.r1 - seq.r0) * a.rep, first = tile * rows;
    if (first + row >= n) return;
    const int64_t stride = chunk_part_bytes(D, rows) / 4;
    const float *part = a.parts + (plan.x + hk * active) * stride;
    float m = kNoMax, l = 0.0f, v[4] = {};
    for (int s0 = 0; s0 < active; s0 += 8) {
        float2 ml[8];
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ml[k] = make_float2(kNoMax, 0.0f), x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s0 + k < active) {
                const float *p = part + (s0 + k) * stride;
                ml[k] = *reinterpret_cast<const float2 *>(p + rows * D + 2 * row);
                x[k] = *reinterpret_cast<const float4 *>(p + (vec * rows + row) * 4);
            }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
        const float f0 = ex2(m - top);
        m = top, l *= f0, v[0] *= f0, v[1] *= f0, v[2] *= f0, v[3] *= f0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = ex2(ml[k].x - m);
            l = fmaf(f, ml[k].y, l);
            v[0] = fmaf(f, x[k].x, v[0]), v[1] = fmaf(f, x[k].y, v[1]), v[2] = fmaf(f, x[k].z, v[2]), v[3] = fmaf(f, x[k].w, v[3]);
        }
    }
    const int i = (first + row) / a.rep;
    const int64_t to = (seq.r0 + i) * a.ldo + (static_cast<int64_t>(hk) * a.rep + first + row - i * a.rep) * D + 4 * vec;
    const int size = a.out_type == QK_F32 ? 4 : 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = l == 0.0f ? 0.0f : v[e] / l;
    if ((reinterpret_cast<uintptr_t>(a.out) | a.ldo * size) % (4 * size) != 0) {
        for (int e = 0; e < 4; ++e) store_float_as(a.out, to + e, a.out_type, v[e]);
    } else if (size == 4) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const bool bf16 = a.out_type == QK_BF16;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to) = make_uint2(pack_as(v[0], v[1], bf16), pack_as(v[2], v[3], bf16));
    }
}

}  // namespace

namespace chunk {

cudaError_t launch_tiles(void (*kern)(const AttnArgs), std::atomic<uint64_t> &done, int smem, int threads, const AttnArgs &a, int D,
                         int rows, int64_t groups, cudaStream_t st)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load(std::memory_order_acquire) >> dev & 1)) {      // two threads that find it undone both do it
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = library_programmatic() ? 1 : 0;
    if (a.cut) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kItems);
        e = cudaLaunchKernelEx(&cfg, plan_kernel, a, D, rows);
        if (e != cudaSuccess) return e;
        cfg.numAttrs = 1;      // what follows may be scheduled while the last kernel still runs: it waits for all of it
    }
    cfg.gridDim = dim3(static_cast<unsigned>(a.cut ? a.cut : groups));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess || !a.cut) return e;
    cfg.gridDim = dim3(static_cast<unsigned>((groups * (rows / 8) * (D / 16) + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel, a, D, rows, groups);
}

}  // namespace chunk

namespace {

template <int G>
cudaError_t launch(const AttnArgs &a, int64_t groups, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    static_assert(ChunkShape<G>::smem <= 227 * 1024, "shared memory of a block");
    return launch_tiles(chunk_kernel<G>, done, ChunkShape<G>::smem, kThreads, a, 32 * G, kChunkRows, groups, st);
}

}  // namespace

namespace attn {

cudaError_t chunk_launch(const AttnArgs &a, int D, int64_t groups, cudaStream_t st)
{
    if (D == 64) return launch<2>(a, groups, st);
    if (D == 96) return launch<3>(a, groups, st);
    if (D == 128) return launch<4>(a, groups, st);
    return cudaErrorInvalidValue;
}

}  // namespace attn
}  // namespace qk
