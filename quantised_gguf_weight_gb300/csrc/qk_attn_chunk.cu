// qk_attn_chunk.cu -- attention over the 4-bit cache for many query rows a
// key/value head (prompt chunks) with 16-bit queries, on the 5th-generation
// tensor cores.
//
// A thread block takes 256 rows (queries x grouped heads) of one key/value
// head as two tiles of 128 and walks the keys in tiles of 128:
//   S = Q K'^T        M 128, N 128, K = D     (Q, K' in shared memory)
//   O += P V'         M 128, N = D, K = 128   (P in tensor memory, V' in shared memory)
// with S, P and O in tensor memory (P takes the place of the S it came from).
// K' and V' are the cache's values in fp16, formed once for both row tiles
// straight in the operands' 128-byte-swizzled layouts.
//
// Scales: K' = K 2^-kk and V' = V 2^-kt, kk and kt the exponents of a
// 16-token block's largest scales, so fp16 holds both whatever their
// magnitude; 2^kk goes to the scores and 2^kt to the exponents of P.  Each row
// keeps a reference M (a whole number, so moving it scales by a power of
// two): P = 2^(z + kt - M) stays below 2^14, and M moves only when that would
// be passed, so most tiles need neither a row maximum nor a rescaling of O.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles (a thread is a row), 8-13
// the dequantisation (each takes every sixth 16-token block), 14 issues the
// MMAs, 15 copies raw blocks into a ring.  While one row tile's softmax runs,
// the other's products do.
#include <atomic>

#include "qk_attn.cuh"
#include "qk_internal.h"
#include "qk_tc.cuh"

namespace qk {
using namespace attn;
namespace {

// Sixteen warps, so that a thread may have 128 registers.
constexpr int kSoftmaxWarps = 8, kDequantWarps = 6, kMmaWarp = 14, kLoadWarp = 15;
constexpr int kThreads = 16 * 32;
constexpr int kTile = 128;                 // keys a tile
constexpr int kTileBlocks = kTile / kBlockTokens;
// Raw blocks in flight: a multiple of the dequantising warps, so that a slot is always the same warp's and its phases
// are waited for one by one (a warp that met a slot only every second time could take an old phase for its own).
constexpr int kSlots = 2 * kDequantWarps;
constexpr float kLimit = 14.0f;            // log2 of the largest P
constexpr float kFresh = 4.0f;             // and of a row's largest when its reference moves

template <int G>
struct ChunkShape {
    static constexpr int D = 32 * G;
    static constexpr int kblocks = (D + 63) / 64;                    // 64-column blocks of a K-major operand row
    static constexpr int block_bytes = 18 * D;
    static constexpr int q_bytes = kblocks * 128 * 128;              // one row tile of Q, one tile of K'
    static constexpr int v_bytes = 2 * D * 128;                      // V' transposed: D rows of 128 keys
    static constexpr int q_at = 0;
    static constexpr int k_at = q_at + 2 * q_bytes;
    static constexpr int v_at = k_at + 2 * q_bytes;
    static constexpr int raw_at = v_at + 2 * v_bytes;
    static constexpr int scale_at = raw_at + kSlots * block_bytes;   // the dequantising warps' scaled scales
    static constexpr int scale_bytes = 2 * 16 * G * 2;
    static constexpr int meta_at = scale_at + kDequantWarps * scale_bytes;       // [tile % 4][block] (2^kk, kt, 2^-kt, 0)
    static constexpr int bars_at = meta_at + 4 * kTileBlocks * 16;
    static constexpr int flags_at = bars_at + (2 * kSlots + 14) * 8;
    static constexpr int bytes = flags_at + 16;
    static_assert(kSlots % kDequantWarps == 0 && kDequantWarps <= kTileBlocks, "every warp meets every phase");
    static constexpr int smem = bytes + 1008;                        // the base is brought to 1024 bytes
    static constexpr int o_col = 256;                                // tensor memory: S 0..255, O after
};

// One operand row's 16-byte chunk (8 elements from element 8 * c) in 128-byte swizzle.
__device__ __forceinline__ uint32_t operand_chunk(int row, int c, int rows)
{
    return static_cast<uint32_t>((c >> 3) * rows * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A wait whose outcome the whole warp shares (a limit may run out for one lane and not another).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit_ns));
}

// Barrier addresses.
struct Bars {
    uint32_t at;
    __device__ __forceinline__ uint32_t rfull(int i) const { return at + 8 * i; }
    __device__ __forceinline__ uint32_t rempty(int i) const { return at + 8 * (kSlots + i); }
    __device__ __forceinline__ uint32_t kfull(int i) const { return at + 8 * (2 * kSlots + i); }
    __device__ __forceinline__ uint32_t kempty(int i) const { return at + 8 * (2 * kSlots + 2 + i); }
    __device__ __forceinline__ uint32_t vfull(int i) const { return at + 8 * (2 * kSlots + 4 + i); }
    __device__ __forceinline__ uint32_t vempty(int i) const { return at + 8 * (2 * kSlots + 6 + i); }
    __device__ __forceinline__ uint32_t sfull(int i) const { return at + 8 * (2 * kSlots + 8 + i); }
    __device__ __forceinline__ uint32_t pfull(int i) const { return at + 8 * (2 * kSlots + 10 + i); }
    __device__ __forceinline__ uint32_t odone(int i) const { return at + 8 * (2 * kSlots + 12 + i); }
};

// Splits of a head that have blocks, at least one: each takes the same number.
__device__ __forceinline__ int active_splits(const AttnArgs &a, int blocks)
{
    const int per = max((blocks + a.splits - 1) / a.splits, a.min_blocks);
    return blocks > per ? (blocks + per - 1) / per : 1;
}

// What a thread block works on.
struct Work {
    int64_t b;
    int hk, tile, split;
    Sequence seq;
    Span span;
    int n, first, rows;          // rows of the sequence and head; this block's
    int active;                  // splits with blocks (at least one)
    int nblk, ntiles;            // 16-token blocks and key tiles of this split
    int64_t blk0;                // its first block in the sequence
    int two;                     // both row tiles hold rows
};

// One row's state and its softmax over 32 columns of a score tile.
struct Row {
    float m, l, to_log2;
    int lo, hi;
};

template <int G, bool MASK>
__device__ __forceinline__ void softmax32(Row &R, uint32_t s_addr, uint32_t o_addr, uint32_t meta, int chunk, int key0,
                                          bool has_o)
{
    constexpr int D = 32 * G;
    uint32_t v[32];
    tmem_ld_32x32b_x32(s_addr + 32 * chunk, v);
    float f[2], kt[2], inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[4];
        lds128(w, meta + 16 * (2 * chunk + h));
        f[h] = R.to_log2 * __uint_as_float(w[0]);
        kt[h] = __uint_as_float(w[1]);
        inv[h] = __uint_as_float(w[2]);
    }
    tmem_ld_wait();
    float big = kNoMax;
    const float base0 = kt[0] - R.m, base1 = kt[1] - R.m;
    float z[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        z[i] = fmaf(__uint_as_float(v[i]), f[i >> 4], i < 16 ? base0 : base1);
        if (MASK && (key0 + i < R.lo || key0 + i >= R.hi)) z[i] = -INFINITY;
        big = fmaxf(big, z[i]);
    }
    if (__any_sync(0xFFFFFFFFu, big > kLimit)) {
        // rows past the limit take a new reference; what they have so far is scaled to it
        float factor = 1.0f;
        if (big > kLimit) {
            float top = kNoMax;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float y = fmaf(__uint_as_float(v[i]), f[i >> 4], kt[i >> 4]);
                if (!MASK || (key0 + i >= R.lo && key0 + i < R.hi)) top = fmaxf(top, y);
            }
            const float m = ceilf(top) - kFresh;
            factor = ex2(R.m - m);
            R.m = m;
            R.l *= factor;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                z[i] = fmaf(__uint_as_float(v[i]), f[i >> 4], kt[i >> 4] - m);
                if (MASK && (key0 + i < R.lo || key0 + i >= R.hi)) z[i] = -INFINITY;
            }
        }
        const uint32_t f2 = pack_half(factor, factor);
        for (int c = 0; c < chunk; ++c) {
            uint32_t w[16];
            tmem_ld_32x32b_x16(s_addr + 16 * c, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = mul_half2(w[i], f2);
            tmem_st_32x32b_x16(s_addr + 16 * c, w);
        }
        if (has_o) {
            for (int c = 0; c < D / 16; ++c) {
                uint32_t w[16];
                tmem_ld_32x32b_x16(o_addr + 16 * c, w);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * factor);
                tmem_st_32x32b_x16(o_addr + 16 * c, w);
            }
        }
        tmem_st_wait();
    }
    uint32_t p[16];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float x = ex2(z[i]), y = ex2(z[i + 1]);
        sum[i >> 4] += x + y;
        p[i >> 1] = pack_half(x, y);
    }
    R.l = fmaf(sum[0], inv[0], fmaf(sum[1], inv[1], R.l));
    tmem_st_32x32b_x16(s_addr + 16 * chunk, p);
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

    // unit: split, row tile, head, sequence
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Work w;
    int64_t u = blockIdx.x;
    w.split = static_cast<int>(u % a.splits);
    u /= a.splits;
    w.hk = static_cast<int>(u % a.n_kv);
    u /= a.n_kv;
    w.tile = static_cast<int>(u % a.tiles);
    w.b = u / a.tiles;
    w.seq = sequence_of(a, w.b);
    if (w.seq.bad) {
        if (w.split == 0) poison_rows(a, w.seq, w.hk, w.tile, a.rep * D);
        return;
    }
    w.n = static_cast<int>(w.seq.r1 - w.seq.r0) * a.rep;
    w.first = w.tile * kChunkRows;
    if (w.first >= w.n) return;
    w.rows = min(kChunkRows, w.n - w.first);
    w.two = w.rows > 128;
    w.span = span_of(a, w.seq, w.first, w.rows);
    const int per = max((w.span.blocks + a.splits - 1) / a.splits, a.min_blocks);
    w.active = active_splits(a, w.span.blocks);
    if (w.split >= w.active) return;
    const int b0 = w.split * per;
    w.nblk = min(w.span.blocks - b0, per);
    w.ntiles = (w.nblk + kTileBlocks - 1) / kTileBlocks;
    w.blk0 = w.span.blk_lo + b0;
    const int64_t base = w.blk0 * kBlockTokens;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(bars.rfull(i), 1), mbar_init(bars.rempty(i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.kfull(i), 8), mbar_init(bars.kempty(i), 1);
            mbar_init(bars.vfull(i), 8), mbar_init(bars.vempty(i), 1);
            mbar_init(bars.sfull(i), 1), mbar_init(bars.pfull(i), 4), mbar_init(bars.odone(i), 1);
        }
        flags[1] = flags[2] = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_1(sb + Sh::flags_at, 512);
        tmem_relinquish_1();
    }

    // softmax threads: their row of Q, scaled by a power of two to [2^10, 2^11), channels 0 4 1 5 2 6 3 7 of each
    // eight (the order in which masks take a word's nibbles apart)
    Row R{kNoMax, 0.0f, 1.2e-38f, 0, INT32_MAX};
    const int half = warp >> 2, my_row = threadIdx.x & 127;
    const bool softmax_warp = warp < 8;
    int64_t row_token = 0, row_head = 0;
    const bool row_in = softmax_warp && half * 128 + my_row < w.rows;
    if (softmax_warp && (half == 0 || w.two)) {
        const int row = w.first + half * 128 + my_row;
        const int i = row_in ? row / a.rep : 0;
        row_token = w.seq.r0 + i;
        row_head = static_cast<int64_t>(w.hk) * a.rep + (row_in ? row - i * a.rep : 0);
        const int64_t at = row_token * a.ldq + row_head * D;
        float big = 0.0f;
        if (row_in)
            for (int c = 0; c < D; ++c) big = fmaxf(big, fabsf(load_as_float(a.q, at + c, a.q_type)));
        int e = 127;
        if (big > 0.0f && big < INFINITY) e = 127 + 10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127);
        e = min(e, 250);
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e) << 23), a.scale_log2);
        R.to_log2 = fmaxf(a.scale_log2 / up, 1.2e-38f);
        if (row_in) {
            const int64_t pos = w.seq.len - (w.seq.r1 - w.seq.r0) + i;
            R.lo = clamp_key(a.window > 0 ? pos - a.window + 1 - base : -1);
            R.hi = clamp_key(pos + 1 - base);
        }
        for (int c = 0; c < D / 8; ++c) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = row_in ? load_as_float(a.q, at + 8 * c + j, a.q_type) * up : 0.0f;
            sts128(sb + Sh::q_at + half * Sh::q_bytes + operand_chunk(my_row, c, 128), pack_half(x[0], x[4]),
                   pack_half(x[1], x[5]), pack_half(x[2], x[6]), pack_half(x[3], x[7]));
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = flags[0];
    bool dead = false, poison = false;

    if (warp == kLoadWarp) {
        // ------------------------------------------------ raw blocks into the ring
        const uint64_t policy = l2_evict_first_policy();
        const uint8_t *addr = nullptr;
        for (int j = 0; j < w.nblk && !dead; ++j) {
            if ((j & 31) == 0) {           // addresses of the next 32 blocks, one a lane
                addr = a.pages;
                if (j + lane < w.nblk) {
                    const int64_t blk = w.blk0 + j + lane, pg = blk / a.page_blocks;
                    const int32_t page = a.page_table[w.b * a.ld_pages + pg];
                    if (page < 0 || page >= a.n_pages) {
                        poison = true;
                        record_error(a.err, kErrBadIndex);
                    } else {
                        addr += ((static_cast<int64_t>(page) * a.n_kv + w.hk) * a.page_blocks +
                                 (blk - pg * a.page_blocks)) * static_cast<int64_t>(Sh::block_bytes);
                    }
                }
            }
            const uint64_t from = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(addr), j & 31);
            const int slot = j % kSlots;
            if (j >= kSlots && !warp_wait(bars.rempty(slot), ((j / kSlots) - 1) & 1, a.wait_ns)) dead = true;
            if (dead || (j == a.skip_block && blockIdx.x == 0)) continue;
            if (lane == 0) {
                mbar_arrive_expect_tx(bars.rfull(slot), Sh::block_bytes);
                bulk_g2s(sb + Sh::raw_at + slot * Sh::block_bytes, reinterpret_cast<const void *>(from), Sh::block_bytes,
                         bars.rfull(slot), policy);
            }
            __syncwarp();
        }
        // a copy in flight when a wait ran out is waited for before the block ends
        if (dead)
            for (int i = 0; i < kSlots; ++i) {
                mbar_wait(bars.rfull(i), 0, a.wait_ns / 16 + 1);
                mbar_wait(bars.rfull(i), 1, a.wait_ns / 16 + 1);
            }
        poison = __any_sync(0xFFFFFFFFu, poison);
        if (poison && lane == 0) flags[1] = 1;
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ the MMAs, one thread
        if (lane == 0 && w.ntiles > 0) {
            constexpr uint32_t idesc_s = idesc_f16_f32(128, kTile), idesc_o = idesc_f16_f32(128, D);
            const int qts = w.two ? 2 : 1;
            auto scores = [&](int x, int i) {
                const uint64_t q0 = smem_desc_sw128_kmajor(sb + Sh::q_at + x * Sh::q_bytes);
                const uint64_t k0 = smem_desc_sw128_kmajor(sb + Sh::k_at + (i & 1) * Sh::q_bytes);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
                    tc_mma_f16(tmem + 128 * x, q0 + off, k0 + off, idesc_s, k > 0);
                }
                tc_commit_1(bars.sfull(x));
                if (x == qts - 1) tc_commit_1(bars.kempty(i & 1));
            };
            dead = !mbar_wait(bars.kfull(0), 0, a.wait_ns);
            tc_fence_after();
            for (int x = 0; x < qts && !dead; ++x) scores(x, 0);
            for (int i = 0; i < w.ntiles && !dead; ++i) {
                const bool more = i + 1 < w.ntiles;
                for (int x = 0; x < qts && !dead; ++x) {
                    if (x == 0 && !mbar_wait(bars.vfull(i & 1), (i >> 1) & 1, a.wait_ns)) { dead = true; break; }
                    if (!mbar_wait(bars.pfull(x), i & 1, a.wait_ns)) { dead = true; break; }
                    tc_fence_after();
                    const uint64_t v0 = smem_desc_sw128_kmajor(sb + Sh::v_at + (i & 1) * Sh::v_bytes);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_f16_tmem_a(tmem + Sh::o_col + D * x, tmem + 128 * x + 8 * k,
                                          v0 + (k >> 2) * (D * 128 / 16) + (k & 3) * 2, idesc_o, i > 0 || k > 0);
                    tc_commit_1(bars.odone(x));
                    if (x == qts - 1) tc_commit_1(bars.vempty(i & 1));
                    if (more) {
                        if (x == 0 && !mbar_wait(bars.kfull((i + 1) & 1), ((i + 1) >> 1) & 1, a.wait_ns)) { dead = true; break; }
                        // the next scores take the place of these probabilities
                        if (!mbar_wait(bars.odone(x), i & 1, a.wait_ns)) { dead = true; break; }
                        tc_fence_after();
                        scores(x, i + 1);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= kSoftmaxWarps) {
        // ------------------------------------------------ dequantisation: block j of the split, 16 tokens
        const int r8 = lane >> 2, c = lane & 3;
        const uint32_t scales = sb + Sh::scale_at + (warp - kSoftmaxWarps) * Sh::scale_bytes;      // keys [token][G], values [G][token]
        const int all_lo = clamp_key(w.span.key_lo - base), all_hi = clamp_key(w.span.key_hi - base);
        for (int j = warp - kSoftmaxWarps; j < w.ntiles * kTileBlocks; j += kDequantWarps) {
            const int i = j / kTileBlocks, bi = j % kTileBlocks;      // key tile, block of it
            const bool have = j < w.nblk;
            const int slot = j % kSlots;
            const uint32_t raw = sb + Sh::raw_at + slot * Sh::block_bytes;
            if (have && !warp_wait(bars.rfull(slot), (j / kSlots) & 1, a.wait_ns)) { dead = true; break; }
            // scales: the block's exponents, and the scales less them as fp16
            uint32_t dk[(16 * G + 31) / 32], dv[(16 * G + 31) / 32], top_k = 0, top_v = 0, odd = 0;
#pragma unroll
            for (int k = 0; k < (16 * G + 31) / 32; ++k) {
                const int at = 32 * k + lane, t = at / G;
                dk[k] = dv[k] = 0;
                const int key = j * kBlockTokens + t;
                if (have && at < 16 * G && key >= all_lo && key < all_hi) {
                    dk[k] = lds16(raw + 16 * D + 2 * at);
                    dv[k] = lds16(raw + 17 * D + 2 * at);
                    if ((dk[k] & 0x7C00u) != 0x7C00u) top_k = max(top_k, dk[k] & 0x7FFFu);
                    if ((dv[k] & 0x7C00u) != 0x7C00u) top_v = max(top_v, dv[k] & 0x7FFFu);
                    else odd = 1;
                }
            }
            top_k = redux_max_u32(0xFFFFFFFFu, top_k);
            top_v = redux_max_u32(0xFFFFFFFFu, top_v);
            odd = __any_sync(0xFFFFFFFFu, odd);
            // largest scale in [2^e, 2^(e+1)); a subnormal or 0 counts as 2^-15
            const int ek = top_k >= 0x0400u ? static_cast<int>(top_k >> 10) - 15 : -15;
            const int ev = top_v >= 0x0400u ? static_cast<int>(top_v >> 10) - 15 : -15;
            const float down_k = __uint_as_float(static_cast<uint32_t>(127 - ek) << 23);
            const float down_v = __uint_as_float(static_cast<uint32_t>(127 - ev) << 23);
#pragma unroll
            for (int k = 0; k < (16 * G + 31) / 32; ++k) {
                const int at = 32 * k + lane, t = at / G, g = at - t * G;
                if (at < 16 * G) {
                    const __half hk = __float2half_rn(half_bits_to_float(dk[k]) * down_k);
                    // a value scale that is not finite: the key's scores become NaN instead (below), and with them
                    // the rows that see it
                    const bool fine = (dv[k] & 0x7C00u) != 0x7C00u;
                    const __half hv = __float2half_rn(fine ? half_bits_to_float(dv[k]) * down_v : 0.0f);
                    *reinterpret_cast<__half *>(sm + (scales - sb) + 2 * at) = hk;
                    *reinterpret_cast<__half *>(sm + (scales - sb) + 32 * G + 2 * (16 * g + t)) = hv;
                }
            }
            if (lane == 0) {
                float4 m;
                m.x = __uint_as_float(static_cast<uint32_t>(127 + ek) << 23);
                m.y = static_cast<float>(ev);
                m.z = down_v, m.w = 0.0f;
                *reinterpret_cast<float4 *>(sm + Sh::meta_at + ((i & 3) * kTileBlocks + bi) * 16) = m;
            }
            __syncwarp();
            if (odd) {
#pragma unroll
                for (int k = 0; k < (16 * G + 31) / 32; ++k) {
                    const int at = 32 * k + lane, t = at / G;
                    if (at < 16 * G && (dv[k] & 0x7C00u) == 0x7C00u)
                        *reinterpret_cast<uint16_t *>(sm + (scales - sb) + 2 * (t * G)) = 0x7FFFu;
                }
                __syncwarp();
            }
            // keys: lane (r, c) has token 4(r/2) + 2h + r%2, channels 32g + 8c..8c+7 a word
            if (i >= 2 && !warp_wait(bars.kempty(i & 1), ((i >> 1) - 1) & 1, a.wait_ns)) { dead = true; break; }
            const uint32_t kb = sb + Sh::k_at + (i & 1) * Sh::q_bytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = 4 * (r8 >> 1) + 2 * h + (r8 & 1);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t word = have ? lds32(raw + h * 128 * G + (lane * G + g) * 4) : 0x88888888u;
                    const uint32_t s1 = lds16(scales + 2 * (t * G + g)), s2 = s1 | s1 << 16;
                    sts128(kb + operand_chunk(bi * kBlockTokens + t, 4 * g + c, 128),
                           mul_half2(signed_nibbles<0>(word), s2), mul_half2(signed_nibbles<1>(word), s2),
                           mul_half2(signed_nibbles<0>(word >> 8), s2), mul_half2(signed_nibbles<1>(word >> 8), s2));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.kfull(i & 1));
            // values: an item is (g, r, half of the block's tokens): 4 words, channels 32g + 4r + j, 8 tokens a chunk
            if (i >= 2 && !warp_wait(bars.vempty(i & 1), ((i >> 1) - 1) & 1, a.wait_ns)) { dead = true; break; }
            const uint32_t vb = sb + Sh::v_at + (i & 1) * Sh::v_bytes;
#pragma unroll
            for (int k = 0; k < (16 * G + 31) / 32; ++k) {
                const int item = 32 * k + lane;
                if (item < 16 * G) {
                    const int g = item >> 4, r = (item >> 1) & 7, kp = item & 1;
                    const uint32_t from = raw + 8 * D + ((r * 4 + 2 * kp) * G + g) * 4;
                    uint32_t word[4];      // tokens 8kp + 0,1 | 2,3 | 4,5 | 6,7
                    word[0] = have ? lds32(from) : 0x88888888u;
                    word[1] = have ? lds32(from + 128 * G) : 0x88888888u;
                    word[2] = have ? lds32(from + 4 * G) : 0x88888888u;
                    word[3] = have ? lds32(from + 4 * G + 128 * G) : 0x88888888u;
                    uint32_t s[4];
                    lds128(s, scales + 32 * G + 2 * (16 * g + 8 * kp));
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t src = jj & 2 ? word[e] >> 8 : word[e];
                            x[e] = mul_half2(jj & 1 ? signed_nibbles<1>(src) : signed_nibbles<0>(src), s[e]);
                        }
                        sts128(vb + operand_chunk(32 * g + 4 * r + jj, 2 * bi + kp, D), x[0], x[1], x[2], x[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bars.vfull(i & 1));
                if (have) mbar_arrive(bars.rempty(slot));
            }
        }
    } else if (half == 0 || w.two) {
        // ------------------------------------------------ softmax: a thread is a row
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;          // 32 lanes a warp, lane in bits 16..
        const uint32_t s_addr = tmem + lanes + 128 * half, o_addr = tmem + lanes + Sh::o_col + D * half;
        // keys that every row of this tile sees
        const int last = min(w.rows, half * 128 + 128) - 1;
        const int64_t p0 = w.seq.len - (w.seq.r1 - w.seq.r0) + (w.first + half * 128) / a.rep;
        const int64_t p1 = w.seq.len - (w.seq.r1 - w.seq.r0) + (w.first + last) / a.rep;
        const int see_lo = clamp_key(a.window > 0 ? p1 - a.window + 1 - base : 0), see_hi = clamp_key(p0 + 1 - base);
        for (int i = 0; i < w.ntiles; ++i) {
            if (!warp_wait(bars.sfull(half), i & 1, a.wait_ns)) { dead = true; break; }
            tc_fence_after();
            const int key0 = i * kTile;
            const uint32_t meta = sb + Sh::meta_at + (i & 3) * kTileBlocks * 16;
            if (key0 >= see_lo && key0 + kTile <= see_hi) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) softmax32<G, false>(R, s_addr, o_addr, meta, c, key0 + 32 * c, i > 0);
            } else {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) softmax32<G, true>(R, s_addr, o_addr, meta, c, key0 + 32 * c, i > 0);
            }
            tmem_st_wait();
            tc_fence_before();
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
    if (softmax_warp && (half == 0 || w.two)) {
        const uint32_t o_addr = tmem + (static_cast<uint32_t>(warp & 3) << 21) + Sh::o_col + D * half;
        if (poison) R.l = __int_as_float(0x7FC00000);
        const float inv = R.l == 0.0f ? 0.0f : 1.0f / R.l;
        float *part = nullptr;
        if (w.active > 1) {
            const int64_t group = (w.b * a.tiles + w.tile) * a.n_kv + w.hk;
            part = a.parts + (group * a.splits + w.split) * (chunk_part_bytes(D) / 4);
            if (row_in) {
                part[kChunkRows * D + 2 * (half * 128 + my_row)] = R.m;
                part[kChunkRows * D + 2 * (half * 128 + my_row) + 1] = R.l;
            }
            part += (half * 128 + my_row) * D;
        }
        const int64_t to = row_token * a.ldo + row_head * D;
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
                    *reinterpret_cast<uint4 *>(part + 16 * c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    store_float_as(a.out, to + 16 * c + i, a.out_type,
                                   R.l == 0.0f ? 0.0f : __uint_as_float(v[i]) * inv);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_1(tmem, 512);
    }
}

// Joins the splits' parts in their order: a warp a row and head.
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a, int D, int64_t groups)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t group = item / kChunkRows;
    if (group >= groups) return;
    const int row = static_cast<int>(item - group * kChunkRows);
    const int hk = static_cast<int>(group % a.n_kv), tile = static_cast<int>(group / a.n_kv % a.tiles);
    const Sequence seq = sequence_of(a, group / a.n_kv / a.tiles);
    if (seq.bad) return;
    const int n = static_cast<int>(seq.r1 - seq.r0) * a.rep, first = tile * kChunkRows;
    if (first + row >= n) return;
    const int active = active_splits(a, span_of(a, seq, first, min(kChunkRows, n - first)).blocks);
    if (active <= 1) return;
    const int64_t stride = chunk_part_bytes(D) / 4;
    const float *part = a.parts + group * a.splits * stride;
    float m = kNoMax;
    for (int s = lane; s < active; s += 32) m = fmaxf(m, part[s * stride + kChunkRows * D + 2 * row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float4 v[2] = {};
    float l = 0.0f;
    const int vecs = D / 4;
#pragma unroll 4
    for (int s = 0; s < active; ++s) {
        const float *p = part + s * stride;
        const float f = ex2(p[kChunkRows * D + 2 * row] - m);
        l = fmaf(f, p[kChunkRows * D + 2 * row + 1], l);
        for (int k = 0; k < 2; ++k)
            if (lane + 32 * k < vecs) {
                const float4 x = *reinterpret_cast<const float4 *>(p + row * D + 4 * (lane + 32 * k));
                v[k].x = fmaf(f, x.x, v[k].x), v[k].y = fmaf(f, x.y, v[k].y);
                v[k].z = fmaf(f, x.z, v[k].z), v[k].w = fmaf(f, x.w, v[k].w);
            }
    }
    const int i = (first + row) / a.rep;
    const int64_t to = (seq.r0 + i) * a.ldo + (static_cast<int64_t>(hk) * a.rep + first + row - i * a.rep) * D;
    for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < vecs) {
            const float x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            for (int e = 0; e < 4; ++e)
                store_float_as(a.out, to + 4 * (lane + 32 * k) + e, a.out_type, l == 0.0f ? 0.0f : x[e] / l);
        }
}

template <int G>
cudaError_t launch(const AttnArgs &a, int64_t groups, cudaStream_t st)
{
    const auto kern = chunk_kernel<G>;
    constexpr int smem = ChunkShape<G>::smem;
    static_assert(smem <= 227 * 1024, "shared memory of a block");
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
    cfg.gridDim = dim3(static_cast<unsigned>(groups * a.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = library_programmatic() ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    // the join may be scheduled while the tiles still run: it waits for all of them
    cfg.gridDim = dim3(static_cast<unsigned>((groups * kChunkRows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel, a, 32 * G, groups);
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
