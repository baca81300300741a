// qk_rope.cu -- per-head RMS norm and position rotation, the append of keys
// and values to the 4-bit cache with both on the way, the cache's read-back,
// and the rotation tables.
//
// Mathematics.  A head x of D channels becomes y_j = x_j w_j / sqrt(mean(x^2) +
// eps), then each pair (a, b) of its first rot channels (a c - b s, b c + a s)
// with its position's (c, s).  A stored group of 32 channels is a scale d =
// fp16(m / -8), m the value of largest magnitude, and nibbles
// clamp(floor(x / d + 8.5), 0, 15).
//
// Heads of 64, 96, 128 and 256 channels whose rows allow 8-byte accesses take
// heads_kernel: a lane has 8 channels of a head, both members of each pair
// among them, so only the norm's sum and a group's extremes cross lanes.  All
// else takes rows_kernel, a warp a head, which is right for every size,
// stride and alignment.
//
// What bounds them: instructions, not the rows' bytes.  8191 tokens of 64 heads
// of 96 in bf16 are 201 MB, 30 us at the memory's rate; the kernel takes 47
// (4.3 TB/s) with the issue slots 70% busy at 38 million warp instructions,
// conversions, products and sums being about half of them.  The append of 8192
// tokens of 48 heads of 128 takes 55 us (100 MB of rows in, 67 out and 9 of
// cache: 26 at the memory's rate; issue slots 78% busy), its read-back 13 (6;
// 78%).
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_kv4.cuh"

namespace qk {
namespace {

constexpr int kRowWarps = 8;

// Page and token of a slot; 32-bit division where the cache is small enough.
struct Slot {
    int64_t page;
    int token;
};
__device__ __forceinline__ Slot slot_of(int64_t slot, int page_tokens, int64_t n_slots)
{
    if (n_slots <= INT32_MAX) {
        const uint32_t p = static_cast<uint32_t>(slot) / static_cast<uint32_t>(page_tokens);
        return {static_cast<int64_t>(p), static_cast<int>(static_cast<uint32_t>(slot) - p * page_tokens)};
    }
    const int64_t p = slot / page_tokens;
    return {p, static_cast<int>(slot - p * page_tokens)};
}

struct RowsArgs {
    // heads [0, n_q) from q with q_weight, the next n_k from k with k_weight, the last n_v from v (append only)
    const void *q, *k, *v;
    void *q_out, *k_out;       // k_out: null in the append
    int64_t ldq, ldk, ldv, ldqo, ldko;
    int in_type, out_type;
    int n_q, n_k, n_v, D;
    const float *q_weight, *k_weight;
    float eps;
    const float2 *table;
    int64_t n_pos;
    int rot, interleaved;
    const int32_t *positions;
    int64_t T;
    bool vec_in, vec_out;      // four elements at a time: rows and bases allow it
    // append
    uint8_t *pages;
    int64_t n_slots;
    int page_tokens;
    const int64_t *slots;
    int *err;
};

__device__ __forceinline__ void load4(const void *p, int64_t i, int type, float (&x)[4])
{
    if (type == QK_F32) {
        const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
        return;
    }
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    if (type == QK_F16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    } else {
        x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void store4(void *p, int64_t i, int type, const float (&x)[4])
{
    if (type == QK_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
        return;
    }
    uint2 w;
    if (type == QK_F16) {
        const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
        w.x = *reinterpret_cast<const uint32_t *>(&a), w.y = *reinterpret_cast<const uint32_t *>(&b);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        w.x = *reinterpret_cast<const uint32_t *>(&a), w.y = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = w;
}

// The row's norm and rotation in place.  Each product and sum is rounded on
// its own (no contraction), so a 4-bit group's nibbles do not depend on how
// the compiler fuses them.
template <int NV>
__device__ __forceinline__ void norm_rotate(float (&x)[NV][4], const RowsArgs &a, const float *weight, bool bad,
                                            const float2 *cs, float *row, int lane)
{
    const int D = a.D;
    if (weight) {
        // the squares in the order of sum_in_order
#pragma unroll
        for (int i = 0; i < NV; ++i)
            *reinterpret_cast<float4 *>(row + (i * 32 + lane) * 4) =
                make_float4(__fmul_rn(x[i][0], x[i][0]), __fmul_rn(x[i][1], x[i][1]), __fmul_rn(x[i][2], x[i][2]),
                            __fmul_rn(x[i][3], x[i][3]));
        __syncwarp();
        float s = 0.0f;
        if (D == 256) {
            for (int e = 0; e < 4; ++e) s = __fadd_rn(s, __fadd_rn(row[4 * lane + e], row[128 + 4 * lane + e]));
        } else {
            for (int ch = lane; ch < D; ch += 32) s = __fadd_rn(s, row[ch]);
        }
        __syncwarp();
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
        const float r = rsqrtf(__fadd_rn(__fmul_rn(s, 1.0f / D), a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ch = (i * 32 + lane) * 4 + e;
                if (ch < D) x[i][e] = __fmul_rn(__fmul_rn(x[i][e], r), weight[ch]);
            }
    }
    if (a.rot > 0 && !bad) {
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int ch = (i * 32 + lane) * 4 + e;
                    if (ch < a.rot) {
                        const float2 t = cs[ch >> 1];
                        const float u = x[i][e], w = x[i][e + 1];
                        x[i][e] = __fsub_rn(__fmul_rn(u, t.x), __fmul_rn(w, t.y));
                        x[i][e + 1] = __fadd_rn(__fmul_rn(u, t.y), __fmul_rn(w, t.x));
                    }
                }
        } else {
            const int half = a.rot >> 1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int ch = (i * 32 + lane) * 4;
                if (ch < a.rot) *reinterpret_cast<float4 *>(row + ch) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int ch = (i * 32 + lane) * 4 + e;
                    if (ch < half) {
                        const float2 t = cs[ch];
                        x[i][e] = __fsub_rn(__fmul_rn(x[i][e], t.x), __fmul_rn(row[ch + half], t.y));
                    } else if (ch < a.rot) {
                        const float2 t = cs[ch - half];
                        x[i][e] = __fadd_rn(__fmul_rn(row[ch - half], t.y), __fmul_rn(x[i][e], t.x));
                    }
                }
            __syncwarp();
        }
    }
    if (bad)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = __int_as_float(0x7FC00000);
}

// Four channels of a head to the cache: the group's scale over its 8 lanes,
// then the lane's four nibbles (the same as nibbles_of's) as two bytes.
__device__ __forceinline__ void store_nibbles(uint8_t *block, int D, int t, int ch, bool active, const float (&x)[4],
                                              bool is_key, int lane)
{
    float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
    bool odd = false;   // a NaN or an infinity
#pragma unroll
    for (int e = 0; e < 4; ++e) odd |= !(fabsf(x[e]) <= FLT_MAX);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    }
    const uint32_t odd_lanes = __ballot_sync(0xFFFFFFFFu, odd);
    if (!active) return;
    const bool group_odd = (odd_lanes >> (lane & 24)) & 0xFFu;
    const float m = hi >= -lo ? hi : lo;
    const float want = fminf(fmaxf(m * -0.125f, -65504.0f), 65504.0f);
    const __half dh = group_odd ? __ushort_as_half(0x7FFF) : __float2half_rn(want);
    const float d = __half2float(dh);
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float n = 8.0f;
        if (d != 0.0f && !group_odd)
            n = fminf(fmaxf(floorf(__fadd_rn(__fdiv_rn(x[e], d), 8.5f)), 0.0f), 15.0f);
        bits |= static_cast<uint32_t>(n) << (4 * e);
    }
    const Kv4Place p = is_key ? kv4_key_place(D, t, ch) : kv4_value_place(D, t, ch);
    *reinterpret_cast<uint16_t *>(block + p.byte + (p.nibble >> 1)) = static_cast<uint16_t>(bits);
    if ((lane & 7) == 0) {
        const int s = is_key ? kv4_key_scale(D, t, ch >> 5) : kv4_value_scale(D, t, ch >> 5);
        *reinterpret_cast<__half *>(block + s) = dh;
    }
}

template <int NV, bool APPEND>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const RowsArgs a)
{
    __shared__ __align__(16) float rows[kRowWarps][NV * 128];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = a.n_q + a.n_k + a.n_v;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (item >= a.T * heads) return;
    const int64_t t = item / heads;
    const int h = static_cast<int>(item - t * heads);
    const bool is_q = h < a.n_q, is_v = h >= a.n_q + a.n_k;
    const int hk = is_q ? h : (is_v ? h - a.n_q - a.n_k : h - a.n_q);
    const void *src = is_q ? a.q : (is_v ? a.v : a.k);
    const int64_t at = t * (is_q ? a.ldq : (is_v ? a.ldv : a.ldk)) + static_cast<int64_t>(hk) * a.D;

    bool bad = false;
    const float2 *cs = a.table;
    if (a.rot > 0 && !is_v) {
        const int32_t p = a.positions[t];
        bad = p < 0 || p >= a.n_pos;
        cs += bad ? 0 : static_cast<int64_t>(p) * (a.rot >> 1);
        if (bad && lane == 0) record_error(a.err, kErrBadIndex);
    }
    float x[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int ch = (i * 32 + lane) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = 0.0f;
        if (a.vec_in) {
            if (ch < a.D) load4(src, at + ch, a.in_type, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ch + e < a.D) x[i][e] = load_as_float(src, at + ch + e, a.in_type);
        }
    }
    if (!is_v) norm_rotate<NV>(x, a, is_q ? a.q_weight : a.k_weight, bad, cs, rows[warp], lane);
    if (APPEND && !is_q) {
        const int64_t slot = a.slots[t];
        if (slot < 0) return;
        if (slot >= a.n_slots) {
            if (lane == 0) record_error(a.err, kErrBadIndex);
            return;
        }
        const int64_t page = slot / a.page_tokens;
        const int off = static_cast<int>(slot - page * a.page_tokens);
        uint8_t *block = a.pages + ((page * a.n_k + hk) * (a.page_tokens / kBlockTokens) + off / kBlockTokens) *
                                       static_cast<int64_t>(18 * a.D);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int ch = (i * 32 + lane) * 4;
            store_nibbles(block, a.D, off % kBlockTokens, ch, ch < a.D, x[i], !is_v, lane);
        }
        return;
    }
    void *dst = is_q ? a.q_out : a.k_out;
    const int64_t to = t * (is_q ? a.ldqo : a.ldko) + static_cast<int64_t>(hk) * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int ch = (i * 32 + lane) * 4;
        if (a.vec_out) {
            if (ch < a.D) store4(dst, to + ch, a.out_type, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ch + e < a.D) store_float_as(dst, to + ch + e, a.out_type, x[i][e]);
        }
    }
}

// ---------------------------------------------------------------- heads of 64, 96, 128 or 256 channels

// Eight channels a lane, two chunks of four.  Interleaved pairs (and values,
// which do not rotate) take eight neighbours; the half layout takes
// 4i..4i+3 and their partners half + 4i.., so a pair is always in one lane and
// nothing is exchanged.  The lanes of a token's heads share its table row and
// keep it in registers over up to heads_per_lane heads; more would share
// more but need registers of the blocks that hide the loads: 8191 tokens of 64
// heads of 96 in 48 us with 4 heads and 4 blocks an SM, 65 with 3 (two blocks
// a token), 52 with 6; the append of 4 x 2048 tokens, 48 heads of 128, 53 us
// with 2 heads and 5 blocks, 57 with 4 and 4, 56 with 3 and 4.
__host__ __device__ constexpr int heads_per_lane(bool append) { return append ? 2 : 4; }
__host__ __device__ constexpr int heads_blocks(bool append) { return append ? 5 : 4; }

template <int D>
constexpr int kRowsPerWarp = D == 96 ? 2 : 256 / D;

// Nibbles floor(x / d + 8.5) of eight values, d != 0, in fp32: the quotient rounded, then the sum, as a plain run of
// the formula has them.  The product with 1/d is within 2^-17 of the quotient; lowered by twice that it gives the floor
// or one less, n, and x - (n - 7.5) d, which fp32 holds to its last bit, how far x lies from the next edge.  That over
// d, added to n - 7.5, is the quotient: correctly rounded near the edge, where it decides, and near enough elsewhere.
__device__ __forceinline__ uint32_t nibbles_of(const float (&x)[8], float d)
{
    // 1/d of a subnormal fp16 is at most 2^24; the quotient is within +-16
    const float step = fabsf(d), inv = __fdividef(1.0f, step);
    const uint32_t sign = __float_as_uint(d) & 0x80000000u;
    const uint64_t inv2 = pack2f(inv, inv), down2 = pack2f(-step, -step);
    float2 w;      // four nibbles each, exact in fp32
#pragma unroll
    for (int e = 3; e >= 0; --e) {
        const uint64_t v = pack2(__float_as_uint(x[e]) ^ sign, __float_as_uint(x[e + 4]) ^ sign);
        const uint64_t low = fma_f32x2(v, inv2, pack2f(8.5f - 1.6e-5f, 8.5f - 1.6e-5f));
        const uint64_t n2 = add_f32x2(add_down_f32x2(low, pack2f(kTwo23, kTwo23)), pack2f(-kTwo23, -kTwo23));
        const uint64_t edge = add_f32x2(n2, pack2f(-7.5f, -7.5f));
        const uint64_t sum = add_f32x2(fma_f32x2(fma_f32x2(edge, down2, v), inv2, edge), pack2f(8.5f, 8.5f));
        float2 n = unpack2f(add_f32x2(add_down_f32x2(sum, pack2f(kTwo23, kTwo23)), pack2f(-kTwo23, -kTwo23)));
        n.x = fminf(fmaxf(n.x, 0.0f), 15.0f), n.y = fminf(fmaxf(n.y, 0.0f), 15.0f);
        w = e == 3 ? n : unpack2f(fma_f32x2(pack2f(w.x, w.y), pack2f(16.0f, 16.0f), pack2f(n.x, n.y)));
    }
    return static_cast<uint32_t>(w.x) | static_cast<uint32_t>(w.y) << 16;
}

// Eight neighbouring channels of a head to the cache: the group's scale over
// 4 lanes, one word of key nibbles or two halves of value words.
template <int D>
__device__ __forceinline__ void store_eight(uint8_t *block, int t, int ch, bool active, const float (&x)[8], bool is_key,
                                            int lane)
{
    float hi = x[0], lo = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) hi = fmaxf(hi, x[e]), lo = fminf(lo, x[e]);
    // a NaN or an infinity: 0 * x is NaN for these alone
    uint64_t zero = 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) zero = fma_f32x2(pack2f(x[e], x[e + 1]), 0, zero);
    const float2 z = unpack2f(zero);
    const bool odd = !(z.x + z.y == 0.0f);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    }
    const uint32_t odd_lanes = __ballot_sync(0xFFFFFFFFu, odd);
    if (!active) return;
    const bool group_odd = (odd_lanes >> (lane & 28)) & 15u;
    const float m = hi >= -lo ? hi : lo;
    const float want = fminf(fmaxf(m * -0.125f, -65504.0f), 65504.0f);
    const __half dh = group_odd ? __ushort_as_half(0x7FFF) : __float2half_rn(want);
    const float d = __half2float(dh);
    const uint32_t bits = d != 0.0f && !group_odd ? nibbles_of(x, d) : 0x88888888u;
    if (is_key) {
        *reinterpret_cast<uint32_t *>(block + kv4_key_place(D, t, ch).byte) = bits;
    } else {
        // the next four channels are one r further
        uint8_t *to = block + kv4_value_place(D, t, ch).byte + 2 * (t & 1);
        *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(bits);
        *reinterpret_cast<uint16_t *>(to + 16 * kv4_gp(D / 32)) = static_cast<uint16_t>(bits >> 16);
    }
    if ((lane & 3) == 0) {
        const int s = is_key ? kv4_key_scale(D, t, ch >> 5) : kv4_value_scale(D, t, ch >> 5);
        *reinterpret_cast<__half *>(block + s) = dh;
    }
}

// The sum of a head's squares in the order that a stored key's norm has wherever its row lies: channels 32 apart one
// after another, then neighbouring sums in pairs; of 256 channels, those 128 apart, then four neighbours one after
// another, then in pairs.  (PyTorch's mean of a row was found to add in this order, so keys are stored as a plain run
// of the formula there stores them.  In another order a norm's last bit moved 7 of 8 million nibbles by a step.)
// row: D floats of shared memory of this head; a lane's channels are ca..ca+3 and cb..cb+3.
template <int D>
__device__ __forceinline__ float sum_in_order(const float (&x)[8], float *row, int ca, int cb, int i, int sub, bool on)
{
    if (on) {
        *reinterpret_cast<float4 *>(row + ca) =
            make_float4(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1]), __fmul_rn(x[2], x[2]), __fmul_rn(x[3], x[3]));
        *reinterpret_cast<float4 *>(row + cb) =
            make_float4(__fmul_rn(x[4], x[4]), __fmul_rn(x[5], x[5]), __fmul_rn(x[6], x[6]), __fmul_rn(x[7], x[7]));
    }
    __syncwarp();
    float s = 0.0f;
    if constexpr (D == 128) {
        float2 t = *reinterpret_cast<const float2 *>(row + 2 * i);
#pragma unroll
        for (int c = 1; c < 4; ++c) {
            const float2 u = *reinterpret_cast<const float2 *>(row + 32 * c + 2 * i);
            t.x = __fadd_rn(t.x, u.x), t.y = __fadd_rn(t.y, u.y);
        }
        s = __fadd_rn(t.x, t.y);
    } else if (D != 96 || (on && i < 8)) {
        constexpr int step = D == 256 ? 128 : 32;
        float4 t = *reinterpret_cast<const float4 *>(row + 4 * i);
#pragma unroll
        for (int c = step; c < D; c += step) {
            const float4 u = *reinterpret_cast<const float4 *>(row + c + 4 * i);
            t.x = __fadd_rn(t.x, u.x), t.y = __fadd_rn(t.y, u.y), t.z = __fadd_rn(t.z, u.z), t.w = __fadd_rn(t.w, u.w);
        }
        s = D == 256 ? __fadd_rn(__fadd_rn(__fadd_rn(t.x, t.y), t.z), t.w) : __fadd_rn(__fadd_rn(t.x, t.y), __fadd_rn(t.z, t.w));
    }
    __syncwarp();
    if constexpr (D == 96) {      // 12 lanes a row, the sums in the first eight
        const int first = sub * 12;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s = __fadd_rn(s, __shfl_sync(0xFFFFFFFFu, s, (first + (i ^ o)) & 31));
        return __shfl_sync(0xFFFFFFFFu, s, first);
    }
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    return s;
}

// Norm and rotation of a lane's eight channels.  Pair e is neighbours 2e,
// 2e + 1 of the eight, or element e of both chunks.  With `sum` the head's
// sum of squares is there already.
template <int D, bool INTER>
__device__ __forceinline__ void turn_eight(float (&x)[8], bool norm, bool weigh, const float (&w)[8], float eps,
                                           bool turn, const float (&c)[4], const float (&s)[4], int sub,
                                           const float *sum = nullptr)
{
    constexpr int LPR = D / 8;
    if (norm) {       // warp-uniform: some row of the call has a weight
        float q;
        if (sum) {
            q = *sum;
        } else {
            uint64_t squares = 0;      // two zeros
#pragma unroll
            for (int e = 0; e < 8; e += 2) squares = fma_f32x2(pack2f(x[e], x[e + 1]), pack2f(x[e], x[e + 1]), squares);
            const float2 two = unpack2f(squares);
            q = two.x + two.y;
            if constexpr (D == 96) {      // 12 lanes a row: groups of four stay inside it
                q += __shfl_xor_sync(0xFFFFFFFFu, q, 1);
                q += __shfl_xor_sync(0xFFFFFFFFu, q, 2);
                const int first = sub * LPR;
                q = __shfl_sync(0xFFFFFFFFu, q, first) + __shfl_sync(0xFFFFFFFFu, q, first + 4) +
                    __shfl_sync(0xFFFFFFFFu, q, (first + 8) & 31);
            } else {
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
            }
        }
        const float r = weigh ? rsqrtf(__fadd_rn(__fmul_rn(q, 1.0f / D), eps)) : 1.0f;   // without: the weights are 1
        const uint64_t r2 = pack2f(r, r);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 y = unpack2f(mul_f32x2(mul_f32x2(pack2f(x[e], x[e + 1]), r2), pack2f(w[e], w[e + 1])));
            x[e] = y.x, x[e + 1] = y.y;
        }
    }
    // each product and sum is rounded by itself, so the stored nibbles do not depend on how a compiler fuses them (which
    // it does where the sums too are in pairs)
    if (turn)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            constexpr int step = INTER ? 2 : 1, other = INTER ? 1 : 4;
            float2 uc, vs, us, vc;
            if constexpr (INTER) {
                uc = make_float2(__fmul_rn(x[2 * e], c[e]), __fmul_rn(x[2 * e + 2], c[e + 1]));
                vs = make_float2(__fmul_rn(x[2 * e + 1], s[e]), __fmul_rn(x[2 * e + 3], s[e + 1]));
                us = make_float2(__fmul_rn(x[2 * e], s[e]), __fmul_rn(x[2 * e + 2], s[e + 1]));
                vc = make_float2(__fmul_rn(x[2 * e + 1], c[e]), __fmul_rn(x[2 * e + 3], c[e + 1]));
            } else {
                const uint64_t u = pack2f(x[e], x[e + 1]), v = pack2f(x[e + 4], x[e + 5]);
                const uint64_t c2 = pack2f(c[e], c[e + 1]), s2 = pack2f(s[e], s[e + 1]);
                uc = unpack2f(mul_f32x2(u, c2)), vs = unpack2f(mul_f32x2(v, s2));
                us = unpack2f(mul_f32x2(u, s2)), vc = unpack2f(mul_f32x2(v, c2));
            }
            x[step * e] = __fsub_rn(uc.x, vs.x), x[step * (e + 1)] = __fsub_rn(uc.y, vs.y);
            x[step * e + other] = __fadd_rn(us.x, vc.x), x[step * (e + 1) + other] = __fadd_rn(us.y, vc.y);
        }
}

__device__ __forceinline__ void load_weights(float (&w)[8], const float *weight, int ca, int cb)
{
    float4 u = make_float4(1.0f, 1.0f, 1.0f, 1.0f), v = u;
    if (weight) u = *reinterpret_cast<const float4 *>(weight + ca), v = *reinterpret_cast<const float4 *>(weight + cb);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
}

// Four elements as they lie in memory, and as floats.
template <int TYPE>
struct Raw {
    using Word = typename std::conditional<TYPE == QK_F32, uint4, uint2>::type;
    static constexpr int size = TYPE == QK_F32 ? 4 : 2;
    Word w;
    __device__ __forceinline__ void load(const uint8_t *p) { w = *reinterpret_cast<const Word *>(p); }
    __device__ __forceinline__ void poison()      // a NaN in every type
    {
        if constexpr (TYPE == QK_F32) w = make_uint4(0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu);
        else w = make_uint2(0x7FFF7FFFu, 0x7FFF7FFFu);
    }
    __device__ __forceinline__ void to(float *x) const
    {
        if constexpr (TYPE == QK_F32) {
            x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y);
            x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
        } else if constexpr (TYPE == QK_F16) {
            const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
            x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
        } else {
            x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
            x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
        }
    }
};

template <int D, int TYPE, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRowWarps * 32, heads_blocks(APPEND)) heads_kernel(const RowsArgs a, int hpl_front, int hpl_back, int q_parts)
{
    constexpr int kHeadsPerLane = heads_per_lane(APPEND);
    constexpr int LPR = D / 8, RPW = kRowsPerWarp<D>, NG = kRowWarps * RPW, size = Raw<TYPE>::size;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, i = lane - sub * LPR;            // row of the warp, lane of the row
    const bool on = sub < RPW;                                   // 96 channels leave 8 lanes idle
    const int part = static_cast<int>(blockIdx.y);
    const uint32_t t_first = blockIdx.x, t_step = gridDim.x;      // T is below 2^31: their sum stays in 32 bits
    const bool front = !APPEND || part < q_parts;                // rows that go out; else rows that are stored
    const int hpl = front ? hpl_front : hpl_back;                // heads a lane
    const int h0 = (front ? part : part - q_parts) * NG * hpl + warp * RPW + sub;
    const int heads = !APPEND ? a.n_q + a.n_k : (front ? a.n_q : 2 * a.n_k);
    const int mine = on && h0 < heads ? min(hpl, (heads - h0 + NG - 1) / NG) : 0;       // heads of this lane
    const int first_mine = front ? a.n_q : a.n_k;                                       // those before it are q, or keys
    const bool turn = on && 8 * i < a.rot;
    const int ca = INTER || !turn ? 8 * i : 4 * i, cb = INTER || !turn ? 8 * i + 4 : (a.rot >> 1) + 4 * i;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const bool norm = a.q_weight || a.k_weight;
    const float *first_weight = h0 < first_mine ? (front ? a.q_weight : a.k_weight) : (front ? a.k_weight : nullptr);
    // a lane's heads may run from queries into keys, or from keys into values: its weights change on the way
    const bool changes = mine > 0 && h0 < first_mine && h0 + (mine - 1) * NG >= first_mine;
    float w[8];
    load_weights(w, mine ? first_weight : nullptr, ca, cb);
    for (uint32_t t = t_first; t < a.T; t += t_step) {
        // rows and position first, together: nothing waits before all of it is on its way
        int32_t pos = a.rot > 0 ? a.positions[t] : 0;
        Raw<TYPE> xa[kHeadsPerLane], xb[kHeadsPerLane];
        {
            const uint8_t *pa = static_cast<const uint8_t *>(front ? a.q : a.k) +
                                (static_cast<int64_t>(t) * (front ? a.ldq : a.ldk) + h0 * D) * size;
            const uint8_t *pv = APPEND && !front ? static_cast<const uint8_t *>(a.v) +
                                                       (static_cast<int64_t>(t) * a.ldv + (h0 - a.n_k) * D + 8 * i) * size
                                                 : nullptr;
#pragma unroll
            for (int k = 0; k < kHeadsPerLane; ++k) {
                xa[k].w = {}, xb[k].w = {};
                if (k < mine) {
                    if (!APPEND || front || h0 + k * NG < a.n_k) {
                        xa[k].load(pa + ca * size + k * (NG * D * size));
                        xb[k].load(pa + cb * size + k * (NG * D * size));
                    } else {
                        xa[k].load(pv + k * (NG * D * size));
                        xb[k].load(pv + 4 * size + k * (NG * D * size));
                    }
                }
            }
        }
        const bool bad = a.rot > 0 && (pos < 0 || pos >= a.n_pos);
        float c[4] = {}, s[4] = {};
        if (turn) {
            const float4 *row = reinterpret_cast<const float4 *>(a.table + static_cast<int64_t>(bad ? 0 : pos) * (a.rot >> 1) +
                                                                 4 * i);
            const float4 u = row[0], v = row[1];
            c[0] = u.x, s[0] = u.y, c[1] = u.z, s[1] = u.w, c[2] = v.x, s[2] = v.y, c[3] = v.z, s[3] = v.w;
        }
        const float *weight = first_weight;
        if (changes && t != t_first) load_weights(w, weight, ca, cb);
        if (bad) {
            if (threadIdx.x == 0) record_error(a.err, kErrBadIndex);
#pragma unroll
            for (int k = 0; k < kHeadsPerLane; ++k)
                if (front || h0 + k * NG < a.n_k) xa[k].poison(), xb[k].poison();
        }
        if (front) {
            uint8_t *to = static_cast<uint8_t *>(a.q_out) +
                          (static_cast<int64_t>(t) * a.ldqo + h0 * D) * (a.out_type == QK_F32 ? 4 : 2);
#pragma unroll
            for (int k = 0; k < kHeadsPerLane; ++k) {
                if (k >= hpl) break;
                float x[8];
                xa[k].to(x), xb[k].to(x + 4);
                if (!APPEND && k > 0 && h0 + k * NG >= first_mine && h0 + (k - 1) * NG < first_mine) {
                    weight = a.k_weight;      // from here the lane's heads are keys
                    load_weights(w, k < mine ? weight : nullptr, ca, cb);
                }
                turn_eight<D, INTER>(x, norm, weight && k < mine, w, a.eps, turn, c, s, sub);
                if (k < mine) {
                    const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
                    if (a.out_type == TYPE) {
                        store4(to + (ca + k * (NG * D)) * size, 0, TYPE, lo);
                        store4(to + (cb + k * (NG * D)) * size, 0, TYPE, hi);
                    } else {
                        store4(to, ca + k * (NG * D), a.out_type, lo);
                        store4(to, cb + k * (NG * D), a.out_type, hi);
                    }
                }
            }
            if constexpr (APPEND) continue;
            else return;
        }
        if constexpr (APPEND) {
            __shared__ __align__(16) float exchange[kRowWarps * RPW][D];
            float *row = exchange[warp * RPW + (on ? sub : 0)];
            const int64_t slot = a.slots[t];
            if (slot < 0) continue;
            if (slot >= a.n_slots) {
                if (threadIdx.x == 0) record_error(a.err, kErrBadIndex);
                continue;
            }
            const Slot at = slot_of(slot, a.page_tokens, a.n_slots);
            const int64_t page = at.page;
            const int off = at.token, tk = off % kBlockTokens;
            const int head_bytes = a.page_tokens / kBlockTokens * (18 * D);
            uint8_t *first = a.pages + page * a.n_k * static_cast<int64_t>(head_bytes) + off / kBlockTokens * (18 * D);
#pragma unroll
            for (int k = 0; k < kHeadsPerLane; ++k) {
                if (k >= hpl) break;
                const int h = h0 + k * NG;
                const bool is_key = h < a.n_k;
                float x[8];
                xa[k].to(x), xb[k].to(x + 4);
                if (changes && !is_key) load_weights(w, nullptr, ca, cb);
                const bool normed = a.k_weight && __any_sync(0xFFFFFFFFu, is_key);      // some row of the warp's
                float sum = 0.0f;
                if (normed) sum = sum_in_order<D>(x, row, ca, cb, i, sub, on);
                turn_eight<D, INTER>(x, normed, weight && k < mine && is_key, w, a.eps, turn && is_key, c, s, sub, &sum);
                if constexpr (!INTER) {      // eight neighbours a lane, as the cache wants them
                    if (on && is_key) {
                        *reinterpret_cast<float4 *>(row + ca) = make_float4(x[0], x[1], x[2], x[3]);
                        *reinterpret_cast<float4 *>(row + cb) = make_float4(x[4], x[5], x[6], x[7]);
                    }
                    __syncwarp();
                    if (on && is_key) {
                        const float4 u = *reinterpret_cast<const float4 *>(row + 8 * i);
                        const float4 v = *reinterpret_cast<const float4 *>(row + 8 * i + 4);
                        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
                    }
                    __syncwarp();
                }
                store_eight<D>(first + static_cast<int64_t>(is_key ? h : h - a.n_k) * head_bytes, tk, 8 * i, k < mine, x,
                               is_key, lane);
            }
        }
    }
}

struct ReadArgs {
    const uint8_t *pages;
    int64_t n_slots;
    int n_kv, D, page_tokens;
    const int64_t *slots;
    int64_t T;
    void *k, *v;
    int64_t ldk, ldv;
    int type;
    bool vec;
    int tokens;              // of a thread block
    int *err;
};

// Eight stored values from their nibbles (in order from the low end) and scale.  A nibble under the bits of 2^23 is
// 2^23 + n 16^e, and one multiply-add gives n - 8 of it exactly.
__device__ __forceinline__ void values_of(uint32_t n, float d, float (&lo)[4], float (&hi)[4])
{
    const uint32_t m = n >> 16;
    lo[0] = __uint_as_float(magic_field<0x000Fu>(n)), hi[0] = __uint_as_float(magic_field<0x000Fu>(m));
    lo[1] = __uint_as_float(magic_field<0x00F0u>(n)), hi[1] = __uint_as_float(magic_field<0x00F0u>(m));
    lo[2] = __uint_as_float(magic_field<0x0F00u>(n)), hi[2] = __uint_as_float(magic_field<0x0F00u>(m));
    lo[3] = __uint_as_float(magic_field<0xF000u>(n)), hi[3] = __uint_as_float(magic_field<0xF000u>(m));
    float down = 1.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e, down *= 0.0625f) {
        const float less = -(kTwo23 * down + 8.0f);
        lo[e] = d * fmaf(lo[e], down, less), hi[e] = d * fmaf(hi[e], down, less);
    }
}

// A lane reads eight channels of a slot's key head and value head.  A thread block takes whole tokens, or (blockIdx.y)
// a part of one.
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) read_kernel(const ReadArgs a)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int lpr = D / 8;
    const int items = a.n_kv * lpr;      // of a token
    int own = 0, item = static_cast<int>(blockIdx.y * (kRowWarps * 32) + threadIdx.x);
    if (a.tokens > 1) own = item / items, item -= own * items;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.tokens + own;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.T || item >= items || own >= a.tokens) return;
    const int h = item / lpr, ch = (item - h * lpr) * 8;
    const int64_t slot = a.slots[t];
    uint32_t nibbles[2] = {0x88888888u, 0x88888888u};
    float scale[2];
    if (slot >= 0 && slot < a.n_slots) {
        const Slot at = slot_of(slot, a.page_tokens, a.n_slots);
        const int tk = at.token % kBlockTokens;
        const uint8_t *block = a.pages + ((at.page * a.n_kv + h) * (a.page_tokens / kBlockTokens) + at.token / kBlockTokens) *
                                             static_cast<int64_t>(18 * D);
        if (a.k) nibbles[0] = *reinterpret_cast<const uint32_t *>(block + kv4_key_place(D, tk, ch).byte);
        if (a.v) {
            const uint8_t *from = block + kv4_value_place(D, tk, ch).byte + 2 * (tk & 1);      // the next four channels are one r further
            nibbles[1] = *reinterpret_cast<const uint16_t *>(from) |
                         static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(from + 16 * kv4_gp(D / 32))) << 16;
        }
        scale[0] = __half2float(*reinterpret_cast<const __half *>(block + kv4_key_scale(D, tk, ch >> 5)));
        scale[1] = __half2float(*reinterpret_cast<const __half *>(block + kv4_value_scale(D, tk, ch >> 5)));
    } else {
        if (slot >= 0) record_error(a.err, kErrBadIndex);
        scale[0] = scale[1] = slot < 0 ? 0.0f : __int_as_float(0x7FC00000);
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        void *dst = kind ? a.v : a.k;
        if (!dst) continue;
        const int64_t to = t * (kind ? a.ldv : a.ldk) + static_cast<int64_t>(h) * D + ch;
        float lo[4], hi[4];
        values_of(nibbles[kind], scale[kind], lo, hi);
        if (a.vec) {
            store4(dst, to, a.type, lo);
            store4(dst, to + 4, a.type, hi);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) store_float_as(dst, to + e, a.type, lo[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) store_float_as(dst, to + 4 + e, a.type, hi[e]);
        }
    }
}

struct TableArgs {
    float2 *table;
    int64_t n_pos;
    int half;
    double base, freq_scale, lo, hi, amplitude;
    bool ramp;
    const float *factors;
};

// Angles p * f_i in 64 bits, reduced to [-pi, pi]; sine and cosine of the
// fp32 part by CUDA's sincosf, the rest of the angle by the first-order term.
__global__ void __launch_bounds__(256) table_kernel(const TableArgs a)
{
    extern __shared__ double freq[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < a.half; i += blockDim.x) {
        double e = pow(a.base, -static_cast<double>(i) / a.half);
        if (a.factors) e /= static_cast<double>(a.factors[i]);
        double s = a.freq_scale;
        if (a.ramp) {
            const double m = 1.0 - fmin(fmax((i - a.lo) / fmax(a.hi - a.lo, 0.001), 0.0), 1.0);
            s = s * (1.0 - m) + m;
        }
        freq[i] = e * s;
    }
    __syncthreads();
    const int64_t n = a.n_pos * a.half;
    const double two_pi = 6.283185307179586476925;
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; j < n;
         j += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t p = j / a.half;
        const double angle = static_cast<double>(p) * freq[j - p * a.half];
        const double r = angle - rint(angle * (1.0 / two_pi)) * two_pi;
        const float rh = static_cast<float>(r), rl = static_cast<float>(r - rh);
        float s, c;
        sincosf(rh, &s, &c);
        const float amp = static_cast<float>(a.amplitude);
        a.table[j] = make_float2(amp * fmaf(-rl, s, c), amp * fmaf(rl, c, s));
    }
}

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Four elements at a time are possible: heads, rows and base on 4-element boundaries.
bool vec_ok(const void *p, int64_t ld, int D, int type)
{
    return D % 4 == 0 && ld % 4 == 0 && multiple(p, type == QK_F32 ? 16 : 8);
}

int64_t blocks_for(int64_t items) { return (items + kRowWarps - 1) / kRowWarps; }

template <class Args>
cudaError_t launch(void (*kern)(const Args), dim3 grid, int threads, size_t smem, cudaStream_t st, const Args &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = library_programmatic() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int TYPE, bool INTER, bool APPEND>
cudaError_t launch_heads(const RowsArgs &a, cudaStream_t st)
{
    constexpr int kHeadsPerLane = heads_per_lane(APPEND);
    constexpr int NG = kRowWarps * kRowsPerWarp<D>;
    int sms = 152, smem = 0;
    device_limits(&sms, &smem);
    const int front = APPEND ? a.n_q : a.n_q + a.n_k, back = APPEND ? 2 * a.n_k : 0;
    // several heads a lane share a table row and keep as many loads going; below two blocks an SM the heads spread over
    // more blocks instead (40 heads of 128: one token 2.7 us with four heads a lane, 2.1 with one, 64 tokens 2.5 and
    // 2.4, 256 tokens 3.1 and 3.7)
    const auto cut = [](int heads, int most, int *per) {
        const int parts = (heads + NG * most - 1) / (NG * most);
        *per = parts ? (heads + NG * parts - 1) / (NG * parts) : 1;
        return parts;
    };
    int hf = 1, hb = 1, fp = cut(front, kHeadsPerLane, &hf), parts = fp + cut(back, kHeadsPerLane, &hb);
    if (a.T * parts < 2 * sms) fp = cut(front, 1, &hf), parts = fp + cut(back, 1, &hb);
    // appending many tokens, thread blocks go from token to token and work out only once what does not change (8192
    // tokens of 32 + 2 x 8 heads of 128: 52 us in six rounds of the blocks that the GPU holds, 53 in four, 62 with a
    // block a token; without the nibbles there is less to save than the waits cost, 57 us against 50 for
    // 8191 x 64 of 96)
    const int64_t most = APPEND ? (6 * heads_blocks(true) * sms + parts - 1) / parts : a.T, tokens = a.T < most ? a.T : most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tokens), static_cast<unsigned>(parts));
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = library_programmatic() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, heads_kernel<D, TYPE, INTER, APPEND>, a, hf, hb, fp);
}

template <int D, int TYPE, bool APPEND>
cudaError_t launch_heads_layout(const RowsArgs &a, cudaStream_t st)
{
    return a.interleaved ? launch_heads<D, TYPE, true, APPEND>(a, st) : launch_heads<D, TYPE, false, APPEND>(a, st);
}

template <int D, bool APPEND>
cudaError_t launch_heads_type(const RowsArgs &a, cudaStream_t st)
{
    if (a.in_type == QK_F32) return launch_heads_layout<D, QK_F32, APPEND>(a, st);
    if (a.in_type == QK_F16) return launch_heads_layout<D, QK_F16, APPEND>(a, st);
    return launch_heads_layout<D, QK_BF16, APPEND>(a, st);
}

template <bool APPEND>
cudaError_t launch_rows(const RowsArgs &a, cudaStream_t st)
{
    const bool wide = a.vec_in && (a.vec_out || (APPEND && !a.n_q)) && a.rot % 8 == 0 && multiple(a.table, 16) &&
                      multiple(a.q_weight, 16) && multiple(a.k_weight, 16);
    if (wide) {
        switch (a.D) {
        case 64: return launch_heads_type<64, APPEND>(a, st);
        case 96: return launch_heads_type<96, APPEND>(a, st);
        case 128: return launch_heads_type<128, APPEND>(a, st);
        case 256: return launch_heads_type<256, APPEND>(a, st);
        }
    }
    const dim3 grid(static_cast<unsigned>(blocks_for(a.T * (a.n_q + a.n_k + a.n_v))));
    if (a.D <= 128) return launch(rows_kernel<1, APPEND>, grid, kRowWarps * 32, 0, st, a);
    if (a.D <= 256) return launch(rows_kernel<2, APPEND>, grid, kRowWarps * 32, 0, st, a);
    if constexpr (!APPEND) return launch(rows_kernel<4, APPEND>, grid, kRowWarps * 32, 0, st, a);
    return cudaErrorInvalidValue;
}

bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }
int size_of(int t) { return t == QK_F32 ? 4 : 2; }

// Rotation arguments shared by the entry points.
int check_rotation(const float *table, int64_t n_pos, int rot, int D, const int32_t *positions)
{
    if (rot < 0 || rot % 2 || rot > D) return QK_ERR_BAD_DIM;
    if (rot > 0) {
        if (!table || !positions) return QK_ERR_NULL;
        if (n_pos <= 0) return QK_ERR_BAD_DIM;
        if (!multiple(table, 8) || !multiple(positions, 4)) return QK_ERR_ALIGN;
    }
    return QK_OK;
}

}  // namespace

int kv4_check_cache(const qk_kv_cache_q4 *c)
{
    if (!c || !c->pages) return QK_ERR_NULL;
    if (c->n_pages <= 0 || c->n_kv_heads <= 0 || c->page_tokens <= 0 || c->page_tokens % kBlockTokens ||
        c->page_tokens > 1024)
        return QK_ERR_BAD_DIM;
    if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256) return QK_ERR_BAD_DIM;
    if (c->n_kv_heads > 65535 || c->n_pages > INT32_MAX) return QK_ERR_TOO_LARGE;
    if (!multiple(c->pages, 16)) return QK_ERR_ALIGN;
    return QK_OK;
}

}  // namespace qk

using namespace qk;

extern "C" {

int qk_rope_table(float *table, int64_t n_pos, int rot, double base, double freq_scale, const float *freq_factors,
                  int64_t orig_ctx, double beta_fast, double beta_slow, double amplitude, qk_stream_t stream)
{
    if (!table) return QK_ERR_NULL;
    if (n_pos <= 0 || rot <= 0 || rot % 2 || !(base > 1.0) || !(freq_scale > 0.0) || orig_ctx < 0) return QK_ERR_BAD_DIM;
    if (orig_ctx > 0 && (!(beta_fast > 0.0) || !(beta_slow > 0.0))) return QK_ERR_BAD_DIM;
    if (rot > 4096 || n_pos > INT64_MAX / 65536) return QK_ERR_TOO_LARGE;
    if (!multiple(table, 8) || (freq_factors && !multiple(freq_factors, 4))) return QK_ERR_ALIGN;
    TableArgs a{};
    a.table = reinterpret_cast<float2 *>(table);
    a.n_pos = n_pos;
    a.half = rot / 2;
    a.base = base, a.freq_scale = freq_scale, a.amplitude = amplitude;
    a.factors = freq_factors;
    a.ramp = orig_ctx > 0;
    if (a.ramp) {
        const auto dim = [&](double turns) {
            return rot * std::log(static_cast<double>(orig_ctx) / (turns * 6.283185307179586476925)) /
                   (2.0 * std::log(base));
        };
        a.lo = std::fmax(0.0, std::floor(dim(beta_fast)));
        a.hi = std::fmin(rot - 1.0, std::ceil(dim(beta_slow)));
    }
    const int64_t want = (n_pos * a.half + 1023) / 1024;
    return launch(table_kernel, dim3(static_cast<unsigned>(want < 1216 ? want : 1216)), 256, sizeof(double) * a.half,
                  reinterpret_cast<cudaStream_t>(stream), a) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

int qk_norm_rope(const void *x, int64_t ldx, int x_type, int n_q_heads, int n_k_heads, int head_dim,
                 const float *q_weight, const float *k_weight, float eps, const float *table, int64_t n_pos, int rot,
                 int interleaved, const int32_t *positions, int64_t T, void *y, int64_t ldy, int y_type,
                 qk_stream_t stream)
{
    if (!type_ok(x_type) || !type_ok(y_type)) return QK_ERR_TYPE;
    if (n_q_heads < 0 || n_k_heads < 0 || n_q_heads + static_cast<int64_t>(n_k_heads) < 1 || head_dim < 2 ||
        head_dim > 512 || head_dim % 2 || T < 0)
        return QK_ERR_BAD_DIM;
    const int64_t heads = static_cast<int64_t>(n_q_heads) + n_k_heads;
    if (heads > 65535) return QK_ERR_TOO_LARGE;
    if (ldx == 0) ldx = heads * head_dim;
    if (ldy == 0) ldy = heads * head_dim;
    if (ldx < heads * head_dim || ldy < heads * head_dim) return QK_ERR_BAD_DIM;
    if (x == y && x && (x_type != y_type || ldx != ldy)) return QK_ERR_BAD_DIM;
    if (T == 0) return QK_OK;
    if (!x || !y) return QK_ERR_NULL;
    const int st = check_rotation(table, n_pos, rot, head_dim, positions);
    if (st != QK_OK) return st;
    if (!multiple(x, size_of(x_type)) || !multiple(y, size_of(y_type)) || !multiple(q_weight, 4) ||
        !multiple(k_weight, 4))
        return QK_ERR_ALIGN;
    if (T > INT32_MAX / blocks_for(heads)) return QK_ERR_TOO_LARGE;
    RowsArgs a{};
    a.q = x, a.q_out = y;
    a.k = static_cast<const char *>(x) + static_cast<int64_t>(n_q_heads) * head_dim * size_of(x_type);
    a.k_out = static_cast<char *>(y) + static_cast<int64_t>(n_q_heads) * head_dim * size_of(y_type);
    a.ldq = a.ldk = ldx, a.ldqo = a.ldko = ldy;
    a.in_type = x_type, a.out_type = y_type;
    a.n_q = n_q_heads, a.n_k = n_k_heads, a.D = head_dim;
    a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps;
    a.table = reinterpret_cast<const float2 *>(table), a.n_pos = n_pos, a.rot = rot, a.interleaved = interleaved;
    a.positions = positions, a.T = T;
    a.vec_in = vec_ok(x, ldx, head_dim, x_type), a.vec_out = vec_ok(y, ldy, head_dim, y_type);
    a.err = library_error_word();
    if (!a.err) return QK_ERR_CUDA;
    return launch_rows<false>(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

int qk_kv_append_q4(const qk_kv_cache_q4 *cache, const void *q, int64_t ldq, int n_q_heads, const void *k, int64_t ldk,
                    const void *v, int64_t ldv, int type, const float *q_weight, const float *k_weight, float eps,
                    const float *table, int64_t n_pos, int rot, int interleaved, const int32_t *positions,
                    const int64_t *slots, int64_t T, void *q_out, int64_t ldqo, int q_out_type, qk_stream_t stream)
{
    int st = kv4_check_cache(cache);
    if (st != QK_OK) return st;
    if (!type_ok(type) || (q && !type_ok(q_out_type))) return QK_ERR_TYPE;
    const int D = cache->head_dim, n_kv = cache->n_kv_heads;
    if (!q) n_q_heads = 0;
    if ((q && n_q_heads < 1) || T < 0) return QK_ERR_BAD_DIM;
    if (n_q_heads > 65535) return QK_ERR_TOO_LARGE;
    const int64_t wq = static_cast<int64_t>(n_q_heads) * D, wk = static_cast<int64_t>(n_kv) * D;
    if (ldq == 0) ldq = wq;
    if (ldqo == 0) ldqo = wq;
    if (ldk == 0) ldk = wk;
    if (ldv == 0) ldv = wk;
    if (ldq < wq || ldqo < wq || ldk < wk || ldv < wk) return QK_ERR_BAD_DIM;
    if (q && q == q_out && (type != q_out_type || ldq != ldqo)) return QK_ERR_BAD_DIM;
    if (T == 0) return QK_OK;
    if (!k || !v || !slots || (q && !q_out)) return QK_ERR_NULL;
    st = check_rotation(table, n_pos, rot, D, positions);
    if (st != QK_OK) return st;
    if (!multiple(k, size_of(type)) || !multiple(v, size_of(type)) || !multiple(slots, 8) || !multiple(q_weight, 4) ||
        !multiple(k_weight, 4) || (q && (!multiple(q, size_of(type)) || !multiple(q_out, size_of(q_out_type)))))
        return QK_ERR_ALIGN;
    const int64_t heads = static_cast<int64_t>(n_q_heads) + 2 * n_kv;
    if (T > INT32_MAX / blocks_for(heads)) return QK_ERR_TOO_LARGE;
    RowsArgs a{};
    a.q = q, a.k = k, a.v = v, a.q_out = q_out;
    a.ldq = ldq, a.ldk = ldk, a.ldv = ldv, a.ldqo = ldqo;
    a.in_type = type, a.out_type = q_out_type;
    a.n_q = n_q_heads, a.n_k = a.n_v = n_kv, a.D = D;
    a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps;
    a.table = reinterpret_cast<const float2 *>(table), a.n_pos = n_pos, a.rot = rot, a.interleaved = interleaved;
    a.positions = positions, a.T = T;
    a.vec_in = vec_ok(k, ldk, D, type) && vec_ok(v, ldv, D, type) && (!q || vec_ok(q, ldq, D, type));
    a.vec_out = q && vec_ok(q_out, ldqo, D, q_out_type);
    a.pages = static_cast<uint8_t *>(cache->pages);
    a.n_slots = cache->n_pages * cache->page_tokens;
    a.page_tokens = cache->page_tokens, a.slots = slots;
    a.err = library_error_word();
    if (!a.err) return QK_ERR_CUDA;
    return launch_rows<true>(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

int qk_kv_read_q4(const qk_kv_cache_q4 *cache, const int64_t *slots, int64_t T, void *k, int64_t ldk, void *v,
                  int64_t ldv, int type, qk_stream_t stream)
{
    const int st = kv4_check_cache(cache);
    if (st != QK_OK) return st;
    if (!type_ok(type)) return QK_ERR_TYPE;
    const int64_t w = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
    if (ldk == 0) ldk = w;
    if (ldv == 0) ldv = w;
    if (T < 0 || ldk < w || ldv < w) return QK_ERR_BAD_DIM;
    if (T == 0) return QK_OK;
    if (!slots || (!k && !v)) return QK_ERR_NULL;
    if (!multiple(slots, 8) || !multiple(k, size_of(type)) || !multiple(v, size_of(type))) return QK_ERR_ALIGN;
    if (T > INT32_MAX / blocks_for(2 * cache->n_kv_heads)) return QK_ERR_TOO_LARGE;
    ReadArgs a{};
    a.pages = static_cast<const uint8_t *>(cache->pages);
    a.n_slots = cache->n_pages * cache->page_tokens;
    a.n_kv = cache->n_kv_heads, a.D = cache->head_dim, a.page_tokens = cache->page_tokens;
    a.slots = slots, a.T = T, a.k = k, a.v = v, a.ldk = ldk, a.ldv = ldv, a.type = type;
    a.vec = (!k || vec_ok(k, ldk, a.D, type)) && (!v || vec_ok(v, ldv, a.D, type));
    a.err = library_error_word();
    if (!a.err) return QK_ERR_CUDA;
    constexpr int kThreads = kRowWarps * 32;
    const int items = a.n_kv * (a.D / 8), parts = (items + kThreads - 1) / kThreads;
    a.tokens = items < kThreads ? kThreads / items : 1;
    const dim3 grid(static_cast<unsigned>((T + a.tokens - 1) / a.tokens), static_cast<unsigned>(parts));
    const auto kern = a.D == 64 ? read_kernel<64> : a.D == 96 ? read_kernel<96> : a.D == 128 ? read_kernel<128> : read_kernel<256>;
    return launch(kern, grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream), a) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

}  // extern "C"
